"""Selection from rows whose logits lie far from zero, as rows of which every word is
banned by the type's lowest value do: score + (x - max) - ln sum exp(x - max) keeps
the logarithm, in 64 bits, whatever max is."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ROWS = [(2, 3, 700), (1, 4, 32000), (50, 1, 128256), (1100, 3, 100)]     # by chunks and in two passes


@pytest.mark.parametrize("G,K,V", ROWS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("end", ["min", "max"])
def test_rows_of_one_extreme_value(cuda_device, G, K, V, dtype, end):
    """Every word as likely: total = score - ln V, to lse's 2^-20 and one rounding."""
    import paged_kv_flashattention_gb300 as pa
    x = torch.full((G * K, V), getattr(torch.finfo(dtype), end), dtype=dtype, device=cuda_device)
    scores = -torch.arange(G * K, device=cuda_device).float().view(G, K) % 7 * 0.5
    n = 5
    total, parents, tokens = pa.beam_select(x, scores, n)
    assert pa.device_error() == 0
    best = scores.double().amax(1, keepdim=True) - math.log(V)
    assert bool(((total.double() - best).abs() <= 2.0 ** -24 * best.abs() + 2.0 ** -20).all())
    assert torch.equal(tokens, torch.arange(n, dtype=torch.int32, device=cuda_device).expand(G, n))
    assert torch.equal(parents.long(), scores.argmax(1, keepdim=True).expand(G, n))      # the first of the best


@pytest.mark.parametrize("G,K,V", ROWS)
@pytest.mark.parametrize("at", [-2.0 ** 60, 2.0 ** 60, -1e38])
def test_rows_around_a_far_value(cuda_device, G, K, V, at):
    """Half of the words at a far value, the others at the lowest one: the first half shares
    the weight."""
    import paged_kv_flashattention_gb300 as pa
    x = torch.full((G * K, V), torch.finfo(torch.float32).min, device=cuda_device)
    x[:, 1::2] = at
    scores = torch.zeros((G, K), device=cuda_device)
    n = 7
    total, parents, tokens = pa.beam_select(x, scores, n)
    want = -math.log(V // 2)
    assert bool(((total.double() - want).abs() <= 2.0 ** -24 * abs(want) + 2.0 ** -20).all())
    assert not bool(parents.any()) and tokens.tolist() == [[1, 3, 5, 7, 9, 11, 13]] * G
