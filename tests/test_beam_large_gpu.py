"""Selection above 3000 tiles of 2048 logits (csrc/beam.cu: (maximum, sum) of 32
columns first, then a CTA per row that reads the few blocks again that hold its n
largest), against a plain implementation in 64 bits.  Beams and tokens are exact,
whatever is equal; a total is one rounding to fp32 and lse's error, below 2^-20,
off."""
import pytest
import torch

pytestmark = pytest.mark.gpu

NEG = float("-inf")
# groups, beams, vocabulary: all over 3000 tiles; the last two have rows of one tile
SHAPES = [(47, 4, 32000), (50, 1, 128256), (25, 2, 128255), (100, 4, 16411), (1100, 3, 100), (60000, 1, 7)]


def plain(logits, scores, n, finished=None, pad=0):
    """(totals, parents, tokens), each [G, n]; equal totals by k * V + v."""
    G, K = scores.shape
    V = logits.shape[-1]
    bad = lambda t: t.double().nan_to_num(nan=NEG, posinf=NEG, neginf=NEG)
    x, sc = bad(logits), bad(scores)
    top = x.amax(1, keepdim=True)
    top = torch.where(top > NEG, top, torch.zeros_like(top))
    total = sc.view(-1, 1) + ((x - top) - (x - top).exp().sum(1, keepdim=True).log())
    total = torch.where(torch.isnan(total) | (x == NEG), NEG, total)
    if finished is not None:
        done = finished.view(-1) != 0
        total[done] = NEG
        total[done, pad] = sc.view(-1)[done]
    total = total.view(G, K * V)
    value, at = torch.sort(total, dim=1, descending=True, stable=True)
    return value[:, :n], at[:, :n] // V, at[:, :n] % V


def check(logits, scores, n, finished=None, pad=0):
    import paged_kv_flashattention_gb300 as pa
    rows, V = logits.shape
    assert rows * -(-V // 2048) > 3000
    got = pa.beam_select(logits, scores, n, finished=finished, pad_token=pad)
    want = plain(logits, scores, n, finished, pad)
    assert pa.device_error() == 0
    for a, b, what in ((got[1], want[1], "parents"), (got[2], want[2], "tokens")):
        wrong = (a != b).any(1).nonzero().flatten()
        assert wrong.numel() == 0, f"{what} of {wrong.numel()} groups, first {int(wrong[0])}: {a[wrong[0]].tolist()}, " \
            f"due {b[wrong[0]].tolist()}"
    t, fin = got[0].double(), want[0] > NEG
    assert torch.equal(t > NEG, fin) and bool((t[~fin] == NEG).all())
    assert bool(((t - want[0])[fin].abs() <= 2.0 ** -24 * want[0][fin].abs() + 2.0 ** -20).all())
    return got


def randn(dev, shape, seed, spread=1.0):
    return torch.randn(shape, generator=torch.Generator(device=dev).manual_seed(seed), device=dev) * spread


def scores_of(dev, G, K, seed):
    return -20 * torch.rand((G, K), generator=torch.Generator(device=dev).manual_seed(seed), device=dev)


def counts(V):
    return [n for n in (1, 8, 10, 128) if n <= V] + ([V] if V < 128 else [])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("G,K,V", SHAPES)
@pytest.mark.parametrize("slack", [0, 3, 8])
def test_vocabularies(cuda_device, G, K, V, slack, dtype):
    """Row distances of every alignment; NaN lies behind the rows."""
    x = randn(cuda_device, (G * K, V + slack), V + slack, 3.0)
    x[:, V:] = float("nan")
    x = x.to(dtype)[:, :V]
    for n in counts(V):
        check(x, scores_of(cuda_device, G, K, n), n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("levels", [1, 2, 8, 16, 32, 64, 300])
@pytest.mark.parametrize("G,K,V", [(47, 4, 32000), (50, 1, 128256), (100, 4, 16411), (1100, 3, 100)])
def test_few_values(cuda_device, G, K, V, levels, dtype):
    """Rows of a few values, so that equal ones lie on both sides of what is kept."""
    g = torch.Generator(device=cuda_device).manual_seed(levels * 7 + V)
    x = torch.randint(0, levels, (G * K, V), generator=g, device=cuda_device).float() * 0.25
    x = x.to(dtype)
    for n in [8, 10, 16, 64] + ([128] if V >= 128 else []):
        check(x, scores_of(cuda_device, G, K, n), n)


@pytest.mark.parametrize("low", [-1.0, NEG, float("nan"), float("inf")])
@pytest.mark.parametrize("G,K,V", [(47, 4, 32000), (50, 1, 128256), (100, 4, 16411)])
@pytest.mark.parametrize("head", [1, 8, 255, 256, 257, 2048, 8192])
def test_equal_logits_behind_lower_ones(cuda_device, G, K, V, head, low):
    """Equal logits of which the first are lower or banned: the due ones begin inside a
    block, behind the first block, tile or span."""
    x = torch.full((G * K, V), 0.5, dtype=torch.bfloat16, device=cuda_device)
    x[:, :head] = low
    for n in (1, 4, 8, 128):
        check(x, scores_of(cuda_device, G, K, n), n)


@pytest.mark.parametrize("where", [100.0, -3.0])
def test_narrow_rows(cuda_device, where):
    """bf16 rows around a value with few steps between."""
    x = (randn(cuda_device, (60, 128256), 3, 0.1) + where).bfloat16()
    for n in (4, 8, 64):
        check(x, scores_of(cuda_device, 60, 1, n), n)


@pytest.mark.parametrize("G,K,V", [(47, 4, 32000), (25, 2, 128255)])
def test_equal_rows(cuda_device, G, K, V):
    """Beams whose rows are the same, at every alignment: ties go to the lower beam."""
    x = randn(cuda_device, (1, V), 4, 2.0).expand(G * K, -1).contiguous()
    for dtype in (torch.float32, torch.bfloat16):
        wide = torch.zeros((G * K, V + 1), dtype=dtype, device=cuda_device)
        wide[:, :V] = x
        check(wide[:, :V], torch.full((G, K), -1.5, device=cuda_device), 16)


@pytest.mark.parametrize("how", ["rising", "falling", "steps", "peak_last", "peaks_apart"])
def test_orders(cuda_device, how):
    V = 70001
    i = torch.arange(V, device=cuda_device, dtype=torch.float32)
    row = {"rising": i * 1e-3, "falling": -i * 1e-3, "steps": torch.floor(i / 1000) * 0.125,
           "peak_last": torch.where(i == V - 1, 50.0, 0.0), "peaks_apart": torch.where(i % 2048 == 7, 3.0, 0.0)}[how]
    x = torch.stack([row, row * 0.5, row.flip(0)] * 30)
    for n in (4, 64):
        check(x, scores_of(cuda_device, 30, 3, n), n)
        check(x * 100, scores_of(cuda_device, 30, 3, n), n)


@pytest.mark.parametrize("keep", [0, 1, 3, 60, 3000])
@pytest.mark.parametrize("G,K,V", [(47, 4, 32000), (100, 4, 16411), (1100, 3, 100)])
def test_banned_words(cuda_device, G, K, V, keep):
    """Rows of which a few words are left, or none; NaN and +inf among them."""
    keep = min(keep, V)
    x = randn(cuda_device, (G * K, V), keep, 3.0)
    rank = torch.argsort(torch.argsort(randn(cuda_device, (G * K, V), keep + 1), 1), 1)
    x = x.masked_fill(rank >= keep, NEG)
    x[1, 5], x[2, 7], x[3, :], x[4, 50:] = float("nan"), float("inf"), NEG, float("nan")
    for n in (1, 6, 64):
        check(x, scores_of(cuda_device, G, K, n), n)


@pytest.mark.parametrize("pad", [0, 3, 31999])
def test_finished_and_dead_beams(cuda_device, pad):
    G, K, V = 47, 4, 32000
    x = randn(cuda_device, (G * K, V), pad).bfloat16()
    s = scores_of(cuda_device, G, K, pad)
    f = torch.zeros((G, K), dtype=torch.uint8, device=cuda_device)
    f[0, 1], f[1], f[2, 0], f[5, ::2] = 1, 1, 7, 1
    s[0, 0], s[2, 0], s[2, 3], s[3] = NEG, float("nan"), float("inf"), NEG
    x[4:8] = float("nan")                                # logits of ended beams are not read
    for n in (1, 5, 64):
        check(x, s, n, f, pad)
        check(x, s, n, f.bool(), pad)


def test_equal_calls_give_equal_bits(cuda_device):
    import paged_kv_flashattention_gb300 as pa
    x = randn(cuda_device, (200, 32000), 1).bfloat16()
    x[:100] = (torch.arange(32000, device=cuda_device) % 4099).float() * 0.003
    s = scores_of(cuda_device, 50, 4, 0)
    ref = pa.beam_select(x, s, 100)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(ref, pa.beam_select(x, s, 100)))
