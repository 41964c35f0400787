"""Decode over shared prefixes in FP8 pools, to the bounds of its arithmetic: q is
exact in f16, the K scale is a factor of the scores in 32 bits.

Tolerances (A = the attention over |V|): a score sums 128 products or fewer, exact in
32 bits, of which sum |q k| scale is below 10 for these inputs; it is off by at most
128 * 2^-23 * 10 = 1.5e-4, and a weight, relative to the sum of weights, by twice that,
3.1e-4.  P is rounded to f16: 2^-11 of a weight.  Together below
(2^-11 + 2^-12 + 2^-13) A, beside the output's rounding of 2^-8 |o|.  lse is off by a
score's error and the logarithm's own, below 3e-4.
"""
import pytest
import torch

from test_shared_decode_gpu import FP8, SHAPES, make, reference, run

pytestmark = pytest.mark.gpu


def check(s, got):
    want, want_l, mag = reference(s)
    out, lse = got[0].double(), got[1].double()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -13) * mag
    over = (out - want).abs() - tol
    assert bool((over <= 0).all()), f"{int((~(over <= 0)).sum())} of {over.numel()} outputs off, worst {float(over.max()):.3g}"
    empty = torch.isneginf(want_l)
    assert torch.equal(torch.isneginf(lse), empty) and not bool(out[empty].any())
    assert bool(((lse - want_l)[~empty].abs() <= 3e-4).all())


def batch(dev, shape):
    hq, hkv, d, page = shape
    return make(dev, 17, [5, 1, 0, 17, 2], [300, 129, 64, 1000, 128], [b * 7 % 41 for b in range(28)], hq, hkv, d, page, FP8, loose=3)


@pytest.mark.parametrize("shape", SHAPES)
def test_groups(cuda_device, shape):
    check(*((lambda s: (s, run(s)))(batch(cuda_device, shape))))


@pytest.mark.parametrize("n", [1, 31, 33, 64, 65])
@pytest.mark.parametrize("prefix", [0, 1, 127, 129, 3000])
def test_sizes(cuda_device, n, prefix):
    s = make(cuda_device, n + prefix, [n, 2], [prefix, prefix // 2], [b % 9 + (prefix == 0) for b in range(n + 2)], 8, 2, 128, 16, FP8)
    check(s, run(s))


@pytest.mark.parametrize("q_up,k_up", [(13, -13), (13, 0), (13, 9), (0, 20), (0, -20), (-4, 0)])
def test_scales_are_no_part_of_q(cuda_device, q_up, k_up):
    """Powers of two moved between q, the K scales and the softmax scale change no bit, also
    where |q| comes near f16's range and q * k_scale passes it."""
    s = batch(cuda_device, (16, 4, 128, 16))
    s["q"] = torch.where(s["q"].abs() < 2.0 ** -9, torch.full_like(s["q"], 2.0 ** -9), s["q"])       # stays normal in f16
    base = run(s, scale=128 ** -0.5)
    check(s, base)
    q, k = s["q"], s["scales"]["k_scale"]
    s["q"] = q * 2.0 ** q_up
    s["scales"]["k_scale"] = k * 2.0 ** k_up
    assert float(s["q"].abs().max()) < 65504
    if (q_up, k_up) == (13, 9):
        assert float((s["q"].abs().max() * s["scales"]["k_scale"].max())) > 65504
    moved = run(s, scale=128 ** -0.5 * 2.0 ** -(q_up + k_up))
    assert torch.equal(moved[0], base[0]) and torch.equal(moved[1], base[1])
