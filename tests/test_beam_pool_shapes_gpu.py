"""Reordering over every shape of pool that the stores and decode take: paged and flat
ones, bf16, FP8 as uint8 or float8_e4m3fn, and 4-bit rows, with as many heads as a page
has slots and with other numbers."""
import numpy as np
import pytest
import torch

from test_beam_gpu import plain_reorder, reorder_case

pytestmark = pytest.mark.gpu

BF16, FP8, FP4 = 0, 1, 2


def layouts():
    import itertools
    out = []
    for heads, d, page in itertools.product((2, 16), (64, 128), (1, 16)):
        for kind, flat, told in itertools.product(("bf16", "uint8", "e4m3", "fp4"), (False, True), (False, True)):
            if page == 1 and heads == 16 and d == 128:
                continue                             # (nothing that the others do not have)
            out.append((kind, flat, told, heads, d, page))
    return out


@pytest.mark.parametrize("search", [False, True])
@pytest.mark.parametrize("kind,flat,told,heads,d,page", layouts())
def test_layouts(cuda_device, kind, flat, told, heads, d, page, search):
    """page_size is given, as BeamSearch does it; ``told``: kv_dtype too."""
    import paged_kv_flashattention_gb300 as pa
    if search and not told and kind == "fp4":
        pytest.skip("4-bit pools are asked for by kv_dtype everywhere")
    rng = np.random.default_rng(heads + d + page)
    row = {"bf16": 2 * heads * d, "uint8": heads * d, "e4m3": heads * d, "fp4": pa.fp4_row_bytes(heads, d)}[kind]
    parents, table, idx, lens, spare, pools, _ = reorder_case(rng, 3, 4, page, 70, layers=1, row=(row,), dtype=torch.uint8)
    shape = (heads, d) if kind != "fp4" else (row,)
    dp = []
    for p in pools:
        t = p.to(cuda_device)
        t = t.view(torch.bfloat16) if kind == "bf16" else t.view(torch.float8_e4m3fn) if kind == "e4m3" else t
        dp.append(t.reshape((-1,) + shape) if flat else t.reshape(tuple(p.shape[:2]) + shape))
    dev = lambda a: torch.from_numpy(np.array(a)).to(cuda_device)
    t, s = dev(table), dev(spare)
    kv = {"bf16": BF16, "uint8": FP8, "e4m3": FP8, "fp4": FP4}[kind]
    if search:
        scales = None if kind == "bf16" else [torch.ones(heads, device=cuda_device)]
        b = pa.BeamSearch([dp[0]], [dp[1]], t, dev(idx), num_groups=3, beams=4, num_q_heads=heads, head_dim=d, vocab=100,
                          max_seqlen_k=table.shape[1], page_size=page, spare_pages=s, k_scales=scales, v_scales=scales,
                          kv_dtype=kv if told else None)
        b.parents.copy_(dev(parents))
        b.lens.copy_(dev(lens))
        b.advance()
    else:
        kw = dict(page_size=page, kv_dtype=kv if told else None)
        pa.beam_reorder(dev(parents), t, dev(idx), dev(lens), s, dp[:1], dp[1:], **kw)
    assert pa.device_error() == 0
    want = [p.flatten(2).numpy().copy() for p in pools]
    table, spare = table.copy(), spare.copy()
    plain_reorder(parents, table, idx, lens, spare, want, page)
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(s.cpu().numpy(), spare)
    for p, w in zip(dp, want):
        assert np.array_equal(p.contiguous().view(torch.uint8).reshape(w.shape).cpu().numpy(), w)
