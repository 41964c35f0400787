"""What the binding of the reordering makes of a pool's shape: the pages, slots and row
bytes that reach the C call (captured in place of it), and what is refused."""
import pytest
import torch

BF16, FP8, FP4 = 0, 1, 2


def arguments(monkeypatch, pool, **kw):
    import paged_kv_flashattention_gb300 as pa
    from paged_kv_flashattention_gb300 import api
    seen = []
    monkeypatch.setattr(api, "_call", lambda fn, t, p: seen.append(p._obj))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    pools = pool if isinstance(pool, list) else [pool]
    pa.beam_reorder(i32(2, 3), i32(6, 50), i32(6), i32(6), i32(6), pools, pools, **kw)
    p = seen[0]
    return p.num_pages, p.page_size, p.row_bytes


def pool(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype)


@pytest.mark.parametrize("shape,dtype,kw,want", [
    ((100, 16, 16, 128), torch.uint8, {}, (100, 16, 2048)),
    ((1600, 16, 128), torch.uint8, dict(page_size=16, kv_dtype=FP8), (100, 16, 2048)),
    ((1600, 16, 128), torch.uint8, dict(page_size=16), (100, 16, 2048)),
    ((1600, 16, 64), torch.uint8, dict(page_size=16), (100, 16, 1024)),
    ((100, 16, 144), torch.uint8, dict(page_size=16), (100, 16, 144)),
    ((1600, 16, 128), torch.float8_e4m3fn, dict(page_size=16), (100, 16, 2048)),
    ((1600, 8, 128), torch.uint8, dict(page_size=16), (100, 16, 1024)),
    ((1600, 16, 128), torch.bfloat16, dict(page_size=16), (100, 16, 4096)),
    ((1600, 16, 128), torch.bfloat16, dict(page_size=16, kv_dtype=BF16), (100, 16, 4096)),
    ((100, 16, 144), torch.uint8, {}, (100, 16, 144)),
    ((100, 16, 144), torch.uint8, dict(page_size=16, kv_dtype=FP4), (100, 16, 144)),
    ((100, 16, 144), torch.uint8, dict(kv_dtype=FP4), (100, 16, 144)),
    ((1600, 144), torch.uint8, dict(page_size=16, kv_dtype=FP4), (100, 16, 144)),
    ((1600, 144), torch.uint8, dict(page_size=16), (100, 16, 144)),
    ((1600, 1, 128), torch.uint8, dict(page_size=1), (1600, 1, 128)),
    ((1600, 1, 144), torch.uint8, dict(page_size=1, kv_dtype=FP4), (1600, 1, 144)),
])
def test_geometry(monkeypatch, shape, dtype, kw, want):
    assert arguments(monkeypatch, pool(*shape, dtype=dtype), **kw) == want


@pytest.mark.parametrize("shape,dtype,kw", [
    ((1600, 16, 128), torch.bfloat16, {}),                               # slots without a page size
    ((1600, 16, 128), torch.float8_e4m3fn, {}),
    ((1600, 16, 128), torch.uint8, dict(kv_dtype=FP8)),
    ((1600, 144), torch.uint8, dict(kv_dtype=FP4)),
    ((100, 16, 144), torch.uint8, dict(page_size=1, kv_dtype=FP4)),
    ((100, 16, 16, 128), torch.uint8, dict(page_size=1)),
    ((2, 100, 16, 2, 64), torch.bfloat16, dict(page_size=16)),
    ((1600,), torch.uint8, dict(page_size=16)),
])
def test_refused(monkeypatch, shape, dtype, kw):
    with pytest.raises(ValueError):
        arguments(monkeypatch, pool(*shape, dtype=dtype), **kw)


@pytest.mark.parametrize("dtype,kv", [(torch.bfloat16, FP8), (torch.uint8, BF16), (torch.bfloat16, FP4), (torch.uint8, 7)])
@pytest.mark.parametrize("shape", [(100, 16, 144), (100, 16, 2, 64), (1600, 144)])
def test_kv_dtype_of_another_type(monkeypatch, shape, dtype, kv):
    with pytest.raises(ValueError if kv == 7 else TypeError):
        arguments(monkeypatch, pool(*shape, dtype=dtype), page_size=16, kv_dtype=kv)


def test_no_row_of_four_bits_is_a_head_long():
    """What tells FP8 slots of 16 heads from 4-bit pages of 16 rows."""
    import paged_kv_flashattention_gb300 as pa
    sizes = {pa.fp4_row_bytes(h, d) for d in (64, 128) for h in range(1, 4096 // d + 1)}     # (all that there are)
    assert not sizes & {64, 128}


@pytest.mark.parametrize("place", range(4))
@pytest.mark.parametrize("other", [(200, 8, 2, 64), (50, 32, 2, 64), (100, 16, 1, 128), (1600, 2, 64), (204800,)])
def test_every_pool_has_the_same_shape(monkeypatch, place, other):
    """Pools of as many bytes but of another geometry would be copied at wrong offsets."""
    pools = [pool(100, 16, 2, 64) for _ in range(4)]
    assert arguments(monkeypatch, pools) == (100, 16, 128)
    pools[place] = pool(*other)
    assert pools[place].nbytes == pools[place - 1].nbytes
    with pytest.raises(ValueError, match="one shape"):
        arguments(monkeypatch, pools)
