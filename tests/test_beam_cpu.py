"""Refusals of decode over shared prefixes and of beam search on the host: the
C calls run in a child process that sees no GPU (their pointers are made up),
the binding's checks on CPU tensors; sizes of workspaces."""
import json
import os
import subprocess
import sys

import pytest
import torch

import beam_reject_cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rejections():
    from paged_kv_flashattention_gb300 import build
    build.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "beam_reject_cases.py")],
                       capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.parametrize("case", sorted(beam_reject_cases.expected()))
def test_rejects_before_launch(rejections, case):
    status, message = rejections[case]
    want = beam_reject_cases.expected()[case]
    assert status == want, f"{case}: status {status} ({message}), expected {want}"
    if want != 0:
        assert message, f"{case}: no error message"


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_shared_checks():
    import paged_kv_flashattention_gb300 as pa
    kc = torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((4, 8, 64), dtype=torch.bfloat16)
    good = dict(page_table=ints(4, 8), cache_seqlens=ints(4), max_seqlen_k=100, cu_groups=ints(2), prefix_lens=ints(4))

    def call(**kw):
        a = {**good, **kw}
        extra = {k: a.pop(k) for k in list(a) if k not in good}
        return pa.decode_shared(extra.pop("q", q), kc, extra.pop("v", kc), a["page_table"], a["cache_seqlens"], a["max_seqlen_k"],
                                a["cu_groups"], a["prefix_lens"], **extra)

    for bad in (dict(q=q[0]), dict(cache_seqlens=ints(3)), dict(prefix_lens=ints(5)), dict(page_table=ints(3, 8)),
                dict(page_table=ints(4, 6)), dict(cu_groups=ints(0)), dict(out=q[:3]), dict(lse=torch.zeros(4, 7)),
                dict(max_prefix=101), dict(max_group=5), dict(max_suffix=-1), dict(page_table=ints(4, 16)[:, ::2]),
                dict(v=kc[:8]), dict(q=q[..., :32].contiguous())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=q.float()), dict(cu_groups=ints(2).long()), dict(prefix_lens=torch.zeros(4)), dict(lse=torch.zeros(4, 8).double())):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(ValueError, match="CUDA"):
        call()


def test_binding_select_checks():
    import paged_kv_flashattention_gb300 as pa
    x, s = torch.zeros((8, 50)), torch.zeros((2, 4))
    for args, kw in (((x[:7], s), {}), ((x, s[0]), {}), ((x.t().contiguous().t(), s), {}), ((x, s, 51), {}), ((x, s, 0), {}),
                     ((x, s), dict(finished=torch.zeros((2, 3), dtype=torch.uint8))), ((x, s), dict(parents=ints(2, 5))),
                     ((x, s, 5), dict(out_scores=s)), ((x.view(4, 2, 50), s), {}),
                     ((torch.zeros((2, 5, 50))[:, :4], s), {})):
        with pytest.raises(ValueError):
            pa.beam_select(*args, **kw)
    for args, kw in (((x.double(), s), {}), ((x, s.double()), {}), ((x, s), dict(finished=ints(2, 4))),
                     ((x, s), dict(tokens=ints(2, 4).long()))):
        with pytest.raises(TypeError):
            pa.beam_select(*args, **kw)
    with pytest.raises(ValueError):
        pa.beam_select_workspace_size(1, 65, 100, 4)


def test_binding_reorder_checks():
    import paged_kv_flashattention_gb300 as pa
    kc = torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16)
    good = dict(parents=ints(2, 3), token_table=ints(6, 50), table_idx=ints(6), seqlens=ints(6), spare_pages=ints(6), k=[kc], v=[kc])

    def call(**kw):
        a = {**good, **kw}
        extra = {k: a.pop(k) for k in list(a) if k not in good}
        pa.beam_reorder(a["parents"], a["token_table"], a["table_idx"], a["seqlens"], a["spare_pages"], a["k"], a["v"], **extra)

    for bad in (dict(parents=ints(6)), dict(table_idx=ints(5)), dict(seqlens=ints(7)), dict(spare_pages=None), dict(v=[]), dict(k=[], v=[]),
                dict(v=[kc[:8]]), dict(page_size=8), dict(max_seqlen_k=51), dict(history=ints(5, 9)), dict(prefix_lens=ints(5)),
                dict(token_table=ints(6, 100)[:, ::2]), dict(k=[kc.view(-1, 128)], v=[kc.view(-1, 128)])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(parents=ints(2, 3).long()), dict(v=[kc.float()]), dict(history=torch.zeros((6, 9)))):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(ValueError, match="CUDA"):
        call()


@pytest.mark.parametrize("kv_dtype", [None, 2])
def test_shared_workspace_serves_smaller_calls(kv_dtype):
    import itertools

    import paged_kv_flashattention_gb300 as pa
    kc = torch.empty((9, 16, 8, 128), dtype=torch.bfloat16) if kv_dtype is None else \
        torch.empty((9, 16, pa.fp4_row_bytes(8, 128)), dtype=torch.uint8)

    def size(B, groups, group, prefix, suffix):
        return pa.decode_shared_workspace_size((B, 32, 128), kc, 40000, groups, max_prefix=prefix, max_suffix=suffix,
                                               max_group=min(group, B), kv_dtype=kv_dtype, num_kv_heads=8)

    for top in (2100, 4096):
        most = size(64, 8, 64, 32768, top)
        for B, groups, group, prefix, suffix in itertools.product((1, 3, 33, 64), (1, 5, 8), (1, 32, 33, 64), (0, 1, 129, 5000, 32768),
                                                                  (0, 1, 63, 64, 65, 1000, 2047, top)):
            assert size(B, groups, group, prefix, suffix) <= most


def _search(**change):
    import paged_kv_flashattention_gb300 as pa
    dtype = change.pop("dtype", torch.bfloat16)
    pool = lambda: torch.zeros((9, 16, 2, 64), dtype=dtype)
    args = dict(k_caches=[pool(), pool()], v_caches=[pool(), pool()], token_table=torch.zeros((6, 64), dtype=torch.int32),
                table_idx=torch.arange(6, dtype=torch.int32), num_groups=2, beams=3, num_q_heads=4, head_dim=64, vocab=500,
                max_seqlen_k=64, spare_pages=torch.arange(6, dtype=torch.int32))
    args.update(change)
    return pa.BeamSearch(args.pop("k_caches"), args.pop("v_caches"), args.pop("token_table"), args.pop("table_idx"), **args)


@pytest.mark.parametrize("change", [
    dict(k_caches=[]), dict(v_caches=[torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16)]), dict(num_groups=0), dict(beams=0),
    dict(beams=4), dict(spare_pages=None), dict(dtype=torch.uint8), dict(vocab=2), dict(k_scales=[torch.ones(2)]),
    dict(num_q_heads=3), dict(max_prefix=65), dict(head_dim=96),
])
def test_search_refuses(change):
    with pytest.raises((ValueError, TypeError)):
        _search(**change)


def test_search_state():
    s = _search()
    s.start(torch.tensor([37, 0]))
    assert s.lens.tolist() == [37] * 3 + [0] * 3 and s.prefix_lens.tolist() == [32] * 3 + [0] * 3
    assert s.scores.tolist() == [[0.0, float("-inf"), float("-inf")]] * 2
    assert s.cu_groups.tolist() == [0, 3, 6]
    with pytest.raises(ValueError):
        s.start(torch.tensor([1]))
    with pytest.raises(ValueError):
        s.attend(0, torch.zeros((6, 4, 64), dtype=torch.bfloat16))
