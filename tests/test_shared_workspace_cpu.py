"""The workspace of decode over shared prefixes on the host: a size reported for a call
serves every call with bounds and counts up to its own, none of them (no groups, no prefix,
no keys behind one) excepted."""
import ctypes
import itertools
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GRID = dict(B=(1, 3, 64), keys=(1, 2000, 2112, 2113, 8256), groups=(0, 1, 7, 64), prefix=(0, 129, 8192), suffix=(0, 64, 2111),
            group=(0, 1, 64))


def cases():
    for c in itertools.product(*GRID.values()):
        c = dict(zip(GRID, c))
        if c["prefix"] <= c["keys"] and c["suffix"] <= c["keys"] and c["group"] <= c["B"]:
            yield c


def params(c, kv, chunk, **change):
    from paged_kv_flashattention_gb300 import _lib
    dec = dict(q=0x1000, k_cache=0x2000, v_cache=0x3000, page_table=0x4000, page_table_stride=1024, cache_seqlens=0x5000, num_seqs=c["B"],
               max_seqlen_k=c["keys"], num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, num_pages=100, scale=0.125,
               out=0x6000, workspace=0x10000, kv_chunk=chunk, kv_dtype=kv, k_scale=0x7000, v_scale=0x7000)
    return _lib.DecodeSharedParams(_lib.DecodeParams(**{**dec, **change}), 0x8000, 0x9000, c["groups"], c["group"], c["prefix"], c["suffix"])


@pytest.mark.parametrize("kv,chunk", [(0, 0), (1, 0), (2, 0), (0, 256)])
def test_reported_size_never_falls(kv, chunk):
    from paged_kv_flashattention_gb300 import _lib
    lib = _lib.load()
    size = {}
    for c in cases():
        size[tuple(c.values())] = lib.pa_decode_shared_workspace_size(ctypes.byref(params(c, kv, chunk)))
    assert all(v > 0 for v in size.values())
    for a, b in itertools.product(size, size):
        if all(x <= y for x, y in zip(a, b)):
            assert size[a] <= size[b], (a, b)


def calls():
    """[bounds reported for, bounds called with, message] where a workspace was refused."""
    from paged_kv_flashattention_gb300 import _lib
    lib = _lib.load()
    out, n = [], 0
    tops = [dict(B=64, keys=8256, groups=1, prefix=8192, suffix=64, group=64), dict(B=64, keys=2113, groups=64, prefix=129, suffix=2111, group=1),
            dict(B=3, keys=2113, groups=7, prefix=129, suffix=0, group=1), dict(B=64, keys=2112, groups=0, prefix=0, suffix=0, group=0)]
    for kv, top in itertools.product((0, 1, 2), tops):
        size = lib.pa_decode_shared_workspace_size(ctypes.byref(params(top, kv, 0)))
        for c in cases():
            if all(c[k] <= top[k] for k in top):
                lib.pa_decode_shared(ctypes.byref(params(c, kv, 0, workspace_bytes=size)), None)
                n += 1
                if b"workspace" in lib.pa_last_error():
                    out.append((top, c, lib.pa_last_error().decode()))
    return n, out


def test_smaller_calls_are_served():
    """In a process that sees no GPU: a workspace is refused before anything is launched."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr
    n, refused = json.loads(r.stdout.strip().splitlines()[-1])
    assert n > 200 and not refused, refused[0]


if __name__ == "__main__":
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    print(json.dumps(calls()))
