"""Selection's workspace on the host: a size reported for a call serves every smaller
one.  The call refuses a workspace before it launches anything, so without a GPU and
with made-up pointers it answers whether a size is enough (in a process of its own that
sees no GPU)."""
import ctypes
import itertools
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def sizes():
    """(groups, beams, vocabulary, num_out), small to large in each."""
    return [c for c in itertools.product((1, 2, 3, 12, 47, 64, 700), (1, 4, 64), (100, 2048, 2049, 8193, 32000, 128256),
                                         (1, 8, 64, 100)) if c[0] * c[1] <= 65535]


def test_reported_size_never_falls():
    import paged_kv_flashattention_gb300 as pa
    need = {c: pa.beam_select_workspace_size(*c) for c in sizes()}
    by_rows = {}
    for (g, k, v, n), b in need.items():
        by_rows.setdefault((g * k, v, n), set()).add(b)
    assert all(len(b) == 1 for b in by_rows.values())
    keys = sorted(by_rows)
    for a in keys:
        for b in keys:
            if all(x <= y for x, y in zip(a, b)):
                assert min(by_rows[a]) <= min(by_rows[b]), (a, b)


def calls():
    """(reported for, called with, status): 0 would launch; 1 is a workspace refused."""
    from paged_kv_flashattention_gb300 import _lib
    import paged_kv_flashattention_gb300 as pa
    lib = _lib.load()
    out = []
    for top in ((3, 4, 128256, 8), (64, 4, 128256, 8), (47, 64, 2049, 100), (700, 4, 2048, 64)):
        size = pa.beam_select_workspace_size(*top)
        for g, k, v, n in sizes():
            if g * k > top[0] * top[1] or v > top[2] or n > top[3]:
                continue
            p = _lib.BeamSelectParams(logits=0x1000, logits_stride=v, scores=0x2000, num_groups=g, beams=k, vocab=v, num_out=n,
                                      out_scores=0x3000, out_parents=0x4000, out_tokens=0x5000, workspace=0x6000, workspace_bytes=size)
            out.append((top, (g, k, v, n), int(lib.pa_beam_select(ctypes.byref(p), None)), lib.pa_last_error().decode()))
    return out


def test_smaller_calls_are_served():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr
    answers = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(answers) > 100
    refused = [a for a in answers if "workspace" in a[3]]
    assert not refused, refused[0]


if __name__ == "__main__":
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    print(json.dumps(calls()))
