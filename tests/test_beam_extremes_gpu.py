"""The ends of the ranges that selection, reordering and decode over shared prefixes allow,
and calls on two streams at once."""
import numpy as np
import pytest
import torch

from test_beam_gpu import plain_reorder, reorder_case
from test_beam_large_gpu import plain
from test_shared_decode_gpu import FP4, check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,K,V,n", [(1, 1, (1 << 24) - 1, 128), (65535, 1, 2, 2), (1023, 64, 130, 128), (1, 64, 140000, 128),
                                     (1, 1, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select(cuda_device, G, K, V, n, dtype):
    import paged_kv_flashattention_gb300 as pa
    g = torch.Generator(device=cuda_device).manual_seed(V)
    x = torch.randn((G * K, V), generator=g, device=cuda_device).to(dtype)
    s = -torch.rand((G, K), generator=g, device=cuda_device) * 5
    got, want = pa.beam_select(x, s, n), plain(x, s, n)
    assert pa.device_error() == 0
    assert torch.equal(got[1].long(), want[1]) and torch.equal(got[2].long(), want[2])
    assert bool(((got[0].double() - want[0]).abs() <= 2.0 ** -24 * want[0].abs() + 2.0 ** -20).all())


@pytest.mark.parametrize("kv", [0, FP4])
@pytest.mark.parametrize("sizes,prefix", [([1] * 16384, 17), ([16384], 16), ([0] * 16383 + [3], 17)])
def test_shared(cuda_device, sizes, prefix, kv):
    """As many groups and sequences as a call takes; some of the rows are compared."""
    s = make(cuda_device, 3, sizes, [prefix] * len(sizes), [b % 3 for b in range(sum(sizes))], 4, 2, 64, 16, kv)
    out, lse = run(s)
    lens, table, page, hkv = s["host"]
    rows = list(range(0, len(lens), max(1, len(lens) // 200))) + [len(lens) - 1]
    some = dict(s, q=s["q"][rows], host=([lens[r] for r in rows], table[rows], page, hkv))
    check(some, (out[rows], lse[rows]))


def test_selections_on_two_streams(cuda_device):
    """Scores and flags in place, step after step, a workspace each."""
    import paged_kv_flashattention_gb300 as pa
    shapes = [(1, 4, 32000), (47, 4, 32000), (9, 5, 5008)]
    dev, steps = cuda_device, 12
    x = [torch.randn((steps, g * k, v), generator=torch.Generator(device=dev).manual_seed(v + g), device=dev).bfloat16()
         for g, k, v in shapes]
    start = [(torch.zeros((g, k), device=dev), torch.zeros((g, k), dtype=torch.uint8, device=dev)) for g, k, _ in shapes]
    for s, _ in start:
        s[:, 1:] = float("-inf")

    def search(i, out):
        s, f = (t.clone() for t in start[i])
        ws = torch.empty(pa.beam_select_workspace_size(*shapes[i], shapes[i][1]), dtype=torch.uint8, device=dev)
        for n in range(steps):
            _, parents, tokens = pa.beam_select(x[i][n], s, finished=f, pad_token=1, out_scores=s, out_finished=f, workspace=ws)
            f |= tokens % 7 == 0
            out += [s.clone(), parents, tokens, f.clone()]

    alone = [[] for _ in shapes]
    for i in range(len(shapes)):
        search(i, alone[i])
    torch.cuda.synchronize()
    for _ in range(3):
        together, streams = [[] for _ in shapes], [torch.cuda.Stream(dev) for _ in shapes]
        for i, st in enumerate(streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                search(i, together[i])
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            assert len(a) == len(b) and all(torch.equal(u, v) for u, v in zip(a, b))


def test_reorder_captured_and_on_two_streams(cuda_device):
    """Two states, a captured call each, replayed at once on two streams."""
    import paged_kv_flashattention_gb300 as pa
    dev = cuda_device
    work = []
    for seed, (G, K, longest) in enumerate(((5, 4, 200), (2, 16, 90))):
        rng = np.random.default_rng(seed)
        parents, table, idx, lens, spare, pools, dtype = reorder_case(rng, G, K, 16, longest, layers=3)
        d = lambda a: torch.from_numpy(np.array(a)).to(dev)
        state = dict(parents=d(parents), table=d(table), idx=d(idx), lens=d(lens), spare=d(spare),
                     pools=[p.to(dev).view(dtype) for p in pools])
        stream = torch.cuda.Stream(dev)

        def call(s=state):
            pa.beam_reorder(s["parents"], s["table"], s["idx"], s["lens"], s["spare"], s["pools"][:3], s["pools"][3:])

        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
        host = (parents, table.copy(), idx, lens, spare.copy(), [p.flatten(2).numpy().copy() for p in pools])
        work.append((graph, stream, state, host))
    for _ in range(7):
        torch.cuda.synchronize()
        for graph, stream, _, _ in work:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert pa.device_error() == 0
        for _, _, s, (parents, table, idx, lens, spare, pools) in work:
            plain_reorder(parents, table, idx, lens, spare, pools, 16)
            assert np.array_equal(s["table"].cpu().numpy(), table) and np.array_equal(s["spare"].cpu().numpy(), spare)
            for p, w in zip(s["pools"], pools):
                assert np.array_equal(p.view(torch.uint8).flatten(2).cpu().numpy(), w)
