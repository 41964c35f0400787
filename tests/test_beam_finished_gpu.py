"""``finished`` goes where the beams go: selection gives each chosen beam its parent's
entry, and a search whose caller only ORs in the end token keeps every ended beam
ended and no other."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,K,V,n", [(3, 5, 700, 5), (1, 4, 32000, 9), (1100, 3, 100, 3), (47, 4, 32000, 4), (2, 64, 90, 64)])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.bool])
def test_entries_of_the_parents(cuda_device, G, K, V, n, dtype):
    import paged_kv_flashattention_gb300 as pa
    g = torch.Generator(device=cuda_device).manual_seed(K + V)
    x = torch.randn((G * K, V), generator=g, device=cuda_device).bfloat16()
    s = -torch.rand((G, K), generator=g, device=cuda_device)
    s[0, 0] = float("-inf")
    f = torch.randint(0, 2 if dtype == torch.bool else 200, (G, K), generator=g, device=cuda_device).to(dtype)
    f[torch.rand((G, K), generator=g, device=cuda_device) < 0.5] = 0
    before = f.clone()
    plain = pa.beam_select(x, s, n, finished=f)
    assert torch.equal(f, before)
    out = torch.full((G, n), 1, dtype=dtype, device=cuda_device)
    got = pa.beam_select(x, s, n, finished=f, out_finished=out)
    assert all(torch.equal(a, b) for a, b in zip(plain, got)) and torch.equal(f, before)
    assert torch.equal(out, before.gather(1, got[1].long()))
    if n == K:
        got = pa.beam_select(x, s, n, finished=f, out_finished=f)
        assert all(torch.equal(a, b) for a, b in zip(plain, got))
        assert torch.equal(f, before.gather(1, got[1].long()))
    out.fill_(1)
    pa.beam_select(x, s, n, out_finished=out)            # none has ended
    assert not bool(out.any())
    assert pa.device_error() == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("page,prompts,beams", [(16, (5, 37, 16), 4), (1, (9,), 6), (16, (20, 3), 64)])
def test_search(cuda_device, page, prompts, beams, captured):
    import paged_kv_flashattention_gb300 as pa
    dev, G, K, V, EOS, PAD, steps = cuda_device, len(prompts), beams, 150, 7, 2, 24
    N, longest = G * K, max(prompts) + steps + 1
    rng = np.random.default_rng(beams)
    ids = list(range(sum(-(-p // page) for p in prompts) * K + N * (steps // page + 3)))
    table = np.zeros((N, longest), np.int32)
    for g, m in enumerate(prompts):
        whole = [ids.pop() for _ in range(m // page)]
        for i in range(K):
            own = whole + ([ids.pop()] if m % page else [])
            j = np.arange(m)
            table[g * K + i, :m] = np.array(own, np.int64)[j // page] * page + j % page
    spare = torch.tensor([ids.pop() for _ in range(N)], dtype=torch.int32, device=dev) if page > 1 else None
    pools = [torch.zeros((sum(-(-p // page) for p in prompts) * K + N * (steps // page + 3), page, 2, 64), dtype=torch.bfloat16,
                         device=dev) for _ in range(2)]
    search = pa.BeamSearch([pools[0]], [pools[1]], torch.from_numpy(table).to(dev), torch.arange(N, dtype=torch.int32, device=dev),
                           num_groups=G, beams=K, num_q_heads=4, head_dim=64, vocab=V, max_seqlen_k=longest, page_size=page,
                           spare_pages=spare, pad_token=PAD)
    search.start(torch.tensor(prompts))
    free, cursor = torch.tensor(ids, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    logits = torch.zeros((N, V), dtype=torch.float32, device=dev)

    def step():
        search.select(logits)
        search.finished |= search.tokens == EOS          # all that the caller does
        search.advance()
        search.plan(free, cursor)

    graph, told, ended_once = None, [[] for _ in range(N)], 0
    for n in range(steps):
        x = rng.normal(size=(N, V)).astype(np.float32) * 2
        x[:, EOS] += 3.0
        logits.copy_(torch.from_numpy(x))
        if captured and n == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=torch.cuda.Stream(dev)):
                step()
        graph.replay() if graph is not None else step()
        assert pa.device_error() == 0
        parents, tokens = search.parents.cpu().numpy(), search.tokens.cpu().numpy()
        told = [told[g * K + parents[g, i]] + [int(tokens[g, i])] for g in range(G) for i in range(K)]
        ended = [EOS in t for t in told]
        assert search.finished.view(-1).cpu().bool().tolist() == ended, n
        for t in told:
            if EOS in t:
                assert set(t[t.index(EOS) + 1:]) <= {PAD}
        ended_once += sum(ended) not in (0, N)
    assert ended_once > 2                                # steps with beams of both kinds
