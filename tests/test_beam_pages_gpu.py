"""Whose the pages of a beam search are: a request's rows and spare pages name, after every
step, only what they named at the start and what the plan has given its beams since."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,prompts,beams", [(16, (5, 37, 16, 0), 4), (1, (9, 2), 6), (16, (31, 3), 16)])
def test_pages_of_a_request(cuda_device, page, prompts, beams):
    import paged_kv_flashattention_gb300 as pa
    dev, G, K, V, steps = cuda_device, len(prompts), beams, 80, 50
    N, longest = G * K, max(prompts) + steps + 1
    rng = np.random.default_rng(beams)
    pages = sum(-(-p // page) for p in prompts) * K + N * (steps // page + 3)
    ids = list(rng.permutation(pages))
    table, owned = np.zeros((N, longest), np.int32), [set() for _ in range(G)]
    for g, m in enumerate(prompts):
        whole = [ids.pop() for _ in range(m // page)]
        for i in range(K):
            own = whole + ([ids.pop()] if m % page else [])
            owned[g] |= set(own)
            j = np.arange(m)
            if m:
                table[g * K + i, :m] = np.array(own, np.int64)[j // page] * page + j % page
    spare = None
    if page > 1:
        spare = np.array([ids.pop() for _ in range(N)], np.int32)
        for g in range(G):
            owned[g] |= set(spare[g * K:(g + 1) * K])
        spare = torch.from_numpy(spare).to(dev)
    pools = [torch.zeros((pages, page, 2, 64), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    search = pa.BeamSearch(pools[:1], pools[1:], torch.from_numpy(table).to(dev), torch.arange(N, dtype=torch.int32, device=dev),
                           num_groups=G, beams=K, num_q_heads=4, head_dim=64, vocab=V, max_seqlen_k=longest, page_size=page,
                           spare_pages=spare)
    search.start(torch.tensor(prompts))
    free, cursor = torch.tensor(ids, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    given, dropped = set(), 0
    for n in range(steps):
        search.select(torch.from_numpy(rng.normal(size=(N, V)).astype(np.float32)).to(dev))
        search.advance()
        b = search.plan(free, cursor)
        assert pa.device_error() == 0
        position, slot = b.positions[:N].cpu().numpy(), b.slot_mapping[:N].cpu().numpy()
        for s in range(N):
            if position[s] % page == 0:
                owned[s // K].add(slot[s] // page)
                given.add(slot[s] // page)
        assert given == set(ids[:int(cursor[0])])
        rows, lens = search.token_table.cpu().numpy(), search.lens.cpu().numpy()
        for g in range(G):
            seqs = range(g * K, (g + 1) * K)
            named = set().union(*(set(rows[s, :lens[s]] // page) for s in seqs))
            if spare is not None:
                named |= set(search.spare_pages.cpu().numpy()[g * K:(g + 1) * K])
                # pages that are still written to belong to one sequence each
                written = [rows[s, lens[s] - 1] // page for s in seqs] + list(search.spare_pages.cpu().numpy()[g * K:(g + 1) * K])
                assert len(set(written)) == 2 * K
            assert named <= owned[g], n
            dropped += len(owned[g] - named)
    assert dropped > 0                                   # pages that no row names are the request's all the same
    assert sum(map(len, owned)) == len(set().union(*owned))
