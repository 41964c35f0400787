"""Beam search as it is run: slots, stores, attention over the shared prompt,
selection, reordering, step after step over one paged pool, eager and as a
replayed graph.  A small model of two layers takes K, V and q of a token from
tables.  Each step is checked against the beams' own histories in 64 bits: the
attention by its rounding (the bounds of test_shared_decode_gpu), beams and
tokens exactly.
"""
import numpy as np
import pytest
import torch

from test_beam_gpu import plain_select
from test_shared_decode_gpu import FP4, FP8

pytestmark = pytest.mark.gpu

LAYERS, VOCAB, EOS = 2, 997, 3


class Model:
    def __init__(self, dev, hq, hkv, d, kv, seed):
        import paged_kv_flashattention_gb300 as pa
        g = torch.Generator(device=dev).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=dev)
        self.pa, self.kv, self.d, self.hkv, self.dev = pa, kv, d, hkv, dev
        self.q = [r(VOCAB, hq, d).bfloat16() for _ in range(LAYERS)]
        self.k = [r(VOCAB, hkv, d).bfloat16() for _ in range(LAYERS)]
        self.v = [r(VOCAB, hkv, d).bfloat16() for _ in range(LAYERS)]
        self.w = [(r(hq * d, VOCAB) * 0.2).bfloat16() for _ in range(LAYERS)]
        self.ks = self.vs = None
        if kv:
            s = 4.5 / (448 if kv == FP8 else 2688) * (0.8 + 0.4 * torch.rand((2, LAYERS, hkv), generator=g, device=dev))
            self.ks, self.vs = list(s[0].unbind(0)), list(s[1].unbind(0))
        # what the pools hold of each token, in 64 bits
        slot = torch.arange(VOCAB, dtype=torch.int32, device=dev)
        self.vals = []
        for l in range(LAYERS):
            pools = self.pools(VOCAB, 1)
            self.store(l, slot.long(), slot, *pools)
            pools = [p.flatten(0, 1) for p in pools]
            if kv == 0:
                vals = [p.double() for p in pools]
            elif kv == FP8:
                vals = [p.view(torch.float8_e4m3fn).double() * s.double()[:, None] for p, s in zip(pools, (self.ks[l], self.vs[l]))]
            else:
                from oracle import fp4
                vals = [torch.from_numpy(fp4.unpack(p.cpu().numpy(), hkv, d, s.cpu().numpy())).double().to(dev)
                        for p, s in zip(pools, (self.ks[l], self.vs[l]))]
            self.vals.append(vals)

    def pools(self, pages, page):
        shape = (pages, page, self.pa.fp4_row_bytes(self.hkv, self.d)) if self.kv == FP4 else (pages, page, self.hkv, self.d)
        dtype = torch.bfloat16 if self.kv == 0 else torch.uint8
        return [torch.zeros(shape, dtype=dtype, device=self.dev) for _ in range(2)]

    def store(self, layer, tokens, slots, kc, vc):
        k, v = self.k[layer][tokens], self.v[layer][tokens]
        if self.kv == 0:
            self.pa.store_kv(k, v, slots, kc, vc)
        else:
            (self.pa.store_kv_fp8 if self.kv == FP8 else self.pa.store_kv_fp4)(k, v, slots, kc, vc, self.ks[layer], self.vs[layer])


def attention(model, layer, tokens, q):
    """(out, attention over |V|) of one sequence in 64 bits."""
    k, v = (x[tokens].permute(1, 0, 2) for x in model.vals[layer])
    hq = q.shape[0]
    w = torch.softmax((q.double().view(model.hkv, hq // model.hkv, -1) @ k.transpose(1, 2)) * model.d ** -0.5, -1)
    return (w @ v).reshape(hq, -1), (w @ v.abs()).reshape(hq, -1)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kv,page,hq,hkv,d,prompts,beams", [
    (0, 16, 8, 2, 128, (1, 16, 37, 300), 5),
    (0, 1, 6, 3, 64, (5, 130), 4),
    (FP8, 16, 4, 4, 64, (47, 15, 64), 4),
    (FP4, 16, 8, 2, 64, (33, 140), 3),
    (0, 16, 4, 1, 64, (200,), 64),
    (0, 16, 4, 2, 64, (20, 31), 1),
])
def test_beam_search(cuda_device, kv, page, hq, hkv, d, prompts, beams, captured):
    import paged_kv_flashattention_gb300 as pa
    dev, G, K, steps = cuda_device, len(prompts), beams, 37
    N, rng = G * K, np.random.default_rng(kv * 7 + page + beams)
    model = Model(dev, hq, hkv, d, kv, 11 + beams)
    longest = max(prompts) + steps + 1
    # pages: the prompts' full ones once, every sequence a last page and a spare page of
    # its own, the rest free
    ids = list(rng.permutation(sum(-(-p // page) for p in prompts) + 2 * N + N * (steps // page + 2)))
    pages, table = len(ids), np.full((N + 1, longest), -5, np.int32)
    idx = rng.permutation(N + 1)[:N].astype(np.int32)
    for g, n in enumerate(prompts):
        whole = [ids.pop() for _ in range(n // page)]
        for i in range(K):
            own = whole + ([ids.pop()] if n % page else [])
            j = np.arange(n)
            table[idx[g * K + i], :n] = np.array(own, np.int64)[j // page] * page + j % page
    spare = torch.tensor([ids.pop() for _ in range(N)], dtype=torch.int32, device=dev) if page > 1 else None
    free = torch.tensor(ids, dtype=torch.int32, device=dev)
    cursor = torch.zeros(2, dtype=torch.int32, device=dev)
    kcs, vcs = zip(*(model.pools(pages, page) for _ in range(LAYERS)))
    table_d, idx_d = torch.from_numpy(table).to(dev), torch.from_numpy(idx).to(dev)
    search = pa.BeamSearch(kcs, vcs, table_d, idx_d, num_groups=G, beams=K, num_q_heads=hq, head_dim=d, vocab=VOCAB,
                           max_seqlen_k=longest, max_prefix=max(prompts), max_suffix=page + steps, page_size=page,
                           spare_pages=spare, pad_token=EOS, k_scales=model.ks, v_scales=model.vs, kv_dtype=FP4 if kv == FP4 else None)
    # the prompts, through the rows of beam 0
    told = [list(rng.integers(0, VOCAB, n)) for n in prompts]
    for g, n in enumerate(prompts):
        slots = table_d[int(idx[g * K]), :n].contiguous()
        for l in range(LAYERS):
            model.store(l, torch.tensor(told[g], device=dev), slots, kcs[l], vcs[l])
    search.start(torch.tensor(prompts, dtype=torch.int32))
    beams_told = [list(told[g]) for g in range(G) for _ in range(K)]
    history = torch.full((N, steps + 1), -1, dtype=torch.int32, device=dev)
    at = torch.zeros((1, 1), dtype=torch.int64, device=dev)

    outs = [torch.zeros((N, hq, d), dtype=torch.bfloat16, device=dev) for _ in range(LAYERS)]
    logits = torch.zeros((N, VOCAB), dtype=torch.bfloat16, device=dev)

    def choose():
        search.select(logits)
        search.advance(history)
        history.scatter_(1, at.expand(N, 1), search.tokens.view(N, 1))
        at.add_(1)
        search.finished.copy_(search.finished.gather(1, search.parents.long()) | (search.tokens == EOS))

    def step():
        tokens = search.tokens.view(N).long()
        batch = search.plan(free, cursor)
        total = 0
        for l in range(LAYERS):
            model.store(l, tokens, batch.slot_mapping, kcs[l], vcs[l])
            search.attend(l, model.q[l][tokens], out=outs[l])
            total = total + outs[l].view(N, -1) @ model.w[l]
        logits.copy_(total)
        choose()

    def check_choice(scores, finished):
        """The selection from ``logits``, and the histories behind it."""
        nonlocal beams_told
        want = plain_select(logits.double().cpu().numpy(), scores, K, finished, EOS)
        parents, tokens = search.parents.cpu().numpy(), search.tokens.cpu().numpy()
        assert np.array_equal(parents, want[1]) and np.array_equal(tokens, want[2])
        got = search.scores.double().cpu().numpy()
        fin = np.isfinite(want[0])
        assert np.array_equal(np.isfinite(got), fin)
        assert bool((np.abs(got - want[0])[fin] <= 2.0 ** -24 * np.abs(want[0][fin]) + 2.0 ** -20).all())
        beams_told = [beams_told[g * K + parents[g, i]] + [int(tokens[g, i])] for g in range(G) for i in range(K)]

    logits.copy_(torch.randn(logits.shape, generator=torch.Generator(device=dev).manual_seed(5), device=dev) * 2)
    scores, finished = search.scores.cpu().numpy(), search.finished.cpu().numpy()
    choose()
    check_choice(scores, finished)
    graph = None
    for n in range(steps):
        scores, finished = search.scores.cpu().numpy(), search.finished.cpu().numpy()
        tokens = search.tokens.view(N).long().clone()
        if captured and n == 1:
            torch.cuda.synchronize()
            stream = torch.cuda.Stream(dev)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
        if graph is not None:
            graph.replay()
        else:
            step()
        assert pa.device_error() == 0
        assert search.lens.cpu().tolist() == [len(t) for t in beams_told]
        for l in range(LAYERS):
            q = model.q[l][tokens]
            for b in range(N):
                want, mag = attention(model, l, torch.tensor(beams_told[b], device=dev), q[b])
                tol = 2.0 ** -8 * want.abs() + {0: 2.0 ** -8 + 2.0 ** -11, FP8: 2.0 ** -11 * 42,
                                                FP4: 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -13}[kv] * mag
                assert bool(((outs[l][b].double() - want).abs() <= tol).all()), (n, l, b)
        check_choice(scores, finished)
        if n % 6 == 0 or n == steps - 1:
            assert history[:, :n + 2].cpu().tolist() == [t[len(told[b // K]):] for b, t in enumerate(beams_told)]
    assert int(cursor[0]) <= free.numel()
