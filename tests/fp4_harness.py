"""Shared helpers of the 4-bit GPU tests: a workloads.Problem over 4-bit pools,
and the comparison with the fp64 oracle.

Tolerances, from the arithmetic.  With A = the attention over |V| (the
oracle's ``mag``):
  - the output is rounded to bf16 once: half a step, 2^-8 |o| at most;
  - P is rounded to f16: 2^-11 of each weight, so 2^-11 A at most (weights
    below f16's normal range lose 2^-25 of the largest weight: with at most
    2^15 keys, 2^-10 A over all of them even if each lost it one-sided; the
    tests' widest spread of scores keeps that below 2^-13 A);
  - fp32 accumulation, the exponential (2^-22) and score errors: a score is a
    sum of 128 products in fp32, off by at most 128 * 2^-24 sum|q k| scale;
    with sum|q k| scale below 40 that is 3e-4 in the worst case and 2^-16 in
    the mean, relative in p: 2^-12 A covers it;
  - lse: the same score errors, 3e-4.
"""
from __future__ import annotations

import numpy as np
import torch

import workloads as W
from oracle import fp4
from oracle_pins import _meta

TOL_A = 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -13
TOL_LSE = 3e-4


def dev_np(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def random_rows(rng, slots, hkv, d):
    """Rows of random codes, their scales around 2^4 .. 2^7 (values of order
    1 with head scales near 2^-8); the padding random."""
    rows = rng.integers(0, 256, (slots, fp4.layout(hkv, d)[-1]), dtype=np.uint8)
    scales = rng.integers(0x58, 0x70, (slots, hkv, d // 16)).astype(np.uint8)
    codes = rng.integers(0, 16, (slots, hkv, d)).astype(np.uint8)
    return fp4.pack(codes, scales, rows)


class FP4Problem:
    """The Problem p over 4-bit pools on the device: random rows, the poison
    page and the unwritten tail slots all ones (their scales read as NaN), the
    new tokens stored by the 4-bit store on both sides."""

    def __init__(self, p: W.Problem, dev, seed: int):
        import paged_kv_flashattention_gb300 as pa
        from paged_kv_flashattention_gb300 import metadata
        from pa_harness import bf16_dev
        self.p, self.dev = p, dev
        rng = np.random.default_rng(seed)
        hkv, d, P = p.num_kv_heads, p.head_dim, p.page_size
        slots = p.num_pages * P
        self.kr, self.vr = random_rows(rng, slots, hkv, d), random_rows(rng, slots, hkv, d)
        tails = W.tail_slots(p.meta["page_lists"], p.device_len, p.token_table, P)
        for r in (self.kr, self.vr):
            r[(p.num_pages - 1) * P:] = 255
            r[tails] = 255
        self.ks = rng.uniform(0.003, 0.006, hkv).astype(np.float32)
        self.vs = rng.uniform(0.003, 0.006, hkv).astype(np.float32)
        self.q = bf16_dev(p.q, dev)
        self.k_scale, self.v_scale = dev_np(self.ks, dev), dev_np(self.vs, dev)
        self.k_cache = dev_np(self.kr, dev).view(p.num_pages, P, -1)
        self.v_cache = dev_np(self.vr, dev).view(p.num_pages, P, -1)
        pa.store_kv_fp4(bf16_dev(p.k_new, dev), bf16_dev(p.v_new, dev), dev_np(p.slot_mapping, dev), self.k_cache,
                        self.v_cache, self.k_scale, self.v_scale)
        fp4.store(W.bf16_bits_to_f32(p.k_new), p.slot_mapping, self.kr, self.ks)
        fp4.store(W.bf16_bits_to_f32(p.v_new), p.slot_mapping, self.vr, self.vs)
        self.meta = metadata.prepare(p.cached_len, p.extend_len, dev_np(p.token_table, dev),
                                     dev_np(p.table_idx, dev), P)

    def decode(self, **kw):
        import paged_kv_flashattention_gb300 as pa
        m = self.meta
        lse = torch.empty(self.q.shape[:2], dtype=torch.float32, device=self.dev)
        out = pa.decode(self.q, self.k_cache, self.v_cache, m.page_table, m.cache_seqlens, m.max_seqlen_k,
                        scale=self.p.scale, lse=lse, k_scale=self.k_scale, v_scale=self.v_scale,
                        kv_dtype=pa.PA_KV_FP4, **kw)
        return out, lse

    def prefill(self, **kw):
        import paged_kv_flashattention_gb300 as pa
        m = self.meta
        lse = torch.empty((self.p.num_q_heads, max(self.q.shape[0], 1)), dtype=torch.float32, device=self.dev)
        out = pa.prefill(self.q, self.k_cache, self.v_cache, m.page_table, m.cu_seqlens_q, m.cu_seqlens_k,
                         m.max_seqlen_q, m.max_seqlen_k, causal=self.p.causal, scale=self.p.scale, lse=lse,
                         k_scale=self.k_scale, v_scale=self.v_scale, kv_dtype=pa.PA_KV_FP4, **kw)
        return out, lse[:, :self.q.shape[0]].t()

    def oracle(self, **kw):
        p = self.p
        cu_q, cu_k, _, pt = _meta(p)
        return fp4.attention(W.bf16_bits_to_f32(p.q), self.kr, self.vr, pt, cu_q, cu_k, num_kv_heads=p.num_kv_heads,
                             page_size=p.page_size, k_scale=self.ks, v_scale=self.vs, scale=p.scale, causal=p.causal, **kw)


def check(out, lse, ref, what):
    """Device (out, lse [rows, Hq]) against the oracle's (out, lse, mag)."""
    want, want_l, mag = ref
    got = out.detach().float().cpu().numpy().astype(np.float64).reshape(want.shape)
    gl = lse.detach().cpu().numpy().astype(np.float64).reshape(want_l.shape)
    assert np.all(np.isfinite(got)), f"{what}: NaN or Inf in the output"
    over = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + TOL_A * mag + 1e-30)
    worst = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over.max() <= 0, (f"{what}: {np.count_nonzero(over > 0)} of {over.size} outputs off, worst at "
                                               f"{worst}: {got[worst]!r}, expected {want[worst]!r} (mag {mag[worst]!r})")
    empty = np.isneginf(want_l)
    assert np.array_equal(np.isneginf(gl), empty), f"{what}: lse of empty rows"
    if not empty.all():
        err = np.abs(gl[~empty] - want_l[~empty]).max()
        assert err <= TOL_LSE, f"{what}: lse off by {err:.3g}"
    assert not got[empty].any(), f"{what}: empty rows must be zero"
