"""Beam search over a paged pool: fixed device buffers for the steps of a batch
of requests, a group of beams each.

A step is ``plan`` (a slot for every beam's new token), the model's layers with
``attend`` in place of decode attention (the keys that a request's beams share
are read once), ``select`` (the best continuations over beams and vocabulary)
and ``advance`` (page tables and partly filled pages follow the chosen beams).
Lengths, pages, scores and parents stay on the device and nothing waits for it,
so a whole step can be captured as a CUDA graph and replayed while the lengths
grow.  ``select`` takes ``finished`` along with the beams, as it does ``scores``:
the caller ORs in its own rule for the tokens just chosen, within the step or
between replays.  Between replays it may also look at ``tokens`` and ``parents``
and refill the list of free pages.

Pages stay the caller's.  A request has the pages that its rows and spare pages
named at ``start`` and those that ``plan`` has given its beams since
(``slot_mapping`` // page size where ``positions`` is a multiple of it).  Full
pages of beams that were dropped are among them and named by no row, so all of
them return to the free list when the request ends, and not before.
"""
from __future__ import annotations

import torch

from . import api
from .metadata import BatchPlanner


class BeamSearch:
    """``beams`` beams for each of ``num_groups`` requests over the pools of
    every layer (``k_caches``, ``v_caches``: one tensor per layer).

    Sequence g * beams + i is beam i of request g, and row table_idx[sequence]
    of ``token_table`` (int32 [rows, >= max_seqlen_k]) its slots.  Buffers:
    ``lens`` (keys stored of each sequence), ``prefix_lens`` (keys that a
    request's beams share, whole pages), ``spare_pages`` (page size 16: a page
    of its own for every sequence, which ``advance`` exchanges for the last page
    of a beam that moves), ``scores`` (fp32) and ``finished`` (uint8), both
    [num_groups, beams], ``parents`` and ``tokens`` (int32, of the last
    ``select``).  ``max_prefix`` and ``max_suffix`` bound the keys of a sequence
    in its prefix and behind it."""

    def __init__(self, k_caches, v_caches, token_table: torch.Tensor, table_idx: torch.Tensor, *, num_groups: int, beams: int,
                 num_q_heads: int, head_dim: int, vocab: int, max_seqlen_k: int, max_prefix: int | None = None,
                 max_suffix: int | None = None, page_size: int = 16, spare_pages: torch.Tensor | None = None, pad_token: int = 0,
                 scale: float | None = None, k_scales=None, v_scales=None, kv_dtype: int | None = None):
        self.k_caches, self.v_caches = list(k_caches), list(v_caches)
        layers = len(self.k_caches)
        if not layers or len(self.v_caches) != layers:
            raise ValueError("k_caches and v_caches must hold one pool per layer")
        self.k_scales = [None] * layers if k_scales is None else list(k_scales)
        self.v_scales = [None] * layers if v_scales is None else list(v_scales)
        if len(self.k_scales) != layers or len(self.v_scales) != layers:
            raise ValueError("k_scales and v_scales must hold one tensor per layer")
        self.kv_dtype = api._kv_dtype(self.k_caches[0], self.v_caches[0], kv_dtype)
        self.num_groups, self.beams, self.vocab = int(num_groups), int(beams), int(vocab)
        self.max_seqlen_k, self.page_size, self.pad_token = int(max_seqlen_k), int(page_size), int(pad_token)
        self.scale = scale
        n, dev = self.num_groups * self.beams, token_table.device
        if self.num_groups < 1 or self.beams < 1:
            raise ValueError("num_groups and beams must be positive")
        if table_idx.numel() != n:
            raise ValueError(f"table_idx must hold one entry per sequence ({n})")
        if self.page_size > 1 and spare_pages is None:
            raise ValueError("spare_pages is required for page sizes over 1")
        if self.kv_dtype != api.PA_KV_BF16 and (k_scales is None or v_scales is None):
            raise ValueError("k_scales and v_scales are required for FP8 and 4-bit pools")
        self.token_table, self.table_idx, self.spare_pages = token_table, table_idx, spare_pages
        self.bounds = dict(max_prefix=self.max_seqlen_k if max_prefix is None else int(max_prefix),
                           max_suffix=self.max_seqlen_k if max_suffix is None else int(max_suffix), max_group=self.beams)
        self.lens = torch.zeros(n, dtype=torch.int32, device=dev)
        self.prefix_lens = torch.zeros(n, dtype=torch.int32, device=dev)
        self.scores = torch.zeros((self.num_groups, self.beams), dtype=torch.float32, device=dev)
        self.finished = torch.zeros((self.num_groups, self.beams), dtype=torch.uint8, device=dev)
        self.parents = torch.zeros((self.num_groups, self.beams), dtype=torch.int32, device=dev)
        self.tokens = torch.zeros((self.num_groups, self.beams), dtype=torch.int32, device=dev)
        self.cu_groups = torch.arange(0, n + 1, self.beams, dtype=torch.int32, device=dev)
        self.one = torch.ones(n, dtype=torch.int32, device=dev)
        self.planner = BatchPlanner(dev, n, n, self.max_seqlen_k, self.page_size)
        self.batch = None
        # (the heads of a 4-bit pool are counted by the scales)
        heads = self.k_scales[0].numel() if self.kv_dtype == api.PA_KV_FP4 else self.k_caches[0].shape[-2]
        need = api.decode_shared_workspace_size(
            (n, int(num_q_heads), int(head_dim)), self.k_caches[0], self.max_seqlen_k, self.num_groups, page_size=self.page_size,
            kv_dtype=self.kv_dtype, num_kv_heads=heads, **self.bounds)
        # one workspace: its calls follow one another
        need = max(need, api.beam_select_workspace_size(self.num_groups, self.beams, self.vocab, self.beams))
        self.workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)

    def start(self, prompt_lens: torch.Tensor) -> None:
        """New requests with prompts of ``prompt_lens`` tokens (int32
        [num_groups], on the host or the device), whose K and V are stored
        through the row of beam 0 or will be before ``advance``; every row
        names the prompt's full pages, and of its partly filled last page a page
        of its own.  Beam 0 alone has a score: the first ``select`` takes every
        beam from the prompt's logits in its row."""
        if prompt_lens.numel() != self.num_groups:
            raise ValueError(f"prompt_lens must hold one entry per request ({self.num_groups})")
        per = prompt_lens.to(device=self.lens.device, dtype=torch.int32).repeat_interleave(self.beams)
        self.lens.copy_(per)
        self.prefix_lens.copy_(per // self.page_size * self.page_size)
        self.scores.fill_(float("-inf"))
        self.scores[:, 0] = 0.0
        self.finished.zero_()

    def plan(self, free_pages: torch.Tensor, free_cursor: torch.Tensor):
        """A slot for every beam's new token, new pages from ``free_pages``
        (int32) where the device cursor stands (``BatchPlanner.build``).
        Returns the batch: positions, slot_mapping, page_table."""
        self.batch = self.planner.build(self.lens, self.one, self.token_table, self.table_idx, free_pages=free_pages,
                                        free_cursor=free_cursor)
        self.lens.copy_(self.batch.cache_seqlens)
        return self.batch

    def attend(self, layer: int, q: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of the new tokens, q bf16 [num_groups * beams, Hq, d],
        over ``layer``'s pools (``decode_shared``), after ``plan`` and the
        layer's store."""
        if self.batch is None:
            raise ValueError("attend needs a plan")
        return api.decode_shared(
            q, self.k_caches[layer], self.v_caches[layer], self.batch.page_table, self.batch.cache_seqlens, self.max_seqlen_k,
            self.cu_groups, self.prefix_lens, scale=self.scale, page_size=self.page_size, out=out, workspace=self.workspace,
            k_scale=self.k_scales[layer], v_scale=self.v_scales[layer], kv_dtype=self.kv_dtype, **self.bounds)

    def select(self, logits: torch.Tensor):
        """The best ``beams`` continuations of each request, into ``scores``,
        ``parents`` and ``tokens`` (``beam_select``); a beam's entry of ``finished``
        becomes its parent's."""
        return api.beam_select(logits, self.scores, self.beams, finished=self.finished, pad_token=self.pad_token,
                               out_scores=self.scores, parents=self.parents, tokens=self.tokens, workspace=self.workspace,
                               out_finished=self.finished)

    def advance(self, history: torch.Tensor | None = None) -> None:
        """Sequences become the continuations of their parents, in every
        layer's pools (``beam_reorder``); rows of ``history`` (int32
        [num_groups * beams, T]) follow."""
        api.beam_reorder(self.parents, self.token_table, self.table_idx, self.lens, self.spare_pages, self.k_caches,
                         self.v_caches, page_size=self.page_size, prefix_lens=self.prefix_lens, history=history,
                         max_seqlen_k=self.max_seqlen_k, kv_dtype=self.kv_dtype)
