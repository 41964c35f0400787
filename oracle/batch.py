"""Oracle of the batch plan (plain Python loops over requests and tokens).
TEST INFRASTRUCTURE ONLY: written from the definition in ``include/pa.h``."""
from __future__ import annotations

import numpy as np


def build(cached, extend, token_table, table_idx, page_size, max_seqlen_k, num_tokens, page_table, free_pages=None):
    """Returns a dict of the outputs; token_table and page_table are copied and
    returned with what the call writes.  ``error``: the names raised."""
    P = page_size
    tt, pt = token_table.copy(), page_table.copy()
    B = len(cached)
    err = set()
    cq, ck, lens = [0], [0], []
    pos, slot = np.zeros(num_tokens, np.int32), np.full(num_tokens, -1, np.int32)
    taken, most_q, most_k = 0, 0, 0
    for b in range(B):
        c, e, r = int(cached[b]), int(extend[b]), int(table_idx[b])
        if c < 0 or e < 0 or c + e > max_seqlen_k:
            err.add("SEQLENS")
            c = e = 0
        known = 0 <= r < tt.shape[0]
        if not known:
            err.add("TABLE_INDEX")
        held = -(-c // P)
        pages = []
        for col in range(-(-(c + e) // P)):
            if not known:
                pages.append(-1)
            elif free_pages is not None and col >= held:
                if taken < len(free_pages):
                    pages.append(int(free_pages[taken]))
                else:
                    err.add("NO_PAGES")
                    pages.append(-1)
                taken += 1
            else:
                pages.append(int(tt[r, col * P]) // P)
        for i in range(e):
            p, t = c + i, cq[-1] + i
            if not known:
                s = -1
            elif free_pages is None:
                s = int(tt[r, p])
            else:
                page = pages[p // P] if p // P >= held else int(tt[r, c - 1]) // P
                s = page * P + p % P if page >= 0 else -1
            if t < num_tokens:
                pos[t], slot[t] = p, s
                if known and free_pages is not None:
                    tt[r, p] = s
        pt[b, :len(pages)] = pages
        cq.append(cq[-1] + e)
        ck.append(ck[-1] + c + e)
        lens.append(c + e)
        most_q, most_k = max(most_q, e), max(most_k, c + e)
    if cq[-1] > num_tokens:
        err.add("SEQLENS")
    return dict(cu_seqlens_q=cq, cu_seqlens_k=ck, cache_seqlens=lens, positions=pos, slot_mapping=slot, page_table=pt,
                token_table=tt, totals=[cq[-1], most_q, most_k, taken], error=err)
