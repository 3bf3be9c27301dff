"""Building paged caches and ragged batches for the serving tests."""
import numpy as np

import oracle
from helpers import torch_dev


def rand16(g, *shape):
    return g.standard_normal(shape).astype(np.float16)


class Batch:
    """A paged cache with `ctx` cached positions and `n` new rows per sequence.

    Pages are dealt in random order; `spare` pages belong to nobody.  Rows
    that hold no position are NaN, so that a read of one shows."""

    def __init__(self, g, ctx, n, Hkv, d, page, spare=2, layers=1):
        self.ctx, self.n, self.Hkv, self.d, self.page = list(ctx), list(n), Hkv, d, page
        self.S, self.rows = len(ctx), sum(n)
        per = [-(-(c + k) // page) for c, k in zip(ctx, n)]
        self.n_pages, self.max_pages = sum(per) + spare, max(1, max(per))
        order = g.permutation(self.n_pages)
        self.table = np.full((self.S, self.max_pages), -1, np.int32)  # unused places hold no page
        at = 0
        for i, p in enumerate(per):
            self.table[i, :p] = order[at:at + p]
            at += p
        self.start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        shape = (layers, self.n_pages, Hkv, page, d)
        self.k, self.v = np.full(shape, np.nan, np.float16), np.full(shape, np.nan, np.float16)
        for i in range(self.S):
            pos = np.arange(ctx[i] + n[i])
            for pool in (self.k, self.v):
                pool[:, self.table[i][pos // page], :, pos % page] = rand16(g, len(pos), layers, Hkv, d)

    def rows_of(self, pool, s, positions):
        return oracle.paged_rows(pool, self.table[s], positions)

    def to_device(self, q4):
        self.dk, self.dv, self.dtable = torch_dev(self.k), torch_dev(self.v), torch_dev(self.table)
        self.dctx, self.dstart = torch_dev(np.array(self.ctx, np.int32)), torch_dev(self.start)
        return q4.PagedCache(self.dk, self.dv, self.n_pages, self.page, self.Hkv, self.d, self.dtable, self.S,
                             self.max_pages)


def mask_words(rows, words):
    """bool rows [T][<= 32 words] -> uint32 [T][words]."""
    out = np.zeros((len(rows), words), np.uint32)
    for i, r in enumerate(rows):
        for j in np.flatnonzero(r):
            out[i, j // 32] |= np.uint32(1 << int(j) % 32)
    return out


def random_tree(g, n, fan=4):
    return [-1] + [int(g.integers(max(0, i - 1 - fan * 3), i)) for i in range(1, n)]
