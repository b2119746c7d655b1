"""Paged caches and calls for the KV-cache tests: numpy arrays for the oracle, and the same
values as tensors for the library."""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv_oracle
from w4a4_mixed_precision_b200 import atom, inputs


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


class Call:
    """`new[b]` new tokens (queries) and `lens[b]` cached tokens of each sequence, in a pool of
    shuffled pages; `garbage` fills the scales of slots that no sequence has."""

    def __init__(self, seed, new, lens, q_heads=8, heads=2, page=16, token_major=False,
                 pad_rows=0, spare_pages=2, garbage=np.nan, q_size=1.5):
        rng = np.random.default_rng(seed)
        self.new, self.lens = np.asarray(new, np.int32), np.asarray(lens, np.int32)
        self.q_heads, self.heads, self.page, self.token_major = q_heads, heads, page, token_major
        need = -(-self.lens // page)
        pages = int(need.sum()) + spare_pages
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(1, int(need.max(initial=0)))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu_q = starts(self.new)
        self.rows = int(self.cu_q[-1]) + pad_rows
        self.cache = []
        for i in range(2):
            x = inputs.kv_cache(seed * 2 + i + 1, pages * page, heads).reshape(pages, page, heads, 128)
            self.cache += kv_oracle.quantize(x)
        if garbage is not None:
            used = np.zeros((pages, page), bool)
            for b, n in enumerate(self.lens):
                p = np.arange(n)
                used[self.table[b, p // page], p % page] = True
            for i in (1, 3):
                self.cache[i][~used] = garbage
        # keys differ in size over decades: queries small enough that the scores stay moderate
        self.q = (rng.standard_normal((self.rows, q_heads, 128)) * q_size).astype(np.float16)
        self.k = inputs.kv_cache(seed + 77, self.rows, heads)
        self.v = inputs.kv_cache(seed + 78, self.rows, heads)

    def sequences(self):
        return self.table, self.lens, self.cu_q

    def device_cache(self, arrays=None):
        out = []
        for a in arrays or self.cache:
            t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
            if not self.token_major:
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            out.append(t)
        return atom.KV4Cache(*out)

    def device_batch(self, max_q="exact"):
        if max_q == "exact":
            max_q = int(self.new.max(initial=0))
        return atom.KV4Batch(dev(self.table), dev(self.lens), dev(self.cu_q), max_q=max_q)


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.float16:
        return torch.from_numpy(a.view(np.int16)).cuda().view(torch.float16)
    return torch.from_numpy(a).cuda()


def host(t):
    torch.cuda.synchronize()
    t = t.detach().cpu()
    if t.dtype == torch.float16:
        return t.contiguous().view(torch.int16).numpy().view(np.float16)
    return t.numpy()


def assert_within(got, want, tol, what=""):
    got = np.asarray(got, np.float64)
    same = np.isinf(want)
    assert np.array_equal(got[same], want[same]), f"{what}: infinities differ"
    with np.errstate(invalid="ignore"):
        off = np.abs(got[~same] - want[~same]) - tol[~same]
    bad = ~(off <= 0) & ~(np.isinf(tol[~same]) & ~np.isnan(got[~same]))
    if bad.any():
        i = int(np.argmax(np.where(np.isnan(off), np.inf, off)))
        raise AssertionError(
            f"{what}: {bad.sum()} of {bad.size} out of tolerance, worst {got[~same][i]} against "
            f"{want[~same][i]} (tolerance {tol[~same][i]})")
