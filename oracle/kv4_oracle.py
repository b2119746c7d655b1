"""Paged INT4 KV cache in numpy, 64 bits -- TEST INFRASTRUCTURE ONLY (the GPU path never uses it).

A cache is its four arrays k4 [pages, page_size, heads, 64], ks [pages, page_size, heads], v4,
vs (any strides); a call's sequences are (block_table, kv_lens, cu_q) as the library takes them.
Beside its values the attention returns bounds on what fp32 arithmetic may change, computed from
the same inputs, so that tests need no guessed tolerance.
"""
from __future__ import annotations

import numpy as np

from . import kv_oracle

HEAD_DIM = 128


def _slots(table, page_size, b, positions):
    return table[b, positions // page_size], positions % page_size


def append(k, v, cache, table, kv_lens, cu_q):
    """Writes fp16 k, v [rows, heads, 128] into the cache's arrays, in place."""
    k4, ks, v4, vs = cache
    for b, length in enumerate(kv_lens):
        rows = np.arange(cu_q[b], cu_q[b + 1])
        page, slot = _slots(table, k4.shape[1], b, length - len(rows) + np.arange(len(rows)))
        for x, q4, s in ((k, k4, ks), (v, v4, vs)):
            q4[page, slot], s[page, slot] = kv_oracle.quantize(x[rows])


def sequence(q4, scales, table, b, length):
    """(codes, scales) of one sequence in 64 bits: [length, heads, 128] and [length, heads]."""
    page, slot = _slots(table, q4.shape[1], b, np.arange(length))
    return kv_oracle.codes(q4[page, slot]).astype(np.float64), scales[page, slot].astype(np.float64)


def gather(cache, table, kv_lens, cu_q, rows):
    """fp16 (k, v) [rows, heads, 128]; rows without a sequence are zero."""
    out = []
    for q4, s in ((cache[0], cache[1]), (cache[2], cache[3])):
        x = np.zeros((rows,) + q4.shape[2:3] + (HEAD_DIM,), np.float16)
        for b, length in enumerate(kv_lens):
            n = cu_q[b + 1] - cu_q[b]
            page, slot = _slots(table, q4.shape[1], b, np.arange(length - n, length))
            x[cu_q[b]:cu_q[b + 1]] = kv_oracle.dequantize(q4[page, slot], s[page, slot])
        out.append(x)
    return out


def scores(q, codes, scales, scale):
    """Scores [n, length] of queries q [n, 128], and what fp32 may add to each.

    A product of 128 terms is summed by the matrix instructions in fp32, 16 terms at a time and at
    worst truncated: 128 terms stay within 2^-20 of the sum of their sizes. The scale of the token
    and of the call, their product and the score's own product are rounded once each: 2^-22."""
    s = scale * (q @ codes.T) * scales
    size = abs(scale) * (np.abs(q) @ np.abs(codes).T) * scales
    return s, size * 2.0 ** -20 + np.abs(s) * 2.0 ** -22


def limits(n, length, causal):
    if not causal:
        return np.full(n, length)
    return np.maximum(0, length - n + 1 + np.arange(n))


def attention(q, cache, table, kv_lens, cu_q, causal, scale):
    """(out, out bound, lse, lse bound) in 64 bits, rows [cu_q[0], cu_q[-1]).

    out's bound: half a step of fp16 (2^-11 of the value, 2^-25 near zero), and of the sum of
    p |v| as much as the weights may be off: a score's error e makes 2e of weight and total, an
    exponential 2^-21, a weight p vs rounded to fp16 2^-11, sums of n terms made 16 at a time and
    over four or more partial sums (n / 16 + 64) 2^-24. A weight below fp16's normal range is off
    by half its smallest step, 2^-25, in units in which 2^4 stands for the largest, over the 64
    tokens that share them and those before, of what the row sees: its largest weight there times
    the power of two above the largest value scale there. Of the row's n codes of at most 7 that is
    at most n * 7 * 2^-29 * 2 max(p vs)."""
    k4, ks, v4, vs = cache
    rows, hq = q.shape[:2]
    group = hq // k4.shape[2]
    q = q.astype(np.float64)
    out, lse = np.zeros((rows, hq, HEAD_DIM)), np.full((rows, hq), -np.inf)
    out_tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
    for b, length in enumerate(kv_lens):
        mine = slice(cu_q[b], cu_q[b + 1])
        n = cu_q[b + 1] - cu_q[b]
        if n == 0 or length == 0:
            continue
        kc, ksc = sequence(k4, ks, table, b, length)
        vc, vsc = sequence(v4, vs, table, b, length)
        seen = np.arange(length)[None] < limits(n, length, causal)[:, None]
        for head in range(hq):
            h = head // group
            s, err = scores(q[mine, head], kc[:, h], ksc[:, h], scale)
            s = np.where(seen, s, -np.inf)
            top = s.max(-1, keepdims=True, initial=-1e300)
            p = np.exp(s - top)
            total = p.sum(-1, keepdims=True)
            some = total[:, 0] > 0
            p = p / np.where(some[:, None], total, 1)
            v = vc[:, h] * vsc[:, h, None]
            out[mine, head] = p @ v
            e = np.where(seen, err, 0).max(-1)
            off = 2 * e + 2.0 ** -21 + 2.0 ** -11 + (length / 16 + 64) * 2.0 ** -24
            groups = np.arange(0, length, 64)
            largest = (np.maximum.reduceat(p, groups, -1) *
                       np.maximum.reduceat(np.where(seen, vsc[:, h], 0), groups, -1)).max(-1)
            floor = seen.sum(-1) * 7 * 2.0 ** -28 * largest
            out_tol[mine, head] = (np.abs(out[mine, head]) * 2.0 ** -11 + 2.0 ** -25 +
                                   floor[:, None] + off[:, None] * (p @ np.abs(v)))
            lse[mine, head] = np.where(some, top[:, 0] + np.log(np.where(some, total[:, 0], 1)),
                                       -np.inf)
            lse_tol[mine, head] = np.where(
                some, e + 2.0 ** -20 + (length / 16 + 64) * 2.0 ** -24 +
                np.abs(np.where(some, lse[mine, head], 0)) * 2.0 ** -21, 0)
    # out is fp16: a sum from 65520 on (half a step above the largest number) rounds to infinity;
    # one so near it that its bound spans both may be either
    over, near = np.abs(out) - 65520 >= out_tol, np.abs(np.abs(out) - 65520) < out_tol
    out[over] = np.copysign(np.inf, out[over])
    out_tol[near] = np.inf
    return out, out_tol, lse, lse_tol


def attention_weights(q, lse, cache, table, kv_lens, cu_q, causal, scale, width):
    """(sums, bound) [batch, heads, width]; elements behind a sequence's length are zero.

    lse (fp32) is an input. A weight is off by its score's error, by the rounding of
    log2(e) * (score - lse) and by the exponential; sums of sums of 64 add 2^-18 at most."""
    k4, ks = cache[:2]
    hq, heads = q.shape[1], k4.shape[2]
    group = hq // heads
    q = q.astype(np.float64)
    sums = np.zeros((len(kv_lens), heads, width))
    tol = np.zeros_like(sums)
    for b, length in enumerate(kv_lens):
        mine = slice(cu_q[b], cu_q[b + 1])
        n = cu_q[b + 1] - cu_q[b]
        if n == 0 or length == 0:
            continue
        kc, ksc = sequence(k4, ks, table, b, length)
        seen = np.arange(length)[None] < limits(n, length, causal)[:, None]
        for head in range(hq):
            h = head // group
            s, err = scores(q[mine, head], kc[:, h], ksc[:, h], scale)
            z = lse[mine, head].astype(np.float64)[:, None]
            some = seen & (z > -np.inf)
            z = np.where(z > -np.inf, z, 0)
            p = np.where(some, np.exp(np.where(some, s - z, 0)), 0)
            sums[b, h, :length] += p.sum(0)
            off = 2 * err + (np.abs(s) + np.abs(z)) * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -18
            tol[b, h, :length] += (p * off).sum(0)
    return sums, tol


def evict(weights, kv_lens, budget, recent):
    """(kept [batch, heads, budget], new_lens): positions that stay, in order, then -1."""
    batch, heads = weights.shape[:2]
    kept = np.full((batch, heads, budget), -1, np.int32)
    new_lens = np.minimum(kv_lens, budget).astype(np.int32)
    for b, length in enumerate(kv_lens):
        n = new_lens[b]
        last = min(recent, n)
        for h in range(heads):
            w = weights[b, h, :length - last].astype(np.float64)
            # by weight, NaN last, then by position
            order = sorted(range(len(w)), key=lambda i: (np.isnan(w[i]), -w[i] if w[i] == w[i] else 0,
                                                         i))
            stay = sorted(order[:n - last]) + list(range(length - last, length))
            kept[b, h, :n] = stay
    return kept, new_lens
