"""Calls of the paged INT4 KV cache's operators that its documentation allows, beside the usual
ones: optional outputs left out, wide tables and rows, views of larger pools, the longest caches."""
import ctypes as ct

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as ko
from w4a4_mixed_precision_b200 import atom

from kv4_util import Call, assert_within, dev, host

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(autouse=True)
def clean_status():
    atom.atom_device_status(clear=True)
    yield
    assert atom.atom_device_status(clear=True) == 0


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("new,heads", [([1, 3, 0], 2), ([150] * 10, 5)])
def test_attention_without_lse_and_with_an_unaligned_workspace(new, heads):
    c = Call(95, new, [200 + i for i in range(len(new))], q_heads=2 * heads, heads=heads, page=16,
             q_size=0.05)
    cache, batch, q = c.device_cache(), c.device_batch(), dev(c.q)
    want = ko.attention(c.q, c.cache, *c.sequences(), True, SCALE)
    out = torch.empty_like(q)
    status = atom.lib().atom_kv4_attention(
        q.data_ptr(), q.stride(0), 128, c.rows, 2 * heads, cache._ref, batch._ref, 1,
        ct.c_float(SCALE), out.data_ptr(), None, None, 0, stream())
    assert status == 0
    assert_within(host(out), want[0], want[1], "out")
    n = atom.atom_kv4_attention_workspace_bytes(c.rows, 2 * heads, heads, c.rows)
    ws = torch.zeros(n + 16, dtype=torch.uint8, device="cuda")[1:]
    got = atom.atom_kv4_attention(q, cache, batch, workspace=ws)      # not shared, as with none
    assert_within(host(got[0]), want[0], want[1], "out")
    assert_within(host(got[1]), want[2], want[3], "lse")


@pytest.mark.parametrize("new,heads", [([1, 3, 0], 2), ([150] * 10, 5)])
def test_wide_tables_rows_and_pools(new, heads):
    """Block tables that are columns of a wider one, caches that are a layer of a pool of several,
    sums wider than the table, a batch whose bound on new tokens is far above them."""
    c = Call(96, new, [200 + i for i in range(len(new))], q_heads=2 * heads, heads=heads, page=24,
             q_size=0.05, garbage=1.0)
    pool = [torch.from_numpy(np.stack([a, np.zeros_like(a), a], 1)).cuda() for a in c.cache]
    cache = atom.KV4Cache(*(t[:, 2] for t in pool))                   # [pages, layers, ...]
    table = torch.full((len(new), c.table.shape[1] + 7), 2 ** 30, dtype=torch.int32, device="cuda")
    table[:, 3:3 + c.table.shape[1]] = dev(c.table)
    batch = atom.KV4Batch(table[:, 3:3 + c.table.shape[1]], dev(c.lens), dev(c.cu_q), max_q=2 ** 31 - 1)
    atom.atom_kv4_append(dev(c.k), dev(c.v), cache, batch)
    ref = [a.copy() for a in c.cache]
    ko.append(c.k, c.v, ref, *c.sequences())
    for t, a, first in zip(pool, ref, c.cache):
        assert np.array_equal(host(t[:, 2]), a)
        assert np.array_equal(host(t[:, 0]), first) and not bool(t[:, 1].any())
    q = dev(c.q)
    out, lse = atom.atom_kv4_attention(q, cache, batch)
    want = ko.attention(c.q, ref, *c.sequences(), True, SCALE)
    assert_within(host(out), want[0], want[1], "out")
    assert_within(host(lse), want[2], want[3], "lse")
    width = c.table.shape[1] * 24 + 1000
    sums = torch.full((len(new), heads, width), 7.0, device="cuda")
    atom.atom_kv4_attention_weights(q, lse, cache, batch, sums)
    s, tol = ko.attention_weights(c.q, host(lse), ref, *c.sequences(), True, SCALE, width)
    inside = np.broadcast_to(np.arange(width)[None, None] < c.lens[:, None, None], s.shape)
    assert_within(host(sums)[inside], s[inside], tol[inside], "sums")
    assert (host(sums)[~inside] == 7).all()
    # evicted into another layer of the pool, new weights wider than the budget
    dst = atom.KV4Cache(*(t[:, 1] for t in pool))
    kept_ref, lens_ref = ko.evict(host(sums), c.lens, 50, 9)
    new_lens = torch.empty(len(new), dtype=torch.int32, device="cuda")
    new_w = torch.full((len(new), heads, 60), 7.0, device="cuda")
    kept, _ = atom.atom_kv4_evict(sums, cache, batch, 50, 9, dst, batch.block_table, new_lens,
                                  new_weights=new_w)
    assert np.array_equal(host(kept), kept_ref) and np.array_equal(host(new_lens), lens_ref)
    to = np.arange(50)
    for b in range(len(new)):
        for h in range(heads):
            at = kept_ref[b, h]
            for t, a in zip(pool, ref):
                assert np.array_equal(host(t[:, 1])[c.table[b, to // 24], to % 24, h],
                                      a[c.table[b, at // 24], at % 24, h])
            assert np.array_equal(host(new_w)[b, h, :50], host(sums)[b, h, at])
    assert bool((new_w[..., 50:] == 7).all())
    for t, a in zip(pool, ref):
        assert np.array_equal(host(t[:, 2]), a)


def test_evict_without_new_weights_and_rows_for_no_sequence():
    c = Call(97, [0, 0], [90, 40], q_heads=3, heads=3, page=16, pad_rows=5)
    cache, batch = c.device_cache(), c.device_batch()
    w = np.random.default_rng(2).random((2, 3, 95)).astype(np.float32)
    kept_ref, lens_ref = ko.evict(w, c.lens, 33, 4)
    new_lens, weights = torch.empty(2, dtype=torch.int32, device="cuda"), dev(w)
    kept = torch.empty((2, 3, 33), dtype=torch.int32, device="cuda")
    table = batch.block_table
    status = atom.lib().atom_kv4_evict(
        weights.data_ptr(), 95, cache._ref, batch._ref, 33, 4, cache._ref, table.data_ptr(),
        table.stride(0), table.shape[1], new_lens.data_ptr(), kept.data_ptr(), None, 0, stream())
    assert status == 0
    assert np.array_equal(host(kept), kept_ref) and np.array_equal(host(new_lens), lens_ref)
    # rows, and a bound that says that no sequence has any: nothing is written
    assert batch.max_q == 0
    out = torch.full((5, 6, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((5, 6), 7.0, device="cuda")
    atom.atom_kv4_attention(torch.zeros_like(out), cache, batch, out=out, lse=lse)
    assert bool((out == 7).all()) and bool((lse == 7).all())
    k = torch.full((5, 3, 128), 7.0, dtype=torch.float16, device="cuda")
    before = [t.clone() for t in (cache.k4, cache.v4)]
    atom.atom_kv4_append(k, k, cache, batch)
    atom.atom_kv4_gather(cache, batch, 5, k, k.clone())
    assert bool((k == 7).all())
    assert torch.equal(before[0], cache.k4) and torch.equal(before[1], cache.v4)


@pytest.mark.parametrize("length", [2 ** 30, 2 ** 30 - 77])
def test_the_longest_cache(length):
    """A token behind up to 2^30 cached ones: one page of 2^17 tokens, listed again and again."""
    if torch.cuda.mem_get_info()[0] < 24 * 2 ** 30:
        pytest.skip("needs 24 GB")
    page = 2 ** 17
    pages = -(-length // page)
    c = Call(98, [1], [page], q_heads=2, heads=1, page=page, q_size=0.05, spare_pages=0)
    table = torch.full((1, pages), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    cache = c.device_cache()
    batch = atom.KV4Batch(table, dev(np.array([length], np.int32)), dev(c.cu_q), max_q=1)
    q = dev(c.q)
    out, lse = atom.atom_kv4_attention(q, cache, batch)
    # whole pages, and the last one's part
    rest = np.array([length - (pages - 1) * page], np.int32)
    want = [ko.attention(c.q, c.cache, c.table, n, c.cu_q, False, SCALE) for n in (c.lens, rest)]
    z = [w[2] + n for w, n in zip(want, (np.log(max(pages - 1, 1)), 0.0))]
    total = np.logaddexp(*z)
    share = np.exp(z[0] - total)[..., None]
    ref = want[0][0] * share + want[1][0] * (1 - share)
    assert np.abs(host(lse) - total).max() <= max(w[3].max() for w in want) + 2.0 ** -18
    assert (np.abs(host(out) - ref) <= want[0][1] + want[1][1] + np.abs(ref) * 2.0 ** -11).all()
    sums = torch.full((1, 1, length + 3), 7.0, device="cuda")
    atom.atom_kv4_attention_weights(q, lse, cache, batch, sums)
    s, tol = ko.attention_weights(c.q, host(lse), c.cache, *c.sequences(), False, SCALE, page)
    got = sums[0, 0, :page]
    assert_within(host(got), s[0, 0], tol[0, 0], "sums")
    whole = sums[0, 0, :(pages - 1) * page].view(-1, page)
    assert bool((whole == got).all())
    assert torch.equal(sums[0, 0, (pages - 1) * page:length], got[:int(rest[0])])
    assert bool((sums[0, 0, length:] == 7).all())
