"""Append and gather with any number of KV heads: rows whose vectors fill a warp's 16 slots and
those that share them with the rows around."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as ko
from w4a4_mixed_precision_b200 import atom

from kv4_util import Call, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    atom.atom_device_status(clear=True)
    yield
    assert atom.atom_device_status(clear=True) == 0


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("heads", [1, 2, 3, 4, 5, 6, 7, 9, 12, 16, 17])
@pytest.mark.parametrize("new,lens,pad", [
    ([1], [1], 0), ([1], [9], 3), ([1] * 7, [5, 1, 80, 33, 17, 16, 2], 1),
    ([0, 3, 0, 0, 11, 0], [4, 30, 0, 9, 11, 70], 5), ([67, 1, 130], [70, 1, 200], 0),
    ([0], [20], 4),
])
def test_any_number_of_heads(new, lens, pad, heads, token_major):
    c = Call(91, new, lens, heads=heads, q_heads=heads, page=16, token_major=token_major,
             pad_rows=pad, garbage=2.0)
    n = int(c.cu_q[-1])
    cache, batch = c.device_cache(), c.device_batch()
    atom.atom_kv4_append(dev(c.k), dev(c.v), cache, batch)
    want = [a.copy() for a in c.cache]
    ko.append(c.k, c.v, want, *c.sequences())
    for got, ref in zip((cache.k4, cache.ks, cache.v4, cache.vs), want):
        assert np.array_equal(host(got), ref)
    k, v = (torch.full((c.rows, heads, 128), 7.0, dtype=torch.float16, device="cuda")
            for _ in range(2))
    atom.atom_kv4_gather(cache, batch, c.rows, k, v)
    for got, ref in zip((k, v), ko.gather(want, *c.sequences(), c.rows)):
        assert np.array_equal(host(got)[:n].view(np.uint16), ref[:n].view(np.uint16))
        assert (host(got)[n:] == 7).all()


@pytest.mark.parametrize("heads", [1, 3, 8, 12])
def test_rows_without_a_slot_leave_their_neighbours_alone(heads):
    """A sequence that contradicts the call, one with a page outside the pool and a pool without
    pages: nothing of theirs is written, the rows that share a warp with theirs are."""
    c = Call(92, [3, 2, 5, 4], [20, 30, 40, 50], heads=heads, q_heads=heads, page=16, garbage=2.0)
    lens, table = c.lens.copy(), c.table.copy()
    lens[1] = -1
    table[2, 2] = len(c.cache[0])            # positions 32 .. 39 of sequence 2, its new tokens
    cache = c.device_cache()
    batch = atom.KV4Batch(dev(table), dev(lens), dev(c.cu_q), max_q=5)
    atom.atom_kv4_append(dev(c.k), dev(c.v), cache, batch)
    assert atom.atom_device_status(clear=True) == 1
    keep = np.r_[0:3, 10:14]
    at = (table[[0, 3]], lens[[0, 3]], np.array([0, 3, 7], np.int32))
    want = [a.copy() for a in c.cache]
    ko.append(c.k[keep], c.v[keep], want, *at)
    for got, ref in zip((cache.k4, cache.ks, cache.v4, cache.vs), want):
        assert np.array_equal(host(got), ref)
    k, v = (torch.full((c.rows, heads, 128), 7.0, dtype=torch.float16, device="cuda")
            for _ in range(2))
    atom.atom_kv4_gather(cache, batch, c.rows, k, v)
    assert atom.atom_device_status(clear=True) == 1
    for got, ref in zip((k, v), ko.gather(want, *at, len(keep))):
        assert np.array_equal(host(got)[keep].view(np.uint16), ref.view(np.uint16))
        assert (host(got)[3:10] == 7).all()
    none = atom.KV4Cache(cache.k4, cache.ks, cache.v4, cache.vs)
    none.struct.pages = 0
    before = [t.clone() for t in (cache.k4, cache.ks, k, v)]
    atom.atom_kv4_append(dev(c.k), dev(c.v), none, batch)
    atom.atom_kv4_gather(none, batch, c.rows, k, v)
    assert atom.atom_device_status(clear=True) == 1
    for t, b in zip((cache.k4, cache.ks, k, v), before):
        assert torch.equal(t, b)


@pytest.mark.parametrize("op", ["append", "gather"])
def test_few_heads_cost_what_their_bytes_cost(op):
    """The same bytes as rows of 1 and of 8 KV heads: within three times the time (1.3 measured;
    with a row's 16 slots 14 of them empty, 6)."""
    def time(heads, rows=2 ** 17):
        rows = rows // heads
        cache = atom.empty_kv4_cache(rows // 64, 64, heads, "cuda")
        batch = atom.KV4Batch(torch.arange(rows // 64, dtype=torch.int32, device="cuda")[None],
                              dev(np.array([rows], np.int32)), dev(np.array([0, rows], np.int32)))
        k = torch.randn((rows, heads, 128), device="cuda").half()
        v, out = k.clone(), (k.clone(), k.clone())
        took = []
        for _ in range(10):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda._sleep(100_000)       # the events and calls are queued behind this
            start.record()
            for _ in range(4):
                if op == "append":
                    atom.atom_kv4_append(k, v, cache, batch)
                else:
                    atom.atom_kv4_gather(cache, batch, rows, *out)
            end.record()
            end.synchronize()
            took.append(start.elapsed_time(end))
        return sorted(took)[len(took) // 2]

    assert time(1) < 3 * time(8)
