"""The paged INT4 KV cache's operators on the GPU beside what they must not see: padding and idle
rows, rows that count for nothing, cached tokens behind a row's own."""
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


def check_weights(c, q, lse, causal=True, prev=None, lse_ref=None):
    """The sums of queries `q` against the oracle's of c.q, and the elements behind the lengths."""
    width = int(c.lens.max()) + 3
    shape = (len(c.lens), c.heads, width)
    sums = torch.full(shape, 7.0, device="cuda")
    atom.atom_kv4_attention_weights(q, lse, c.device_cache(), c.device_batch(), sums, causal=causal)
    want, tol = ko.attention_weights(c.q, host(lse) if lse_ref is None else lse_ref, c.cache,
                                     *c.sequences(), causal, SCALE, width)
    inside = np.broadcast_to(np.arange(width)[None, None] < c.lens[:, None, None], shape)
    assert_within(host(sums)[inside], want[inside], tol[inside], "sums")
    assert (host(sums)[~inside] == 7).all()
    return sums


@pytest.mark.parametrize("fill", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,q_heads,heads", [
    ([1, 3], [40, 90], 8, 2),
    ([1, 1, 2, 1], [200, 0, 77, 0], 8, 8),
    ([200], [700], 16, 2),
    ([9], [9], 7, 1),
    ([150, 1, 40, 1, 133], [150, 0, 300, 0, 500], 10, 5),
    ([150, 7, 20] * 4, [400, 7, 300] * 4, 35, 5),
])
def test_what_padding_and_idle_rows_hold_counts_for_nothing(new, lens, q_heads, heads, causal, fill):
    """Query, key and value rows behind the last sequence, and the query of a slot with nothing
    cached, hold NaN or infinities."""
    c = Call(81, new, lens, q_heads=q_heads, heads=heads, page=16, pad_rows=150, q_size=0.05,
             garbage=1.0)
    n = int(c.cu_q[-1])
    idle = np.zeros(c.rows, bool)
    for b in np.flatnonzero(c.lens == 0):
        idle[c.cu_q[b]:c.cu_q[b + 1]] = True
    nothing = idle | (np.arange(c.rows) >= n)
    q, k, v = (x.copy() for x in (c.q, c.k, c.v))
    for x in (q, k, v):
        x[nothing] = fill
    cache, batch = c.device_cache(), c.device_batch()
    if not idle.any():
        atom.atom_kv4_append(dev(k), dev(v), cache, batch)
        ko.append(c.k, c.v, c.cache, *c.sequences())
        for got, ref in zip((cache.k4, cache.ks, cache.v4, cache.vs), c.cache):
            assert np.array_equal(host(got), ref)
        back = [torch.full((c.rows, heads, 128), 7.0, dtype=torch.float16, device="cuda")
                for _ in range(2)]
        atom.atom_kv4_gather(cache, batch, c.rows, *back)
        for got, ref in zip(back, ko.gather(c.cache, *c.sequences(), c.rows)):
            assert np.array_equal(host(got)[:n], ref[:n]) and (host(got)[n:] == 7).all()
    out = torch.full((c.rows, q_heads, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((c.rows, q_heads), 7.0, device="cuda")
    atom.atom_kv4_attention(dev(q), cache, batch, causal=causal, out=out, lse=lse)
    want = ko.attention(c.q, c.cache, *c.sequences(), causal, SCALE)
    assert_within(host(out)[:n], want[0][:n], want[1][:n], "out")
    assert_within(host(lse)[:n], want[2][:n], want[3][:n], "lse")
    assert (host(out)[n:] == 7).all() and (host(lse)[n:] == 7).all()
    sums = check_weights(c, dev(q), lse, causal)
    # by sums that such rows have no part in the same tokens stay
    budget = max(1, int(c.lens.max()) // 2)
    kept_ref, lens_ref = ko.evict(host(sums), c.lens, budget, 3 if budget > 3 else 0)
    new_lens = torch.empty(len(new), dtype=torch.int32, device="cuda")
    kept, _ = atom.atom_kv4_evict(sums, cache, batch, budget, 3 if budget > 3 else 0, cache,
                                  batch.block_table, new_lens)
    assert np.array_equal(host(kept), kept_ref) and np.array_equal(host(new_lens), lens_ref)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,q_heads,heads", [
    ([1, 6], [40, 90], 4, 4), ([9, 5], [60, 400], 12, 2), ([300], [700], 16, 2),
    ([150, 30, 128], [150, 300, 500], 10, 5),
])
def test_rows_without_a_log_sum_exp_count_for_nothing(new, lens, q_heads, heads, causal):
    """A row whose lse is -infinity adds nothing, whatever its query holds."""
    c = Call(82, new, lens, q_heads=q_heads, heads=heads, page=24, q_size=0.05)
    _, lse = atom.atom_kv4_attention(dev(c.q), c.device_cache(), c.device_batch(), causal=causal)
    rng = np.random.default_rng(4)
    silent = rng.random((c.rows, q_heads)) < 0.2
    silent[-1, -1] = True
    z, q = host(lse).copy(), c.q.copy()
    z[silent] = -np.inf
    q[silent] = np.where(rng.random((int(silent.sum()), 1)) < 0.5, np.nan, np.inf)
    check_weights(c, dev(q), dev(z), causal)


@pytest.mark.parametrize("new,group", [(2, 128), (1, 100)])
def test_weights_of_a_prefix_beyond_2_to_31_query_rows(new, group):
    """A sequence whose cached tokens before the new ones, times the group's query heads, pass
    2^31: all of them are seen by every row. (Its pages are one page, listed again and again.)"""
    page = 64
    pages = 2 ** 31 // group // page + 17
    c = Call(83, [new], [page], q_heads=group, heads=1, page=page, q_size=0.05)
    length = pages * page
    table = torch.full((1, pages), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    batch = atom.KV4Batch(table, dev(np.array([length], np.int32)), dev(c.cu_q), max_q=new)
    z = ko.attention(c.q, c.cache, *c.sequences(), False, SCALE)[2] + np.log(pages)
    z = z.astype(np.float32)
    sums = torch.full((1, 1, length), 7.0, device="cuda")
    atom.atom_kv4_attention_weights(dev(c.q), dev(z), c.device_cache(), batch, sums)
    want, tol = ko.attention_weights(c.q, z, c.cache, *c.sequences(), False, SCALE, page)
    got = sums.view(pages, page)
    assert_within(host(got[0]), want[0, 0], tol[0, 0], "sums")
    assert bool((got[:-1] == got[0]).all())
    # the last page holds the new tokens: the last of them only the last query sees
    want, tol = ko.attention_weights(c.q, z, c.cache, *c.sequences(), True, SCALE, page)
    assert_within(host(got[-1]), want[0, 0], tol[0, 0], "last page")


@pytest.mark.parametrize("size", [2.0 ** -14, 0.0])
@pytest.mark.parametrize("new,lens,q_heads,heads", [
    ([3, 5, 2], [3, 60, 129], 4, 4),
    ([4, 4], [64, 50], 8, 2),
    ([2, 8], [31, 200], 1, 1),
    ([60], [60], 16, 2),
    ([150] * 8, [400, 300, 150, 210, 333, 230, 1000, 151], 8, 8),
    ([1000], [1100], 7, 1),
])
def test_values_behind_a_row_leave_its_output_alone(new, lens, q_heads, heads, size):
    """Later tokens' value scales up to 2^27 times a row's own, or beside zeros (all of them as fp16
    vectors have them): the row does not see them, and its weights keep their precision."""
    c = Call(84, new, lens, q_heads=q_heads, heads=heads, page=16, q_size=0.05, garbage=1.0)
    unit = (c.cache[3] / c.cache[3].max()).astype(np.float32)
    c.cache[3] = unit * np.float32(size)
    want = ko.attention(c.q, c.cache, *c.sequences(), True, SCALE)
    later = [a.copy() for a in c.cache]
    rows = np.zeros(c.rows, bool)            # those that see none of the large values
    for b, n in enumerate(c.new):
        few = (n + 1) // 2
        at = np.arange(c.lens[b] - few, c.lens[b])
        place = (c.table[b, at // 16], at % 16)
        later[3][place] = unit[place] * np.float32(2.0 ** 13)
        rows[c.cu_q[b]:c.cu_q[b + 1] - few] = True
    assert rows.any()
    out, lse = atom.atom_kv4_attention(dev(c.q), c.device_cache(later), c.device_batch())
    assert_within(host(out)[rows], want[0][rows], want[1][rows], "out")
    assert_within(host(lse)[rows], want[2][rows], want[3][rows], "lse")


def test_evict_with_the_largest_budget():
    """A budget of 2^31 - 1: every token stays, and the rest of `kept` is -1."""
    budget = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 24 * 2 ** 30:
        pytest.skip("needs 24 GB")
    c = Call(85, [0], [5000], q_heads=1, heads=1, page=16)
    to = Call(86, [0], [5000], q_heads=1, heads=1, page=64)
    dst = to.device_cache()
    w = np.random.default_rng(1).random((1, 1, 5001)).astype(np.float32)
    new_lens = torch.empty(1, dtype=torch.int32, device="cuda")
    kept, new_w = atom.atom_kv4_evict(dev(w), c.device_cache(), c.device_batch(), budget, 100, dst,
                                      dev(to.table), new_lens)
    assert host(new_lens).tolist() == [5000]
    assert np.array_equal(host(kept[0, 0, :5000]), np.arange(5000))
    assert int(kept[0, 0, 5000:].max()) == int(kept[0, 0, 5000:].min()) == -1
    assert np.array_equal(host(new_w[0, 0, :5000]), w[0, 0, :5000])
    at = np.arange(5000)
    for x, ref in zip((dst.k4, dst.ks, dst.v4, dst.vs), c.cache):
        assert np.array_equal(host(x)[to.table[0, at // 64], at % 64],
                              ref[c.table[0, at // 16], at % 16])


@pytest.mark.parametrize("share", [0.1, 0.5, 1.0])
@pytest.mark.parametrize("most,spread,batch", [(8, 16, 1500), (160, 100, 24)])
def test_zero_values_leave_the_log_sum_exp_its_bound(most, spread, batch, share):
    """Tokens whose values are zero (a scale of 0, as the quantizer writes it) beside value scales
    that jump from token to token, and nothing but such tokens."""
    rng = np.random.default_rng(5)
    new = rng.integers(most // 2 if most > 8 else 1, most + 1, batch)
    c = Call(5, new, new + rng.integers(0, spread, batch), q_heads=8, heads=4, page=16, q_size=0.02,
             garbage=1.0)
    shape = c.cache[3].shape
    jumping = c.cache[3] * np.exp2(rng.integers(-13, 9, shape))
    c.cache[3] = np.where(rng.random(shape) < share, 0, np.minimum(jumping, 9000)).astype(np.float32)
    out, lse = atom.atom_kv4_attention(dev(c.q), c.device_cache(), c.device_batch())
    want = ko.attention(c.q, c.cache, *c.sequences(), True, SCALE)
    assert_within(host(out), want[0], want[1], "out")
    assert_within(host(lse), want[2], want[3], "lse")
