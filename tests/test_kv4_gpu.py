"""The paged INT4 KV cache on the GPU (atom_kv4_append, atom_kv4_gather, atom_kv4_attention,
atom_kv4_attention_weights, atom_kv4_evict) against oracle/kv4_oracle.py: writing, reading and
evicting bit for bit, attention and its weights within the bounds that the oracle derives."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as ko
from w4a4_mixed_precision_b200 import atom

from kv4_util import Call, assert_within, dev, host, starts

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(autouse=True)
def clean_status():
    atom.atom_device_status(clear=True)
    yield
    assert atom.atom_device_status(clear=True) == 0


def check_attention(c, causal=True, scale=SCALE, **kw):
    out, lse = atom.atom_kv4_attention(dev(c.q), c.device_cache(), c.device_batch(), causal=causal,
                                       scale=scale, **kw)
    want = ko.attention(c.q, c.cache, *c.sequences(), causal, scale)
    n = c.cu_q[-1]
    assert_within(host(out)[:n], want[0][:n], want[1][:n], "out")
    assert_within(host(lse)[:n], want[2][:n], want[3][:n], "lse")
    return out, lse


# ------------------------------------------------------------------------------ append, gather

@pytest.mark.parametrize("new,lens,heads,page,token_major", [
    ([1], [1], 1, 16, False),
    ([1, 1, 1], [1, 17, 33], 2, 16, True),
    ([5, 0, 7, 1], [5, 9, 31, 1], 3, 7, False),
    ([40, 3], [100, 3], 8, 24, True),
    ([33], [33], 2, 1, False),
    ([300, 1, 0, 129], [300, 4, 0, 500], 4, 64, False),
])
def test_append_and_gather_bit_exact(new, lens, heads, page, token_major):
    c = Call(3, new, lens, heads=heads, q_heads=heads, page=page, token_major=token_major,
             garbage=2.0)
    cache, batch = c.device_cache(), c.device_batch()
    atom.atom_kv4_append(dev(c.k), dev(c.v), cache, batch)
    want = [a.copy() for a in c.cache]
    ko.append(c.k, c.v, want, *c.sequences())
    for got, ref in zip((cache.k4, cache.ks, cache.v4, cache.vs), want):
        assert np.array_equal(host(got), ref)      # untouched slots included
    k, v = atom.atom_kv4_gather(cache, batch, c.rows)
    for got, ref in zip((k, v), ko.gather(want, *c.sequences(), c.rows)):
        assert np.array_equal(host(got).view(np.uint16), ref.view(np.uint16))


def test_append_takes_slices_of_a_fused_projection():
    c = Call(5, [3, 9], [10, 9], heads=2, page=8)
    fused = dev(np.concatenate([c.q, c.k, c.v], 1))      # [rows, 8 + 2 + 2, 128]
    cache, batch = c.device_cache(), c.device_batch()
    atom.atom_kv4_append(fused[:, 8:10], fused[:, 10:], cache, batch)
    want = [a.copy() for a in c.cache]
    ko.append(c.k, c.v, want, *c.sequences())
    for got, ref in zip((cache.k4, cache.ks, cache.v4, cache.vs), want):
        assert np.array_equal(host(got), ref, equal_nan=got.dtype == torch.float32)


def test_rows_behind_the_last_sequence_are_left():
    c = Call(6, [2, 3], [20, 3], heads=2, page=8, pad_rows=4)
    cache, batch = c.device_cache(), c.device_batch()
    k = torch.full((c.rows, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    v, out = k.clone(), torch.full((c.rows, 8, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((c.rows, 8), 7.0, device="cuda")
    atom.atom_kv4_gather(cache, batch, c.rows, k=k, v=v)
    atom.atom_kv4_attention(dev(c.q), cache, batch, out=out, lse=lse)
    for t in (k, v, out, lse):
        assert bool((t[5:] == 7).all()) and not bool((t[:5] == 7).all())


# ------------------------------------------------------------------------------ attention

LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000]


@pytest.mark.parametrize("page", [1, 16, 24, 100])
@pytest.mark.parametrize("q_heads,heads", [(1, 1), (4, 4), (8, 1), (14, 2)])
def test_single_tokens_of_all_lengths(page, q_heads, heads):
    check_attention(Call(11, [1] * len(LENGTHS), LENGTHS, q_heads=q_heads, heads=heads, page=page,
                         q_size=0.05))


@pytest.mark.parametrize("token_major", [False, True])
def test_empty_sequences_and_rows(token_major):
    """Sequences with nothing cached, without new tokens, and causal rows before the cache's
    first token: zeros and -infinity."""
    c = Call(12, [1, 0, 4, 1, 6, 0], [0, 5, 2, 40, 0, 0], page=8, token_major=token_major,
             q_size=0.05)
    out, lse = check_attention(c)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -torch.inf).all())
    assert bool((out[1:3] == 0).all()) and bool((lse[1:3] == -torch.inf).all())
    assert bool((lse[3:6] > -torch.inf).all())
    check_attention(c, causal=False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,q_heads,heads", [
    ([2, 5, 8], [100, 5, 300], 8, 8),
    ([3, 4, 1, 5], [200, 4, 77, 130], 6, 2),
    ([5] * 4, [128, 129, 640, 31], 16, 4),
    ([16, 17, 33], [16, 100, 700], 8, 8),
    ([7, 100, 64], [7, 333, 64], 14, 2),
    ([130, 1, 257], [400, 900, 257], 4, 2),
    ([300], [300], 8, 1),
    ([1], [1], 40, 1),
    ([3, 70], [30, 200], 130, 1),
    ([2, 3], [30, 200], 128, 1),
    ([50], [60], 96, 2),
    ([17, 0, 1, 300, 40], [17, 30, 0, 777, 20], 4, 4),
    ([1000], [1100], 7, 1),
    ([129, 128, 127, 33], [129, 4096, 128, 1500], 16, 8),
])
def test_several_queries(new, lens, q_heads, heads, causal):
    check_attention(Call(13, new, lens, q_heads=q_heads, heads=heads, page=24, q_size=0.05),
                    causal=causal)


@pytest.mark.parametrize("heads,lens", [(1, [20000]), (2, [9001, 30, 12345]), (8, [4096] * 3)])
def test_long_sequences_shared_between_ctas(heads, lens):
    check_attention(Call(14, [1] * len(lens), lens, q_heads=4 * heads, heads=heads, page=64,
                         q_size=0.05))


def test_without_a_workspace_and_with_a_kept_one():
    c = Call(15, [1, 3, 1], [700, 50, 3000], page=32, q_size=0.05)
    out, lse = check_attention(c, split=False)
    n = atom.atom_kv4_attention_workspace_bytes(c.rows, c.q_heads, c.heads, 3)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # contents do not matter
    first = check_attention(c, workspace=ws)
    again = check_attention(c, workspace=ws)
    short = check_attention(c, workspace=ws[:n - 16])              # too small: not shared
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    for a, b in zip((out, lse), short):
        assert torch.equal(a, b)


def test_many_short_sequences():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 3000)
    check_attention(Call(16, [1] * 3000, lens, q_heads=2, heads=1, page=16, q_size=0.05))


def test_strided_queries_and_sharp_scores():
    """Queries as a slice of a projection, scores of some hundreds (one token takes all)."""
    c = Call(17, [2, 1, 3], [90, 260, 3], q_heads=4, heads=2, page=16, q_size=3.0)
    wide = dev(np.concatenate([c.q, c.k, c.v], 1))
    out, lse = atom.atom_kv4_attention(wide[:, :4], c.device_cache(), c.device_batch(), scale=SCALE)
    want = ko.attention(c.q, c.cache, *c.sequences(), True, SCALE)
    assert_within(host(out), want[0], want[1], "out")
    assert_within(host(lse), want[2], want[3], "lse")


@pytest.mark.parametrize("new", [[1, 2], [200, 60]])
@pytest.mark.parametrize("power", [-20, 13])
def test_values_of_any_size(power, new):
    """Value scales from fp16's smallest to its largest vectors."""
    c = Call(18, new, [400, 300], page=16, q_size=0.05)
    c.cache[3] = (c.cache[3] * np.float32(2.0 ** power) / np.nanmax(c.cache[3])).astype(np.float32)
    check_attention(c)


@pytest.mark.parametrize("new", [1, 250])
def test_value_sizes_that_grow_and_shrink_along_the_sequence(new):
    """Value scales that rise and fall by 2^36 over the sequence, and sharp scores: the running
    reference has to follow what each row's own weights need."""
    c = Call(20, [new, new], [1300, 900], q_heads=4, heads=2, page=16, q_size=0.3)
    for b, n in enumerate(c.lens):
        at = np.arange(n)
        size = np.exp2(18 * np.sin(at / 150.0) - 5)[:, None].astype(np.float32)
        place = (c.table[b, at // 16], at % 16)
        c.cache[3][place] *= size / 8
    check_attention(c)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,q_heads,heads,page", [
    ([200, 1, 0, 129, 128, 127, 17, 300, 113, 112], [200, 30, 9, 700, 128, 127, 0, 300, 2, 500], 6, 6, 16),
    ([64, 17, 0, 1, 30, 65, 16, 200], [64, 1000, 20, 1, 29, 65, 333, 900], 56, 8, 24),
    ([3, 2, 5, 1, 4, 7, 0, 3], [3, 100, 60, 64, 4, 300, 5, 0], 480, 5, 7),
    ([1, 2, 3, 4, 2, 3, 1, 2], [1, 65, 129, 4, 90, 3, 64, 700], 640, 5, 64),
    ([130] * 8, [1000, 130, 2049, 513, 140, 131, 4000, 191], 16, 8, 100),
    ([257, 256, 255, 1, 512, 64, 40, 9], [257, 256, 300, 700, 512, 2000, 40, 9], 10, 5, 1),
])
def test_many_prompts(new, lens, q_heads, heads, page, causal):
    """Batches with rows enough for the kernel that reads the cache once per 256 of them."""
    check_attention(Call(22, new, lens, q_heads=q_heads, heads=heads, page=page, q_size=0.05),
                    causal=causal)


@pytest.mark.parametrize("power", [-20, 13])
def test_many_prompts_with_values_of_any_size(power):
    c = Call(23, [200] * 8, [400, 300, 200, 210, 333, 230, 1000, 201], q_heads=8, heads=8, page=16,
             q_size=0.05, token_major=True)
    c.cache[3] = (c.cache[3] * np.float32(2.0 ** power) / np.nanmax(c.cache[3])).astype(np.float32)
    check_attention(c)


def test_many_prompts_with_value_sizes_that_grow_and_shrink():
    c = Call(24, [210] * 8, [1300, 900, 210, 700, 500, 300, 1000, 800], q_heads=8, heads=8, page=16,
             q_size=0.3)
    for b, n in enumerate(c.lens):
        at = np.arange(n)
        size = np.exp2(18 * np.sin(at / 150.0) - 5)[:, None].astype(np.float32)
        c.cache[3][c.table[b, at // 16], at % 16] *= size / 8
    check_attention(c)


def test_scale_and_larger_bound_on_new_tokens():
    c = Call(19, [1, 2], [40, 50], page=16, q_size=0.05)
    check_attention(c, scale=0.3)
    cache = c.device_cache()
    a = atom.atom_kv4_attention(dev(c.q), cache, c.device_batch(max_q=None))
    want = ko.attention(c.q, c.cache, *c.sequences(), True, SCALE)
    assert_within(host(a[0]), want[0], want[1], "out")


# ------------------------------------------------------------------------------ weights

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,q_heads,heads,page", [
    ([1], [1], 1, 1, 16),
    ([1, 1, 1, 1], [17, 128, 129, 1000], 8, 2, 24),
    ([5, 0, 3], [300, 20, 3], 6, 2, 16),
    ([64, 100], [64, 500], 4, 4, 7),
    ([200], [200], 16, 2, 64),
    ([1, 4], [0, 2], 4, 2, 16),
    ([40, 3, 0, 130], [40, 90, 20, 700], 4, 4, 24),
    ([1000], [1300], 7, 1, 100),
    ([257, 300], [257, 129], 8, 8, 16),
    ([513], [2000], 16, 4, 64),
])
def test_attention_weights(new, lens, q_heads, heads, page, causal):
    c = Call(21, new, lens, q_heads=q_heads, heads=heads, page=page, q_size=0.05)
    cache, batch = c.device_cache(), c.device_batch()
    _, lse = atom.atom_kv4_attention(dev(c.q), cache, batch, causal=causal)
    width = max(lens) + 3
    shape = (len(new), heads, width)
    sums = torch.full(shape, 7.0, device="cuda")
    atom.atom_kv4_attention_weights(dev(c.q), lse, cache, batch, sums, causal=causal)
    want, tol = ko.attention_weights(c.q, host(lse), c.cache, *c.sequences(), causal, SCALE, width)
    inside = np.arange(width)[None, None] < c.lens[:, None, None]
    inside = np.broadcast_to(inside, shape)
    got = host(sums).copy()
    assert_within(got[inside], want[inside], tol[inside], "sums")
    assert (got[~inside] == 7).all()
    # added to what was there, in place
    again = sums.clone()
    atom.atom_kv4_attention_weights(dev(c.q), lse, cache, batch, again, prev=again, causal=causal)
    twice = host(sums) + got
    assert np.array_equal(host(again)[inside], twice[inside])
    assert (host(again)[~inside] == 7).all()


# ------------------------------------------------------------------------------ eviction

@pytest.mark.parametrize("lens,budget,recent,page,to_page,token_major", [
    ([1], 1, 0, 16, 16, False),
    ([5, 100, 64, 0], 64, 16, 16, 24, True),
    ([513, 1000], 100, 100, 24, 16, False),
    ([700, 701], 512, 0, 16, 1, False),
    ([2000, 3], 1999, 1, 100, 64, True),
    ([1500], 1, 1, 64, 64, False),
    ([40000], 3000, 500, 64, 16, False),
    ([9000, 33], 8999, 0, 24, 64, True),
    ([0, 20000], 4096, 4096, 16, 100, False),
])
def test_evict_matches_the_oracle(lens, budget, recent, page, to_page, token_major):
    heads = 3
    c = Call(31, [0] * len(lens), lens, q_heads=heads, heads=heads, page=page,
             token_major=token_major)
    rng = np.random.default_rng(9)
    width = max(lens) + 2
    w = rng.random((len(lens), heads, width)).astype(np.float32)
    w[rng.random(w.shape) < 0.4] = 0.0           # ties
    w[rng.random(w.shape) < 0.1] = -0.0
    w[rng.random(w.shape) < 0.05] = np.nan
    w[rng.random(w.shape) < 0.05] = np.inf
    w[rng.random(w.shape) < 0.05] = -3.0
    kept_ref, lens_ref = ko.evict(w, c.lens, budget, recent)
    to = Call(32, [0] * len(lens), lens_ref, q_heads=heads, heads=heads, page=to_page,
              token_major=not token_major)
    cache, dst = c.device_cache(), to.device_cache()
    new_lens = torch.full((len(lens),), -1, dtype=torch.int32, device="cuda")
    kept, new_w = atom.atom_kv4_evict(dev(w), cache, c.device_batch(), budget, recent, dst,
                                      dev(to.table), new_lens)
    assert np.array_equal(host(new_lens), lens_ref)
    assert np.array_equal(host(kept), kept_ref)
    check_moved(c, w, kept_ref, lens_ref, (dst.k4, dst.ks, dst.v4, dst.vs), to.table, to_page,
                host(new_w))
    # in place: the same pages, the weights too
    new_lens.fill_(-1)
    wd = dev(w)
    kept, new_w = atom.atom_kv4_evict(wd, cache, c.device_batch(), budget, recent, cache,
                                      dev(c.table), new_lens, new_weights=wd if width >= budget
                                      else None)
    assert np.array_equal(host(new_lens), lens_ref)
    assert np.array_equal(host(kept), kept_ref)
    check_moved(c, w, kept_ref, lens_ref, (cache.k4, cache.ks, cache.v4, cache.vs), c.table, page,
                host(new_w))


@pytest.mark.parametrize("budget,recent", [(1, 0), (100, 30), (257, 257), (600, 64)])
def test_evict_many_sequences(budget, recent):
    """More (sequence, head)s than the GPU holds of the larger CTAs at once."""
    rng = np.random.default_rng(11)
    lens = np.concatenate([[0, 1, 2, 3000], rng.integers(0, 700, 200)])
    test_evict_matches_the_oracle(lens.tolist(), budget, recent, 16, 16, False)


def check_moved(c, w, kept, lens, got, table, page, new_w):
    got = [host(x) for x in got]
    for b, n in enumerate(lens):
        to = np.arange(n)
        for h in range(c.heads):
            at = kept[b, h, :n]
            for ref, x in zip(c.cache, got):
                src = ref[c.table[b, at // c.page], at % c.page, h]
                assert np.array_equal(x[table[b, to // page], to % page, h], src)
            assert np.array_equal(new_w[b, h, :n], w[b, h, at], equal_nan=True)


# ------------------------------------------------------------------------------ together

def test_a_served_sequence_from_prompt_to_eviction():
    """Prompts appended and attended, their weights summed, the cache cut in place to a budget,
    two more tokens decoded on what is left: every step against the oracle's."""
    heads, q_heads, page, budget, recent = 2, 8, 16, 48, 12
    new = np.array([70, 20, 133], np.int32)
    c = Call(41, new, new, q_heads=q_heads, heads=heads, page=page, spare_pages=6, q_size=0.05)
    table = np.full((3, c.table.shape[1] + 1), -1, np.int32)
    table[:, :-1] = c.table
    free = np.setdiff1d(np.arange(c.cache[0].shape[0]), c.table)
    table[1, 2] = free[0]                      # sequence 1 grows into a page of its own
    cache = c.device_cache()
    ref = [a.copy() for a in c.cache]
    lens, table_d = dev(new.copy()), dev(table)
    batch = atom.KV4Batch(table_d, lens, dev(c.cu_q), max_q=int(new.max()))
    atom.atom_kv4_append(dev(c.k), dev(c.v), cache, batch)
    ko.append(c.k, c.v, ref, table, new, c.cu_q)
    out, lse = atom.atom_kv4_attention(dev(c.q), cache, batch)
    want = ko.attention(c.q, ref, table, new, c.cu_q, True, SCALE)
    assert_within(host(out), want[0], want[1], "prompt")
    width = 160
    sums = torch.zeros((3, heads, width), device="cuda")
    atom.atom_kv4_attention_weights(dev(c.q), lse, cache, batch, sums, prev=sums)
    w_ref, w_tol = ko.attention_weights(c.q, host(lse), ref, table, new, c.cu_q, True, SCALE, width)
    assert_within(host(sums), w_ref, w_tol, "sums")
    # evict by the sums that the library made
    w = host(sums).copy()
    kept_ref, lens_ref = ko.evict(w, new, budget, recent)
    new_lens = torch.empty_like(lens)
    kept, _ = atom.atom_kv4_evict(sums, cache, batch, budget, recent, cache, table_d, new_lens,
                                  new_weights=sums)
    assert np.array_equal(host(kept), kept_ref)
    lens.copy_(new_lens)
    moved = [a.copy() for a in ref]
    for b, n in enumerate(lens_ref):
        to = np.arange(n)
        for h in range(heads):
            at = kept_ref[b, h, :n]
            for dst, src in zip(moved, ref):
                dst[table[b, to // page], to % page, h] = src[table[b, at // page], at % page, h]
    rng = np.random.default_rng(3)
    one = atom.KV4Batch(table_d, lens, dev(starts([1, 1, 1])), max_q=1)
    for step in range(2):
        lens += 1
        lens_ref = lens_ref + 1
        q = (rng.standard_normal((3, q_heads, 128)) * 0.05).astype(np.float16)
        kv = rng.standard_normal((2, 3, heads, 128)).astype(np.float16)
        atom.atom_kv4_append(dev(kv[0]), dev(kv[1]), cache, one)
        ko.append(kv[0], kv[1], moved, table, lens_ref, starts([1, 1, 1]))
        out, lse = atom.atom_kv4_attention(dev(q), cache, one)
        want = ko.attention(q, moved, table, lens_ref, starts([1, 1, 1]), True, SCALE)
        assert_within(host(out), want[0], want[1], f"decode {step}")
        assert_within(host(lse), want[2], want[3], f"decode {step}")


# ------------------------------------------------------------------------------ streams, graphs

def test_side_stream_and_captured_graph():
    """A step captured into a graph and replayed on new values and lengths (device memory that
    the program updates) gives what the calls give."""
    c = Call(51, [1, 1, 1], [30, 300, 64], page=16, q_size=0.05, spare_pages=8, garbage=1.0)
    table = np.concatenate([c.table, np.full((3, 1), 0, np.int32)], 1)
    cache, lens = c.device_cache(), dev(c.lens)
    batch = atom.KV4Batch(dev(table), lens, dev(c.cu_q), max_q=1)
    q, k, v = dev(c.q), dev(c.k), dev(c.v)
    sums = torch.zeros((3, 2, 400), device="cuda")

    def step():
        atom.atom_kv4_append(k, v, cache, batch)
        out, lse = atom.atom_kv4_attention(q, cache, batch)
        atom.atom_kv4_attention_weights(q, lse, cache, batch, sums)
        return out, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    rng = np.random.default_rng(2)
    for lens_now in ([30, 300, 64], [12, 301, 1], [31, 32, 33]):
        q.copy_(dev((rng.standard_normal(c.q.shape) * 0.05).astype(np.float16)))
        lens.copy_(dev(np.array(lens_now, np.int32)))
        graph.replay()
        got = [t.clone() for t in (out, lse, sums)]
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got[2], sums)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    a = atom.atom_kv4_attention(q, cache, batch, stream=other)
    other.synchronize()
    assert torch.equal(a[0], want[0])


def test_a_captured_step_with_eviction():
    """Append, attention, its weights and an eviction in place in one graph, replayed."""
    c = Call(52, [1, 1], [200, 90], page=16, q_size=0.05, garbage=1.0)
    cache, lens = c.device_cache(), dev(c.lens)
    batch = atom.KV4Batch(dev(c.table), lens, dev(c.cu_q), max_q=1)
    q, k, v = dev(c.q), dev(c.k), dev(c.v)
    first = [t.clone() for t in (cache.k4, cache.ks, cache.v4, cache.vs)]
    sums = torch.zeros((2, 2, 256), device="cuda")
    new_lens = torch.empty(2, dtype=torch.int32, device="cuda")

    def step():
        atom.atom_kv4_append(k, v, cache, batch)
        out, lse = atom.atom_kv4_attention(q, cache, batch)
        atom.atom_kv4_attention_weights(q, lse, cache, batch, sums, prev=sums)
        kept, _ = atom.atom_kv4_evict(sums, cache, batch, 100, 20, cache, batch.block_table,
                                      new_lens, new_weights=sums)
        return out, lse, kept

    def restart():
        for t, f in zip((cache.k4, cache.ks, cache.v4, cache.vs), first):
            t.copy_(f)
        sums.zero_()
        lens.copy_(dev(c.lens))

    def state(outs):
        return [t.clone() for t in (*outs, cache.k4, cache.ks, cache.v4, cache.vs, sums, new_lens)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    runs = []
    for run in (step, lambda: graph.replay() or outs):
        restart()
        one = state(run())
        lens.copy_(new_lens)           # the next step's token is the last that stayed
        runs.append(one + state(run()))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert host(new_lens).tolist() == [100, 90]


def test_weights_of_a_sequence_without_new_tokens():
    """`max_q` is a bound: one sequence may have none, and its sums are still written."""
    c = Call(59, [0], [300], page=16, q_size=0.05, pad_rows=3)
    lse = torch.zeros((3, 8), device="cuda")
    prev = torch.rand((1, 2, 310), device="cuda")
    sums = torch.full_like(prev, 7.0)
    atom.atom_kv4_attention_weights(dev(c.q), lse, c.device_cache(), c.device_batch(max_q=100), sums,
                                    prev=prev)
    assert torch.equal(sums[..., :300], prev[..., :300]) and bool((sums[..., 300:] == 7).all())


def test_between_the_quantizer_and_the_gemm():
    """Layers of a step in one stream, whose kernels' set-ups may overlap: quantize, project
    (the GEMM for few tokens, which holds tensor memory as the prompt kernels do), append,
    attention and weights by the prompt kernels, the next layer's quantizer on the output."""
    K, heads, group = 512, 5, 32
    c = Call(70, [5] * 12, [300 + i for i in range(12)], q_heads=heads * group, heads=heads, page=16,
             garbage=1.0)
    cache, batch = c.device_cache(), c.device_batch()
    first = [t.clone() for t in (cache.k4, cache.ks, cache.v4, cache.vs)]
    gen = torch.Generator(device="cuda").manual_seed(3)
    idx = torch.arange(0, 256, 2, dtype=torch.int32, device="cuda")
    x0 = torch.randn((60, K), generator=gen, device="cuda").half()
    w = torch.randn(((group + 2) * heads * 128, K), generator=gen, device="cuda").half() * 0.02
    qw = atom.atom_quant_weights(w, idx)
    ws = atom.gemm_workspace(60, w.shape[0], K, "cuda")

    def step(between):
        x, sums = x0, torch.zeros((12, heads, 320), device="cuda")
        for _ in range(3):
            qa = atom.atom_reorder_quant(x, idx)
            between()
            y = atom.atom_w4a4_gemm(qa, qw, K, workspace=ws).view(60, -1, 128)
            between()
            q, k, v = y.split([heads * group, heads, heads], 1)
            atom.atom_kv4_append(k, v, cache, batch)
            between()
            out, lse = atom.atom_kv4_attention(q, cache, batch)
            between()
            atom.atom_kv4_attention_weights(q, lse, cache, batch, sums, prev=sums)
            between()
            x = out.view(60, -1)[:, :K]
        return out, lse, sums

    def restart():
        for t, f in zip((cache.k4, cache.ks, cache.v4, cache.vs), first):
            t.copy_(f)

    want = [t.clone() for t in step(torch.cuda.synchronize)]
    assert bool(want[0].isfinite().all())
    for _ in range(5):
        restart()
        for a, b in zip(step(lambda: None), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(lambda: None)
    for _ in range(5):
        restart()
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """The same work on two streams at a time, each call with its own workspace."""
    cases = [Call(60, [1] * 5, [700, 3, 2000, 64, 900], page=16, q_size=0.05),
             Call(61, [130] * 10, [300] * 10, q_heads=8, heads=8, page=16, q_size=0.05)]
    work = [(dev(c.q), c.device_cache(), c.device_batch(),
             torch.zeros((len(c.lens), c.heads, 2000), device="cuda")) for c in cases]

    def run(q, cache, batch, sums, stream):
        out, lse = atom.atom_kv4_attention(q, cache, batch, stream=stream)
        atom.atom_kv4_attention_weights(q, lse, cache, batch, sums, stream=stream)
        return out, lse, sums

    want = [[t.clone() for t in run(*w, None)] for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(20):
        got = [run(*w, s) for w, s in zip(work, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_a_sequence_listed_twice():
    """Sequences that share their pages (a common prefix) read the same tokens."""
    c = Call(62, [2, 2], [300, 300], page=16, q_size=0.05)
    c.table[1] = c.table[0]
    c.q[2:4] = c.q[:2]
    out, lse = check_attention(c)
    assert torch.equal(out[:2], out[2:]) and torch.equal(lse[:2], lse[2:])


@pytest.mark.parametrize("layout", ["heads first", "one head", "one token", "wide"])
@pytest.mark.parametrize("new,heads", [([1, 4, 30], 2), ([150] * 10, 5)])
def test_layouts_of_queries_keys_and_values(new, heads, layout):
    """Row tensors whose strides are not a contiguous tensor's, broadcast ones among them."""
    c = Call(67, new, [200 + i for i in range(len(new))], q_heads=2 * heads, heads=heads, page=16,
             q_size=0.05, garbage=1.0)

    def laid_out(a):
        t = dev(a)
        if layout == "heads first":
            t = t.transpose(0, 1).contiguous().transpose(0, 1)
        elif layout == "one head":
            t = t[:, :1].expand(t.shape)
        elif layout == "one token":
            t = t[:1].expand(t.shape)
        else:
            wide = torch.zeros((t.shape[0], t.shape[1] + 3, 136), dtype=t.dtype, device="cuda")
            wide[:, 1:-2, :128] = t
            t = wide[:, 1:-2, :128]
        return t, host(t)

    (q, qn), (k, kn), (v, vn) = map(laid_out, (c.q, c.k, c.v))
    cache, batch = c.device_cache(), c.device_batch()
    atom.atom_kv4_append(k, v, cache, batch)
    want = [a.copy() for a in c.cache]
    ko.append(kn, vn, want, *c.sequences())
    for got, ref in zip((cache.k4, cache.ks, cache.v4, cache.vs), want):
        assert np.array_equal(host(got), ref)
    out, lse = atom.atom_kv4_attention(q, cache, batch)
    ref = ko.attention(qn, want, *c.sequences(), True, SCALE)
    assert_within(host(out), ref[0], ref[1], "out")
    assert_within(host(lse), ref[2], ref[3], "lse")
    sums = torch.zeros((len(new), heads, 220), device="cuda")
    atom.atom_kv4_attention_weights(q, lse, cache, batch, sums)
    s, tol = ko.attention_weights(qn, host(lse), want, *c.sequences(), True, SCALE, 220)
    inside = np.broadcast_to(np.arange(220)[None, None] < c.lens[:, None, None], s.shape)
    assert_within(host(sums)[inside], s[inside], tol[inside], "sums")


@pytest.mark.parametrize("new,heads", [([1, 3], 2), ([150] * 10, 5)])
def test_the_largest_scale(new, heads):
    """One token takes all (its score is 1e17 above the next), and nothing overflows."""
    c = Call(68, new, [200 + i for i in range(len(new))], q_heads=2 * heads, heads=heads, page=16,
             garbage=1.0)
    out, lse = atom.atom_kv4_attention(dev(c.q), c.device_cache(), c.device_batch(), scale=1e18)
    want = ko.attention(c.q, c.cache, *c.sequences(), True, 1e18)
    lse, ref = host(lse), want[2]
    assert np.isfinite(host(out)).all()
    assert (np.abs(lse - ref) <= np.abs(ref) * 2.0 ** -20 + want[3]).all()


@pytest.mark.parametrize("scale", [0.0, -0.05])
@pytest.mark.parametrize("new,heads", [([1, 3], 2), ([150] * 10, 5)])
def test_scales_of_zero_and_below(scale, new, heads):
    check_attention(Call(63, new, [200 + i for i in range(len(new))], q_heads=2 * heads, heads=heads,
                         page=16, q_size=0.05), scale=scale)


def test_pool_beyond_32_bits():
    """Codes at byte offsets beyond 2^32: the last pages of a pool of 4.6 GB."""
    pages, size, heads = 140_000, 64, 8
    c = Call(64, [3, 70], [150, 200], q_heads=16, heads=heads, page=size, q_size=0.05)
    free, _ = torch.cuda.mem_get_info()
    if free < 12 * 2 ** 30:
        pytest.skip("needs 12 GB")
    base = pages - 1 - int(c.table.max())
    big = [torch.empty((pages, size, heads, n), dtype=t, device="cuda").squeeze(-1) if n == 1 else
           torch.empty((pages, size, heads, n), dtype=t, device="cuda")
           for n, t in ((64, torch.uint8), (1, torch.float32)) * 2]
    for t, a in zip(big, c.cache):
        t[base:base + a.shape[0]].copy_(torch.from_numpy(np.ascontiguousarray(a)).cuda())
    cache = atom.KV4Cache(*big)
    table = np.where(c.table >= 0, c.table + base, -1).astype(np.int32)
    batch = atom.KV4Batch(dev(table), dev(c.lens), dev(c.cu_q), max_q=70)
    want = [a.copy() for a in c.cache]
    atom.atom_kv4_append(dev(c.k), dev(c.v), cache, batch)
    ko.append(c.k, c.v, want, *c.sequences())
    for t, a in zip(big, want):
        assert np.array_equal(host(t[base:base + a.shape[0]]), a, equal_nan=a.dtype == np.float32)
    out, lse = atom.atom_kv4_attention(dev(c.q), cache, batch)
    ref = ko.attention(c.q, want, *c.sequences(), True, SCALE)
    assert_within(host(out), ref[0], ref[1], "out")
    assert_within(host(lse), ref[2], ref[3], "lse")
    sums = torch.zeros((2, heads, 200), device="cuda")
    atom.atom_kv4_attention_weights(dev(c.q), lse, cache, batch, sums)
    s, tol = ko.attention_weights(c.q, host(lse), want, *c.sequences(), True, SCALE, 200)
    inside = np.broadcast_to(np.arange(200)[None, None] < c.lens[:, None, None], s.shape)
    assert_within(host(sums)[inside], s[inside], tol[inside], "sums")
    new_lens = torch.empty(2, dtype=torch.int32, device="cuda")
    kept, _ = atom.atom_kv4_evict(sums, cache, batch, 100, 10, cache, batch.block_table, new_lens)
    at = host(kept)
    for b in range(2):
        for h in range(heads):
            i, j = at[b, h], np.arange(100)
            src, dst = (c.table[b, i // size], i % size, h), (c.table[b, j // size], j % size, h)
            for t, a in zip(big, want):
                assert np.array_equal(host(t[base:base + a.shape[0]])[dst], a[src])


def test_arrays_that_contradict_the_call():
    """What only the device can see: the sequence is skipped or the page's tokens are zeros, the
    others are as ever, and the status says so."""
    good = Call(65, [2, 2, 2, 2], [40, 50, 60, 70], page=16, q_size=0.05, garbage=1.0)
    want = ko.attention(good.q, good.cache, *good.sequences(), True, SCALE)
    lens, table, cu_q = good.lens.copy(), good.table.copy(), good.cu_q.copy()
    lens[1] = 16 * table.shape[1] + 1          # more than the table has
    lens[2] = -3
    cache = good.device_cache()
    batch = atom.KV4Batch(dev(table), dev(lens), dev(cu_q), max_q=2)
    out = torch.full((8, 8, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((8, 8), 7.0, device="cuda")
    sums = torch.full((4, 2, 80), 7.0, device="cuda")
    before = [t.clone() for t in (cache.k4, cache.ks, cache.v4, cache.vs)]

    def status():
        return atom.atom_device_status(clear=True)

    atom.atom_kv4_attention(dev(good.q), cache, batch, out=out, lse=lse)
    assert status() == 1
    for rows in (slice(0, 2), slice(6, 8)):
        assert_within(host(out)[rows], want[0][rows], want[1][rows], "out")
    assert bool((out[2:6] == 7).all()) and bool((lse[2:6] == 7).all())
    atom.atom_kv4_attention_weights(dev(good.q), lse, cache, batch, sums)
    assert status() == 1
    assert bool((sums[1:3] == 7).all()) and not bool((sums[0, :, :40] == 7).any())
    atom.atom_kv4_append(dev(good.k), dev(good.v), cache, batch)
    assert status() == 1
    ref = [a.copy() for a in good.cache]
    keep = (table[[0, 3]], lens[[0, 3]], np.array([0, 2, 4], np.int32))
    ko.append(good.k[[0, 1, 6, 7]], good.v[[0, 1, 6, 7]], ref, *keep)
    for t, a, b in zip((cache.k4, cache.ks, cache.v4, cache.vs), ref, before):
        assert np.array_equal(host(t), a)
        t.copy_(b)
    new_lens = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    atom.atom_kv4_evict(sums, cache, batch, 30, 5, cache, batch.block_table, new_lens)
    assert status() == 1 and host(new_lens).tolist() == [30, 7, 7, 30]
    # too many new tokens, descending starts
    small = atom.KV4Batch(dev(table), dev(good.lens), dev(cu_q), max_q=1)
    atom.atom_kv4_attention(dev(good.q), cache, small, out=out.fill_(7))
    assert status() == 1 and bool((out == 7).all())
    cu_q[2] = 1
    atom.atom_kv4_attention(dev(good.q), cache, atom.KV4Batch(dev(table), dev(good.lens), dev(cu_q),
                                                             max_q=8), out=out)
    assert status() == 1


@pytest.mark.parametrize("new", [1, 20, 130])
@pytest.mark.parametrize("page", [16, 64])
def test_pages_outside_the_pool_read_as_zeros(new, page):
    c = Call(66, [new] * 16, [200] * 16, q_heads=4, heads=4, page=page, q_size=0.05, garbage=1.0)
    cache = c.device_cache()
    bad = c.table.copy()
    bad[3, 1], bad[5, 0], bad[5, 2] = len(c.cache[0]), -1, 2 ** 31 - 1
    batch = atom.KV4Batch(dev(bad), dev(c.lens), dev(c.cu_q), max_q=new)
    # the oracle reads zeros in pages of their own
    arrays = [np.concatenate([a, np.zeros((1, *a.shape[1:]), a.dtype)]) for a in c.cache]
    table = np.where((bad < 0) & (np.arange(bad.shape[1]) * page < 200) | (bad >= len(c.cache[0])),
                     len(c.cache[0]), bad)
    out, lse = atom.atom_kv4_attention(dev(c.q), cache, batch)
    assert atom.atom_device_status(clear=True) == 1
    want = ko.attention(c.q, arrays, table, c.lens, c.cu_q, True, SCALE)
    assert_within(host(out), want[0], want[1], "out")
    assert_within(host(lse), want[2], want[3], "lse")
    sums = torch.zeros((16, 4, 200), device="cuda")
    atom.atom_kv4_attention_weights(dev(c.q), lse, cache, batch, sums)
    assert atom.atom_device_status(clear=True) == 1
    s, tol = ko.attention_weights(c.q, host(lse), arrays, table, c.lens, c.cu_q, True, SCALE, 200)
    assert_within(host(sums), s, tol, "sums")
