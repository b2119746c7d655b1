"""The paged INT4 KV cache without a GPU: the index arithmetic that the kernels share with the
host (csrc/kv4_plan.h, compiled here by the host compiler), the library's refusals and the
binding's checks."""
import ctypes as ct
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from w4a4_mixed_precision_b200 import atom

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
A16, MIS = 0x10000, 0x10001      # device addresses that nothing reads

CHECKS = r"""
#include "kv4_plan.h"
using namespace atomk;
extern "C" {
int div_by(int n, int64_t d) { return kv4_div(n, kv4_div_by(d)); }
int64_t vector_of(int page, int slot, int head, int pages, int ps, int ts, int hs) {
  Kv4Geom g{};
  g.pages = pages; g.page_stride = ps; g.token_stride = ts; g.head_stride = hs;
  return kv4_vector(g, page, slot, head);
}
int seq_ok(int q0, int q1, int len, int rows, int capacity) {
  return kv4_seq_of(q0, q1, len, rows, capacity).ok;
}
int limit(int qn, int len, int qi, int causal) {
  return kv4_limit(Kv4Seq{0, qn, len, true}, qi, causal != 0);
}
uint32_t weight_key(uint32_t bits) { return kv4_weight_key(bits); }
int64_t part_begin(int64_t total, int parts, int i) { return kv4_part_begin(total, parts, i); }
int capacity(int64_t max_pages, int64_t page_size) { return kv4_capacity(max_pages, page_size); }
int64_t few_rows(int64_t pairs, int64_t max_rows, int sms) { return kv4_few_rows(pairs, max_rows, sms); }

// Items' query copies with a wait for an empty buffer that gives up at its
// give_up-th call (0: none does). 0: every copy was started in a buffer that was
// empty, and what was under way at the end was waited for.
int query_copies(int items, int give_up) {
  uint32_t started[2] = {0, 0};
  int waits = 0, copies[2] = {0, 0}, landed[2] = {0, 0}, bad = 0;
  bool ok = true;
  for (int i = 0; ok && i < items; ++i)
    ok = kv4_start_queries(
        started,
        [&](int w, uint32_t parity) {
          // a buffer is empty when its last copy has landed and been used; the
          // barrier's phase before the first reads as odd
          bad |= parity != ((copies[w] & 1u) ^ 1u);
          if (++waits == give_up) return false;
          landed[w] = copies[w];
          return true;
        },
        [&](int w) {
          bad |= landed[w] != copies[w];
          ++copies[w];
        });
  bad |= ok != (give_up == 0 || give_up > 2 * items);
  kv4_drain_queries(started, [&](int w, uint32_t parity) {
    bad |= copies[w] == 0 || parity != ((copies[w] - 1u) & 1u);
    landed[w] = copies[w];
  });
  return bad || landed[0] != copies[0] || landed[1] != copies[1];
}

// The decode kernel's division of a call among `ctas` CTAs, walked through on
// the host. Counts how often every (tile, unit) is computed, checks that a
// tile's shares are exactly the slots that its join reads, and returns 0 where
// all of it holds.
int walk(const int *new_tokens, const int *lens, int batch, int heads, int group, int tile,
         int ctas, int *units_out) {
  int64_t total = 0;
  auto tiles = [&](int b) { return kv4_tiles(Kv4Seq{0, new_tokens[b], lens[b], true}, group, tile); };
  for (int b = 0; b < batch; ++b) total += int64_t(tiles(b)) * heads * kv4_units(lens[b]);
  *units_out = int(total);
  int64_t rows = 0;
  for (int b = 0; b < batch; ++b) rows += int64_t(tiles(b)) * heads;
  const int parts = kv4_parts(total, rows, ctas);
  if (total > 0 && (parts < 1 || parts > ctas || parts > total)) return 7;
  int64_t next = 0;
  // the tile of each place, as the line's order gives it
  struct Tile { int64_t begin, end; };
  int b = 0, h = 0, q = 0;
  int64_t begin = 0;
  auto settle = [&]() { while (b < batch && tiles(b) == 0) ++b; };
  settle();
  int *slots = new int[2 * ctas]();   // 1: written, 2: written and read
  for (; begin < total;) {
    const int64_t end = begin + kv4_units(lens[b]);
    const int first = kv4_part_of(total, parts, begin), last = kv4_part_of(total, parts, end - 1);
    if (kv4_part_begin(total, parts, first) > begin || kv4_part_begin(total, parts, first + 1) <= begin)
      return 1;
    if (kv4_part_begin(total, parts, last + 1) < end) return 2;
    if (first != last)
      for (int i = first; i <= last; ++i) {
        const int64_t lo = kv4_part_begin(total, parts, i), hi = kv4_part_begin(total, parts, i + 1);
        if (lo >= hi) return 3;                       // an empty part would write no share
        const bool starts = lo <= begin;              // (kernel) the share's first unit is the tile's
        const int slot = 2 * i + (starts ? 1 : 0);
        if (slots[slot]++) return 4;                  // two shares in one slot
        if (slot != 2 * i + (i == first ? 1 : 0)) return 5;   // the join reads this one
      }
    next += end - begin;
    begin = end;
    if (++q == tiles(b)) { q = 0; if (++h == heads) { h = 0; ++b; settle(); } }
  }
  delete[] slots;
  return next == total && b == batch ? 0 : 6;
}
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(CHECKS)
    subprocess.run([cc, "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                    os.path.join(ROOT, "w4a4_mixed_precision_b200", "csrc"), str(d / "plan.cpp"),
                    "-o", str(d / "plan.so")], check=True)
    lib = ct.CDLL(str(d / "plan.so"))
    lib.div_by.argtypes = [ct.c_int, ct.c_int64]
    lib.vector_of.argtypes = [ct.c_int] * 7
    lib.vector_of.restype = ct.c_int64
    lib.weight_key.argtypes, lib.weight_key.restype = [ct.c_uint32], ct.c_uint32
    lib.part_begin.argtypes, lib.part_begin.restype = [ct.c_int64, ct.c_int, ct.c_int], ct.c_int64
    return lib


def test_division_by_the_page_size(plan):
    top = 2 ** 31 - 1
    for d in [1, 2, 3, 7, 16, 24, 64, 100, 1000, 65537, 131072, 2 ** 30 - 1, 2 ** 30 + 1, top]:
        for n in {0, 1, d - 1, d, d + 1, 2 * d - 1, 2 * d, top, top - 1, top // d * d,
                  top // d * d - 1, 12345678}:
            if 0 <= n <= top:
                assert plan.div_by(n, d) == n // d, (n, d)


def test_vectors_and_bad_pages(plan):
    assert plan.vector_of(3, 5, 2, 4, 1000, 10, 1) == 3052
    top = 2 ** 31 - 1                                             # far past 32 bits
    assert plan.vector_of(top - 1, top, 7, top, top, top, 1) == (top - 1) * top + top * top + 7
    for page in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        assert plan.vector_of(page, 0, 0, 4, 1000, 10, 1) == -1


def test_sequences_that_contradict_the_call(plan):
    assert plan.seq_ok(0, 5, 9, 5, 9) == 1
    assert plan.seq_ok(5, 5, 0, 5, 9) == 1
    for bad in [(-1, 5, 9, 5, 9), (3, 2, 9, 5, 9), (0, 6, 9, 5, 9), (0, 5, -1, 5, 9),
                (0, 5, 10, 5, 9), (0, 2 ** 31 - 1, 9, 5, 9)]:
        assert plan.seq_ok(*bad) == 0, bad


def test_limits(plan):
    assert [plan.limit(3, 10, i, 1) for i in range(3)] == [8, 9, 10]
    assert [plan.limit(3, 10, i, 0) for i in range(3)] == [10, 10, 10]
    assert [plan.limit(4, 2, i, 1) for i in range(4)] == [0, 0, 1, 2]
    assert plan.limit(2 ** 31 - 1, 0, 0, 1) == 0


def test_positions_stay_below_2_to_30(plan):
    plan.capacity.argtypes = [ct.c_int64, ct.c_int64]
    for pages, size, want in [(0, 16, 0), (0, 2 ** 31 - 1, 0), (3, 16, 48), (2 ** 30, 1, 2 ** 30),
                              (2 ** 30 + 1, 1, 2 ** 30), (1, 2 ** 31 - 1, 2 ** 30),
                              (2 ** 26, 16, 2 ** 30), (2 ** 62, 3, 2 ** 30)]:
        assert plan.capacity(pages, size) == want


def test_rows_that_the_decode_kernel_takes(plan):
    plan.few_rows.argtypes = [ct.c_int64, ct.c_int64, ct.c_int]
    plan.few_rows.restype = ct.c_int64
    for pairs in [1, 2, 7, 36, 64, 128, 148, 149, 300, 512, 10 ** 4, 2 ** 31, 2 ** 62]:
        rows = [plan.few_rows(pairs, m, 148) for m in (1, 16, 17, 300, 10 ** 5, 2 ** 30)]
        assert rows[0] == rows[1] == 16 and rows == sorted(rows) and rows[-1] <= 4096
        assert all(r % 16 == 0 for r in rows)
    assert plan.few_rows(8, 10 ** 6, 148) > plan.few_rows(128, 10 ** 6, 148) >= 48


def test_weight_keys_order_as_the_weights(plan):
    values = np.array([np.nan, -np.inf, -3.0, -1e-40, -0.0, 0.0, 1e-45, 1e-40, 1.0, 3e38, np.inf],
                      np.float32)
    keys = [plan.weight_key(int(b)) for b in values.view(np.uint32)]
    assert keys[4] == keys[5]                          # the two zeros
    assert all(a < b for a, b in zip(keys[:4], keys[1:5])) and all(
        a < b for a, b in zip(keys[5:-1], keys[6:]))
    assert plan.weight_key(0xFFC00001) == 0 and keys[-1] < 0xFFFFFFFF


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 444, 592])
def test_division_of_the_work(plan, ctas):
    rng = np.random.default_rng(ctas)
    for case in range(60):
        batch = int(rng.integers(1, 40))
        new = rng.integers(0, 4, batch) if case % 2 else rng.integers(0, 70, batch)
        lens = np.where(rng.random(batch) < 0.2, 0, rng.integers(0, 10 ** int(rng.integers(1, 6)), batch))
        a = [np.ascontiguousarray(x, np.int32) for x in (new, lens)]
        units = ct.c_int()
        rc = plan.walk(*[x.ctypes.data_as(ct.c_void_p) for x in a], batch, int(rng.integers(1, 9)),
                       int(rng.integers(1, 9)), int(rng.choice([8, 16])), ctas, ct.byref(units))
        assert rc == 0, (rc, new, lens)


def test_parts_of_long_lines(plan):
    for total in (2 ** 40 + 12345, 2 ** 33):
        edges = [plan.part_begin(total, 592, i) for i in range(593)]
        assert edges[0] == 0 and edges[-1] == total
        assert all(b - a in (total // 592, total // 592 + 1) for a, b in zip(edges, edges[1:]))


def test_query_copies_are_waited_for_wherever_a_wait_gives_up(plan):
    for items in range(1, 6):
        for give_up in range(0, 2 * items + 2):
            assert plan.query_copies(items, give_up) == 0, (items, give_up)


# ------------------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def lib():
    from w4a4_mixed_precision_b200 import build
    build.build()
    return atom.lib()


def cache(**kw):
    f = dict(k4=A16, ks=A16, v4=A16, vs=A16, pages=4, page_size=16, heads=2, page_stride=32,
             token_stride=2, head_stride=1)
    f.update(kw)
    return ct.byref(atom._CacheStruct(**f))


def batch(**kw):
    f = dict(block_table=A16, table_stride=2, max_pages=2, kv_lens=A16, cu_q=A16, batch=2, max_q=1)
    f.update(kw)
    return ct.byref(atom._BatchStruct(**f))


def append(lib, k=A16, kt=256, kh=128, v=A16, vt=256, vh=128, rows=2, c=None, b=None):
    return lib.atom_kv4_append(k, kt, kh, v, vt, vh, rows, c or cache(), b or batch(), None)


def attention(lib, q=A16, qt=1024, qh=128, rows=2, q_heads=8, c=None, b=None, scale=0.1, out=A16,
              lse=A16):
    return lib.atom_kv4_attention(q, qt, qh, rows, q_heads, c or cache(), b or batch(), 1, scale, out,
                                  lse, None, 0, None)


def weights(lib, q=A16, rows=2, q_heads=8, lse=A16, c=None, b=None, prev=0, sums=A16, width=32,
            scale=0.1):
    return lib.atom_kv4_attention_weights(q, 1024, 128, rows, q_heads, lse, c or cache(),
                                          b or batch(), 1, scale, prev, sums, width, None)


def evict(lib, w=A16, width=32, c=None, b=None, budget=8, recent=4, dst=None, table=A16, stride=2,
          pages=2, lens=A16 + 64, kept=A16, new_w=A16 + 4096, new_width=8):
    return lib.atom_kv4_evict(w, width, c or cache(), b or batch(), budget, recent, dst or cache(),
                              table, stride, pages, lens, kept, new_w, new_width, None)


def both(lib, kw):
    return append(lib, **kw), attention(lib, **kw), weights(lib, **kw), evict(lib, **kw)


@pytest.mark.parametrize("kw,expect", [
    (dict(c=dict(page_size=0)), SHAPE), (dict(c=dict(heads=0)), SHAPE),
    (dict(c=dict(pages=2 ** 31)), SHAPE), (dict(c=dict(page_size=2 ** 31)), SHAPE),
    (dict(c=dict(token_stride=-1)), INVALID), (dict(c=dict(page_stride=2 ** 31)), SHAPE),
    (dict(c=dict(k4=0)), INVALID),
    (dict(c=dict(vs=0)), INVALID), (dict(c=dict(v4=A16 + 8)), ALIGN),
    (dict(c=dict(ks=MIS)), ALIGN), (dict(b=dict(batch=-1)), INVALID),
    (dict(b=dict(batch=2 ** 31)), SHAPE), (dict(b=dict(table_stride=1)), SHAPE),
    (dict(b=dict(block_table=0)), INVALID), (dict(b=dict(kv_lens=0)), INVALID),
    (dict(b=dict(kv_lens=MIS)), ALIGN), (dict(b=dict(block_table=MIS)), ALIGN),
    (dict(b=dict(max_q=-1)), INVALID), (dict(b=dict(batch=0)), OK),
])
def test_caches_and_batches_are_checked_on_the_host(lib, kw, expect):
    kw = {k: (cache if k == "c" else batch)(**v) for k, v in kw.items()}
    assert both(lib, kw) == (expect,) * 4


def test_null_structs_are_refused(lib):
    n = ct.c_void_p(None)
    assert lib.atom_kv4_append(A16, 256, 128, A16, 256, 128, 2, n, batch(), None) == INVALID
    assert lib.atom_kv4_append(A16, 256, 128, A16, 256, 128, 2, cache(), n, None) == INVALID
    assert lib.atom_kv4_gather(n, batch(), 2, A16, A16, None) == INVALID
    assert lib.atom_kv4_attention(A16, 8, 8, 2, 8, n, batch(), 1, 0.1, A16, A16, None, 0,
                                  None) == INVALID
    assert lib.atom_kv4_evict(A16, 32, n, batch(), 8, 4, cache(), A16, 2, 2, A16 + 64, A16, None, 8,
                              None) == INVALID
    assert lib.atom_kv4_evict(A16, 32, cache(), n, 8, 4, cache(), A16, 2, 2, A16 + 64, A16, None, 8,
                              None) == INVALID


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), INVALID), (dict(rows=2 ** 31), SHAPE), (dict(rows=0), OK),
    (dict(k=0), INVALID), (dict(v=A16 + 8), ALIGN), (dict(kt=4), SHAPE), (dict(vh=-8), INVALID),
])
def test_append_is_checked_on_the_host(lib, kw, expect):
    assert append(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), INVALID), (dict(rows=2 ** 31), SHAPE), (dict(rows=0), OK), (dict(q=0), INVALID),
    (dict(q=MIS), ALIGN), (dict(qt=1028), SHAPE), (dict(q_heads=7), SHAPE), (dict(q_heads=0), SHAPE),
    (dict(q_heads=-2), INVALID), (dict(rows=2 ** 30), SHAPE), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(out=0), INVALID), (dict(out=A16 + 8), ALIGN),
    (dict(lse=MIS), ALIGN),
])
def test_attention_is_checked_on_the_host(lib, kw, expect):
    assert attention(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(width=-1), INVALID), (dict(lse=0), INVALID), (dict(sums=0), INVALID),
    (dict(sums=MIS), ALIGN), (dict(prev=MIS), ALIGN), (dict(q_heads=5), SHAPE),
    (dict(scale=float("nan")), INVALID), (dict(rows=0), OK),
])
def test_weights_are_checked_on_the_host(lib, kw, expect):
    assert weights(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(budget=0), INVALID), (dict(recent=-1), INVALID), (dict(recent=9), INVALID),
    (dict(budget=2 ** 31, new_width=2 ** 31), SHAPE), (dict(new_width=7), SHAPE),
    (dict(w=0), INVALID), (dict(lens=0), INVALID), (dict(lens=A16), INVALID),   # batch's kv_lens
    (dict(kept=0), INVALID), (dict(kept=MIS), ALIGN), (dict(stride=1), SHAPE),
    (dict(new_w=A16, new_width=16), SHAPE),      # in place with rows of another width
    (dict(dst=cache(heads=4)), SHAPE), (dict(dst=cache(k4=A16 + 4)), ALIGN),
])
def test_eviction_is_checked_on_the_host(lib, kw, expect):
    assert evict(lib, **kw) == expect


# ------------------------------------------------------------------------------ binding

def q4(*lead):
    return torch.zeros(*lead, 64, dtype=torch.uint8)


@pytest.mark.parametrize("scale", [1.1e18, -1e30, float("inf"), float("nan")])
def test_scales_that_scores_cannot_hold_are_refused(lib, scale):
    assert attention(lib, scale=scale) == INVALID
    assert weights(lib, scale=scale) == INVALID


def test_more_rows_than_2_to_30_are_refused(lib):
    assert append(lib, rows=2 ** 30 + 1) == SHAPE
    assert attention(lib, rows=2 ** 30 + 1, q_heads=2) == SHAPE
    assert attention(lib, rows=2 ** 28 + 1, q_heads=8) == SHAPE
    assert weights(lib, rows=2 ** 29 + 1, q_heads=4) == SHAPE


def test_more_sequences_than_2_to_30_are_refused(lib):
    """Searches add two sequence numbers, and threads round runs of them up, in 32 bits."""
    for n in (2 ** 30 + 1, 2 ** 31 - 1):
        assert both(lib, dict(b=batch(batch=n))) == (SHAPE,) * 4


def test_binding_checks_a_cache():
    s = torch.zeros(3, 16, 2)
    with pytest.raises(ValueError, match="CUDA"):
        atom.KV4Cache(q4(3, 16, 2), s, q4(3, 16, 2), s)
    with pytest.raises(ValueError, match="shape"):
        atom.KV4Cache(q4(3, 16, 2), s, q4(3, 16, 1), s)
    with pytest.raises(ValueError, match="shape"):
        atom.KV4Cache(q4(3, 16, 2)[..., :32], s, q4(3, 16, 2), s)
    head_major = q4(3, 2, 16).transpose(1, 2)
    with pytest.raises(ValueError, match="layout"):
        atom.KV4Cache(head_major, s, head_major, s)
    with pytest.raises(ValueError, match="CUDA"):
        atom.KV4Cache(head_major, s.view(3, 2, 16).transpose(1, 2), head_major,
                      s.view(3, 2, 16).transpose(1, 2))
    with pytest.raises(ValueError, match="uint8"):
        atom.KV4Cache(q4(3, 16, 2).to(torch.int8), s, q4(3, 16, 2), s)


def test_binding_checks_a_batch():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)   # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        atom.KV4Batch(i(2, 5), i(2), i(3))
    with pytest.raises(ValueError, match="shape"):
        atom.KV4Batch(i(2, 5), i(2), i(2))
    with pytest.raises(ValueError, match="shape"):
        atom.KV4Batch(i(3, 5), i(2), i(3))
    with pytest.raises(ValueError, match="int32"):
        atom.KV4Batch(i(2, 5).long(), i(2), i(3))
    with pytest.raises(ValueError, match="max_q"):
        atom.KV4Batch(i(2, 5), i(2), i(3), max_q=-1)


def test_binding_checks_rows():
    with pytest.raises(ValueError, match="shape"):
        atom._kv4_rows(torch.zeros(4, 2, 64), 2, "q", None)
    with pytest.raises(ValueError, match="shape"):
        atom._kv4_rows(torch.zeros(4, 3, 128, dtype=torch.float16), 2, "q", None)
    with pytest.raises(ValueError, match="float16"):
        atom._kv4_rows(torch.zeros(4, 2, 128), 2, "q", None)
    with pytest.raises(ValueError, match="CUDA"):
        atom._kv4_rows(torch.zeros(4, 2, 128, dtype=torch.float16), 2, "q", None)


def test_a_failed_workspace_query_is_raised_and_not_kept(monkeypatch):
    answers = [0, 4096]
    monkeypatch.setattr(atom, "atom_kv4_attention_workspace_bytes", lambda *a: answers.pop(0))
    sizes = (2 ** 20, 5, 8, 2, 7)          # a device that no other test names
    with pytest.raises(atom.AtomError, match="ATOM_ERR_CUDA"):
        atom._kv4_workspace_bytes(*sizes)
    assert atom._kv4_workspace_bytes(*sizes) == atom._kv4_workspace_bytes(*sizes) == 4096
    # no work, or sizes that the call itself refuses
    monkeypatch.setattr(atom, "atom_kv4_attention_workspace_bytes", lambda *a: 0)
    for rows, q_heads, heads, max_q in [(0, 8, 2, 7), (5, 7, 2, 7), (5, 8, 2, 0), (5, 0, 2, 7)]:
        assert atom._kv4_workspace_bytes(2 ** 20 + 1, rows, q_heads, heads, max_q) == 0
