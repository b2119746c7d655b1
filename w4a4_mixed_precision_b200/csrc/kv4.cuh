// kv4.cuh -- the paged INT4 KV cache: writing new tokens to it (append) and
// reading them back (gather). The encoding is kv.cuh's: one group per (token,
// head) vector of 128 elements.
//
// Token `row` of the call is new token i = row - cu_q[b] of its sequence b and
// sits at position kv_lens[b] - (cu_q[b+1] - cu_q[b]) + i, whose page is
// table[b][position / page_size].
//
// Both kernels stream: 8 lanes own one vector (16 elements each), as the
// contiguous cache kernels do, and a warp 16 vectors at once (four a lane), so
// that the loads overlap and a token's sequence (a binary search of cu_q) and
// page are looked up once for many of them. Where a token's keys and values are a
// multiple of 16 vectors (8 KV heads) the 16 are one token's; else (kLine) they
// are 16 of the line of all tokens' vectors, and each token that they touch is
// looked up by a lane of its own.
//
// What bounds them: bytes (2 x 256 of fp16 and 2 x 68 of cache a token and head)
// and, nearly as much, the instructions that make one of the other (gather: ALU 69
// % busy, DRAM 55; append: issue slots 63 %, DRAM 44). Nine sequences of some 4000
// tokens, 8 heads: append and gather, 255 MB, 54 us, in a replayed graph as in
// calls; the gather of 64 x 1024 tokens 340 MB in 61 us, 5.5 TB/s.
#pragma once

#include "kv.cuh"
#include "kv4_plan.h"

namespace atomk {

struct Kv4Rows {
  uint8_t *k4, *v4;
  float *ks, *vs;
  Kv4Geom geom;
  Kv4Seqs seqs;
  __half *k, *v;                          // append: read; gather: written
  int64_t k_token, k_head, v_token, v_head;   // strides of k and v, in elements
  uint32_t by_vecs;                       // 2^16 / (vectors of a row), rounded up, for fewer than 16
};

// The last sequence that begins at `row` or before (cu_q ascending).
__device__ __forceinline__ int kv4_sequence_of(const Kv4Seqs &s, int row) {
  int lo = 0, hi = s.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(s.cu_q + mid) <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Vector number of head 0 in the row's slot, or -1 where there is none; what the
// device arrays get wrong is recorded in the status word.
__device__ __forceinline__ int64_t kv4_row_vector(const Kv4Rows &p, int row) {
  const Kv4Seqs &q = p.seqs;
  const int b = kv4_sequence_of(q, row);
  const int q0 = __ldg(q.cu_q + b), q1 = __ldg(q.cu_q + b + 1);
  if (row < q0 || row >= q1) return -1;   // behind the last sequence
  const Kv4Seq s = kv4_seq_of(q0, q1, __ldg(q.kv_lens + b), q.rows, q.capacity);
  if (!s.ok || s.qn > s.len) {
    report_status(1 /* ATOM_ERR_INVALID_ARG */);
    return -1;
  }
  const int pos = s.len - s.qn + row - q0;
  const int page_no = kv4_div(pos, p.geom.by_page);
  const int page = __ldg(q.table + b * q.table_stride + page_no);
  const int64_t vec = kv4_vector(p.geom, page, pos - page_no * p.geom.page_size, 0);
  if (vec < 0) report_status(1 /* ATOM_ERR_INVALID_ARG */);
  return vec;
}

constexpr int kKv4RowVecs = 16;   // per warp and step

// Measured at equal bytes, 340 MB (52 us of HBM), append and gather, us: kLine 84
// and 68 with 1 head, 79 and 63 with 4 and with 12, some 80 and 65 with 8; one
// token's vectors a step 68 and 59 with 8 heads, and with slots left empty 417 and
// 385 with 1 head, 115 and 99 with 4, 80 and 64 with 12.
// (At least 3 and 5 CTAs an SM: 80 registers instead of 100 for append's, 9 x 4000
// tokens 62 -> 58 us with the gather.)
template <bool kAppend, bool kLine>
__global__ void __launch_bounds__(kKvThreads, kAppend ? 3 : 5) kv4_rows_kernel(const Kv4Rows p) {
  const int lane = threadIdx.x & 31, sub = lane & 7, team = lane >> 3;
  const unsigned team_mask = 0xFFu << (8 * team);
  const uint32_t heads = p.geom.heads, vecs = 2 * heads;   // keys of all heads, then values
  const int warps = static_cast<int>(gridDim.x) * (kKvThreads / 32);
  const int warp = static_cast<int>(blockIdx.x) * (kKvThreads / 32) + (threadIdx.x >> 5);
  // one vector of each team, four times: loaded, then encoded or decoded
  uint4 a[4], b[4];
  auto load = [&](int u, int row, int64_t vec0, uint32_t i) {
    const bool value = i >= heads;
    const int head = static_cast<int>(value ? i - heads : i);
    if constexpr (kAppend) {
      const __half *x = value ? p.v + row * p.v_token + head * p.v_head
                              : p.k + row * p.k_token + head * p.k_head;
      const uint4 *src = reinterpret_cast<const uint4 *>(x + sub * 16);
      a[u] = __ldg(src);
      b[u] = __ldg(src + 1);
    } else {
      const int64_t vec = vec0 + static_cast<int64_t>(head) * p.geom.head_stride;
      // words `sub` and 8 + `sub`, so that a team writes 128 bytes in one piece
      const uint32_t *q = reinterpret_cast<const uint32_t *>((value ? p.v4 : p.k4) + vec * 64) + sub;
      a[u] = make_uint4(__ldg(q), __ldg(q + 8),
                        __float_as_uint(__ldg((value ? p.vs : p.ks) + vec)), 0u);
    }
  };
  auto finish = [&](int u, int row, int64_t vec0, uint32_t i, bool store) {
    const bool value = i >= heads;
    const int head = static_cast<int>(value ? i - heads : i);
    if constexpr (kAppend) {
      const int64_t vec = vec0 + static_cast<int64_t>(head) * p.geom.head_stride;
      const uint32_t w[8] = {a[u].x, a[u].y, a[u].z, a[u].w, b[u].x, b[u].y, b[u].z, b[u].w};
      float scale;
      const uint2 codes = kv_encode16(w, team_mask, scale);
      if (store) *reinterpret_cast<uint2 *>((value ? p.v4 : p.k4) + vec * 64 + sub * 8) = codes;
      if (store && sub == 0) (value ? p.vs : p.ks)[vec] = scale;
    } else {
      uint32_t o[8];
      kv_decode16(make_uint2(a[u].x, a[u].y), __uint_as_float(a[u].z), o);
      __half *x = value ? p.v + row * p.v_token + head * p.v_head
                        : p.k + row * p.k_token + head * p.k_head;
      uint4 *dst = reinterpret_cast<uint4 *>(x) + sub;
      if (store) {
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[8] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  };
  grid_dependency_wait();
  if constexpr (kLine) {
    // 16 places a step; the rows that they touch are looked up by a lane each
    const int64_t step = static_cast<int64_t>(warps) * kKv4RowVecs;
    const int64_t step_rows = step / vecs, place = static_cast<int64_t>(warp) * kKv4RowVecs;
    const uint32_t step_off = static_cast<uint32_t>(step - step_rows * vecs);
    int64_t row0 = place / vecs;
    uint32_t off = static_cast<uint32_t>(place - row0 * vecs);
    auto row_of = [&](uint32_t at) -> uint32_t {   // at / vecs, for at < vecs + 15
      return vecs < 16 ? at * p.by_vecs >> 16 : (at >= vecs ? 1u : 0u);
    };
    const int last = p.seqs.rows - 1;
    for (; row0 <= last; row0 += step_rows) {
      int64_t mine = -1;
      if (lane <= row_of(off + 15) && row0 + lane <= last)
        mine = kv4_row_vector(p, static_cast<int>(row0) + lane);
      int64_t vec0[4];
      // (append: a team without a vector encodes one of the last row's, and stores
      // nothing, so that no branch stands around it: 1 head 88 -> 84 us)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t at = off + 4 * u + team, r = row_of(at);
        const int row = static_cast<int>(row0 + r <= last ? row0 + r : last);
        vec0[u] = __shfl_sync(0xffffffffu, mine, r);
        a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
        if (kAppend || vec0[u] >= 0) load(u, row, vec0[u], at - r * vecs);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t at = off + 4 * u + team, r = row_of(at);
        finish(u, static_cast<int>(row0 + r), vec0[u], at - r * vecs, vec0[u] >= 0);
      }
      off += step_off;
      if (off >= vecs) {
        off -= vecs;
        ++row0;
      }
    }
  } else {
    for (int64_t row64 = warp; row64 < p.seqs.rows; row64 += warps) {
      const int row = static_cast<int>(row64);
      const int64_t vec0 = kv4_row_vector(p, row);
      if (vec0 < 0) continue;
      for (uint32_t first = blockIdx.y * kKv4RowVecs; first < vecs;
           first += gridDim.y * kKv4RowVecs) {
#pragma unroll
        for (int u = 0; u < 4; ++u) load(u, row, vec0, first + 4 * u + team);
#pragma unroll
        for (int u = 0; u < 4; ++u) finish(u, row, vec0, first + 4 * u + team, true);
      }
    }
  }
}

}  // namespace atomk
