// kv4_evict.cuh -- eviction from the paged INT4 KV cache by accumulated
// attention weight.
//
// Of a sequence's `len` cached tokens, new_len = min(len, budget) stay in each
// KV head: the last recent' = min(recent, new_len), and of the others the
// new_len - recent' with the largest weights (equal weights: the earlier
// token; NaN counts as smaller than everything). They keep their order and move
// to positions 0 .. new_len - 1 of the destination cache.
//
// A cluster of one to eight CTAs per (sequence, head), each with a run of its
// tokens. The smallest weight that stays is found by a radix select over the
// keys (kv4_weight_key) in three passes of 11, 11 and 10 bits: each counts the
// next bits' values among the keys that agree with the bits already known, the
// CTAs add up each other's counts through distributed shared memory, and all
// find the same value. The counts also say how many of each CTA's tokens stay,
// so that one more pass numbers them in order. Then the cluster moves the
// vectors, 8 lanes a token.
//
// In place (or where source and destination memory overlap) the move goes in
// steps: every copy of a step is read before any is written, and a token never
// moves up, so nothing is overwritten that is still to be read.
//
// What bounds it: many sequences, the bytes moved (136 read and written per
// token and head that stays); one long sequence, latency: four passes and a
// dozen cluster barriers.
#pragma once

#include <type_traits>

#include "kv4_plan.h"
#include "ptx.cuh"

namespace atomk {

struct Kv4Evict {
  const float *weights;      // [batch][heads][width]
  int64_t width;
  const uint8_t *k4, *v4;    // source
  const float *ks, *vs;
  Kv4Geom geom;
  Kv4Seqs seqs;              // cu_q is not read
  uint8_t *to_k4, *to_v4;    // destination
  float *to_ks, *to_vs;
  Kv4Geom to_geom;
  const int32_t *to_table;
  int64_t to_table_stride;
  int to_capacity;
  int budget, recent;
  int32_t *new_lens;         // [batch]
  int32_t *kept;             // [batch][heads][budget]
  float *new_weights;        // [batch][heads][new_width], or null
  int64_t new_width;
  int in_steps;              // source and destination memory overlap
};

namespace kv4_evict_cfg {
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kRun = 8;                  // tokens a thread numbers at once
constexpr int kMove = kThreads / 8;      // tokens a CTA moves at once
constexpr int kUnroll = 4;               // ... so many times over, if not in steps
}  // namespace kv4_evict_cfg

__device__ __forceinline__ int ld_shared_cluster_s32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kv4_evict_cfg::kThreads, 2)
kv4_evict_kernel(const __grid_constant__ Kv4Evict p, const int cluster) {
  using namespace kv4_evict_cfg;
  __shared__ int hist[kBins];
  __shared__ int scan[2][kWarps];
  __shared__ int counts[2];                // larger than, equal to `least` among this CTA's
  __shared__ int found_bin, found_above;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cluster > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
  const int row = static_cast<int>(blockIdx.x) / cluster;
  const int head = row % p.geom.heads, b = row / p.geom.heads;
  auto sync_all = [&]() {
    if (cluster > 1) cluster_sync();
    else __syncthreads();
  };
  const int len = __ldg(p.seqs.kv_lens + b);
  const int new_len = len < p.budget ? len : p.budget;
  if (len < 0 || len > p.seqs.capacity || len > p.width || new_len > p.to_capacity) {
    if (tid == 0 && rank == 0) report_status(1 /* ATOM_ERR_INVALID_ARG */);
    return;   // the whole cluster
  }
  const int recent = p.recent < new_len ? p.recent : new_len;
  const int old = len - recent;          // tokens that must earn their place
  const int want = new_len - recent;     // how many of them stay
  const float *w = p.weights + (static_cast<int64_t>(b) * p.geom.heads + head) * p.width;
  int32_t *kept = p.kept + (static_cast<int64_t>(b) * p.geom.heads + head) * p.budget;
  if (head == 0 && tid == 0 && rank == 0) p.new_lens[b] = new_len;
  // this CTA's tokens
  const int share = ((len + cluster - 1) / cluster + kRun - 1) / kRun * kRun;
  const int lo = static_cast<int64_t>(share) * rank < len ? share * rank : len;
  const int hi = len - lo < share ? len : lo + share;
  const int old_hi = hi < old ? hi : old;   // [lo, old_hi) must earn theirs

  // ---- the smallest key that stays, and how many of its equals do
  uint32_t least = 0;    // 0: all equal or above stay
  int same = old;
  int above_here = 0, equal_here = old_hi > lo ? old_hi - lo : 0;   // of this CTA's tokens
  if (want == 0) {
    least = 0xFFFFFFFFu;   // above every key (the largest is that of +infinity)
    same = equal_here = 0;
  } else if (want < old) {
    uint32_t known = 0;
    int need = want;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t bins = pass == 2 ? 1023u : 2047u;
      const uint32_t mask = pass == 0 ? 0u : (pass == 1 ? 0xFFE00000u : 0xFFFFFC00u);
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int i0 = lo; i0 < old_hi; i0 += kThreads) {
        const int i = i0 + tid;
        const uint32_t key = i < old_hi ? kv4_weight_key(__float_as_uint(w[i])) : 0u;
        const bool is = i < old_hi && (key & mask) == known;
        const uint32_t bin = is ? (key >> shift) & bins : kBins;
        // one addition for the lanes of a warp that have the same value (most
        // weights are small, many are zero)
        const unsigned peers = __match_any_sync(0xffffffffu, bin);
        if (is && lane == __ffs(peers) - 1) atomicAdd(&hist[bin], __popc(peers));
      }
      sync_all();
      // the bin at which the count from above reaches `need`; thread t has the
      // bins kBins - 1 - 4t .. - 3
      int mine[4], total = 0, own = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = kBins - 1 - 4 * tid - j;
        mine[j] = hist[at];
        for (int c = 1; c < cluster; ++c)
          mine[j] += ld_shared_cluster_s32(cluster_map(&hist[at], (rank + c) % cluster));
        total += mine[j];
      }
      int upto = total;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
      }
      if (lane == 31) scan[0][warp] = upto;
      __syncthreads();
      for (int v = 0; v < warp; ++v) upto += scan[0][v];
      int above = upto - total;
      if (above < need && upto >= need) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (above < need && above + mine[j] >= need) {
            found_bin = kBins - 1 - 4 * tid - j;
            found_above = above;
          }
          above += mine[j];
        }
      }
      __syncthreads();
      const int bin = found_bin;
      known |= static_cast<uint32_t>(bin) << shift;
      need -= found_above;
      // this CTA's own tokens above it
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (kBins - 1 - 4 * tid - j > bin) own += hist[kBins - 1 - 4 * tid - j];
      own = __reduce_add_sync(0xffffffffu, own);
      if (lane == 0) scan[1][warp] = own;
      __syncthreads();
      for (int v = 0; v < kWarps; ++v) above_here += scan[1][v];
      equal_here = hist[bin];
      sync_all();   // the counts have been read
    }
    least = known;
    same = need;
  }

  // ---- number the tokens that stay: as many as are above `least` before them,
  // and of its equals the first `same`
  int above_before = 0, equal_before = 0;
  if (cluster > 1) {
    if (tid == 0) {
      counts[0] = above_here;
      counts[1] = equal_here;
    }
    cluster_sync();
    for (int c = 0; c < rank; ++c) {
      above_before += ld_shared_cluster_s32(cluster_map(&counts[0], c));
      equal_before += ld_shared_cluster_s32(cluster_map(&counts[1], c));
    }
  }
#pragma unroll 1
  for (int base = lo; base < hi; base += kThreads * kRun) {
    const int i0 = base + tid * kRun;
    unsigned above = 0, equal = 0;   // bits: tokens i0 ..
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int i = i0 + j;
      if (i >= hi || i >= old) continue;
      const uint32_t key = kv4_weight_key(__float_as_uint(w[i]));
      above |= (key > least ? 1u : 0u) << j;
      equal |= (key == least ? 1u : 0u) << j;
    }
    const int mine_a = __popc(above), mine_e = __popc(equal);
    int a = mine_a, e = mine_e;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int va = __shfl_up_sync(0xffffffffu, a, d), ve = __shfl_up_sync(0xffffffffu, e, d);
      if (lane >= d) {
        a += va;
        e += ve;
      }
    }
    if (lane == 31) {
      scan[0][warp] = a;
      scan[1][warp] = e;
    }
    __syncthreads();
    a += above_before - mine_a;
    e += equal_before - mine_e;
    for (int v = 0; v < kWarps; ++v) {
      if (v < warp) {
        a += scan[0][v];
        e += scan[1][v];
      }
      above_before += scan[0][v];
      equal_before += scan[1][v];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int i = i0 + j;
      if (i >= hi) continue;
      if (i >= old) {
        kept[want + i - old] = i;
      } else if ((above >> j) & 1u) {
        kept[a + (e < same ? e : same)] = i;
        ++a;
      } else if ((equal >> j) & 1u) {
        if (e < same) kept[a + e] = i;
        ++e;
      }
    }
  }
  for (int i = new_len + rank * kThreads + tid; i < p.budget; i += cluster * kThreads) kept[i] = -1;
  sync_all();

  // ---- move them: 8 lanes a token, 4 for the key's and 4 for the value's codes
  const int part = tid & 7;
  const bool value = part >= 4;
  const uint8_t *codes = (value ? p.v4 : p.k4) + (part & 3) * 16;
  uint8_t *to_codes = (value ? p.to_v4 : p.to_k4) + (part & 3) * 16;
  const float *scales = value ? p.vs : p.ks;
  float *to_scales = value ? p.to_vs : p.to_ks;
  float *new_w = p.new_weights == nullptr
                     ? nullptr
                     : p.new_weights + (static_cast<int64_t>(b) * p.geom.heads + head) * p.new_width;
  const bool has_scale = (part & 3) == 0, has_weight = part == 1 && new_w != nullptr;
  auto move = [&](auto unroll, int base, auto between) {
    constexpr int U = decltype(unroll)::value;
    int from[U], page[U], to_page[U];
    int64_t dst[U];
    uint4 c[U];
    float s[U], weight[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int to = base + u * kMove + (tid >> 3);
      from[u] = to < new_len ? kept[to] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int to = base + u * kMove + (tid >> 3);
      page[u] = to_page[u] = -1;
      if (from[u] < 0) continue;
      page[u] = __ldg(p.seqs.table + b * p.seqs.table_stride + kv4_div(from[u], p.geom.by_page));
      to_page[u] = __ldg(p.to_table + b * p.to_table_stride + kv4_div(to, p.to_geom.by_page));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int to = base + u * kMove + (tid >> 3);
      dst[u] = -1;
      c[u] = make_uint4(0u, 0u, 0u, 0u);
      s[u] = weight[u] = 0.f;
      if (from[u] < 0) continue;
      if (has_weight) weight[u] = w[from[u]];
      const int64_t src = kv4_vector(p.geom, page[u], from[u] - kv4_div(from[u], p.geom.by_page) *
                                                                    p.geom.page_size, head);
      dst[u] = kv4_vector(p.to_geom, to_page[u],
                          to - kv4_div(to, p.to_geom.by_page) * p.to_geom.page_size, head);
      if (src < 0 || dst[u] < 0) {
        report_status(1 /* ATOM_ERR_INVALID_ARG */);
        dst[u] = -1;
        continue;
      }
      c[u] = *reinterpret_cast<const uint4 *>(codes + src * 64);
      if (has_scale) s[u] = scales[src];
    }
    between();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int to = base + u * kMove + (tid >> 3);
      if (dst[u] >= 0) {
        *reinterpret_cast<uint4 *>(to_codes + dst[u] * 64) = c[u];
        if (has_scale) to_scales[dst[u]] = s[u];
      }
      if (from[u] >= 0 && has_weight) new_w[to] = weight[u];
    }
  };
  if (p.in_steps) {
    for (int base = 0; base < new_len; base += cluster * kMove) {
      move(std::integral_constant<int, 1>{}, base + rank * kMove, sync_all);
      sync_all();
    }
  } else {
    for (int base = rank * kUnroll * kMove; base < new_len; base += cluster * kUnroll * kMove)
      move(std::integral_constant<int, kUnroll>{}, base, [] {});
  }
}

}  // namespace atomk
