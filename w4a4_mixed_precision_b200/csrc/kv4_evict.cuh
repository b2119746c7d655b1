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
// vectors.
//
// In place (or where source and destination memory overlap) the move goes in
// steps: every copy of a step is read before any is written, and a token never
// moves up, so nothing is overwritten that is still to be read.
//
// What bounds it: many sequences, the latencies of three passes and the move, for
// DRAM is half busy (136 bytes read and written per token and head that stays: 64 x
// 2048 tokens to 1024, 8 heads, 42 us in a replayed graph, 3.5 TB/s); one long
// sequence, four passes and a dozen cluster barriers (65537 to 4097 tokens, 8
// heads, 28 us).
#pragma once

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
  int keys;                  // that the launch's shared memory holds
  int in_steps;              // source and destination memory overlap
};

namespace kv4_evict_cfg {
constexpr int kThreads = 512;
constexpr int kFewThreads = 256;         // where there are many (sequence, head)s
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kRun = 8;                  // tokens a thread numbers at once
constexpr int kKeys = 12288;             // keys kept in shared memory, at most
}  // namespace kv4_evict_cfg

__device__ __forceinline__ int4 ld_shared_cluster_v4s(uint32_t cluster_addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}
__device__ __forceinline__ int ld_shared_cluster_s32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// T threads; with kFewThreads no cluster.
template <int T>
__global__ void __launch_bounds__(T, 1024 / T)
kv4_evict_kernel(const __grid_constant__ Kv4Evict p, const int cluster_size) {
  using namespace kv4_evict_cfg;
  constexpr int kWarps = T / 32, kOwnBins = kBins / T;
  const int cluster = T == kThreads ? cluster_size : 1;
  extern __shared__ __align__(16) uint8_t kv4_smem[];
  uint32_t *keys = reinterpret_cast<uint32_t *>(kv4_smem);
  __shared__ __align__(16) int hist[kBins];
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
  // sum of the values of the warps before this one
  auto warps_before = [&](const int (&of)[kWarps]) {
    return static_cast<int>(__reduce_add_sync(0xffffffffu, lane < warp ? of[lane & (kWarps - 1)] : 0));
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

  // The keys of [lo, old_hi), read once, where they fit. Loads of a batch are in
  // flight together.
  const bool in_smem = old_hi - lo <= p.keys;
  if (in_smem && want > 0 && want < old) {
    for (int i0 = lo; i0 < old_hi; i0 += 8 * T) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * T + tid;
        v[j] = i < old_hi ? w[i] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * T + tid;
        if (i < old_hi) keys[i - lo] = kv4_weight_key(__float_as_uint(v[j]));
      }
    }
  }
  auto key_of = [&](int i) {
    return in_smem ? keys[i - lo] : kv4_weight_key(__float_as_uint(w[i]));
  };

  // ---- the smallest key that stays, and how many of its equals do
  uint32_t least = 0;    // 0: all stay
  int same = 0;
  int above_here = old_hi > lo ? old_hi - lo : 0, equal_here = 0;   // of this CTA's tokens
  if (want == 0) {
    least = 0xFFFFFFFFu;   // above every key (the largest is that of +infinity)
    above_here = 0;
  } else if (want < old) {
    uint32_t known = 0;
    int need = want;
    above_here = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t bins = pass == 2 ? 1023u : 2047u;
      const uint32_t mask = pass == 0 ? 0u : (pass == 1 ? 0xFFE00000u : 0xFFFFFC00u);
      for (int i = tid; i < kBins; i += T) hist[i] = 0;
      __syncthreads();
#pragma unroll 8
      for (int i0 = lo; i0 < old_hi; i0 += T) {
        const int i = i0 + tid;
        const uint32_t key = i < old_hi ? key_of(i) : 0u;
        const bool is = i < old_hi && (key & mask) == known;
        if (is) atomicAdd(&hist[(key >> shift) & bins], 1);
      }
      sync_all();
      // the bin at which the count from above reaches `need`; thread t has the
      // kOwnBins below kBins - kOwnBins * t
      const int top_bin = kBins - 1 - kOwnBins * tid;
      int mine[kOwnBins], own = 0;
#pragma unroll
      for (int j = 0; j < kOwnBins; j += 4) {
        const int4 here = *reinterpret_cast<const int4 *>(&hist[top_bin - 3 - j]);
        mine[j] = here.w;
        mine[j + 1] = here.z;
        mine[j + 2] = here.y;
        mine[j + 3] = here.x;
      }
      if (cluster > 1) {   // (kOwnBins is 4)
        int4 v[kMaxCluster - 1];
#pragma unroll
        for (int c = 1; c < kMaxCluster; ++c)
          v[c - 1] = c < cluster ? ld_shared_cluster_v4s(cluster_map(&hist[top_bin - 3], (rank + c) % cluster))
                                 : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int c = 1; c < kMaxCluster; ++c) {
          mine[0] += v[c - 1].w;
          mine[1] += v[c - 1].z;
          mine[2] += v[c - 1].y;
          mine[3] += v[c - 1].x;
        }
      }
      int total = 0;
#pragma unroll
      for (int j = 0; j < kOwnBins; ++j) total += mine[j];
      int upto = total;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
      }
      if (lane == 31) scan[0][warp] = upto;
      __syncthreads();
      upto += warps_before(scan[0]);
      int above = upto - total;
      if (above < need && upto >= need) {
#pragma unroll
        for (int j = 0; j < kOwnBins; ++j) {
          if (above < need && above + mine[j] >= need) {
            found_bin = top_bin - j;
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
      for (int j = 0; j < kOwnBins; ++j)
        if (top_bin - j > bin) own += hist[top_bin - j];
      own = __reduce_add_sync(0xffffffffu, own);
      if (lane == 0) scan[1][warp] = own;
      __syncthreads();
      above_here += __reduce_add_sync(0xffffffffu, lane < kWarps ? scan[1][lane] : 0);
      equal_here = hist[bin];
      sync_all();   // the counts have been read
    }
    least = known;
    same = need;
  }

  // ---- number the tokens that stay: as many as are above `least` before them,
  // and of its equals the first `same`
  const bool searched = want > 0 && want < old;
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
  for (int base = lo; base < old_hi; base += T * kRun) {
    const int i0 = base + tid * kRun;
    unsigned above = 0, equal = 0;   // bits: tokens i0 ..
    uint32_t run[kRun];
    if (searched && in_smem && i0 + kRun <= old_hi) {   // (lo and i0 are multiples of kRun apart)
#pragma unroll
      for (int j = 0; j < kRun; j += 4) {
        const uint4 k = *reinterpret_cast<const uint4 *>(keys + i0 - lo + j);
        run[j] = k.x;
        run[j + 1] = k.y;
        run[j + 2] = k.z;
        run[j + 3] = k.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kRun; ++j)   // (without a search all or none of them stay)
        run[j] = searched && i0 + j < old_hi ? key_of(i0 + j) : 1u;
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      if (i0 + j >= old_hi) continue;
      above |= (run[j] > least ? 1u : 0u) << j;
      equal |= (run[j] == least ? 1u : 0u) << j;
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
    a += above_before - mine_a + warps_before(scan[0]);
    e += equal_before - mine_e + warps_before(scan[1]);
    above_before += __reduce_add_sync(0xffffffffu, lane < kWarps ? scan[0][lane] : 0);
    equal_before += __reduce_add_sync(0xffffffffu, lane < kWarps ? scan[1][lane] : 0);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int is_above = (above >> j) & 1, is_equal = (equal >> j) & 1;
      if (is_above | (is_equal & (e < same ? 1 : 0))) kept[a + (e < same ? e : same)] = i0 + j;
      a += is_above;
      e += is_equal;
    }
  }
  for (int i = old + rank * T + tid; i < len; i += cluster * T) kept[want + i - old] = i;
  for (int64_t i = new_len + rank * T + tid; i < p.budget; i += cluster * T)   // (to 2^31 - 1)
    kept[i] = -1;
  sync_all();

  // ---- move them. A warp takes 32 tokens at a time: a lane finds the addresses
  // of one of them (and moves its scales and weight), then 8 lanes move a token's
  // codes, 4 the key's and 4 the value's. The addresses of the next 32 are looked
  // up while the codes are on their way.
  float *new_w = p.new_weights == nullptr
                     ? nullptr
                     : p.new_weights + (static_cast<int64_t>(b) * p.geom.heads + head) * p.new_width;
  const uint8_t *codes = ((lane & 4) != 0 ? p.v4 : p.k4) + (lane & 3) * 16;
  uint8_t *to_codes = ((lane & 4) != 0 ? p.to_v4 : p.to_k4) + (lane & 3) * 16;
  const int32_t *table = p.seqs.table + b * p.seqs.table_stride;
  const int32_t *to_table = p.to_table + b * p.to_table_stride;
  int from = -1, page_no = 0, to_page_no = 0, page = -1, to_page = -1;
  auto look_up = [&](int to) {   // token `to` of those that stay
    from = to < new_len ? kept[to] : -1;
    if (from < 0) return;
    page_no = kv4_div(from, p.geom.by_page);
    to_page_no = kv4_div(to, p.to_geom.by_page);
    page = __ldg(table + page_no);
    to_page = __ldg(to_table + to_page_no);
  };
  // steps: as many warps as the cluster has, 32 tokens each
  const int step = cluster * T;
  const int first = (rank * kWarps + warp) * 32 + lane;
  look_up(first);
  for (int base = 0; base < new_len; base += step) {
    const int to = base + first;
    int64_t src = -1, dst = -1;
    float ks = 0.f, vs = 0.f, weight = 0.f;
    const bool mine = from >= 0;
    if (mine) {
      src = kv4_vector(p.geom, page, from - page_no * p.geom.page_size, head);
      dst = kv4_vector(p.to_geom, to_page, to - to_page_no * p.to_geom.page_size, head);
      if (new_w != nullptr) weight = w[from];
      if (src < 0 || dst < 0) {
        report_status(1 /* ATOM_ERR_INVALID_ARG */);
        src = dst = -1;
      } else {
        ks = p.ks[src];
        vs = p.vs[src];
      }
    }
    uint4 c[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t at = __shfl_sync(0xffffffffu, src, 4 * u + (lane >> 3));
      c[u] = make_uint4(0u, 0u, 0u, 0u);
      if (at >= 0) c[u] = *reinterpret_cast<const uint4 *>(codes + at * 64);
    }
    look_up(to + step);
    if (p.in_steps) sync_all();   // all of the step's copies have been read
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t at = __shfl_sync(0xffffffffu, dst, 4 * u + (lane >> 3));
      if (at >= 0) *reinterpret_cast<uint4 *>(to_codes + at * 64) = c[u];
    }
    if (dst >= 0) {
      p.to_ks[dst] = ks;
      p.to_vs[dst] = vs;
    }
    if (mine && new_w != nullptr) new_w[to] = weight;
    if (p.in_steps) sync_all();   // ... and written
  }
}

}  // namespace atomk
