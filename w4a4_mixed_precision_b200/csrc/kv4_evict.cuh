// kv4_evict.cuh -- eviction from the paged INT4 KV cache by accumulated
// attention weight.
//
// Of a sequence's `len` cached tokens, new_len = min(len, budget) stay in each
// KV head: the last recent' = min(recent, new_len), and of the others the
// new_len - recent' with the largest weights (equal weights: the earlier
// token; NaN counts as smaller than everything). They keep their order and move
// to positions 0 .. new_len - 1 of the destination cache.
//
// One CTA per (sequence, head). The smallest weight that stays is found by a
// radix select: four passes over the keys (kv4_weight_key), each of which
// counts one byte's values among the keys that agree with the bytes already
// known. Then one pass in order numbers the tokens that stay, and the move
// copies 64 tokens at a time: a token never moves up, and every copy of a step
// is read before any is written, so source and destination may be the same.
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
};

constexpr int kKv4EvictThreads = 512;

__global__ void __launch_bounds__(kKv4EvictThreads) kv4_evict_kernel(const __grid_constant__ Kv4Evict p) {
  constexpr int kWarps = kKv4EvictThreads / 32;
  __shared__ int hist[256];
  __shared__ int warp_keep[kWarps], warp_same[kWarps];
  __shared__ int found_byte, found_above;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = static_cast<int>(blockIdx.x) % p.geom.heads;
  const int b = static_cast<int>(blockIdx.x) / p.geom.heads;
  const int len = __ldg(p.seqs.kv_lens + b);
  const int new_len = len < p.budget ? len : p.budget;
  if (len < 0 || len > p.seqs.capacity || len > p.width || new_len > p.to_capacity) {
    if (tid == 0) report_status(1 /* ATOM_ERR_INVALID_ARG */);
    return;
  }
  const int recent = p.recent < new_len ? p.recent : new_len;
  const int old = len - recent;          // tokens that must earn their place
  const int want = new_len - recent;     // how many of them stay
  const float *w = p.weights + (static_cast<int64_t>(b) * p.geom.heads + head) * p.width;
  int32_t *kept = p.kept + (static_cast<int64_t>(b) * p.geom.heads + head) * p.budget;
  if (head == 0 && tid == 0) p.new_lens[b] = new_len;

  // ---- the smallest key that stays, and how many of its equals do
  uint32_t least = 0;   // everything is kept where want == old
  int same = old;       // equals of `least` that stay
  if (want < old) {
    uint32_t known = 0;
    int need = want;
    if (want == 0) {
      least = 0xFFFFFFFFu;   // above every key (the largest is that of +infinity)
      same = 0;
    } else {
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kKv4EvictThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
        for (int i = tid; i < old; i += kKv4EvictThreads) {
          const uint32_t key = kv4_weight_key(__float_as_uint(w[i]));
          if ((key & mask) == known) atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (warp == 0) {   // the byte at which the count from above reaches `need`
          int mine[8], total = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            mine[j] = hist[255 - (lane * 8 + j)];
            total += mine[j];
          }
          int upto = total;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
          }
          int above = upto - total;
          if (above < need && upto >= need) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (above < need && above + mine[j] >= need) {
                found_byte = 255 - (lane * 8 + j);
                found_above = above;
                break;
              }
              above += mine[j];
            }
          }
        }
        __syncthreads();
        known |= static_cast<uint32_t>(found_byte) << shift;
        need -= found_above;
      }
      least = known;
      same = need;
    }
  }

  // ---- number the tokens that stay
  int kept_before = 0, same_before = 0;
  for (int base = 0; base < len; base += kKv4EvictThreads) {
    const int i = base + tid;
    uint32_t key = 0;
    if (i < old) key = kv4_weight_key(__float_as_uint(w[i]));
    const bool equal = i < old && key == least;
    const unsigned equals = __ballot_sync(0xffffffffu, equal);
    if (lane == 0) warp_same[warp] = __popc(equals);
    __syncthreads();
    int at = same_before + __popc(equals & ((1u << lane) - 1));
    for (int v = 0; v < kWarps; ++v) {
      if (v < warp) at += warp_same[v];
      same_before += warp_same[v];
    }
    const bool keep = i < len && (i >= old || key > least || (equal && at < same));
    const unsigned keeps = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) warp_keep[warp] = __popc(keeps);
    __syncthreads();
    int to = kept_before + __popc(keeps & ((1u << lane) - 1));
    for (int v = 0; v < kWarps; ++v) {
      if (v < warp) to += warp_keep[v];
      kept_before += warp_keep[v];
    }
    if (keep) kept[to] = i;
  }
  for (int i = new_len + tid; i < p.budget; i += kKv4EvictThreads) kept[i] = -1;
  __syncthreads();

  // ---- move them: 8 lanes a token, 4 for the key's and 4 for the value's codes
  const int part = tid & 7;
  const bool value = part >= 4;
  for (int base = 0; base < new_len; base += kKv4EvictThreads / 8) {
    const int to = base + (tid >> 3);
    int64_t src = -1, dst = -1;
    uint4 codes = make_uint4(0u, 0u, 0u, 0u);
    float scale = 0.f, weight = 0.f;
    if (to < new_len) {
      const int from = kept[to];
      int page_no = kv4_div(from, p.geom.by_page);
      src = kv4_vector(p.geom, __ldg(p.seqs.table + b * p.seqs.table_stride + page_no),
                       from - page_no * p.geom.page_size, head);
      page_no = kv4_div(to, p.to_geom.by_page);
      dst = kv4_vector(p.to_geom, __ldg(p.to_table + b * p.to_table_stride + page_no),
                       to - page_no * p.to_geom.page_size, head);
      if (src < 0 || dst < 0) {
        report_status(1 /* ATOM_ERR_INVALID_ARG */);
      } else {
        codes = *reinterpret_cast<const uint4 *>((value ? p.v4 : p.k4) + src * 64 + (part & 3) * 16);
        if ((part & 3) == 0) scale = value ? p.vs[src] : p.ks[src];
      }
      if (part == 1 && p.new_weights != nullptr) weight = w[from];
    }
    __syncthreads();
    if (src >= 0 && dst >= 0) {
      *reinterpret_cast<uint4 *>((value ? p.to_v4 : p.to_k4) + dst * 64 + (part & 3) * 16) = codes;
      if ((part & 3) == 0) (value ? p.to_vs : p.to_ks)[dst] = scale;
    }
    if (to < new_len && part == 1 && p.new_weights != nullptr)
      p.new_weights[(static_cast<int64_t>(b) * p.geom.heads + head) * p.new_width + to] = weight;
    __syncthreads();
  }
}

}  // namespace atomk
