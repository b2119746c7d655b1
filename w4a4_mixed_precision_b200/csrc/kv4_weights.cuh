// kv4_weights.cuh -- the attention weight that every cached token received:
//
//   sums[b][h][t] = prev[b][h][t] + sum over the new tokens i of sequence b and
//                   the query heads of KV head h of exp(s[i][t] - lse[i])
//
// with the scores s of kv4_attn.cuh and the log-sum-exps that the attention
// returned. Only keys are read. A warp holds the key fragments of 32 tokens and
// passes all query rows that see one of them by, 8 at a time, so every sum is
// made by one warp in a fixed order: no atomics, the same result every time.
#pragma once

#include "kv4_attn.cuh"

namespace atomk {

struct Kv4Weights {
  const __half *q;
  int64_t q_token, q_head;
  const float *lse;      // [rows][q_heads]
  const uint8_t *k4;
  const float *ks;
  Kv4Geom geom;
  Kv4Seqs seqs;
  int q_heads, group;
  float scale_log2;
  int causal;
  const float *prev;     // [batch][heads][width], or null
  float *sums;           // [batch][heads][width]
  int64_t width;
};

constexpr int kKv4WeightThreads = 128;

__global__ void __launch_bounds__(kKv4WeightThreads, 4)
kv4_weights_kernel(const __grid_constant__ Kv4Weights p) {
  constexpr int kWarps = kKv4WeightThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  grid_dependency_wait();
  auto units_of = [&](const Kv4Seq &s) { return s.len > 0 ? kv4_units(s.len) : 0; };
  auto weight = [&](const Kv4Seq &s) -> int64_t {
    return static_cast<int64_t>(units_of(s)) * p.geom.heads;
  };
  const Kv4Part part = kv4_find_part<kWarps>(p.seqs, weight);
  if (part.count == 0) return;
  int b = part.b;
  Kv4Seq s = kv4_load_seq(p.seqs, b);
  int units = units_of(s);
  int head = static_cast<int>(part.rest / units);
  int unit = static_cast<int>(part.rest - static_cast<int64_t>(head) * units);
  for (int64_t left = part.count; left > 0; --left) {
    const int tok0 = unit * kKv4Unit + warp * 32;
    if (tok0 < s.len) {
      // ---- key fragments of 32 tokens: rows g, g + 8 of two halves
      uint32_t kf[2][8][4];
      float ks[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int pos = tok0 + 16 * h + 8 * i + g;
          w[i] = make_uint4(0u, 0u, 0u, 0u);
          ks[h][i] = 0.f;
          if (pos < s.len) {
            const int page_no = kv4_div(pos, p.geom.by_page);
            const int page = __ldg(p.seqs.table + b * p.seqs.table_stride + page_no);
            const int64_t vec =
                kv4_vector(p.geom, page, pos - page_no * p.geom.page_size, head);
            if (vec < 0) {
              report_status(1 /* ATOM_ERR_INVALID_ARG */);
            } else {
              w[i] = __ldg(reinterpret_cast<const uint4 *>(p.k4 + vec * 64 + t * 16));
              ks[h][i] = __ldg(p.ks + vec) * p.scale_log2;
            }
          }
        }
        const uint32_t wa[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
        const uint32_t wb[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t ca[4], cb[4];
          codes_f16_word(wa[j], ca);
          codes_f16_word(wb[j], cb);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            kf[h][2 * j + k][0] = ca[2 * k];
            kf[h][2 * j + k][1] = cb[2 * k];
            kf[h][2 * j + k][2] = ca[2 * k + 1];
            kf[h][2 * j + k][3] = cb[2 * k + 1];
          }
        }
      }
      // ---- all query rows that see the first of the tokens, and those after
      const int rows = s.qn * p.group;
      int qi0 = p.causal ? tok0 - (s.len - s.qn) : 0;
      if (qi0 < 0) qi0 = 0;
      float sum[2][2] = {}, far[2][2] = {};
      int since = 0;
      for (int r0 = qi0 * p.group / 8 * 8; r0 < rows; r0 += 8) {
        uint32_t qf[16];
        {
          const int r = r0 + g;
          const bool valid = r < rows;
          const int qi = valid ? r / p.group : 0;
          const int hq = head * p.group + (valid ? r - qi * p.group : 0);
          kv4_query_fragments(p.q + (s.q0 + qi) * p.q_token + hq * p.q_head, t, valid, qf);
        }
        float lse[2];
        int limit[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = r0 + 2 * t + c;
          limit[c] = 0;
          lse[c] = 0.f;
          if (r < rows) {
            const int qi = r / p.group, hq = head * p.group + r - qi * p.group;
            limit[c] = kv4_limit(s, qi, p.causal != 0);
            const float z = __ldg(p.lse + static_cast<int64_t>(s.q0 + qi) * p.q_heads + hq);
            lse[c] = z * 1.44269504088896341f;
            if (z == -INFINITY) limit[c] = 0;   // a row that saw nothing
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[4] = {};
#pragma unroll
          for (int k = 0; k < 8; ++k) mma_f16_16816(x, kf[h][k], qf[2 * k], qf[2 * k + 1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int pos = tok0 + 16 * h + 8 * (e >> 1) + g;
            const float w = exp2_approx(fmaf(x[e], ks[h][e >> 1], -lse[e & 1]));
            sum[h][e >> 1] += pos < limit[e & 1] ? w : 0.f;
          }
        }
        if (++since == 32) {   // sums of sums: the rounding of long sums stays small
          since = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            far[i >> 1][i & 1] += sum[i >> 1][i & 1];
            sum[i >> 1][i & 1] = 0.f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = far[i >> 1][i & 1] + sum[i >> 1][i & 1];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        const int pos = tok0 + 16 * (i >> 1) + 8 * (i & 1) + g;
        if (t == 0 && pos < s.len) {
          const int64_t at = (static_cast<int64_t>(b) * p.geom.heads + head) * p.width + pos;
          p.sums[at] = p.prev != nullptr ? p.prev[at] + v : v;
        }
      }
    }
    if (left > 1 && ++unit == units) {
      unit = 0;
      if (++head == p.geom.heads) {
        head = 0;
        do {
          ++b;
          s = kv4_load_seq(p.seqs, b);
          units = units_of(s);
        } while (units == 0);
      }
    }
  }
}

}  // namespace atomk
