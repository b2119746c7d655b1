// kv4_weights.cuh -- the attention weight that every cached token received:
//
//   sums[b][h][t] = prev[b][h][t] + sum over the new tokens i of sequence b and
//                   the query heads of KV head h of exp(s[i][t] - lse[i])
//
// with the scores s of kv4_attn.cuh and the log-sum-exps that the attention
// returned. Only keys are read. Every sum is made in a fixed order: no atomics,
// the same result every time.
//
// Few query rows (single and drafted tokens), kv4_weights_kernel: a warp expands
// the keys of 16 tokens at a time and passes the query rows that see one of them
// by, 8 at a time. 64 sequences of up to 8192 tokens, 64 heads over 8: 237 MB in 62
// us in a replayed graph, 3.8 TB/s; 65 to 68 a call. No unit is full (issue slots 61
// %, ALU 43 %, DRAM 43 %): a warp's chains of copies, expansion and products.
//
// Many (prompts), kv4_weights_prompt_kernel: the transposed product K Q^T on the
// tcgen05 tensor cores. A CTA takes 128 tokens of a (sequence, KV head) and all
// query rows that see one of them in tiles of 128. A token is a row of the
// product, that is a TMEM lane and a thread: its scale is one register, its sum
// another, and nothing is reduced across threads. The expanded keys stay in TMEM
// as the A operand (read from shared memory for each product, A costs 105
// cycles a 128x128x16 MMA instead of 74). What bounds it: the exponentials, 1024
// cycles of the SM per 128x128 tile, against 592 of the tensor core (4096 tokens,
// 64 heads over 8: 180 us in a replayed graph, 188 to 193 a call, with the
// exponential unit 79 % busy; an earlier form took 181, and with an eighth to a half
// of them as a polynomial on the FMA units 187 to 213).
#pragma once

#include "kv4_prompt.cuh"

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
  Kv4Div by_group;
  int tile_rows;         // query rows of a tile: whole tokens' rows, up to 128
  float scale_log2;
  int causal;
  int whole;             // as in Kv4Attn
  int few_rows;          // sequences of up to so many rows a KV head go to the first
                         // kernel, the others to the second
  const float *prev;     // [batch][heads][width], or null
  float *sums;           // [batch][heads][width]
  int64_t width;
  Kv4Magic magic;
};

namespace kv4_wdecode_cfg {
constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kTok = 64;             // tokens per warp and stage
constexpr int kUnit = kWarps * kTok;
constexpr int kStages = 2;
constexpr uint32_t kCodeBytes = kTok * 64;
constexpr uint32_t kStage = kCodeBytes + 2 * kTok * 4;   // codes, scales, earlier sums
constexpr uint32_t kSmemBytes = kWarps * kStages * kStage;
}  // namespace kv4_wdecode_cfg

// A unit of 256 tokens of a (sequence, KV head), with its sequence's facts.
struct Kv4WUnit {
  int b, head, unit, units;
  Kv4Seq s;
};

__device__ __forceinline__ int kv4_wdecode_units(const Kv4Seq &s, const Kv4Weights &p) {
  return s.len > 0 && static_cast<int64_t>(s.qn) * p.group <= p.few_rows ? (s.len - 1) / kv4_wdecode_cfg::kUnit + 1
                                                                             : 0;
}
__device__ __forceinline__ void kv4_next_unit(Kv4WUnit &u, const Kv4Weights &p) {
  if (++u.unit < u.units) return;
  u.unit = 0;
  if (++u.head < p.geom.heads) return;
  u.head = 0;
  do {
    ++u.b;
    u.s = kv4_load_seq(p.seqs, u.b);
    u.units = kv4_wdecode_units(u.s, p);
  } while (u.units == 0);
}

__global__ void __launch_bounds__(kv4_wdecode_cfg::kThreads, 5)
kv4_weights_kernel(const __grid_constant__ Kv4Weights p) {
  using namespace kv4_wdecode_cfg;
  __shared__ __align__(16) uint8_t ring_all[kSmemBytes];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  grid_dependency_wait();
  const Kv4Part part = kv4_find_part<kWarps>(
      p.seqs,
      [&](const Kv4Seq &s) { return static_cast<int64_t>(kv4_wdecode_units(s, p)) * p.geom.heads; },
      [&](const Kv4Seq &s) { return kv4_wdecode_units(s, p) > 0 ? p.geom.heads : 0; });
  if (part.count == 0) return;
  Kv4WUnit u;    // what is computed
  u.b = part.b;
  u.s = kv4_load_seq(p.seqs, u.b);
  u.units = kv4_wdecode_units(u.s, p);
  u.head = static_cast<int>(part.rest / u.units);
  u.unit = static_cast<int>(part.rest - static_cast<int64_t>(u.head) * u.units);

  // ---- the copies, kStages units ahead of the arithmetic (as kv4_attn.cuh's)
  Kv4WUnit l = u;
  int to_load = static_cast<int>(part.count);
  const uint8_t *ring = ring_all + warp * kStages * kStage;
  const uint32_t k_dst = smem_addr(ring) + lane * 16, s_dst = smem_addr(ring) + kCodeBytes + lane * 4;
  const int64_t lane_scale = static_cast<int64_t>(lane) * p.geom.token_stride;
  const int64_t lane_code = static_cast<int64_t>(g) * p.geom.token_stride * 64 + t * 16;
  const int64_t step = static_cast<int64_t>(p.geom.token_stride) * 512;
  int page_no, page;   // of the next stage's first token (whole)
  auto fetch_page = [&]() {
    const int pos = l.unit * kUnit + warp * kTok;
    page_no = kv4_div(pos, p.geom.by_page);
    page = pos < l.s.len ? __ldg(p.seqs.table + l.b * p.seqs.table_stride + page_no) : -1;
  };
  if (p.whole) fetch_page();
  auto issue = [&](int stage) {
    if (to_load > 0) {
      const int pos0 = l.unit * kUnit + warp * kTok;
      const uint32_t at = stage * kStage;
      if (pos0 < l.s.len && p.prev != nullptr) {
        const float *src = p.prev + (static_cast<int64_t>(l.b) * p.geom.heads + l.head) * p.width + pos0;
#pragma unroll
        for (int i = 0; i < kTok; i += 32) {
          const bool is = pos0 + i + lane < l.s.len;
          cp_async_4z(s_dst + at + kTok * 4 + i * 4, is ? src + i + lane : p.prev, is ? 4u : 0u);
        }
      }
      if (pos0 >= l.s.len) {
        // none of the sequence's tokens
      } else if (p.whole) {
        int n = l.s.len - pos0;
        int64_t vec = kv4_vector(p.geom, page, pos0 - page_no * p.geom.page_size, l.head);
        if (vec < 0) {
          report_status(1 /* ATOM_ERR_INVALID_ARG */);
          vec = 0;
          n = 0;
        }
#pragma unroll
        for (int i = 0; i < kTok; i += 32) {
          const bool is = i + lane < n;
          cp_async_4z(s_dst + at + i * 4,
                      p.ks + vec + (is ? lane_scale + static_cast<int64_t>(i) * p.geom.token_stride : 0),
                      is ? 4u : 0u);
        }
        const uint8_t *kp = p.k4 + lane_code + vec * 64;
        if (n >= kTok && step == 512) {   // (a head's tokens together need no address sums: 64 -> 63 us)
#pragma unroll
          for (int i = 0; i < kTok / 8; ++i)
            cp_async_16(k_dst + at + i * 512, kp + i * 512, 16u);
        } else {
#pragma unroll
          for (int i = 0; i < kTok / 8; ++i) {
            const bool is = 8 * i + g < n;
            cp_async_16(k_dst + at + i * 512, is ? kp : p.k4, is ? 16u : 0u);
            kp += step;
          }
        }
      } else {
        for (int j = 0; j < kTok; j += 32) {
          const int pos = pos0 + j + lane;
          int64_t vec = -1;
          if (pos < l.s.len) {
            const int no = kv4_div(pos, p.geom.by_page);
            vec = kv4_vector(p.geom, __ldg(p.seqs.table + l.b * p.seqs.table_stride + no),
                             pos - no * p.geom.page_size, l.head);
            if (vec < 0) report_status(1 /* ATOM_ERR_INVALID_ARG */);
          }
          cp_async_4z(s_dst + at + j * 4, p.ks + (vec < 0 ? 0 : vec), vec < 0 ? 0u : 4u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t v = __shfl_sync(0xffffffffu, vec, 8 * i + g);
            cp_async_16(k_dst + at + j * 64 + i * 512, p.k4 + (v < 0 ? 0 : v) * 64 + t * 16,
                        v < 0 ? 0u : 16u);
          }
        }
      }
      if (--to_load > 0) {
        kv4_next_unit(l, p);
        if (p.whole) fetch_page();
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) issue(i);

  // ---- query rows r0 .. r0 + 7 of the unit's (sequence, head): fragments, and
  // the log-sum-exps and limits of this lane's two columns
  uint32_t qf[16];
  float lse[2];
  int limit[2], least = 0;   // least: of the warp's columns that count
  auto queries = [&](int r0, int rows) {
    const int r = r0 + g;
    const bool valid = r < rows;
    const int qi = valid ? kv4_div(r, p.by_group) : 0;
    const int hq = u.head * p.group + (valid ? r - qi * p.group : 0);
    kv4_query_fragments(p.q + (u.s.q0 + qi) * p.q_token + hq * p.q_head, t, valid, qf);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int rc = r0 + 2 * t + c;
      limit[c] = INT32_MAX;
      lse[c] = INFINITY;   // of a column that counts for nothing
      if (rc < rows) {
        const int qc = kv4_div(rc, p.by_group);
        const float z = __ldg(p.lse + static_cast<int64_t>(u.s.q0 + qc) * p.q_heads +
                              u.head * p.group + rc - qc * p.group);
        // (a row that saw nothing is masked too: its query may hold anything)
        const bool some = z != -INFINITY;
        limit[c] = some ? kv4_limit(u.s, qc, p.causal != 0) : 0;
        if (some) lse[c] = z * 1.44269504088896341f;
      }
    }
    least = __reduce_min_sync(0xffffffffu, limit[0] < limit[1] ? limit[0] : limit[1]);
  };

  int had_b = -1, had_head = -1;   // whose rows the fragments hold, if it has one tile
  int stage = 0;
  for (int left = static_cast<int>(part.count);;) {
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const int tok0 = u.unit * kUnit + warp * kTok;
    if (tok0 < u.s.len) {
      const uint8_t *st = ring + stage * kStage;
      const float *sc = reinterpret_cast<const float *>(st + kCodeBytes);
      const int rows = u.s.qn * p.group;
      // all query rows that see the first of the tokens, and those after
      const int qi0 = p.causal ? tok0 - (u.s.len - u.s.qn) : 0;
      const int first = (qi0 < 0 ? 0 : qi0) * p.group / 8 * 8;
      if (rows <= 8 && (u.b != had_b || u.head != had_head)) {
        queries(0, rows);
        had_b = u.b;
        had_head = u.head;
      }
      float *to = p.sums + (static_cast<int64_t>(u.b) * p.geom.heads + u.head) * p.width + tok0;
      // keys of 16 tokens as A fragments: rows g and g + 8
      auto expand = [&](int row, uint32_t (&kf)[8][4]) {
        const uint4 ka = *reinterpret_cast<const uint4 *>(st + row * 64 + t * 16);
        const uint4 kb = *reinterpret_cast<const uint4 *>(st + (row + 8) * 64 + t * 16);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t ca[4], cb[4];
          codes_f16_word(wa[j], p.magic, ca);
          codes_f16_word(wb[j], p.magic, cb);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            kf[2 * j + k][0] = ca[2 * k];
            kf[2 * j + k][1] = cb[2 * k];
            kf[2 * j + k][2] = ca[2 * k + 1];
            kf[2 * j + k][3] = cb[2 * k + 1];
          }
        }
      };
      // weights of 16 tokens for 8 query rows
      auto weigh = [&](const uint32_t (&kf)[8][4], int row, float s0, float s1, bool mask,
                       float (&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) mma_f16_16816(x, kf[k], qf[2 * k], qf[2 * k + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = exp2_approx(fmaf(x[e], e < 2 ? s0 : s1, -lse[e & 1]));
        if (mask) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (tok0 + row + 8 * (e >> 1) >= limit[e & 1]) x[e] = 0.f;
        }
      };
      auto over_columns = [](float w) {
        w += __shfl_xor_sync(0xffffffffu, w, 1);
        return w + __shfl_xor_sync(0xffffffffu, w, 2);
      };
      // lane (g, t) stores token 8 t + g of 32, v: sums of the tokens 8 i + g
      auto store = [&](int q, const float (&v)[4]) {
        const int tok = q + 8 * t + g;
        float w = t < 2 ? (t == 0 ? v[0] : v[1]) : (t == 2 ? v[2] : v[3]);
        if (p.prev != nullptr) w += sc[kTok + tok];
        if (tok0 + tok < u.s.len) to[tok] = w;
      };
      if (rows <= 8) {   // (without the loop over rows: 64 sequences of 8192 tokens: 77 us with it, 64
                         // without)
        const bool mask = tok0 + kTok > least;
#pragma unroll
        for (int q = 0; q < kTok; q += 32) {
          float v[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = q + 16 * h + g;
            uint32_t kf[8][4];
            expand(row, kf);
            float x[4];
            weigh(kf, row, sc[row] * p.scale_log2, sc[row + 8] * p.scale_log2, mask, x);
            v[2 * h] = over_columns(x[0] + x[1]);
            v[2 * h + 1] = over_columns(x[2] + x[3]);
          }
          store(q, v);
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < kTok; q += 32) {
          float v[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = q + 16 * h + g;
            uint32_t kf[8][4];
            expand(row, kf);
            const float s0 = sc[row] * p.scale_log2, s1 = sc[row + 8] * p.scale_log2;
            // (sums of sums: the rounding of long ones stays small)
            float sum[2] = {0.f, 0.f}, far[2] = {0.f, 0.f};
            for (int r0 = first; r0 < rows; r0 += 8) {
              queries(r0, rows);
              had_b = -1;
              float x[4];
              weigh(kf, row, s0, s1, tok0 + q + 32 > least, x);
              sum[0] += x[0] + x[1];
              sum[1] += x[2] + x[3];
              if (((r0 >> 3) & 31) == 31) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  far[i] += sum[i];
                  sum[i] = 0.f;
                }
              }
            }
            v[2 * h] = over_columns(far[0] + sum[0]);
            v[2 * h + 1] = over_columns(far[1] + sum[1]);
          }
          store(q, v);
        }
      }
    }
    if (--left == 0) break;
    kv4_next_unit(u, p);
    __syncwarp();
    issue(stage);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------ many rows

namespace kv4_wprompt_cfg {
constexpr int kThreads = 448;
constexpr int kLoadWarp = 8;         // .. 11: queries, keys
constexpr int kMmaWarp = 12;
constexpr int kItemWarp = 13;
constexpr int kTok = 128;            // tokens of an item
constexpr int kRows = 128;           // query rows of a tile, at most
constexpr int kStages = 4;           // query tiles in shared memory
constexpr int kLseStages = 16;       // their log-sum-exps
constexpr int kBufs = 3;             // of the product, in TMEM
constexpr int kItems = 4;
constexpr int kItemReaders = 8 + 4 + 1;
constexpr uint32_t kTile = kRows * 256, kHalf = kTile / 2;
constexpr uint32_t kQOff = 1024;
constexpr uint32_t kLseOff = kQOff + kStages * kTile;
constexpr uint32_t kKsOff = kLseOff + kLseStages * kRows * 4;   // [2][128] key scales
constexpr uint32_t kSumOff = kKsOff + 2 * kTok * 4;             // [2][128] sums of half the tiles
constexpr uint32_t kNoneOff = kSumOff + 2 * kTok * 4;   // [kLseStages][4]: of 32 rows each, whether
                                                        // one of the tile counts for nothing
constexpr uint32_t kSmemBytes = kNoneOff + kLseStages * 16 + 1024;   // + alignment slack
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemK = 0, kTmemS = 128;   // 2 x 64 columns of keys, 3 x 128 of products
constexpr uint32_t kIdesc = idesc_f16(128, 128);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
}  // namespace kv4_wprompt_cfg

// Tiles of kTok tokens in the order sequence, tile (the first, which most rows
// see, first), head; taken in turns as the prompt attention's items are.
struct Kv4WItem {
  int b, head, tok0, more;
  int q0, qn, len, row0;   // row0: first row of the first tile of rows
  int tiles;               // of rows
};

__device__ __forceinline__ int64_t kv4_wprompt_weight(const Kv4Seq &s, const Kv4Weights &p) {
  if (static_cast<int64_t>(s.qn) * p.group <= p.few_rows) return 0;
  return static_cast<int64_t>((s.len + kv4_wprompt_cfg::kTok - 1) / kv4_wprompt_cfg::kTok) *
         p.geom.heads;
}

__device__ __forceinline__ Kv4WItem kv4_wprompt_item(const Kv4Weights &p, int &b, int64_t &rest) {
  using namespace kv4_wprompt_cfg;
  Kv4Seq s;
  for (;;) {
    s = kv4_load_seq(p.seqs, b);
    const int64_t w = kv4_wprompt_weight(s, p);
    if (rest < w) break;
    rest -= w;
    ++b;
  }
  Kv4WItem it;
  it.b = b;
  const int at = static_cast<int>(rest / p.geom.heads);
  it.head = static_cast<int>(rest - static_cast<int64_t>(at) * p.geom.heads);
  it.tok0 = at * kTok;
  it.q0 = s.q0;
  it.qn = s.qn;
  it.len = s.len;
  // the first query that sees the first token
  int qi = p.causal ? it.tok0 - (s.len - s.qn) : 0;
  if (qi < 0) qi = 0;
  it.row0 = qi * p.group / p.tile_rows * p.tile_rows;
  it.tiles = (s.qn * p.group - it.row0 + p.tile_rows - 1) / p.tile_rows;
  it.more = 1;
  return it;
}

__global__ void __launch_bounds__(kv4_wprompt_cfg::kThreads, 1)
kv4_weights_prompt_kernel(const __grid_constant__ CUtensorMap q_map,
                          const __grid_constant__ Kv4Weights p) {
  using namespace kv4_wprompt_cfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem);   // [kStages] query tile stored
  uint64_t *q_empty = q_full + kStages;     // [kStages] its product complete
  uint64_t *s_full = q_empty + kStages;     // [kBufs] product complete
  uint64_t *s_empty = s_full + kBufs;       // [kBufs] product read
  uint64_t *k_full = s_empty + kBufs;       // [2] keys in TMEM
  uint64_t *k_empty = k_full + 2;           // [2] last product with them complete, scales read
  uint64_t *sum_full = k_empty + 2;         // [2] second warpgroup's sums stored
  uint64_t *sum_empty = sum_full + 2;       // [2] and read
  uint64_t *item_full = sum_empty + 2;      // [kItems]
  uint64_t *item_empty = item_full + kItems;
  uint64_t *done = item_empty + kItems;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  Kv4WItem *ring = reinterpret_cast<Kv4WItem *>(tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&q_full[i], 4);      // one arrival per warp, here and below (+ the copies' bytes)
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1 + 8);   // the last product, and the scales read
      mbar_init(&sum_full[i], 4);
      mbar_init(&sum_empty[i], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kItemReaders);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // rows of the query tiles that no copy reaches
  for (uint32_t i = threadIdx.x; i < kStages * kTile / 16; i += kThreads)
    st_shared_v4(smem + kQOff + 16 * i, 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  grid_dependency_wait();
  // (not before: a CTA of the kernel before this one, on the same SM, may still be
  // about to allocate, and would wait for a CTA that waits for it)
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  const Kv4Line line = kv4_find_place<kThreads / 32>(
      p.seqs, [&](const Kv4Seq &s) { return kv4_wprompt_weight(s, p); },
      [](const Kv4Seq &) { return 0; },
      [](int64_t total, int64_t) -> int64_t {
        return blockIdx.x < total ? static_cast<int64_t>(blockIdx.x) : -1;
      });
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  auto fail = [&]() {
    report_status(6 /* ATOM_ERR_TIMEOUT */);
    *abort_flag = 1;
  };
  uint32_t item_no = 0;
  auto take_item = [&](Kv4WItem &it) -> bool {
    const int slot = item_no % kItems;
    const bool ok =
        mbar_wait_idle(&item_full[slot], (item_no / kItems) & 1, abort_flag, 64, kItemLooks);
    if (!__all_sync(0xffffffffu, ok)) return false;
    it = ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[slot]);
    ++item_no;
    return true;
  };
  bool ok = true;

  if (warp < 8) {
    // ================================================================ sums
    const int w = warp >> 2;                 // takes every second tile of rows
    const int tid = threadIdx.x & 127;       // token of the item, TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    uint32_t tiles = 0, items = 0;           // so far, over all items
    for (;;) {
      Kv4WItem it;
      if (!(ok = take_item(it)) || !it.more) break;
      const int pos = it.tok0 + tid;
      const bool valid = pos < it.len;
      // first row that sees the token (a prefix times the group can pass 2^31)
      const int first_qi = pos - (it.len - it.qn);
      const int sees = p.causal && first_qi > 0 ? first_qi * p.group : 0;
      ok = mbar_wait_idle(&k_full[items & 1], (items >> 1) & 1, abort_flag, 32);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const float k = reinterpret_cast<const float *>(smem + kKsOff)[(items & 1) * kTok + tid];
      const float2 k2 = make_float2(k, k);
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_empty[items & 1]);
      float sum = 0.f;
      for (int i = (w - tiles) & 1; i < it.tiles; i += 2) {
        const uint32_t no = tiles + i, buf = no % kBufs;
        ok = mbar_wait_spin(&s_full[buf], (no / kBufs) & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after_sync();
        const uint32_t s_addr = tbase + lane_base + kTmemS + kRows * buf;
        const float4 *lse = reinterpret_cast<const float4 *>(smem + kLseOff) +
                            (no % kLseStages) * (kRows / 4);
        const int from = sees - (it.row0 + i * p.tile_rows);   // first column that counts
        // A row that counts for nothing may hold anything (the copy of a sequence's
        // last tile also brings the rows behind it), and a score of NaN minus an
        // infinite log-sum-exp is still NaN. Tiles with such rows, and those with rows
        // that do not see all of the warp's tokens, select, in a short loop over the
        // columns that the tile has: the loop below is the faster for having no
        // selection in it. (Prompt of 4096 tokens 180 us; with the rows before `from`
        // left to the loop below 188, with all selections there 225. Clearing the
        // rows' elements before the product, for which the copy has to land first,
        // took 16 sequences with 32 rows from 45 us to 65.)
        const int4 none = reinterpret_cast<const int4 *>(smem + kNoneOff)[no % kLseStages];
        if (__any_sync(0xffffffffu, from > 0 || (none.x | none.y | none.z | none.w) != 0)) {
          const int rows = it.qn * p.group - (it.row0 + i * p.tile_rows);
          const int columns = rows < p.tile_rows ? rows : p.tile_rows;
          float own[4] = {};
#pragma unroll 1
          for (int c = 0; c < columns; c += 32) {
            uint32_t r[32];
            tmem_ld_x32(s_addr + c, r);
            tmem_ld_wait(r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 z = lse[c / 4 + j];   // (behind `columns` -infinity too)
              const float z4[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float y = fmaf(__uint_as_float(r[4 * j + e]), k, z4[e]);
                own[e] += exp2_approx(c + 4 * j + e < from || z4[e] == -INFINITY ? -INFINITY : y);
              }
            }
          }
          sum += (own[0] + own[1]) + (own[2] + own[3]);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[buf]);
          continue;
        }
        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t raw[2][32];
        tmem_ld_x32(s_addr, raw[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // the next columns are on their way meanwhile
          tmem_ld_wait(raw[c & 1]);
          if (c < 3) {
            tmem_ld_x32(s_addr + 32 * (c + 1), raw[(c + 1) & 1]);
          } else {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[buf]);
          }
          const uint32_t (&r)[32] = raw[c & 1];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 z = lse[8 * c + j];   // negative
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2 y = f2_fma(make_float2(__uint_as_float(r[4 * j + 2 * h]),
                                            __uint_as_float(r[4 * j + 2 * h + 1])),
                                k2, h == 0 ? make_float2(z.x, z.y) : make_float2(z.z, z.w));
              y.x = exp2_approx(y.x);
              y.y = exp2_approx(y.y);
              part[h] = f2_add(part[h], y);
            }
          }
        }
        const float2 both = f2_add(part[0], part[1]);
        sum += both.x + both.y;
      }
      if (!ok) break;
      // ---- the two warpgroups' sums
      float *other = reinterpret_cast<float *>(smem + kSumOff) + (items & 1) * kTok + tid;
      if (w == 1) {
        ok = mbar_wait_idle(&sum_empty[items & 1], ((items >> 1) & 1) ^ 1u, abort_flag, 32);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        *other = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sum_full[items & 1]);
      } else {
        ok = mbar_wait_idle(&sum_full[items & 1], (items >> 1) & 1, abort_flag, 32);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        sum += *other;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sum_empty[items & 1]);
        if (valid) {
          const int64_t at = (static_cast<int64_t>(it.b) * p.geom.heads + it.head) * p.width + pos;
          p.sums[at] = p.prev != nullptr ? p.prev[at] + sum : sum;
        }
      }
      tiles += it.tiles;
      ++items;
    }
    if (!ok && lane == 0) fail();
  } else if (warp < kMmaWarp) {
    // ================================================================ load
    const int lt = threadIdx.x - 32 * kLoadWarp;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    uint32_t tiles = 0, items = 0;
    for (;;) {
      Kv4WItem it;
      if (!(ok = take_item(it)) || !it.more) break;
      // ---- keys: a thread expands a token's vector into its TMEM lane
      {
        const int pos = it.tok0 + lt;
        uint4 q[4] = {};
        float k = 0.f;
        if (pos < it.len) {
          const int page_no = kv4_div(pos, p.geom.by_page);
          const int page = __ldg(p.seqs.table + it.b * p.seqs.table_stride + page_no);
          const int64_t vec = kv4_vector(p.geom, page, pos - page_no * p.geom.page_size, it.head);
          if (vec < 0) {
            report_status(1 /* ATOM_ERR_INVALID_ARG */);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              q[i] = __ldg(reinterpret_cast<const uint4 *>(p.k4 + vec * 64) + i);
            k = __ldg(p.ks + vec) * p.scale_log2;
          }
        }
        ok = mbar_wait_idle(&k_empty[items & 1], ((items >> 1) & 1) ^ 1u, abort_flag, 32);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after_sync();
        const uint32_t k_addr = tbase + lane_base + kTmemK + 64 * (items & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t words[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 c = codes_f16_chunk(words[j], p.magic, true);
            o[4 * j] = c.x;
            o[4 * j + 1] = c.y;
            o[4 * j + 2] = c.z;
            o[4 * j + 3] = c.w;
          }
          tmem_st_x16(k_addr + 16 * i, o);
        }
        reinterpret_cast<float *>(smem + kKsOff)[(items & 1) * kTok + lt] = k;
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[items & 1]);
      }
      // ---- query tiles, and this thread's row's log-sum-exp
      const int rows = it.qn * p.group;
      auto row_lse = [&](int i) -> float {
        const int r = it.row0 + i * p.tile_rows + lt;
        if (i >= it.tiles || lt >= p.tile_rows || r >= rows) return INFINITY;
        const int qi = kv4_div(r, p.by_group);
        const float z = __ldg(p.lse + static_cast<int64_t>(it.q0 + qi) * p.q_heads +
                              it.head * p.group + r - qi * p.group);
        return z == -INFINITY ? INFINITY : z * 1.44269504088896341f;   // one that saw nothing
      };
      float next = row_lse(0);
      for (int i = 0; i < it.tiles; ++i, ++tiles) {
        const uint32_t st = tiles % kStages;
        const float z = next;
        next = row_lse(i + 1);
        ok = mbar_wait_idle(&q_empty[st], ((tiles / kStages) & 1) ^ 1u, abort_flag, 20);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        // (the stage was last read for the tile 16 before, t: the product that freed
        // this tile's stage, of tile t + 12, waited until product t + 9 was read, so
        // the warps that take t's turn are past it)
        reinterpret_cast<float *>(smem + kLseOff)[(tiles % kLseStages) * kRows + lt] = -z;
        const bool some = __any_sync(0xffffffffu, z == INFINITY && lt < p.tile_rows);
        if (lane == 0)
          reinterpret_cast<int *>(smem + kNoneOff)[(tiles % kLseStages) * 4 + (warp & 3)] = some;
        __syncwarp();
        if (lt == 0) {
          mbar_arrive_expect_tx(&q_full[st], p.tile_rows * 256);
          const int tok = it.q0 + kv4_div(it.row0 + i * p.tile_rows, p.by_group);
          for (int h = 0; h < 2; ++h)
            tma_load_3d(smem + kQOff + st * kTile + h * kHalf, &q_map, 64 * h, it.head * p.group,
                        tok, &q_full[st]);
        } else if (lane == 0) {
          mbar_arrive(&q_full[st]);
        }
      }
      if (!ok) break;
      ++items;
    }
    // copies in flight land before shared memory is released
    if (!ok && lt == 0)
      for (uint32_t no = tiles > kStages ? tiles - kStages : 0; no < tiles; ++no)
        (void)mbar_wait(&q_full[no % kStages], (no / kStages) & 1, nullptr);
    if (!ok && lane == 0) fail();
  } else if (warp == kMmaWarp) {
    // ================================================================ MMA issuer
    uint32_t tiles = 0, items = 0;
    const uint32_t q_lo = desc_lo_k(smem_addr(smem + kQOff));
    const bool leader = elect_one();
    for (;;) {
      Kv4WItem it;
      if (!(ok = take_item(it)) || !it.more) break;
      ok = mbar_wait(&k_full[items & 1], (items >> 1) & 1, abort_flag);
      if (it.tiles == 0 && leader) tc_commit(&k_empty[items & 1]);   // no new tokens
      for (int i = 0; ok && i < it.tiles; ++i, ++tiles) {
        const uint32_t st = tiles % kStages, buf = tiles % kBufs;
        ok = mbar_wait(&s_empty[buf], ((tiles / kBufs) & 1) ^ 1u, abort_flag) &&
             mbar_wait(&q_full[st], (tiles / kStages) & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after_sync();
        if (leader) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_f16_ts(tbase + kTmemS + kRows * buf, tbase + kTmemK + 64 * (items & 1) + 8 * k,
                       q_lo + ((st * kTile + (k >> 2) * kHalf + (k & 3) * 32) >> 4), kIdesc,
                       k > 0 ? 1u : 0u);
          tc_commit(&s_full[buf]);
          tc_commit(&q_empty[st]);
          if (i + 1 == it.tiles) tc_commit(&k_empty[items & 1]);
        }
        __syncwarp();
      }
      if (!ok) break;
      ++items;
    }
    if (!ok && lane == 0) fail();
    // nothing may still write TMEM or read shared memory when they are released
    if (leader) tc_commit(done);
    (void)mbar_wait(done, 0, nullptr);
  } else if (threadIdx.x == 32 * kItemWarp) {
    // ================================================================ items
    int b = line.b, turn = 0;
    int64_t place = blockIdx.x, rest = line.rest;
    for (uint32_t made = 0;; ++made) {
      const int slot = made % kItems;
      ok = mbar_wait_idle(&item_empty[slot], ((made / kItems) & 1) ^ 1u, abort_flag, 64, kItemLooks);
      if (!ok) break;
      Kv4WItem it{};
      if (place < line.total) {
        it = kv4_wprompt_item(p, b, rest);
        const int grid = static_cast<int>(gridDim.x), i = static_cast<int>(blockIdx.x);
        const int step = ++turn & 1 ? 2 * (grid - 1 - i) + 1 : 2 * i + 1;
        place += step;
        rest += step;
      }
      ring[slot] = it;
      mbar_arrive(&item_full[slot]);
      if (!it.more) break;
    }
    if (!ok) fail();
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, kTmemCols);
  }
}

}  // namespace atomk
