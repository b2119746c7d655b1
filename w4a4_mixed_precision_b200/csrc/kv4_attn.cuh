// kv4_attn.cuh -- attention of a few query rows a sequence over the paged INT4
// KV cache (single tokens, drafted tokens), without expanding the cache.
//
//   s[r][t] = scale * ks[t] * sum_d q[r][d] kc[t][d]        t < limit(r)
//   out[r]  = sum_t p[r][t] vs[t] vc[t][:] / sum_t p[r][t],  p = exp(s - max s)
//   lse[r]  = log sum_t exp(s[r][t])
//
// kc, vc are the signed 4-bit codes and ks, vs the vectors' scales. A scale
// belongs to a token, which is a row of the products below, so it multiplies a
// score or a weight instead of 128 elements, and the matrix instructions see
// the codes themselves, which fp16 holds exactly.
//
// The weights p * vs go into the second product as fp16 (2^-11 relative, as wide
// as the output's own rounding; nothing else is rounded to 16 bits). vs spans
// what the values spanned, so the scales of each 64 tokens are divided by 2^e, e
// the exponent of their maximum, and a row's reference R is the running maximum
// of (its largest x among them) + e, x = s log2(e): the weight 2^(x + e - R + 4)
// vs 2^-e is then at most 2^15 (R lags by up to 11 before the sums are rescaled)
// whatever the scales are. It keeps fp16's full precision down to 2^-18 of R's
// own, and an absolute error of 2^-29 of the tokens' largest value below. Where a
// row does not see all of the 64 tokens, R follows its largest x + log2 vs
// instead (the weights' bound is the same): with e, a token that the row does not
// see, its value scale 2^28 times the others', left them 2^-24 of themselves,
// fp16's last bit. The sum of weights uses the same reference.
//
// What bounds it: 136 bytes per cached token and KV head (64 + 4 each of keys
// and values) against 4 * 128 * rows operations, far below the tensor cores'
// balance for the tiles of 8 or 16 rows taken here. So the matrix instructions are
// warp-wide mma.sync, whose operands are made in registers from the loaded
// words, with no expanded copy of a tile in shared memory (which a tcgen05
// operand would need: twice the loaded bytes written, then read). It measures
// 4.1 TB/s (64 sequences of up to 8192 tokens, 64 heads over 8: 419 MB in 101 us
// in a replayed graph, 105 to 109 a call). No unit is full: DRAM 50 %, issue slots
// 57 %, ALU 47 %, with the twelve warps an SM that the rings leave room for. A
// warp issues 300 instructions for 16 tokens, half of them turning codes into
// fp16; their chains of dependent steps, three warps to a scheduler, take the time.
//
// The products. M is the side of the tokens (first product) or of the elements
// (second), N is the query rows, 8 per n-tile. A contraction's order is free,
// so the first product takes a vector's elements in the order in which masking
// a word gives pairs (nibbles i and i + 4), and the query's fragments follow
// it; the second takes words of two tokens, exchanges their halves, and the
// same masks give pairs of one element for the two tokens.
//
// The work. A call's units of 256 tokens (kv4_plan.h) are divided evenly over
// all CTAs, whatever the lengths are. A CTA walks its part; the four warps take
// 64 tokens each of a unit through rings of their own in shared memory, filled
// by asynchronous copies that run ahead across the ends of sequences. At the
// end of a tile's share the warps' maxima, sums and outputs are joined. A share
// that is a whole tile is written out; the others go to the workspace, and the
// second kernel joins each tile's shares.
#pragma once

#include "kv4_plan.h"
#include "ptx.cuh"

namespace atomk {

// A nibble n is the code (n ^ 8) - 8. fp16 pairs of nibbles 0 and 4 of w: the
// bits 0x6400 | (n ^ 8) are 1024 + (n ^ 8), exactly, and 1032 is subtracted; of
// nibbles 1 and 5: 0x6400 | 16 (n ^ 8) is 1024 + 16 (n ^ 8), and / 16 - 72 is
// exact. One LOP3 masks and sets the upper bits, if the latter come from a
// register: it takes one immediate. The compiler, which knows constants, makes
// two of it (142 instead of 64 LOP3 per 16 tokens of the decode kernel, on the
// pipe that bounded it), so the two words come with the kernel's arguments.
struct Kv4Magic {
  uint32_t lo, hi;   // 0x64086408, 0x64806480
};
constexpr Kv4Magic kKv4Magic{0x64086408u, 0x64806480u};

struct Kv4Attn {
  const __half *q;
  int64_t q_token, q_head;      // strides in elements
  __half *out;                  // [rows][q_heads][128]
  float *lse;                   // [rows][q_heads], or null
  const uint8_t *k4, *v4;
  const float *ks, *vs;
  Kv4Geom geom;
  Kv4Seqs seqs;
  int q_heads, group;
  Kv4Div by_group;
  int tile_rows;                // query rows of a prompt tile: whole tokens' rows, up to 128
  float scale_log2;             // scale * log2(e)
  int causal;
  int max_q;                    // largest qn of the call, as its caller says
  int few_rows;                 // sequences of up to so many rows a KV head go to the decode
                                // kernel, the others to the prompt kernel
  int split;                    // tiles may be shared between CTAs
  int whole;                    // 64 tokens that begin at a multiple of 64 share a page
  float *ws;                    // the shares (kv4_decode_cfg)
  Kv4Magic magic;
};

// Reference of a row that has seen nothing.
constexpr float kKv4NoMax = -1e30f;
// Weights are raised by 2^kKv4Raise over the reference, which may lag by
// 2^kKv4Lag behind the largest.
constexpr float kKv4Raise = 4.f, kKv4Lag = 11.f;

// Exponent e of a positive number's (its bits): the number < 2^e; and 2^-e. Not
// below that of the smallest value scale but 0, 2^-24 / 7: references and sums stay
// near 1, and a log-sum-exp, their two logarithms' sum, keeps its last bits (0.5 of
// its bound where half of the values are zero; with -60 it passed that).
constexpr int kKv4LeastExponent = -26;
__device__ __forceinline__ int kv4_exponent(uint32_t bits) {
  const int e = static_cast<int>(bits >> 23) - 126;
  return e < kKv4LeastExponent ? kKv4LeastExponent : (e > 100 ? 100 : e);
}
__device__ __forceinline__ float kv4_down(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// log2 of a value scale that has been multiplied by 2^-e, at least `least`: with e
// not below the least exponent, as e itself is not, and with any e not below -100
// (the weights are summed in units of 2^e: a token's is then below 2^115).
__device__ __forceinline__ float kv4_level(float scaled, float least) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(scaled));
  return fmaxf(y, least);
}
__device__ __forceinline__ float kv4_least_level(float e) {
  return fmaxf(kKv4LeastExponent - e, -100.f);
}

namespace kv4_decode_cfg {
constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kTok = 64;        // tokens per warp and stage
constexpr int kStages = 2;
constexpr uint32_t kCodeBytes = kTok * 64;
constexpr uint32_t kStage = 2 * kCodeBytes + 2 * kTok * 4;   // keys, values, their scales
constexpr uint32_t kRing = kStages * kStage;                 // per warp
constexpr int kORow = 132;      // floats of an output row in shared memory
constexpr uint32_t kSmemBytes = kWarps * kRing;
// The warps' shares of a tile are joined in the stages that its last unit left.
static_assert(8 * 2 * (kORow + 2) * 4 <= kStage, "a share of 16 rows fits a stage");
// Workspace: for each CTA two slots of 8 nt rows (128 outputs, maximum, sum),
// then a descriptor {first CTA, sequence, head, tile} of the tile that ends in
// it and began in an earlier CTA (first CTA = -1: none).
__host__ __device__ constexpr int64_t slot_floats(int nt) { return 8 * nt * 130; }
constexpr int64_t ws_bytes(int ctas, int nt) {
  return ctas * (2 * slot_floats(nt) * 4 + 16);
}
static_assert(kWarps * kTok == kKv4Unit, "a unit is one stage of every warp");
}  // namespace kv4_decode_cfg

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_4z(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// D (16 x 8, fp32) += A (16 x 16) * B (16 x 8).
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held as mma fragments.
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t codes_f16_lo(uint32_t w, const Kv4Magic &c) {
  const uint32_t m = (w & 0x000F000Fu) ^ c.lo;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&m),
                            __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408)));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t w, const Kv4Magic &c) {
  const uint32_t m = (w & 0x00F000F0u) ^ c.hi;
  const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&m),
                            __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00)),
                            __halves2half2(__ushort_as_half(0xD480), __ushort_as_half(0xD480)));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// The four pairs of a word: nibbles (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ void codes_f16_word(uint32_t w, const Kv4Magic &c, uint32_t (&o)[4]) {
  const uint32_t w8 = w >> 8;
  o[0] = codes_f16_lo(w, c);
  o[1] = codes_f16_hi(w, c);
  o[2] = codes_f16_lo(w8, c);
  o[3] = codes_f16_hi(w8, c);
}

// Query fragments (B operand) of 8 query rows for codes_f16_word's order: lane
// (g, t) holds row g's elements 32t .. 32t + 31.
__device__ __forceinline__ void kv4_query_fragments(const __half *row, int t, bool valid,
                                                    uint32_t (&b)[16]) {
  const uint4 *src = reinterpret_cast<const uint4 *>(row + 32 * t);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 x = valid ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
    // elements 8j + {0,1} {2,3} {4,5} {6,7}
    b[4 * j + 0] = __byte_perm(x.x, x.z, 0x5410);   // 0, 4
    b[4 * j + 1] = __byte_perm(x.x, x.z, 0x7632);   // 1, 5
    b[4 * j + 2] = __byte_perm(x.y, x.w, 0x5410);   // 2, 6
    b[4 * j + 3] = __byte_perm(x.y, x.w, 0x7632);   // 3, 7
  }
}

__device__ __forceinline__ Kv4Seq kv4_load_seq(const Kv4Seqs &q, int b) {
  return kv4_seq_of(__ldg(q.cu_q + b), __ldg(q.cu_q + b + 1), __ldg(q.kv_lens + b), q.rows,
                    q.capacity);
}

// A place on the line on which sequence b takes weight(b) places: the line's
// length, the sequence and the places into it (b = -1: no place was asked for).
struct Kv4Line {
  int64_t total, rest;
  int b;
};

// Finds place_of(total, tiles) (negative: none), `tiles` the sum of tiles_of.
// Every thread of the CTA calls it; each sums a run of the sequences.
template <int kWarps, class Weight, class Tiles, class Place>
__device__ __forceinline__ Kv4Line kv4_find_place(const Kv4Seqs &seqs, const Weight &weight_of,
                                                  const Tiles &tiles_of, const Place &place_of) {
  __shared__ int64_t warp_sums[kWarps], warp_tiles[kWarps];
  __shared__ int64_t found_rest;
  __shared__ int found_b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = (seqs.batch + 32 * kWarps - 1) / (32 * kWarps);
  const int64_t run_lo = static_cast<int64_t>(threadIdx.x) * run;
  const int b_lo = run_lo < seqs.batch ? static_cast<int>(run_lo) : seqs.batch;
  const int b_hi = seqs.batch - b_lo < run ? seqs.batch : b_lo + run;
  int64_t mine = 0, tiles = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Kv4Seq s = kv4_load_seq(seqs, b);
    if (!s.ok && blockIdx.x == 0) report_status(1 /* ATOM_ERR_INVALID_ARG */);
    mine += weight_of(s);
    tiles += tiles_of(s);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, d);
  if (lane == 0) warp_tiles[warp] = tiles;
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  Kv4Line line{0, 0, -1};
  tiles = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += warp_sums[w];
    line.total += warp_sums[w];
    tiles += warp_tiles[w];
  }
  const int64_t place = place_of(line.total, tiles);   // the same for the whole CTA
  if (place < 0) return line;
  if (place >= upto - mine && place < upto) {
    int64_t rest = place - (upto - mine);
    for (int b = b_lo; b < b_hi; ++b) {
      const int64_t w = weight_of(kv4_load_seq(seqs, b));
      if (rest < w) {
        found_b = b;
        found_rest = rest;
        break;
      }
      rest -= w;
    }
  }
  __syncthreads();
  line.b = found_b;
  line.rest = found_rest;
  return line;
}

// This CTA's part of the line: where it begins and how many places it has.
struct Kv4Part {
  int64_t total, begin, count, rest;
  int parts, b;
};

template <int kWarps, class Weight, class Tiles>
__device__ __forceinline__ Kv4Part kv4_find_part(const Kv4Seqs &seqs, const Weight &weight_of,
                                                 const Tiles &tiles_of) {
  Kv4Part part{};
  const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  const Kv4Line line = kv4_find_place<kWarps>(seqs, weight_of, tiles_of, [&](int64_t total,
                                                                             int64_t tiles) -> int64_t {
    part.parts = kv4_parts(total, tiles, ctas);
    if (cta >= part.parts) return -1;
    part.begin = kv4_part_begin(total, part.parts, cta);
    part.count = kv4_part_begin(total, part.parts, cta + 1) - part.begin;
    return part.begin;
  });
  part.total = line.total;
  part.b = line.b;
  part.rest = line.rest;
  return part;
}

// A place on the line of units (kv4_plan.h), with its sequence's facts.
struct Kv4Walk {
  int b, head, tile, unit;
  int tiles, units;
  Kv4Seq s;
};

// Whether a sequence has more new tokens than the call allows: it is skipped.
__device__ __forceinline__ bool kv4_too_many(const Kv4Seq &s, const Kv4Attn &p) {
  if (s.qn <= p.max_q) return false;
  if (blockIdx.x == 0) report_status(1 /* ATOM_ERR_INVALID_ARG */);
  return true;
}
// Tiles per head of a sequence that this kernel takes: one with few query rows.
__device__ __forceinline__ int kv4_own_tiles(const Kv4Seq &s, const Kv4Attn &p, int tile) {
  if (kv4_too_many(s, p) || static_cast<int64_t>(s.qn) * p.group > p.few_rows) return 0;
  return kv4_tiles(s, p.group, tile);
}

template <int NT>
__device__ __forceinline__ void kv4_enter_sequence(Kv4Walk &w, const Kv4Attn &p) {
  for (; w.b < p.seqs.batch; ++w.b) {
    w.s = kv4_load_seq(p.seqs, w.b);
    w.tiles = kv4_own_tiles(w.s, p, 8 * NT);
    w.units = kv4_units(w.s.len);
    if (w.tiles > 0) return;
  }
}
template <int NT>
__device__ __forceinline__ void kv4_next_tile(Kv4Walk &w, const Kv4Attn &p) {
  w.unit = 0;
  if (++w.tile < w.tiles) return;
  w.tile = 0;
  if (++w.head < p.geom.heads) return;
  w.head = 0;
  ++w.b;
  kv4_enter_sequence<NT>(w, p);
}
// Cached positions that the rows of the walk's tile see between them.
template <int NT>
__device__ __forceinline__ int kv4_tile_end(const Kv4Walk &w, const Kv4Attn &p) {
  int last = (w.tile + 1) * 8 * NT - 1;
  const int rows = w.s.qn * p.group;
  if (last >= rows) last = rows - 1;
  return kv4_limit(w.s, last / p.group, p.causal != 0);
}

// Elements [d, d + 8) of an output row from their sums, and (with d = 0) the
// row's log-sum-exp. A row that saw nothing has sum 0: zeros and -infinity.
__device__ __forceinline__ void kv4_write_row(const Kv4Attn &p, int64_t row, int d,
                                              const float (&acc)[8], float top, float sum) {
  const float inv = sum > 0.f ? __fdiv_rn(exp2_approx(-kKv4Raise), sum) : 0.f;
  *reinterpret_cast<uint4 *>(p.out + row * 128 + d) =
      make_uint4(pack_half2_rn(acc[0] * inv, acc[1] * inv), pack_half2_rn(acc[2] * inv, acc[3] * inv),
                 pack_half2_rn(acc[4] * inv, acc[5] * inv), pack_half2_rn(acc[6] * inv, acc[7] * inv));
  if (d == 0 && p.lse != nullptr)
    p.lse[row] = sum > 0.f ? (top + log2f(sum)) * 0.693147180559945309f : -INFINITY;
}

template <int NT>
__global__ void __launch_bounds__(kv4_decode_cfg::kThreads, NT == 1 ? 3 : 2)
kv4_decode_kernel(const __grid_constant__ Kv4Attn p) {
  using namespace kv4_decode_cfg;
  constexpr int R = 8 * NT;
  extern __shared__ __align__(16) uint8_t kv4_smem[];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cta = static_cast<int>(blockIdx.x);
  launch_dependents();
  grid_dependency_wait();

  // ---- this CTA's part of the line
  auto tiles = [&](const Kv4Seq &q) -> int64_t {
    return static_cast<int64_t>(kv4_own_tiles(q, p, R)) * p.geom.heads;
  };
  auto weight = [&](const Kv4Seq &q) -> int64_t {
    return tiles(q) * (p.split ? kv4_units(q.len) : 1);
  };
  const Kv4Part part = kv4_find_part<kWarps>(p.seqs, weight, tiles);
  int *desc = p.split ? reinterpret_cast<int *>(p.ws + gridDim.x * 2 * slot_floats(NT)) + 4 * cta
                      : nullptr;
  if (part.count == 0) {
    if (desc != nullptr && threadIdx.x == 0) desc[0] = -1;
    return;
  }
  int64_t left = part.count;   // units, or tiles if not split

  Kv4Walk cw;   // what is computed
  cw.b = part.b;
  cw.head = cw.tile = cw.unit = 0;
  kv4_enter_sequence<NT>(cw, p);
  {
    const int64_t per_tile = p.split ? cw.units : 1, per_head = per_tile * cw.tiles;
    int64_t rest = part.rest;
    cw.head = static_cast<int>(rest / per_head);
    rest -= cw.head * per_head;
    cw.tile = static_cast<int>(rest / per_tile);
    cw.unit = static_cast<int>(rest - cw.tile * per_tile);
  }

  // ---- the copies: they run kStages units ahead of the arithmetic
  Kv4Walk lw = cw;
  int64_t to_load = left;
  int l_end = kv4_tile_end<NT>(lw, p);
  uint8_t *ring = kv4_smem + warp * kRing;
  const uint32_t ring_addr = smem_addr(ring);
  // Lane (g, t) copies chunk t of the tokens g, g + 8, ... Token i of 16 (bits
  // k t1 t0 j) of the values goes to row (k t1 j t0), chunks exchanged by t1: the
  // 8-byte loads below then meet no bank twice.
  const uint32_t k_dst = ring_addr + lane * 16;
  const uint32_t v_dst = ring_addr + kCodeBytes +
                         (((g & ~3) | ((g & 1) << 1) | ((g >> 1) & 1)) << 6) + ((t ^ ((g >> 1) & 2)) << 4);
  const uint32_t s_dst = ring_addr + 2 * kCodeBytes + lane * 4;
  const int64_t lane_scale = static_cast<int64_t>(lane) * p.geom.token_stride;
  const int64_t lane_code = static_cast<int64_t>(g) * p.geom.token_stride * 64 + t * 16;
  const int64_t step = static_cast<int64_t>(p.geom.token_stride) * 512;
  int page_no, page;   // of the next stage's first token (whole)
  auto fetch_page = [&]() {
    const int pos = lw.unit * kKv4Unit + warp * kTok;
    page_no = kv4_div(pos, p.geom.by_page);
    page = pos < l_end ? __ldg(p.seqs.table + lw.b * p.seqs.table_stride + page_no) : -1;
  };
  if (p.whole) fetch_page();
  auto issue = [&](int stage) {
    if (to_load > 0) {
      const int pos0 = lw.unit * kKv4Unit + warp * kTok;
      const uint32_t at = stage * kStage;
      if (pos0 >= l_end) {
        // nothing of this warp's share is seen
      } else if (p.whole) {
        // the stage's tokens are in one page
        int n = l_end - pos0;
        int64_t vec = kv4_vector(p.geom, page, pos0 - page_no * p.geom.page_size, lw.head);
        if (vec < 0) {
          report_status(1 /* ATOM_ERR_INVALID_ARG */);
          vec = 0;
          n = 0;
        }
#pragma unroll
        for (int i = 0; i < kTok; i += 32) {
          const bool is = i + lane < n;
          const int64_t scale =
              vec + (is ? lane_scale + static_cast<int64_t>(i) * p.geom.token_stride : 0);
          cp_async_4z(s_dst + at + i * 4, p.ks + scale, is ? 4u : 0u);
          cp_async_4z(s_dst + at + (kTok + i) * 4, p.vs + scale, is ? 4u : 0u);
        }
        const uint8_t *kp = p.k4 + lane_code + vec * 64, *vp = p.v4 + lane_code + vec * 64;
        if (n >= kTok) {
#pragma unroll
          for (int i = 0; i < kTok / 8; ++i) {
            cp_async_16(k_dst + at + i * 512, kp, 16u);
            cp_async_16(v_dst + at + i * 512, vp, 16u);
            kp += step;
            vp += step;
          }
        } else {
#pragma unroll
          for (int i = 0; i < kTok / 8; ++i) {
            const bool is = 8 * i + g < n;
            cp_async_16(k_dst + at + i * 512, is ? kp + i * step : p.k4, is ? 16u : 0u);
            cp_async_16(v_dst + at + i * 512, is ? vp + i * step : p.v4, is ? 16u : 0u);
          }
        }
      } else {
        for (int j = 0; j < kTok; j += 32) {
          const int pos = pos0 + j + lane;
          int64_t vec = -1;
          if (pos < l_end) {
            const int no = kv4_div(pos, p.geom.by_page);
            vec = kv4_vector(p.geom, __ldg(p.seqs.table + lw.b * p.seqs.table_stride + no),
                             pos - no * p.geom.page_size, lw.head);
            if (vec < 0) report_status(1 /* ATOM_ERR_INVALID_ARG */);
          }
          const int64_t safe = vec < 0 ? 0 : vec;
          cp_async_4z(s_dst + at + j * 4, p.ks + safe, vec < 0 ? 0u : 4u);
          cp_async_4z(s_dst + at + (kTok + j) * 4, p.vs + safe, vec < 0 ? 0u : 4u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t v = __shfl_sync(0xffffffffu, vec, 8 * i + g);
            const int64_t off = (v < 0 ? 0 : v) * 64 + t * 16;
            const uint32_t bytes = v < 0 ? 0u : 16u;
            cp_async_16(k_dst + at + j * 64 + i * 512, p.k4 + off, bytes);
            cp_async_16(v_dst + at + j * 64 + i * 512, p.v4 + off, bytes);
          }
        }
      }
      const bool last = lw.unit + 1 >= lw.units;
      if (p.split || last) --to_load;
      if (to_load > 0) {
        if (last) {
          kv4_next_tile<NT>(lw, p);
          l_end = kv4_tile_end<NT>(lw, p);
        } else {
          ++lw.unit;
        }
        if (p.whole) fetch_page();
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) issue(s);

  int stage = 0;
  int4 ended = make_int4(-1, 0, 0, 0);   // descriptor: the tile that ends here and began earlier
  while (left > 0) {
    // ---- one tile's share: units [cw.unit, cw.unit + count)
    const bool starts = cw.unit == 0;
    int count = cw.units - cw.unit;
    if (p.split && count > left) count = static_cast<int>(left);
    const bool ends = cw.unit + count == cw.units;
    const int end = kv4_tile_end<NT>(cw, p);
    const int rows = cw.s.qn * p.group, row0 = cw.tile * R;

    uint32_t qf[NT][16];
    int limit[NT][2];       // of this lane's two columns (query rows) of each n-tile
    float m[NT][2], l[NT][2], o[NT][8][4];
    int least = end;        // every row sees the positions before it
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + 8 * n + g;
      const bool valid = r < rows;
      const int qi = valid ? r / p.group : 0, head = cw.head * p.group + (valid ? r - qi * p.group : 0);
      kv4_query_fragments(p.q + (cw.s.q0 + qi) * p.q_token + head * p.q_head, t, valid, qf[n]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rc = row0 + 8 * n + 2 * t + c;
        limit[n][c] = rc < rows ? kv4_limit(cw.s, rc / p.group, p.causal != 0) : 0;
        if (rc < rows && limit[n][c] < least) least = limit[n][c];
        m[n][c] = kKv4NoMax;
        l[n][c] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    }

    for (int u = 0; u < count; ++u) {
      const int tok0 = (cw.unit + u) * kKv4Unit + warp * kTok;
      cp_async_wait<kStages - 1>();
      __syncwarp();
      if (tok0 < end) {
        const uint8_t *st = ring + stage * kStage;
        const float *sc = reinterpret_cast<const float *>(st + 2 * kCodeBytes);
        // scores of 64 tokens: rows g and g + 8 of four times 16
        float x[NT][kTok / 16][4];
#pragma unroll
        for (int h = 0; h < kTok / 16; ++h) {
          const uint4 ka = *reinterpret_cast<const uint4 *>(st + (16 * h + g) * 64 + t * 16);
          const uint4 kb = *reinterpret_cast<const uint4 *>(st + (16 * h + g + 8) * 64 + t * 16);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][h][e] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t ca[4], cb[4];
            codes_f16_word(wa[j], p.magic, ca);
            codes_f16_word(wb[j], p.magic, cb);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {ca[2 * k], cb[2 * k], ca[2 * k + 1], cb[2 * k + 1]};
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16_16816(x[n][h], a, qf[n][4 * j + 2 * k], qf[n][4 * j + 2 * k + 1]);
            }
          }
          const float s0 = sc[16 * h + g] * p.scale_log2, s1 = sc[16 * h + g + 8] * p.scale_log2;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            x[n][h][0] *= s0;
            x[n][h][1] *= s0;
            x[n][h][2] *= s1;
            x[n][h][3] *= s1;
          }
        }
        const int e = kv4_exponent(__reduce_max_sync(
            0xffffffffu, __float_as_uint(fmaxf(sc[kTok + lane], sc[kTok + 32 + lane]))));
        const float ef = static_cast<float>(e), down = kv4_down(e);
        // what the references of the columns follow
        float mx[NT][2];
        if (__any_sync(0xffffffffu, tok0 + kTok > least)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY;
          const float least_level = kv4_least_level(ef);
#pragma unroll
          for (int h = 0; h < kTok / 16; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int row = 16 * h + 8 * k + g;
              const float level = kv4_level(sc[kTok + row] * down, least_level);
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  if (tok0 + row >= limit[n][c]) x[n][h][2 * k + c] = -INFINITY;
                  mx[n][c] = fmaxf(mx[n][c], x[n][h][2 * k + c] + level);
                }
            }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float v = fmaxf(x[n][0][c], x[n][0][c + 2]);
#pragma unroll
              for (int h = 1; h < kTok / 16; ++h) v = max3(v, x[n][h][c], x[n][h][c + 2]);
              mx[n][c] = v;
            }
        }
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = mx[n][c];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            mx[n][c] = v + ef;
            rise |= mx[n][c] > m[n][c] + kKv4Lag;
          }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float top = fmaxf(m[n][c], mx[n][c]);
              const float f = exp2_approx(m[n][c] - top);
              m[n][c] = top;
              l[n][c] *= f;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                o[n][i][c] *= f;
                o[n][i][c + 2] *= f;
              }
            }
        }
        // weights in their references, in the units 2^(e + kKv4Raise)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float add[2] = {ef + kKv4Raise - m[n][0], ef + kKv4Raise - m[n][1]};
#pragma unroll
          for (int h = 0; h < kTok / 16; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][h][i] = exp2_approx(x[n][h][i] + add[i & 1]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float step = 0.f;
#pragma unroll
            for (int h = 0; h < kTok / 16; ++h) step += x[n][h][c] + x[n][h][c + 2];
            l[n][c] = fmaf(step, exp2_approx(-ef - kKv4Raise), l[n][c]);
          }
        }
        const uint8_t *vt = st + kCodeBytes + (4 * (t >> 1) + (t & 1)) * 64 +
                            (((g >> 1) ^ (t & 2)) << 4) + ((g & 1) << 3);
#pragma unroll
        for (int h = 0; h < kTok / 16; ++h) {
          const float v0 = sc[kTok + 16 * h + g] * down, v1 = sc[kTok + 16 * h + g + 8] * down;
          // weights times value scales, as B operands
          uint32_t wf[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            wf[n][0] = movmatrix(pack_half2_rn(x[n][h][0] * v0, x[n][h][1] * v0));
            wf[n][1] = movmatrix(pack_half2_rn(x[n][h][2] * v1, x[n][h][3] * v1));
          }
          // values: two words (16 elements) of the tokens 2t, 2t+1, 2t+8, 2t+9
          uint2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = *reinterpret_cast<const uint2 *>(vt + h * 1024 + (i >> 1) * 512 + (i & 1) * 128);
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // word i / 2, its lower or upper half
            const bool up = (i & 1) != 0;
            const uint32_t a0 = i < 2 ? v[0].x : v[0].y, a1 = i < 2 ? v[1].x : v[1].y;
            const uint32_t a2 = i < 2 ? v[2].x : v[2].y, a3 = i < 2 ? v[3].x : v[3].y;
            uint32_t ab[4], cd[4];   // elements 4i .. 4i + 3 of two tokens each
            codes_f16_word(__byte_perm(a0, a1, up ? 0x7632 : 0x5410), p.magic, ab);
            codes_f16_word(__byte_perm(a2, a3, up ? 0x7632 : 0x5410), p.magic, cd);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {ab[2 * k], ab[2 * k + 1], cd[2 * k], cd[2 * k + 1]};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16_16816(o[n][2 * i + k], a, wf[n][0], wf[n][1]);
            }
          }
        }
      }
      __syncwarp();
      if (u + 1 < count) {
        issue(stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
      }
    }

    // ---- join the warps' shares, each in the stage that it left last
    float *share = reinterpret_cast<float *>(kv4_smem + warp * kRing + stage * kStage);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[n][c];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int r = 8 * n + 2 * t + c;
        if (g == 0) {
          share[R * kORow + 2 * r] = m[n][c];
          share[R * kORow + 2 * r + 1] = sum;
        }
        // o[n][i][c], o[n][i][c + 2]: elements 16 g + 2 i, + 1
        float *dst = share + r * kORow + 16 * g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4 *>(dst + 4 * i) =
              make_float4(o[n][2 * i][c], o[n][2 * i][c + 2], o[n][2 * i + 1][c],
                          o[n][2 * i + 1][c + 2]);
      }
    __syncthreads();
    auto share_of = [&](int w) {
      return reinterpret_cast<const float *>(kv4_smem + w * kRing + stage * kStage);
    };
    const bool whole = starts && ends;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + static_cast<int>(threadIdx.x >> 4), d = (threadIdx.x & 15) * 8;
      float top = kKv4NoMax;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, share_of(w)[R * kORow + 2 * r]);
      float sum = 0.f, acc[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float *theirs = share_of(w);
        const float f = exp2_approx(theirs[R * kORow + 2 * r] - top);
        sum += f * theirs[R * kORow + 2 * r + 1];
        const float *src = theirs + r * kORow + d;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f * src[e];
      }
      if (row0 + r >= rows) continue;
      if (whole) {
        const int qi = (row0 + r) / p.group, head = cw.head * p.group + row0 + r - qi * p.group;
        kv4_write_row(p, static_cast<int64_t>(cw.s.q0 + qi) * p.q_heads + head, d, acc, top, sum);
      } else {
        float *slot = p.ws + (2 * static_cast<int64_t>(cta) + (starts ? 1 : 0)) * slot_floats(NT);
        *reinterpret_cast<float4 *>(slot + r * 128 + d) =
            make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4 *>(slot + r * 128 + d + 4) =
            make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (d == 0) *reinterpret_cast<float2 *>(slot + R * 128 + 2 * r) = make_float2(top, sum);
      }
    }
    if (ends && !starts && threadIdx.x == 0)   // only the first share of a part can
      ended = make_int4(kv4_part_of(part.total, part.parts, part.begin - cw.unit), cw.b, cw.head, cw.tile);
    left -= p.split ? count : 1;
    if (left > 0) {
      __syncthreads();   // the shares have been read
      issue(stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      kv4_next_tile<NT>(cw, p);
    }
  }
  if (desc != nullptr && threadIdx.x == 0) *reinterpret_cast<int4 *>(desc) = ended;
}

// Joins the shares of the tile that ends in CTA blockIdx.x and began earlier:
// slot 2i+1 of the CTA where it begins, slots 2i of the others.
constexpr int kKv4JoinThreads = 512;

template <int NT>
__global__ void __launch_bounds__(kKv4JoinThreads) kv4_join_kernel(const __grid_constant__ Kv4Attn p) {
  using namespace kv4_decode_cfg;
  constexpr int R = 8 * NT;
  constexpr int kTeams = kKv4JoinThreads / 128;   // each takes every kTeams-th share
  __shared__ float part[kTeams][R][132];
  __shared__ float part_ml[kTeams][R][2];
  grid_dependency_wait();
  const int cta = static_cast<int>(blockIdx.x);
  const int4 desc = *reinterpret_cast<const int4 *>(
      reinterpret_cast<const int *>(p.ws + gridDim.x * 2 * slot_floats(NT)) + 4 * cta);
  if (desc.x < 0) return;
  const int first = desc.x, shares = cta - first + 1;
  const Kv4Seq s = kv4_load_seq(p.seqs, desc.y);
  const int rows = s.qn * p.group, row0 = desc.w * R;
  auto slot_of = [&](int i) {
    return p.ws + (2 * static_cast<int64_t>(first + i) + (i == 0 ? 1 : 0)) * slot_floats(NT);
  };
  const int team = static_cast<int>(threadIdx.x >> 7), tid = threadIdx.x & 127;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = 8 * n + (tid >> 4), d = (tid & 15) * 8;
    float top = kKv4NoMax, sum = 0.f, acc[8] = {};
    if (row0 + r < rows) {
#pragma unroll 4
      for (int i = team; i < shares; i += kTeams) {
        const float *slot = slot_of(i);
        const float2 ml = *reinterpret_cast<const float2 *>(slot + R * 128 + 2 * r);
        const float4 a = *reinterpret_cast<const float4 *>(slot + r * 128 + d);
        const float4 b = *reinterpret_cast<const float4 *>(slot + r * 128 + d + 4);
        const float up = fmaxf(top, ml.x);
        const float f = exp2_approx(top - up), fi = exp2_approx(ml.x - up);
        top = up;
        sum = sum * f + ml.y * fi;
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = acc[e] * f + v[e] * fi;
      }
    }
    if ((tid & 15) == 0) {
      part_ml[team][r][0] = top;
      part_ml[team][r][1] = sum;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[team][r][d + e] = acc[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < R * 16; i += kKv4JoinThreads) {
    const int r = i >> 4, d = (i & 15) * 8;
    if (row0 + r >= rows) continue;
    float top = kKv4NoMax;
#pragma unroll
    for (int w = 0; w < kTeams; ++w) top = fmaxf(top, part_ml[w][r][0]);
    float sum = 0.f, acc[8] = {};
#pragma unroll
    for (int w = 0; w < kTeams; ++w) {
      const float f = exp2_approx(part_ml[w][r][0] - top);
      sum += f * part_ml[w][r][1];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f * part[w][r][d + e];
    }
    const int qi = (row0 + r) / p.group, head = desc.z * p.group + row0 + r - qi * p.group;
    kv4_write_row(p, static_cast<int64_t>(s.q0 + qi) * p.q_heads + head, d, acc, top, sum);
  }
}

}  // namespace atomk
