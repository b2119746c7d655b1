// kv4_prompt.cuh -- attention of many query rows a sequence (prompts, chunks of
// prompts) over the paged INT4 KV cache, on the tcgen05 tensor cores. The
// formulas are kv4_attn.cuh's.
//
// A CTA takes up to 256 query rows of a (sequence, KV head) as two tiles of 128
// (of as many whole tokens' rows as fit: a tile is one box of a tensor copy), and
// the cached tokens that they see in tiles of 64. Per KV tile and query tile:
//   S = Q K^T     128x64x128, fp16 codes of K from shared memory, fp32 S in TMEM
//   W = 2^(x - R) * vs, x = S * ks * scale * log2(e)   (one thread a row; fp16, into TMEM
//                                                       over S)
//   O += W V      128x128x64, W from TMEM, codes of V from shared memory
// S has two buffers a query tile, so that the scores of the next KV tile are
// there when a row's weights are done (with tiles of 128 tokens TMEM, 512
// columns, has room for one, and the softmax waited for the tensor core).
// The codes are exact in fp16 and every scale belongs to a token, that is to a
// column of S and W, so it multiplies there, in fp32. What is rounded to 16 bits
// is W alone (2^-11 relative, as wide as the output's own rounding; an exact sum
// of two halves would cost half as many matrix instructions again).
//
// The references R and the exponents e of the value scales are kv4_attn.cuh's.
// (One row of 32 that outgrows R costs its warp the wait for the output so far:
// with a lag of 2^4 two warps in five did so in every tile of the 4096-token
// prompt, with 2^8 one in ten, with 2^11 one in fifty.)
//
// Roles (640 threads, one CTA per SM, a persistent loop over the work):
//   warps 0..3, 4..7     softmax of query tile 0 and 1: thread = row = TMEM lane
//   warps 8..11, 12..15  load packed keys and values, expand them to operand tiles
//   warps 16, 17         issue the MMAs of query tile 0 and 1
//   warp 18, lane 0      finds the work items, starts the copies of their queries
// While the tensor core multiplies for one query tile, the other tile's weights
// are made. A prompt of 4096 tokens, 64 heads over 8, takes 321 us in a replayed
// graph (856 TFLOP/s), 329 to 340 a call. What bounds it (parts left out in
// copies, of then 334 us): of the clocks of a KV tile and two query tiles, some
// 2200, the tensor core works 1776 (74 for each instruction of S, 16 x 128 x 64,
// which its operands' way out of shared memory costs, and 74 for each of O), the
// exponential unit 1056, and the issue slots are half full. With nearly all
// products left out it takes 6 per cent less, with the exponentials left out 15:
// it is the softmax warps' own chain, two of them on each scheduler, that takes
// the time (alone, a tile's scores take a warp 250 clocks and its weights 630;
// two warps together 1370). What was tried against it and was not faster: four
// softmax warps a scheduler with half the columns each (394 us for the 4096-token
// prompt against 340), weights before the tile's own maximum is known (476), the
// two warps taking turns at the exponentials (337 against 334), the next tile's
// scores read ahead (356 against 334).
//
// Operand layouts. K and V tiles are 64 rows (tokens) of 256 bytes as two
// halves of 128-byte rows with the 128-byte swizzle: for S they are a K-major B
// operand, for O an MN-major one. A word of 8 codes becomes one 16-byte chunk:
// of keys in its own order, as the queries are copied; of values in the order
// 0 4 1 5 2 6 3 7 that masking gives, which the epilogue undoes.
#pragma once

#include "kv4_attn.cuh"

namespace atomk {

namespace kv4_prompt_cfg {
constexpr int kThreads = 640;
constexpr int kMmaWarp = 16;         // and 17: one for each query tile
constexpr int kQWarp = 18;
constexpr int kItems = 4;            // ring of work items
constexpr int kItemReaders = 8 + 8 + 2 + 1;   // softmax, expanding, MMA warps, queries
// registers: 144 * 256 + 64 * 256 + 64 * 128 = 96 * 640, what the launch has
constexpr int kSoftRegs = 144, kExpandRegs = 64, kOtherRegs = 64;
constexpr int kTok = 64;             // tokens of a KV tile
constexpr int kStages = 4;           // of key and of value tiles
constexpr int kScStages = 8;         // of their scales
constexpr uint32_t kQTile = 128 * 256, kQHalf = kQTile / 2;   // fp16 operand tiles
constexpr uint32_t kTile = kTok * 256, kHalf = kTile / 2;
constexpr uint32_t kQOff = 1024;
constexpr uint32_t kKOff = kQOff + 2 * kQTile;
constexpr uint32_t kVOff = kKOff + kStages * kTile;
constexpr uint32_t kScOff = kVOff + kStages * kTile;   // ks, vs of a tile's tokens, 2 exponents,
constexpr uint32_t kScStage = 3 * kTok * 4 + 16;       // log2 of the vs
constexpr uint32_t kOutOff = kScOff + kScStages * kScStage;      // 2 KB for each softmax warp
constexpr uint32_t kSmemBytes = kOutOff + 8 * 2048 + 1024;   // + alignment slack
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0, kTmemO = 256;       // + 128 * query tile; S + 64 * (tile & 1)
constexpr uint32_t kIdescS = idesc_f16(128, kTok);
constexpr uint32_t kIdescO = idesc_f16(128, 128) | (1u << 16);   // B is MN-major
constexpr float kRaise = kKv4Raise, kLag = kKv4Lag;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
}  // namespace kv4_prompt_cfg

// 32 lanes x 32 columns of TMEM.
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               :
               : "memory");
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Operand descriptors of tiles of 128-byte rows with the 128-byte swizzle, as
// their lower words; the upper one is the same for all: 1024 bytes between
// groups of 8 rows, descriptor version 1 (sm_100), swizzle mode 2. Kept in
// halves, and joined where they are used, they cost the issuing thread one
// register each. K-major: rows are MN, 64 elements of K in a row. MN-major: rows
// are K, and blocks of 64 MN elements are `lbo` bytes apart.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo_k(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (1u << 16);
}
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

// What the items of the persistent loops wait for can be as long as an item takes
// (one of a cache of 2^26 tokens some seconds) or as finding one among many idle
// sequences: 32 times the other waits' limit. A role that gives up ends them too.
constexpr uint32_t kItemLooks = 32 * kWaitLooks;

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// D (+)= A * B, fp16 with an fp32 accumulator, A and B in shared memory.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}
// The same with A (fp16 pairs, one row a lane) in TMEM.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

// A word of codes as a 16-byte chunk: in the order 0 4 1 5 2 6 3 7 that masking
// gives, or in its own.
__device__ __forceinline__ uint4 codes_f16_chunk(uint32_t w, const Kv4Magic &magic, bool in_order) {
  uint32_t o[4];
  codes_f16_word(w, magic, o);
  if (!in_order) return make_uint4(o[0], o[1], o[2], o[3]);
  return make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                    __byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632));
}

// The items of the persistent loop: pairs of query tiles in the order sequence,
// pair (the last, which sees most, first), head. Of each `grid` places in turn
// CTA i takes the i-th, of every second turn the i-th from the end, so that
// large and small items meet in a CTA. One thread finds them and hands them on
// through a ring in shared memory.
struct Kv4Item {
  int b, head, row0, rows;   // rows: query rows of the sequence and head
  int kv_tiles, last;        // KV tiles and cached positions that the tile's rows see
  int q0, qn, len, more;     // more = 0: no item, the end
};

__device__ __forceinline__ int64_t kv4_prompt_weight(const Kv4Seq &s, const Kv4Attn &p) {
  if (kv4_too_many(s, p) || static_cast<int64_t>(s.qn) * p.group <= p.few_rows) return 0;
  return static_cast<int64_t>(kv4_tiles(s, p.group, 2 * p.tile_rows)) * p.geom.heads;
}

// The item `rest` places into sequence b; both move on to the sequence that
// holds it.
__device__ __forceinline__ Kv4Item kv4_prompt_item(const Kv4Attn &p, int &b, int64_t &rest) {
  using namespace kv4_prompt_cfg;
  Kv4Seq s;
  for (;;) {
    s = kv4_load_seq(p.seqs, b);
    const int64_t w = kv4_prompt_weight(s, p);
    if (rest < w) break;
    rest -= w;
    ++b;
  }
  Kv4Item it;
  it.b = b;
  it.rows = s.qn * p.group;
  const int item_rows = 2 * p.tile_rows, tiles = kv4_tiles(s, p.group, item_rows);
  const int at = static_cast<int>(rest / p.geom.heads);
  it.head = static_cast<int>(rest - static_cast<int64_t>(at) * p.geom.heads);
  it.row0 = (tiles - 1 - at) * item_rows;
  const int last_row = (it.rows - it.row0 > item_rows ? it.row0 + item_rows : it.rows) - 1;
  it.last = kv4_limit(s, last_row / p.group, p.causal != 0);
  it.kv_tiles = (it.last + kTok - 1) / kTok;
  it.q0 = s.q0;
  it.qn = s.qn;
  it.len = s.len;
  it.more = 1;
  return it;
}

// A row's scores of a KV tile in the exponent's units (x, -infinity where the
// row does not see), and what the reference follows: the largest of each 32
// tokens plus their e, or (kMask) the largest x + log2 vs, to which tokens that
// the row does not see add nothing. `sc`, in shared memory: ks, vs (scaled by
// 2^-e), the e's, one per 32 tokens, and kv4_level of the vs. (A tile of 64 also keeps this code, unrolled, short enough for the
// instruction caches beside that of the other roles; at 128 columns half of the
// softmax's time went into waiting for instructions.)
template <bool kMask>
__device__ __forceinline__ float kv4_row_scores(uint32_t s_addr, const float4 *sc, int seen,
                                                float2 (&x)[32]) {
  using namespace kv4_prompt_cfg;
  uint32_t raw[2][32];
  tmem_ld_x32(s_addr, raw[0]);
  tmem_ld_x32(s_addr + 32, raw[1]);
  const float2 e = *reinterpret_cast<const float2 *>(sc + 2 * kTok / 4);
  tmem_ld_wait(raw[0]);
  tmem_ld_wait(raw[1]);
  float mx = -INFINITY;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 k = sc[8 * c + i];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t *r = &raw[c][4 * i + 2 * h];
        float2 y = f2_mul(make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])),
                          h == 0 ? make_float2(k.x, k.y) : make_float2(k.z, k.w));
        if (kMask) {
          const int left = seen - 32 * c - 4 * i - 2 * h;
          if (left <= 0) y.x = -INFINITY;
          if (left <= 1) y.y = -INFINITY;
        }
        x[16 * c + 2 * i + h] = y;
        if (kMask) {
          const float4 v = sc[2 * kTok / 4 + 1 + 8 * c + i];
          y = f2_add(y, h == 0 ? make_float2(v.x, v.y) : make_float2(v.z, v.w));
        }
        m4[2 * (i & 1) + h] = max3(m4[2 * (i & 1) + h], y.x, y.y);
      }
    }
    mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) + (c == 0 ? e.x : e.y));
  }
  return mx;
}

// Weights in the reference `top`, times the value scales, as fp16 pairs over the
// scores; returns their sum.
__device__ __forceinline__ float kv4_row_weights(uint32_t s_addr, const float4 *sc, float top,
                                                 const float2 (&x)[32]) {
  using namespace kv4_prompt_cfg;
  const float2 e = *reinterpret_cast<const float2 *>(sc + 2 * kTok / 4);
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float ec = c == 0 ? e.x : e.y, add = ec + kRaise - top;
    const float2 add2 = make_float2(add, add);
    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t packed[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = sc[kTok / 4 + 8 * c + i];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 y = f2_add(x[16 * c + 2 * i + h], add2);
        y.x = exp2_approx(y.x);
        y.y = exp2_approx(y.y);
        part[h] = f2_add(part[h], y);
        y = f2_mul(y, h == 0 ? make_float2(v.x, v.y) : make_float2(v.z, v.w));
        packed[2 * i + h] = pack_half2_rn(y.x, y.y);
      }
    }
    tmem_st_x16(s_addr + 16 * c, packed);
    const float2 both = f2_add(part[0], part[1]);
    sum = fmaf(both.x + both.y, exp2_approx(-ec - kRaise), sum);
  }
  return sum;
}

__global__ void __launch_bounds__(kv4_prompt_cfg::kThreads, 1)
kv4_prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ Kv4Attn p) {
  using namespace kv4_prompt_cfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem);   // [2] query tile stored
  uint64_t *q_empty = q_full + 2;   // [2] its last product complete
  uint64_t *s_full = q_empty + 2;   // [2][2] S of the query tile (and buffer) complete
  uint64_t *p_full = s_full + 4;    // [2][2] W stored over S (and O rescaled)
  uint64_t *o_full = p_full + 4;    // [2][2] W V complete
  uint64_t *k_full = o_full + 4;    // [kStages] key tile expanded
  uint64_t *k_empty = k_full + kStages;   // [kStages] both products with it complete
  uint64_t *v_full = k_empty + kStages;
  uint64_t *v_empty = v_full + kStages;
  uint64_t *item_full = v_empty + kStages;   // [kItems]
  uint64_t *item_empty = item_full + kItems; // [kItems] read by every role
  uint64_t *done = item_empty + kItems;      // [2]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 2);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  Kv4Item *ring = reinterpret_cast<Kv4Item *>(tmem_slot + 2);   // [kItems]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);     // + the copies' bytes
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&o_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);   // one arrival per warp, here and below
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&k_full[i], 2);
      mbar_init(&k_empty[i], 2);
      mbar_init(&v_full[i], 2);
      mbar_init(&v_empty[i], 2);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kItemReaders);
    }
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // rows of the query tiles that no copy reaches
  for (uint32_t i = threadIdx.x; i < 2 * kQTile / 16; i += kThreads)
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
      p.seqs, [&](const Kv4Seq &s) { return kv4_prompt_weight(s, p); },
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
  // The next item for a warp, in turn; false: a wait gave up.
  uint32_t item_no = 0;
  auto take_item = [&](Kv4Item &it) -> bool {
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

  if (warp < 8) {
    // ================================================================ softmax
    regs_increase<kSoftRegs>();
    const int w = warp >> 2;                     // query tile
    const int tid = threadIdx.x & 127;           // row of it, TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_base = tbase + lane_base + kTmemS + 128 * w;
    const uint32_t o_addr = tbase + lane_base + kTmemO + 128 * w;
    uint32_t tiles = 0;                          // KV tiles so far, over all items
    bool ok = true;
    // The output of the no-th tile. (Two barriers, as S has two buffers: the
    // scores of a tile are complete after the output of the tile two before, so
    // that a parity names one phase.)
    auto o_wait = [&](uint32_t no) {
      return mbar_wait_spin(&o_full[2 * w + (no & 1)], (no >> 1) & 1, abort_flag);
    };
    for (;;) {
      Kv4Item it;
      if (!(ok = take_item(it)) || !it.more) break;
      const int r = it.row0 + p.tile_rows * w + tid;
      const bool valid = tid < p.tile_rows && r < it.rows;
      const int qi = valid ? kv4_div(r, p.by_group) : 0;
      const int hq = it.head * p.group + (valid ? r - qi * p.group : 0);
      // (a row that is none computes on what the copy brought, or on the zeros
      // that the tile began with, and is not written)
      const int limit =
          valid ? kv4_limit(Kv4Seq{it.q0, it.qn, it.len, true}, qi, p.causal != 0) : INT32_MAX;
      const int n = it.kv_tiles;
      float top = kKv4NoMax, sum = 0.f;
      for (int j = 0; j < n; ++j, ++tiles) {
        const uint32_t buf = tiles & 1, s_addr = s_base + 64 * buf;
        ok = mbar_wait_spin(&s_full[2 * w + buf], (tiles >> 1) & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after_sync();
        const float4 *sc = reinterpret_cast<const float4 *>(smem + kScOff + (tiles % kScStages) * kScStage);
        const int seen = limit - j * kTok;   // columns of this tile that the row sees
        const bool mask = __any_sync(0xffffffffu, seen < kTok);
        float2 x[32];
        const float mx = mask ? kv4_row_scores<true>(s_addr, sc, seen, x)
                              : kv4_row_scores<false>(s_addr, sc, seen, x);
        if (__any_sync(0xffffffffu, mx > top + kLag)) {
          const float up = fmaxf(top, mx);
          const float f = exp2_approx(top - up);
          top = up;
          sum *= f;
          if (j > 0) {   // the output so far, in the new reference
            ok = o_wait(tiles - 1);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld_x16(o_addr + 16 * c, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st_x16(o_addr + 16 * c, o);
            }
          }
        }
        sum += kv4_row_weights(s_addr, sc, top, x);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * w + buf]);
      }
      if (!ok) break;
      // ---- the rows' outputs
      const int64_t row = static_cast<int64_t>(it.q0 + qi) * p.q_heads + hq;
      const float inv = sum > 0.f ? __fdiv_rn(exp2_approx(-kRaise), sum) : 0.f;
      if (n > 0) {
        ok = o_wait(tiles - 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after_sync();
      }
      // 32 columns at a time through shared memory, so that four lanes write 64
      // bytes of a row together
      uint8_t *stage = smem + kOutOff + warp * 2048;
      const int64_t my_row = valid ? row : -1;
      auto write = [&](const uint32_t (&o)[32], int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // 8 columns, in the order 0 4 1 5 2 6 3 7
          float2 y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[k] = make_float2(__uint_as_float(o[8 * i + 2 * k]), __uint_as_float(o[8 * i + 2 * k + 1]));
            y[k] = n > 0 ? f2_fma(y[k], make_float2(inv, inv), make_float2(0.f, 0.f))
                         : make_float2(0.f, 0.f);
          }
          st_shared_v4(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4),
                       pack_half2_rn(y[0].x, y[1].x), pack_half2_rn(y[2].x, y[3].x),
                       pack_half2_rn(y[0].y, y[1].y), pack_half2_rn(y[2].y, y[3].y));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int src = 8 * i + (lane >> 2), ch = lane & 3;
          const int64_t to = __shfl_sync(0xffffffffu, my_row, src);
          const uint4 v = *reinterpret_cast<const uint4 *>(stage + src * 64 +
                                                           ((ch ^ ((src >> 1) & 3)) << 4));
          if (to >= 0) *reinterpret_cast<uint4 *>(p.out + to * 128 + 32 * c + 8 * ch) = v;
        }
        __syncwarp();
      };
      // (each 32 columns are read while those before them are written)
      uint32_t o[2][32];
      tmem_ld_x32(o_addr, o[0]);
      tmem_ld_wait(o[0]);
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        tmem_ld_x32(o_addr + 32 * c + 32, o[1]);
        write(o[0], c);
        tmem_ld_wait(o[1]);
        tmem_ld_x32(o_addr + (32 * c + 64) % 128, o[0]);
        write(o[1], c + 1);
        tmem_ld_wait(o[0]);
      }
      if (valid && p.lse != nullptr)
        p.lse[row] = sum > 0.f ? (top + log2f(sum)) * 0.693147180559945309f : -INFINITY;
      tc_fence_before_sync();
    }
    if (!ok && lane == 0) fail();
  } else if (warp < 16) {
    // ================================================================ expand
    regs_decrease<kExpandRegs>();
    const bool value = warp >= 12;   // warps 8..11 keys, 12..15 values;
    const int turn = (warp >> 1) & 1, ew = warp & 1;   // two warps a tile, in turn
    const int g = lane >> 2, t = lane & 3;
    const uint8_t *codes = value ? p.v4 : p.k4;
    const float *scales = value ? p.vs : p.ks;
    uint64_t *full = value ? v_full : k_full, *empty = value ? v_empty : k_empty;
    uint8_t *tile0 = smem + (value ? kVOff : kKOff);
    uint32_t tiles = 0;
    bool ok = true;
    for (;;) {
      Kv4Item it;
      if (!(ok = take_item(it)) || !it.more) break;
      const int n = it.kv_tiles;
      const int32_t *table = p.seqs.table + it.b * p.seqs.table_stride;
      int page_no = 0, page = -1;      // of the token whose address is made next
      auto fetch_page = [&](int j) {
        const int pos = j * kTok + 32 * ew + lane;
        page_no = kv4_div(pos, p.geom.by_page);
        page = pos < it.last ? __ldg(table + page_no) : -1;
      };
      uint4 q[4];
      float scale = 0.f;
      auto load = [&](int j) {
        const int pos = j * kTok + 32 * ew + lane;
        int64_t vec = -1;
        scale = 0.f;
        if (pos < it.last) {
          vec = kv4_vector(p.geom, page, pos - page_no * p.geom.page_size, it.head);
          if (vec < 0)
            report_status(1 /* ATOM_ERR_INVALID_ARG */);
          else
            scale = __ldg(scales + vec);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // chunk t of token 8i + g
          const int64_t v = __shfl_sync(0xffffffffu, vec, 8 * i + g);
          q[i] = make_uint4(0u, 0u, 0u, 0u);
          if (v >= 0) q[i] = __ldg(reinterpret_cast<const uint4 *>(codes + v * 64 + t * 16));
        }
      };
      const int first = (turn - tiles) & 1;   // of the item's tiles, for these warps
      if (first < n) {
        fetch_page(first);
        load(first);
        if (first + 2 < n) fetch_page(first + 2);
      }
      for (int j = first; j < n; j += 2) {
        const uint32_t no = tiles + j, st = no % kStages;
        ok = mbar_wait_idle(&empty[st], ((no / kStages) & 1) ^ 1u, abort_flag, 64);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        // scales of this warp's 32 tokens, those of the values divided by 2^e
        // (a stage of scales was last read for the tile eight before, whose weights
        // were complete before the product that freed this operand stage began)
        float *sc = reinterpret_cast<float *>(smem + kScOff + (no % kScStages) * kScStage);
        if (value) {
          const uint32_t largest = __reduce_max_sync(0xffffffffu, __float_as_uint(scale));
          const int e = kv4_exponent(largest);
          const float ef = static_cast<float>(e), scaled = scale * kv4_down(e);
          sc[kTok + 32 * ew + lane] = scaled;
          sc[2 * kTok + 4 + 32 * ew + lane] = kv4_level(scaled, kv4_least_level(ef));
          if (lane == 0) sc[2 * kTok + ew] = ef;
        } else {
          sc[32 * ew + lane] = scale * p.scale_log2;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 32 * ew + 8 * i + g;
          uint8_t *dst = tile0 + st * kTile + (t >> 1) * kHalf + row * 128;
          const uint32_t words[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 c = codes_f16_chunk(words[k], p.magic, !value);
            st_shared_v4(dst + (((4 * (t & 1) + k) ^ (row & 7)) << 4), c.x, c.y, c.z, c.w);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        if (j + 2 < n) {
          load(j + 2);
          if (j + 4 < n) fetch_page(j + 4);
        }
      }
      if (!ok) break;
      tiles += n;
    }
    if (!ok && lane == 0) fail();
  } else {
    regs_decrease<kOtherRegs>();
    if (warp >= kQWarp) {
      // ============================================================== queries
      // Finds the items and starts the copy of each query tile as soon as the
      // last product with the previous one is complete.
      if (warp == kQWarp && lane == 0) {
        int b = line.b, turn = 0;
        int64_t place = blockIdx.x, rest = line.rest;
        uint32_t started[2] = {0, 0};
        bool ok = true;
        const uint32_t bytes = p.tile_rows * 256;
        for (uint32_t made = 0;; ++made) {
          const int slot = made % kItems;
          ok = mbar_wait_idle(&item_empty[slot], ((made / kItems) & 1) ^ 1u, abort_flag, 64, kItemLooks);
          if (!ok) break;
          Kv4Item it{};
          if (place < line.total) {
            it = kv4_prompt_item(p, b, rest);
            const int grid = static_cast<int>(gridDim.x), i = static_cast<int>(blockIdx.x);
            const int step = ++turn & 1 ? 2 * (grid - 1 - i) + 1 : 2 * i + 1;
            place += step;
            rest += step;
          }
          ring[slot] = it;
          mbar_arrive(&item_full[slot]);
          mbar_arrive(&item_empty[slot]);   // as one of its readers
          if (!it.more) break;
          if (it.kv_tiles == 0) continue;
          ok = kv4_start_queries(
              started,
              [&](int w, uint32_t parity) {
                return mbar_wait_idle(&q_empty[w], parity, abort_flag, 32, kItemLooks);
              },
              [&](int w) {
                mbar_arrive_expect_tx(&q_full[w], bytes);
                const int tok = it.q0 + kv4_div(it.row0 + p.tile_rows * w, p.by_group);
                for (int h = 0; h < 2; ++h)
                  tma_load_3d(smem + kQOff + w * kQTile + h * kQHalf, &q_map, 64 * h,
                              it.head * p.group, tok, &q_full[w]);
              });
          if (!ok) break;
        }
        if (!ok) {
          fail();
          // copies in flight land before shared memory is released
          kv4_drain_queries(started, [&](int w, uint32_t parity) {
            (void)mbar_wait(&q_full[w], parity, nullptr);
          });
        }
      }
    } else {
      // ============================================================== MMA issuer
      uint32_t tiles = 0, items = 0;
      bool ok = true;
      const uint32_t q_lo = desc_lo_k(smem_addr(smem + kQOff));
      const uint32_t k_lo = desc_lo_k(smem_addr(smem + kKOff));
      const uint32_t v_lo = desc_lo_mn(smem_addr(smem + kVOff), kHalf);
      // The warp stays together and one lane issues: the operands' descriptors
      // are then known to be the same for the whole warp.
      const bool leader = elect_one();
      const int w = warp - kMmaWarp;
      const uint32_t s_tmem = tbase + kTmemS + 128 * w, o_tmem = tbase + kTmemO + 128 * w;
      for (;;) {
        Kv4Item it;
        if (!(ok = take_item(it)) || !it.more) break;
        const int n = it.kv_tiles;
        if (n == 0) continue;
        ok = mbar_wait(&q_full[w], items & 1, abort_flag);
        // step j: the output of tile j - 2, when its weights are there, then S of
        // tile j in the buffer that they leave
        for (int j = 0; ok && j < n + 2; ++j) {
          const uint32_t no = tiles + j, st = no % kStages, s_buf = s_tmem + 64 * (no & 1);
          if (j >= 2) {
            const uint32_t old = no - 2, ost = old % kStages;
            ok = mbar_wait(&p_full[2 * w + (old & 1)], (old >> 1) & 1, abort_flag);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
              for (int k = 0; k < kTok / 16; ++k)
                mma_f16_ts(o_tmem, s_buf + 8 * k, v_lo + ((ost * kTile + k * 2048) >> 4), kIdescO,
                           j > 2 || k > 0 ? 1u : 0u);
              tc_commit(&o_full[2 * w + (old & 1)]);
              tc_commit(&v_empty[ost]);
            }
            __syncwarp();
          }
          if (j < n) {
            // (the values' scales are needed as soon as the scores are there)
            ok = mbar_wait(&k_full[st], (no / kStages) & 1, abort_flag) &&
                 mbar_wait(&v_full[st], (no / kStages) & 1, abort_flag);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_f16_ss(s_buf, q_lo + ((w * kQTile + (k >> 2) * kQHalf + (k & 3) * 32) >> 4),
                           k_lo + ((st * kTile + (k >> 2) * kHalf + (k & 3) * 32) >> 4), kIdescS,
                           k > 0 ? 1u : 0u);
              tc_commit(&s_full[2 * w + (no & 1)]);
              tc_commit(&k_empty[st]);
              if (j + 1 == n) tc_commit(&q_empty[w]);
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        tiles += n;
        ++items;
      }
      if (!ok && lane == 0) fail();
      // nothing may still write TMEM or read shared memory when they are released
      if (leader) tc_commit(&done[w]);
      (void)mbar_wait(&done[w], 0, nullptr);
    }
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, kTmemCols);
  }
}

}  // namespace atomk
