// kv4_prompt.cuh -- attention of many query rows a sequence (prompts, chunks of
// prompts) over the paged INT4 KV cache, on the tcgen05 tensor cores. The
// formulas are kv4_attn.cuh's.
//
// A CTA takes 256 query rows of a (sequence, KV head) as two tiles of 128, and
// the cached tokens that they see in tiles of 128. Per KV tile and query tile:
//   S = Q K^T     128x128x128, fp16 codes of K from shared memory, fp32 S in TMEM
//   W = 2^(x - R) * vs, x = S * ks * scale * log2(e)   (one thread a row; fp16, into TMEM
//                                                       over S)
//   O += W V      128x128x128, W from TMEM, codes of V from shared memory
// The codes are exact in fp16 and every scale belongs to a token, that is to a
// column of S and W, so it multiplies there, in fp32. What is rounded to 16 bits
// is W alone (2^-11 relative, as wide as the output's own rounding; an exact sum
// of two halves would cost half as many matrix instructions again).
//
// The range of W. vs spans what the values spanned, so each KV tile's scales are
// divided by 2^e, e the exponent of their maximum, and a row's reference R is
// the running maximum of (row maximum of x in the tile) + e: the largest W of a
// tile is then at most 2^15 (R lags by up to 4 before the output is rescaled,
// W is raised by 2^11) whatever the scales are, and W keeps fp16's full
// precision down to 2^-25 of that and an absolute error of 2^-36 of the tile's
// largest value below. The sum of weights uses the same reference.
//
// Roles (512 threads, one CTA per SM, a persistent loop over the work):
//   warps 0..3, 4..7   softmax of query tile 0 and 1: thread = row = TMEM lane
//   warps 8..11        load packed tiles, expand them to fp16 operand tiles
//   warp 12, lane 0    issues the MMAs
// While the tensor core multiplies for one query tile, the other tile's
// weights are made. What bounds it: the exponentials, 16 per clock and SM (1024
// clocks per 128x128 tile), as much as the two products (1024 clocks).
//
// Operand layouts. K and V tiles are 128 rows (tokens) of 256 bytes as two
// halves of 128-byte rows with the 128-byte swizzle: for S they are a K-major B
// operand, for O an MN-major one. A word of 8 codes becomes one 16-byte chunk
// in the order 0 4 1 5 2 6 3 7 that masking gives; Q's chunks are stored in the
// same order, and the epilogue undoes it for the output's columns.
#pragma once

#include "kv4_attn.cuh"

namespace atomk {

namespace kv4_prompt_cfg {
constexpr int kThreads = 512;
constexpr int kRows = 256;           // query rows of a CTA's work item
constexpr int kTok = 128;            // tokens of a KV tile
constexpr uint32_t kTile = 128 * 256;    // an fp16 operand tile
constexpr uint32_t kHalf = kTile / 2;
constexpr uint32_t kQOff = 1024;
constexpr uint32_t kKOff = kQOff + 2 * kTile;
constexpr uint32_t kVOff = kKOff + 2 * kTile;
constexpr uint32_t kScOff = kVOff + 2 * kTile;     // 4 stages: ks, vs of 128 tokens, exponent
constexpr uint32_t kScStage = 2 * kTok * 4 + 16;
constexpr uint32_t kSmemBytes = kScOff + 4 * kScStage + 1024;   // + alignment slack
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0, kTmemO = 256;       // + 128 * query tile
constexpr uint32_t kIdescS = idesc_f16(128, 128);
constexpr uint32_t kIdescO = idesc_f16(128, 128) | (1u << 16);   // B is MN-major
constexpr float kRaise = 11.f, kLag = 4.f;
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
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
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

// 16 bytes from shared memory, in program order with the TMEM accesses (loads
// that the compiler moves together do not fit in the softmax's registers).
__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// D += A * B with A (fp16) in TMEM.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of an MN-major tile stored as K rows of 128 bytes (64 elements of
// MN) with the 128-byte swizzle: `lbo` bytes between blocks of 64 MN elements,
// `sbo` between groups of 8 K rows.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lbo >> 4) << 16;
  d |= static_cast<uint64_t>(sbo >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;   // descriptor version (sm_100)
  d |= static_cast<uint64_t>(2) << 61;   // 128-byte swizzle
  return d;
}

__device__ __forceinline__ float2 f2_mul(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
  return d;
}
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
  return d;
}

// A word of codes as a 16-byte chunk, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 codes_f16_chunk(uint32_t w) {
  uint32_t o[4];
  codes_f16_word(w, o);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The items of the persistent loop: query tiles of kRows rows in the order
// sequence, tile (the last, which sees most, first), head. CTA i takes places
// i, i + grid, ...
struct Kv4Item {
  int b, head, row0, rows, kv_tiles;   // rows: query rows of the sequence and head
  int64_t place, rest;
  Kv4Seq s;
};

__device__ __forceinline__ int64_t kv4_prompt_weight(const Kv4Seq &s, const Kv4Attn &p) {
  if (kv4_too_many(s, p) || static_cast<int64_t>(s.qn) * p.group <= p.few_rows) return 0;
  return static_cast<int64_t>(kv4_tiles(s, p.group, kv4_prompt_cfg::kRows)) * p.geom.heads;
}

// The item at `rest` places into sequence it.b.
__device__ __forceinline__ void kv4_prompt_locate(Kv4Item &it, const Kv4Attn &p) {
  using namespace kv4_prompt_cfg;
  for (;;) {
    it.s = kv4_load_seq(p.seqs, it.b);
    const int64_t w = kv4_prompt_weight(it.s, p);
    if (it.rest < w) break;
    it.rest -= w;
    ++it.b;
  }
  it.rows = it.s.qn * p.group;
  const int tiles = kv4_tiles(it.s, p.group, kRows);
  const int at = static_cast<int>(it.rest / p.geom.heads);
  it.head = static_cast<int>(it.rest - static_cast<int64_t>(at) * p.geom.heads);
  it.row0 = (tiles - 1 - at) * kRows;
  const int last = (it.row0 + kRows < it.rows ? it.row0 + kRows : it.rows) - 1;
  it.kv_tiles = (kv4_limit(it.s, last / p.group, p.causal != 0) + kTok - 1) / kTok;
}

__global__ void __launch_bounds__(kv4_prompt_cfg::kThreads, 1)
kv4_prompt_kernel(const __grid_constant__ Kv4Attn p) {
  using namespace kv4_prompt_cfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem);   // [2] query tile stored
  uint64_t *s_full = q_full + 2;    // [2] S of the query tile complete
  uint64_t *p_full = s_full + 2;    // [2] W stored over S (and O rescaled)
  uint64_t *o_full = p_full + 2;    // [2] W V complete
  uint64_t *k_full = o_full + 2;    // [2] key tile expanded
  uint64_t *k_empty = k_full + 2;   // [2] both products with it complete
  uint64_t *v_full = k_empty + 2;
  uint64_t *v_empty = v_full + 2;
  uint64_t *done = v_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint32_t *tile_max = tmem_slot + 4;   // [2][4] largest value scale of each expanding warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  const Kv4Line line = kv4_find_place<kThreads / 32>(
      p.seqs, [&](const Kv4Seq &s) { return kv4_prompt_weight(s, p); },
      [](int64_t total) -> int64_t { return blockIdx.x < total ? static_cast<int64_t>(blockIdx.x) : -1; });
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  auto fail = [&]() {
    report_status(6 /* ATOM_ERR_TIMEOUT */);
    *abort_flag = 1;
  };
  Kv4Item it;
  it.place = blockIdx.x;
  it.b = line.b;
  it.rest = line.rest;
  auto next_item = [&]() {
    it.place += gridDim.x;
    it.rest += gridDim.x;
  };

  if (warp < 8) {
    // ================================================================ softmax
    const int w = warp >> 2;                     // query tile
    const int tid = threadIdx.x & 127;           // row of it, TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_addr = tbase + lane_base + kTmemS + 128 * w;
    const uint32_t o_addr = tbase + lane_base + kTmemO + 128 * w;
    uint32_t tiles = 0;                          // KV tiles so far, over all items
    bool ok = true;
    for (; ok && it.place < line.total; next_item()) {
      kv4_prompt_locate(it, p);
      const int r = it.row0 + 128 * w + tid;
      const bool valid = r < it.rows;
      const int qi = valid ? r / p.group : 0;
      const int hq = it.head * p.group + (valid ? r - qi * p.group : 0);
      const int limit = valid ? kv4_limit(it.s, qi, p.causal != 0) : 0;
      const int n = it.kv_tiles;
      float top = kKv4NoMax, sum = 0.f;
      if (n > 0) {
        // ---- this row of Q, in the codes' order
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (it.s.q0 + qi) * p.q_token +
                                                           hq * p.q_head);
        uint8_t *dst = smem + kQOff + w * kTile + tid * 128;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint4 x = valid ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
          st_shared_v4(dst + (c >> 3) * kHalf + (((c & 7) ^ (tid & 7)) << 4),
                       __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                       __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_full[w]);
      }
      for (int j = 0; j < n; ++j, ++tiles) {
        if (!__all_sync(0xffffffffu, mbar_wait_inline(&s_full[w], tiles & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint8_t *sc = smem + kScOff + (tiles & 3) * kScStage;
        const uint32_t ks = smem_addr(sc), vs = ks + kTok * 4;
        const float e = *reinterpret_cast<const float *>(sc + 2 * kTok * 4);
        float4 kq;
        const int seen = limit - j * kTok;   // columns of this tile that the row sees
        const bool mask = __any_sync(0xffffffffu, seen < kTok);
        // ---- first pass over S: the maximum. (S is read again below: 128
        // scores a thread do not fit beside the rest of its registers.)
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t raw[32];
          tmem_ld_x32(s_addr + 32 * c, raw);
          tmem_ld_wait(raw);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 k;
            if ((i & 1) == 0) kq = ld_shared_v4(ks + 16 * (8 * c + i / 2));
            k = (i & 1) == 0 ? make_float2(kq.x, kq.y) : make_float2(kq.z, kq.w);
            float2 x = f2_mul(
                make_float2(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1])), k);
            if (mask) {
              if (32 * c + 2 * i >= seen) x.x = -INFINITY;
              if (32 * c + 2 * i + 1 >= seen) x.y = -INFINITY;
            }
            m4[i & 3] = fmaxf(m4[i & 3], fmaxf(x.x, x.y));
          }
        }
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        if (__any_sync(0xffffffffu, mx + e > top + kLag)) {
          const float up = fmaxf(top, mx + e);
          const float f = exp2_approx(top - up);
          top = up;
          sum *= f;
          if (j > 0) {   // the output so far, in the new reference
            if (!__all_sync(0xffffffffu, mbar_wait_inline(&o_full[w], (tiles - 1) & 1, abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
#pragma unroll
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
        const float add = e + kRaise - top;
        const float2 add2 = make_float2(add, add);
        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // ---- second pass: weights, their sum, and W over S (columns 16c .. of W
        // are columns 32c .. of S, which has been read by then)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t raw[32], packed[16];
          tmem_ld_x32(s_addr + 32 * c, raw);
          tmem_ld_wait(raw);
          float4 v;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const bool even = (i & 1) == 0;
            if (even) {
              kq = ld_shared_v4(ks + 16 * (8 * c + i / 2));
              v = ld_shared_v4(vs + 16 * (8 * c + i / 2));
            }
            float2 y = f2_fma(
                make_float2(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1])),
                even ? make_float2(kq.x, kq.y) : make_float2(kq.z, kq.w), add2);
            y.x = exp2_approx(y.x);
            y.y = exp2_approx(y.y);
            if (mask) {
              if (32 * c + 2 * i >= seen) y.x = 0.f;
              if (32 * c + 2 * i + 1 >= seen) y.y = 0.f;
            }
            part[i & 1] = f2_add(part[i & 1], y);
            y = f2_mul(y, even ? make_float2(v.x, v.y) : make_float2(v.z, v.w));
            packed[i] = pack_half2_rn(y.x, y.y);
          }
          tmem_st_x16(s_addr + 16 * c, packed);
        }
        const float2 both = f2_add(part[0], part[1]);
        sum += (both.x + both.y) * exp2_approx(-e - kRaise);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&p_full[w]);
      }
      if (!ok) break;
      // ---- the rows' outputs
      const int64_t row = static_cast<int64_t>(it.s.q0 + qi) * p.q_heads + hq;
      const float inv = sum > 0.f ? __fdiv_rn(exp2_approx(-kRaise), sum) : 0.f;
      if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait_inline(&o_full[w], (tiles - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld_x32(o_addr + 32 * c, o);
          tmem_ld_wait(o);
        }
        if (valid) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // 8 columns, in the order 0 4 1 5 2 6 3 7
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              v[(k >> 1) + 4 * (k & 1)] = sum > 0.f ? __uint_as_float(o[8 * i + k]) * inv : 0.f;
            *reinterpret_cast<uint4 *>(p.out + row * 128 + 32 * c + 8 * i) =
                make_uint4(pack_half2_rn(v[0], v[1]), pack_half2_rn(v[2], v[3]),
                           pack_half2_rn(v[4], v[5]), pack_half2_rn(v[6], v[7]));
          }
        }
      }
      if (valid && p.lse != nullptr)
        p.lse[row] = sum > 0.f ? (top + log2f(sum)) * 0.693147180559945309f : -INFINITY;
      tc_fence_before_sync();
    }
    if (!ok && lane == 0) fail();
  } else if (warp < 12) {
    // ================================================================ expand
    const int ew = warp - 8, g = lane >> 2, t = lane & 3;
    uint32_t tiles = 0;
    bool ok = true;
    uint4 kq[4], vq[4];
    float ks = 0.f, vs = 0.f;
    int64_t last = 0;   // cached positions that the item's rows see
    auto load = [&](int j) {
      const int pos = j * kTok + 32 * ew + lane;
      int64_t vec = -1;
      ks = vs = 0.f;
      if (pos < last) {
        const int page_no = kv4_div(pos, p.geom.by_page);
        const int page = __ldg(p.seqs.table + it.b * p.seqs.table_stride + page_no);
        vec = kv4_vector(p.geom, page, pos - page_no * p.geom.page_size, it.head);
        if (vec < 0) {
          report_status(1 /* ATOM_ERR_INVALID_ARG */);
        } else {
          ks = __ldg(p.ks + vec) * p.scale_log2;
          vs = __ldg(p.vs + vec);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // chunk t of token 8i + g
        const int64_t v = __shfl_sync(0xffffffffu, vec, 8 * i + g);
        kq[i] = vq[i] = make_uint4(0u, 0u, 0u, 0u);
        if (v >= 0) {
          kq[i] = __ldg(reinterpret_cast<const uint4 *>(p.k4 + v * 64 + t * 16));
          vq[i] = __ldg(reinterpret_cast<const uint4 *>(p.v4 + v * 64 + t * 16));
        }
      }
    };
    auto expand = [&](const uint4 (&q)[4], uint8_t *tile) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 32 * ew + 8 * i + g;
        uint8_t *dst = tile + (t >> 1) * kHalf + row * 128;
        const uint32_t words[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 c = codes_f16_chunk(words[k]);
          st_shared_v4(dst + (((4 * (t & 1) + k) ^ (row & 7)) << 4), c.x, c.y, c.z, c.w);
        }
      }
      fence_proxy_async_smem();
    };
    for (; ok && it.place < line.total; next_item()) {
      kv4_prompt_locate(it, p);
      const int n = it.kv_tiles;
      const int last_row = (it.row0 + kRows < it.rows ? it.row0 + kRows : it.rows) - 1;
      last = kv4_limit(it.s, last_row / p.group, p.causal != 0);
      if (n > 0) load(0);
      for (int j = 0; j < n; ++j, ++tiles) {
        const int st = tiles & 1;
        const uint32_t ph = (tiles >> 1) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&k_empty[st], ph ^ 1u, abort_flag))) {
          ok = false;
          break;
        }
        // the stage's scales were last read four tiles ago
        uint8_t *sc = smem + kScOff + (tiles & 3) * kScStage;
        const uint32_t largest = __reduce_max_sync(0xffffffffu, __float_as_uint(vs));
        if (lane == 0) tile_max[4 * st + ew] = largest;
        expand(kq, smem + kKOff + st * kTile);
        named_bar_sync(1, 128);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = tile_max[4 * st + i] > m ? tile_max[4 * st + i] : m;
        int e = static_cast<int>(m >> 23) - 126;   // m < 2^e
        e = e < -60 ? -60 : (e > 100 ? 100 : e);
        reinterpret_cast<float *>(sc)[32 * ew + lane] = ks;
        reinterpret_cast<float *>(sc)[kTok + 32 * ew + lane] =
            vs * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        if (threadIdx.x == 8 * 32)
          *reinterpret_cast<float *>(sc + 2 * kTok * 4) = static_cast<float>(e);
        mbar_arrive(&k_full[st]);
        if (!__all_sync(0xffffffffu, mbar_wait(&v_empty[st], ph ^ 1u, abort_flag))) {
          ok = false;
          break;
        }
        expand(vq, smem + kVOff + st * kTile);
        mbar_arrive(&v_full[st]);
        if (j + 1 < n) load(j + 1);
      }
    }
    if (!ok && lane == 0) fail();
  } else {
    // ================================================================ MMA issuer
    if (warp == 12 && lane == 0) {
      uint32_t tiles = 0, items = 0;
      bool ok = true;
      const uint32_t q_addr = smem_addr(smem + kQOff), k_addr = smem_addr(smem + kKOff);
      const uint32_t v_addr = smem_addr(smem + kVOff);
      auto scores = [&](int w, int st) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (k >> 2) * kHalf + (k & 3) * 32;
          mma_f16(tbase + kTmemS + 128 * w, smem_desc_k_sw128(q_addr + w * kTile + off),
                  smem_desc_k_sw128(k_addr + st * kTile + off), kIdescS, k > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[w]);
      };
      auto outputs = [&](int w, int st, bool first) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_f16_ts(tbase + kTmemO + 128 * w, tbase + kTmemS + 128 * w + 8 * k,
                     smem_desc_mn_sw128(v_addr + st * kTile + k * 2048, kHalf, 1024), kIdescO,
                     !first || k > 0 ? 1u : 0u);
        tc_commit(&o_full[w]);
      };
      for (; ok && it.place < line.total; next_item()) {
        kv4_prompt_locate(it, p);
        const int n = it.kv_tiles;
        if (n == 0) continue;
        if (!mbar_wait(&k_full[tiles & 1], (tiles >> 1) & 1, abort_flag) ||
            !mbar_wait(&q_full[0], items & 1, abort_flag) ||
            !mbar_wait(&q_full[1], items & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        scores(0, tiles & 1);
        scores(1, tiles & 1);
        tc_commit(&k_empty[tiles & 1]);
        for (int j = 0; j < n; ++j, ++tiles) {
          const int st = tiles & 1, nst = (tiles + 1) & 1;
          if (!mbar_wait(&v_full[st], (tiles >> 1) & 1, abort_flag) ||
              !mbar_wait(&p_full[0], tiles & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          outputs(0, st, j == 0);
          if (j + 1 < n) {
            if (!mbar_wait(&k_full[nst], ((tiles + 1) >> 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            scores(0, nst);
          }
          if (!mbar_wait(&p_full[1], tiles & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          outputs(1, st, j == 0);
          tc_commit(&v_empty[st]);
          if (j + 1 < n) {
            scores(1, nst);
            tc_commit(&k_empty[nst]);
          }
        }
        ++items;
      }
      if (!ok) fail();
      // nothing may still write TMEM or read shared memory when they are released
      tc_commit(done);
      (void)mbar_wait(done, 0, nullptr);
    }
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, kTmemCols);
  }
}

}  // namespace atomk
