// kv4_api.cuh -- host side of the paged INT4 KV cache's entry points: argument
// checks and launches. Part of the translation unit atom_lib.cu.
#pragma once

namespace {

bool kv4_fits(int64_t v) { return v <= INT32_MAX; }
// Rows, heads and sequences leave room for the loops that step past them, and sums
// of two of them, in 32 bits.
bool kv4_fits_rows(int64_t v) { return v <= atomk::kKv4MaxPositions; }

// Sizes and strides, then (with `touched`) pointers.
atom_status_t kv4_check_cache(const atom_kv4_cache_t *c, bool touched) {
  if (!c || c->pages < 0 || c->heads < 0 || c->page_stride < 0 || c->token_stride < 0 ||
      c->head_stride < 0)
    return ATOM_ERR_INVALID_ARG;
  if (c->page_size < 1 || c->heads < 1 || !kv4_fits(c->pages) || !kv4_fits(c->page_size) ||
      !kv4_fits_rows(c->heads) || !kv4_fits(c->page_stride) || !kv4_fits(c->token_stride) ||
      !kv4_fits(c->head_stride))
    return ATOM_ERR_SHAPE;
  if (!touched) return ATOM_OK;
  if (!c->k4 || !c->ks || !c->v4 || !c->vs) return ATOM_ERR_INVALID_ARG;
  if (!aligned(c->k4, 16) || !aligned(c->v4, 16) || !aligned(c->ks, 4) || !aligned(c->vs, 4))
    return ATOM_ERR_ALIGN;
  return ATOM_OK;
}

// Whether two runs of memory share a byte.
bool kv4_overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}
bool kv4_caches_overlap(const atom_kv4_cache_t *a, const atom_kv4_cache_t *b) {
  auto vectors = [](const atom_kv4_cache_t *c) {
    return c->pages < 1 ? 0 : (c->pages - 1) * c->page_stride + (c->page_size - 1) * c->token_stride +
                                  (c->heads - 1) * c->head_stride + 1;
  };
  const int64_t x = vectors(a), y = vectors(b);
  const struct { const void *p; int64_t bytes; } src[4] = {
      {a->k4, x * 64}, {a->v4, x * 64}, {a->ks, x * 4}, {a->vs, x * 4}};
  const struct { const void *p; int64_t bytes; } dst[4] = {
      {b->k4, y * 64}, {b->v4, y * 64}, {b->ks, y * 4}, {b->vs, y * 4}};
  for (const auto &s : src)
    for (const auto &d : dst)
      if (kv4_overlap(s.p, s.bytes, d.p, d.bytes)) return true;
  return false;
}

atom_status_t kv4_check_table(const int32_t *table, int64_t stride, int64_t max_pages) {
  if (max_pages < 0 || stride < 0) return ATOM_ERR_INVALID_ARG;
  if (stride < max_pages) return ATOM_ERR_SHAPE;
  if (!table && max_pages > 0) return ATOM_ERR_INVALID_ARG;
  return aligned(table, 4) ? ATOM_OK : ATOM_ERR_ALIGN;
}

atom_status_t kv4_check_batch(const atom_kv4_batch_t *b, bool rows_read) {
  if (!b || b->batch < 0 || b->max_q < 0) return ATOM_ERR_INVALID_ARG;
  if (!kv4_fits_rows(b->batch)) return ATOM_ERR_SHAPE;
  if (b->batch == 0) return ATOM_OK;
  const atom_status_t st = kv4_check_table(b->block_table, b->table_stride, b->max_pages);
  if (st != ATOM_OK) return st;
  if (!b->kv_lens || (rows_read && !b->cu_q)) return ATOM_ERR_INVALID_ARG;
  if (!aligned(b->kv_lens, 4) || !aligned(b->cu_q, 4)) return ATOM_ERR_ALIGN;
  return ATOM_OK;
}

// fp16 row tensors [rows][heads][128]
atom_status_t kv4_check_rows(const void *x, int64_t token, int64_t head) {
  if (token < 0 || head < 0) return ATOM_ERR_INVALID_ARG;
  if (token % 8 != 0 || head % 8 != 0) return ATOM_ERR_SHAPE;
  if (!x) return ATOM_ERR_INVALID_ARG;
  return aligned(x, 16) ? ATOM_OK : ATOM_ERR_ALIGN;
}

atomk::Kv4Geom kv4_geom(const atom_kv4_cache_t *c) {
  atomk::Kv4Geom g;
  // (a dimension of one has no stride)
  g.page_stride = c->pages > 1 ? static_cast<int>(c->page_stride) : 0;
  g.token_stride = c->page_size > 1 ? static_cast<int>(c->token_stride) : 0;
  g.head_stride = c->heads > 1 ? static_cast<int>(c->head_stride) : 0;
  g.pages = static_cast<int>(c->pages);
  g.page_size = static_cast<int>(c->page_size);
  g.heads = static_cast<int>(c->heads);
  g.by_page = atomk::kv4_div_by(c->page_size);
  return g;
}

atomk::Kv4Seqs kv4_seqs(const atom_kv4_batch_t *b, const atom_kv4_cache_t *c, int64_t rows) {
  atomk::Kv4Seqs s;
  s.table = b->block_table;
  s.table_stride = b->table_stride;
  s.kv_lens = b->kv_lens;
  s.cu_q = b->cu_q;
  s.batch = static_cast<int>(b->batch);
  s.rows = static_cast<int>(rows);
  s.capacity = atomk::kv4_capacity(b->max_pages, c->page_size);
  return s;
}

// Launch that may overlap the end of the kernel before it in the stream (the
// kernel waits for that one before it touches memory).
template <class... P>
cudaError_t kv4_launch(void (*fn)(P...), dim3 grid, int threads, size_t smem,
                       atom_stream_t stream, const P &...p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p...);
}

atom_status_t kv4_rows(bool append, const void *k, int64_t k_token, int64_t k_head, const void *v,
                       int64_t v_token, int64_t v_head, int64_t rows, const atom_kv4_cache_t *cache,
                       const atom_kv4_batch_t *batch, atom_stream_t stream) {
  if (rows < 0) return ATOM_ERR_INVALID_ARG;
  if (!kv4_fits_rows(rows)) return ATOM_ERR_SHAPE;
  const bool touched = rows > 0 && batch != nullptr && batch->batch > 0;
  atom_status_t st;
  if ((st = kv4_check_cache(cache, touched)) != ATOM_OK) return st;
  if ((st = kv4_check_batch(batch, touched)) != ATOM_OK) return st;
  if (!touched) return ATOM_OK;
  if ((st = kv4_check_rows(k, k_token, k_head)) != ATOM_OK) return st;
  if ((st = kv4_check_rows(v, v_token, v_head)) != ATOM_OK) return st;
  DeviceState *dev = nullptr;
  if ((st = current_device(&dev)) != ATOM_OK) return st;
  atomk::Kv4Rows p;
  p.k4 = cache->k4;
  p.v4 = cache->v4;
  p.ks = cache->ks;
  p.vs = cache->vs;
  p.geom = kv4_geom(cache);
  p.seqs = kv4_seqs(batch, cache, rows);
  p.k = static_cast<__half *>(const_cast<void *>(k));
  p.v = static_cast<__half *>(const_cast<void *>(v));
  p.k_token = k_token;
  p.k_head = k_head;
  p.v_token = v_token;
  p.v_head = v_head;
  const int64_t vecs = 2 * cache->heads, step = atomk::kKv4RowVecs;
  p.by_vecs = static_cast<uint32_t>((65536 + vecs - 1) / vecs);
  // 15 CTAs an SM, a multiple of the three or five that it holds at once
  const int64_t cap = static_cast<int64_t>(dev->sm_count) * 15, warps = atomk::kKvThreads / 32;
  const bool line = vecs % step != 0;   // (measured at the kernel)
  // a warp 16 places of the line, or a row, whose parts of 16 grid_y may divide
  const int64_t steps = line ? (rows * vecs + step - 1) / step : rows;
  const int64_t ctas = (steps + warps - 1) / warps, parts = line ? 1 : vecs / step;
  const int grid_x = static_cast<int>(ctas < cap ? ctas : cap);
  int64_t grid_y = cap / grid_x;
  if (grid_y > parts) grid_y = parts;
  void (*const fn)(atomk::Kv4Rows) =
      append ? (line ? atomk::kv4_rows_kernel<true, true> : atomk::kv4_rows_kernel<true, false>)
             : (line ? atomk::kv4_rows_kernel<false, true> : atomk::kv4_rows_kernel<false, false>);
  const cudaError_t err =
      kv4_launch(fn, dim3(static_cast<unsigned>(grid_x), static_cast<unsigned>(grid_y), 1),
                 atomk::kKvThreads, 0, stream, p);
  return err == cudaSuccess ? ATOM_OK : ATOM_ERR_CUDA;
}

// Largest number of query rows of a KV head that goes to the first kernel of the
// attention weights (kv4_few_rows is the attention's). Both measured, us: 16 sequences of
// 3000 tokens, 8 heads, 16 rows 34 and 42, 24 rows 45 and 42, 32 rows 57 and 43; four of
// 20000, 16 rows 49 and 66, 24 rows 66 and 67, 32 rows 85 and 67.
constexpr int kKv4WeightFewRows = 24;

// Query rows a CTA of the decode kernel takes at once, 8 or 16: the smallest
// that holds every sequence's rows of a KV head, so that the cache is read once.
int kv4_decode_nt(int64_t max_q, int64_t group) { return max_q * group <= 8 ? 1 : 2; }

// CTAs of the decode kernel: all that the GPU holds at once.
atom_status_t kv4_decode_ctas(DeviceState *dev, int nt, int *ctas) {
  using namespace atomk::kv4_decode_cfg;
  if (!dev->kv4_attr[nt - 1].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!dev->kv4_attr[nt - 1].load(std::memory_order_relaxed)) {
      const void *fn = nt == 1 ? reinterpret_cast<const void *>(atomk::kv4_decode_kernel<1>)
                               : reinterpret_cast<const void *>(atomk::kv4_decode_kernel<2>);
      int per_sm = 0;
      if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSmemBytes)) != cudaSuccess ||
          cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, kThreads, kSmemBytes) !=
              cudaSuccess ||
          per_sm < 1)
        return ATOM_ERR_CUDA;
      dev->kv4_ctas[nt - 1] = per_sm * dev->sm_count;
      dev->kv4_attr[nt - 1].store(true, std::memory_order_release);
    }
  }
  *ctas = dev->kv4_ctas[nt - 1];
  return ATOM_OK;
}

// Tensor map of fp16 queries [rows][q_heads][128] whose boxes are the rows of as
// many whole tokens of a KV head as make at most 128, half a vector wide.
bool kv4_query_map(CUtensorMap *map, const void *q, int64_t q_token, int64_t q_head, int64_t rows,
                   int64_t q_heads, int group) {
  EncodeTiledFn fn = encode_fn();
  // (a tensor map's strides are not zero)
  if (!fn || (q_heads > 1 && q_head == 0) || (rows > 1 && q_token == 0)) return false;
  // (a dimension of one has no stride of its own)
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(q_heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(q_heads > 1 ? q_head * 2 : 256),
                                 static_cast<cuuint64_t>(rows > 1 ? q_token * 2 : 256)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the prompt kernels can take a call: its longest sequence has more rows
// than the decode kernel should take, its tokens' rows fit a tile, and a tensor
// map describes its queries.
bool kv4_prompt_call(CUtensorMap *map, const void *q, int64_t q_token, int64_t q_head, int64_t rows,
                     int64_t q_heads, int group, int64_t max_q, int64_t few_rows) {
  return max_q * group > few_rows && group <= 128 &&
         kv4_query_map(map, q, q_token, q_head, rows, q_heads, group);
}

constexpr float kLog2e = 1.44269504088896341f;

// Sizes shared by the two attention entry points.
atom_status_t kv4_check_queries(int64_t rows, int64_t q_heads, float scale,
                                const atom_kv4_cache_t *cache, const atom_kv4_batch_t *batch,
                                bool *touched) {
  if (rows < 0 || q_heads < 0) return ATOM_ERR_INVALID_ARG;
  // With vectors of fp16 numbers no score times log2(e) then passes 1e30, which
  // stands for a row that has seen nothing (kKv4NoMax).
  if (!(fabsf(scale) <= 1e18f)) return ATOM_ERR_INVALID_ARG;
  *touched = rows > 0 && batch != nullptr && batch->batch > 0;
  atom_status_t st;
  if ((st = kv4_check_cache(cache, *touched)) != ATOM_OK) return st;
  if ((st = kv4_check_batch(batch, *touched)) != ATOM_OK) return st;
  if (!kv4_fits_rows(rows) || q_heads < 1 || q_heads % cache->heads != 0 || !kv4_fits(q_heads) ||
      !kv4_fits_rows(rows * (q_heads / cache->heads)))   // query rows of a KV head
    return ATOM_ERR_SHAPE;
  return ATOM_OK;
}

}  // namespace

extern "C" {

atom_status_t atom_kv4_append(const void *k, int64_t k_token, int64_t k_head, const void *v,
                              int64_t v_token, int64_t v_head, int64_t rows,
                              const atom_kv4_cache_t *cache, const atom_kv4_batch_t *batch,
                              atom_stream_t stream) {
  return kv4_rows(true, k, k_token, k_head, v, v_token, v_head, rows, cache, batch, stream);
}

atom_status_t atom_kv4_gather(const atom_kv4_cache_t *cache, const atom_kv4_batch_t *batch,
                              int64_t rows, void *k_out, void *v_out, atom_stream_t stream) {
  const int64_t token = cache != nullptr ? cache->heads * 128 : 0;
  return kv4_rows(false, k_out, token, 128, v_out, token, 128, rows, cache, batch, stream);
}

size_t atom_kv4_attention_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads,
                                          int64_t max_q) {
  if (rows <= 0 || q_heads < 1 || heads < 1 || q_heads % heads != 0 || max_q < 1) return 0;
  DeviceState *dev = nullptr;
  if (current_device(&dev) != ATOM_OK) return 0;
  const int nt = kv4_decode_nt(max_q < rows ? max_q : rows, q_heads / heads);
  int ctas = 0;
  if (kv4_decode_ctas(dev, nt, &ctas) != ATOM_OK) return 0;
  return static_cast<size_t>(atomk::kv4_decode_cfg::ws_bytes(ctas, nt));
}

atom_status_t atom_kv4_attention(const void *q, int64_t q_token, int64_t q_head, int64_t rows,
                                 int64_t q_heads, const atom_kv4_cache_t *cache,
                                 const atom_kv4_batch_t *batch, int32_t causal, float scale,
                                 void *out, float *lse, void *workspace, size_t workspace_bytes,
                                 atom_stream_t stream) {
  bool touched = false;
  atom_status_t st = kv4_check_queries(rows, q_heads, scale, cache, batch, &touched);
  if (st != ATOM_OK || !touched) return st;
  if ((st = kv4_check_rows(q, q_token, q_head)) != ATOM_OK) return st;
  if (!out) return ATOM_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(lse, 4)) return ATOM_ERR_ALIGN;
  DeviceState *dev = nullptr;
  if ((st = current_device(&dev)) != ATOM_OK) return st;
  atomk::Kv4Attn p;
  p.q = static_cast<const __half *>(q);
  p.q_token = q_token;
  p.q_head = q_head;
  p.out = static_cast<__half *>(out);
  p.lse = lse;
  p.k4 = cache->k4;
  p.v4 = cache->v4;
  p.ks = cache->ks;
  p.vs = cache->vs;
  p.geom = kv4_geom(cache);
  p.seqs = kv4_seqs(batch, cache, rows);
  p.q_heads = static_cast<int>(q_heads);
  p.group = static_cast<int>(q_heads / cache->heads);
  p.by_group = atomk::kv4_div_by(p.group);
  p.magic = atomk::kKv4Magic;
  p.scale_log2 = scale * kLog2e;
  p.causal = causal != 0 ? 1 : 0;
  // One address a stage instead of one a token (64x8192: 103 us with pages of 64, 111
  // with pages of 16).
  p.whole = cache->page_size % atomk::kv4_decode_cfg::kTok == 0;
  p.max_q = static_cast<int>(batch->max_q < rows ? batch->max_q : rows);
  // Sequences with few query rows a KV head go to the decode kernel, those with
  // more to the prompt kernel; one that no sequence can need is not launched.
  CUtensorMap q_map;
  const int64_t few_rows = atomk::kv4_few_rows(batch->batch * cache->heads,
                                        static_cast<int64_t>(p.max_q) * p.group, dev->sm_count);
  const bool prompts =
      kv4_prompt_call(&q_map, q, q_token, q_head, rows, q_heads, p.group, p.max_q, few_rows);
  const bool decode = !prompts || batch->batch > 1;
  p.tile_rows = prompts ? 128 / p.group * p.group : 0;
  p.few_rows = !prompts ? INT32_MAX : (decode ? static_cast<int>(few_rows) : 0);
  cudaError_t err = cudaSuccess;
  if (prompts) {
    using namespace atomk::kv4_prompt_cfg;
    if (!dev->kv4_prompt_attr.load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(atomk::kv4_prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSmemBytes)) != cudaSuccess)
        return ATOM_ERR_CUDA;
      dev->kv4_prompt_attr.store(true, std::memory_order_release);
    }
    err = kv4_launch(atomk::kv4_prompt_kernel, dev->sm_count, kThreads, kSmemBytes, stream, q_map, p);
  }
  if (err == cudaSuccess && decode) {
    using namespace atomk::kv4_decode_cfg;
    const int nt = kv4_decode_nt(p.max_q, p.group);
    int ctas = 0;
    if ((st = kv4_decode_ctas(dev, nt, &ctas)) != ATOM_OK) return st;
    p.split = workspace != nullptr && aligned(workspace, 16) &&
              workspace_bytes >= static_cast<size_t>(ws_bytes(ctas, nt));
    p.ws = p.split ? static_cast<float *>(workspace) : nullptr;
    err = nt == 1 ? kv4_launch(atomk::kv4_decode_kernel<1>, ctas, kThreads, kSmemBytes, stream, p)
                  : kv4_launch(atomk::kv4_decode_kernel<2>, ctas, kThreads, kSmemBytes, stream, p);
    if (err == cudaSuccess && p.split)
      err = nt == 1
                ? kv4_launch(atomk::kv4_join_kernel<1>, ctas, atomk::kKv4JoinThreads, 0, stream, p)
                : kv4_launch(atomk::kv4_join_kernel<2>, ctas, atomk::kKv4JoinThreads, 0, stream, p);
  }
  return err == cudaSuccess ? ATOM_OK : ATOM_ERR_CUDA;
}

atom_status_t atom_kv4_attention_weights(const void *q, int64_t q_token, int64_t q_head,
                                         int64_t rows, int64_t q_heads, const float *lse,
                                         const atom_kv4_cache_t *cache,
                                         const atom_kv4_batch_t *batch, int32_t causal, float scale,
                                         const float *prev, float *sums, int64_t width,
                                         atom_stream_t stream) {
  bool touched = false;
  if (width < 0) return ATOM_ERR_INVALID_ARG;
  atom_status_t st = kv4_check_queries(rows, q_heads, scale, cache, batch, &touched);
  if (st != ATOM_OK || !touched) return st;
  if ((st = kv4_check_rows(q, q_token, q_head)) != ATOM_OK) return st;
  if (!lse || (!sums && width > 0)) return ATOM_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(sums, 4) || !aligned(prev, 4)) return ATOM_ERR_ALIGN;
  DeviceState *dev = nullptr;
  if ((st = current_device(&dev)) != ATOM_OK) return st;
  atomk::Kv4Weights p;
  p.q = static_cast<const __half *>(q);
  p.q_token = q_token;
  p.q_head = q_head;
  p.lse = lse;
  p.k4 = cache->k4;
  p.ks = cache->ks;
  p.geom = kv4_geom(cache);
  p.seqs = kv4_seqs(batch, cache, rows);
  if (p.seqs.capacity > width) p.seqs.capacity = static_cast<int>(width);
  p.q_heads = static_cast<int>(q_heads);
  p.group = static_cast<int>(q_heads / cache->heads);
  p.scale_log2 = scale * kLog2e;
  p.causal = causal != 0 ? 1 : 0;
  p.by_group = atomk::kv4_div_by(p.group);
  p.magic = atomk::kKv4Magic;
  p.whole = cache->page_size % atomk::kv4_wdecode_cfg::kTok == 0;
  p.prev = prev;
  p.sums = sums;
  p.width = width;
  // as in atom_kv4_attention (a larger sequence than max_q says costs time here,
  // nothing else)
  const int64_t max_q = batch->max_q < rows ? batch->max_q : rows;
  CUtensorMap q_map;
  const bool prompts = kv4_prompt_call(&q_map, q, q_token, q_head, rows, q_heads, p.group, max_q,
                                       kKv4WeightFewRows);
  const bool few = !prompts || batch->batch > 1;
  p.tile_rows = prompts ? 128 / p.group * p.group : 0;
  // (alone, the second kernel also takes a sequence without new tokens)
  p.few_rows = !prompts ? INT32_MAX : (few ? kKv4WeightFewRows : -1);
  cudaError_t err = cudaSuccess;
  if (prompts) {
    using namespace atomk::kv4_wprompt_cfg;
    if (!dev->kv4_wprompt_attr.load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(atomk::kv4_weights_prompt_kernel,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSmemBytes)) != cudaSuccess)
        return ATOM_ERR_CUDA;
      dev->kv4_wprompt_attr.store(true, std::memory_order_release);
    }
    err = kv4_launch(atomk::kv4_weights_prompt_kernel, dev->sm_count, kThreads, kSmemBytes, stream,
                     q_map, p);
  }
  if (err == cudaSuccess && few)
    err = kv4_launch(atomk::kv4_weights_kernel, 5 * dev->sm_count,
                     atomk::kv4_wdecode_cfg::kThreads, 0, stream, p);
  return err == cudaSuccess ? ATOM_OK : ATOM_ERR_CUDA;
}

atom_status_t atom_kv4_evict(const float *weights, int64_t width, const atom_kv4_cache_t *cache,
                             const atom_kv4_batch_t *batch, int64_t budget, int64_t recent,
                             const atom_kv4_cache_t *dst, const int32_t *to_table,
                             int64_t to_table_stride, int64_t to_max_pages, int32_t *new_lens,
                             int32_t *kept, float *new_weights, int64_t new_width,
                             atom_stream_t stream) {
  if (width < 0 || new_width < 0 || budget < 1 || recent < 0 || recent > budget)
    return ATOM_ERR_INVALID_ARG;
  if (!kv4_fits(budget) || (new_weights && new_width < budget)) return ATOM_ERR_SHAPE;
  const bool touched = batch != nullptr && batch->batch > 0;
  atom_status_t st;
  if ((st = kv4_check_cache(cache, touched)) != ATOM_OK) return st;
  if ((st = kv4_check_cache(dst, touched)) != ATOM_OK) return st;
  if (cache->heads != dst->heads) return ATOM_ERR_SHAPE;
  if ((st = kv4_check_batch(batch, false)) != ATOM_OK) return st;
  if (!touched) return ATOM_OK;
  if (batch->batch * cache->heads > INT32_MAX) return ATOM_ERR_SHAPE;
  if ((st = kv4_check_table(to_table, to_table_stride, to_max_pages)) != ATOM_OK) return st;
  if ((!weights && width > 0) || !new_lens || !kept || new_lens == batch->kv_lens)
    return ATOM_ERR_INVALID_ARG;
  if (new_weights == weights && new_weights != nullptr && new_width != width) return ATOM_ERR_SHAPE;
  if (!aligned(weights, 4) || !aligned(new_lens, 4) || !aligned(kept, 4) || !aligned(new_weights, 4))
    return ATOM_ERR_ALIGN;
  DeviceState *dev = nullptr;
  if ((st = current_device(&dev)) != ATOM_OK) return st;
  atomk::Kv4Evict p;
  p.weights = weights;
  p.width = width;
  p.k4 = cache->k4;
  p.v4 = cache->v4;
  p.ks = cache->ks;
  p.vs = cache->vs;
  p.geom = kv4_geom(cache);
  p.seqs = kv4_seqs(batch, cache, 0);
  p.to_k4 = dst->k4;
  p.to_v4 = dst->v4;
  p.to_ks = dst->ks;
  p.to_vs = dst->vs;
  p.to_geom = kv4_geom(dst);
  p.to_table = to_table;
  p.to_table_stride = to_table_stride;
  p.to_capacity = atomk::kv4_capacity(to_max_pages, dst->page_size);
  p.budget = static_cast<int>(budget);
  p.recent = static_cast<int>(recent);
  p.new_lens = new_lens;
  p.kept = kept;
  p.new_weights = new_weights;
  p.new_width = new_width;
  p.in_steps = kv4_caches_overlap(cache, dst) ||
               (new_weights != nullptr &&
                kv4_overlap(weights, batch->batch * cache->heads * width * 4, new_weights,
                            batch->batch * cache->heads * new_width * 4));
  // CTAs a (sequence, head): as many as leave none without an SM of its own, and
  // at least 2048 of the widest sequence's tokens to each (1 x 65537, 8 heads:
  // with the gather of what stays 173 us with one CTA, 33 with eight)
  const int64_t rows = batch->batch * cache->heads;
  int64_t tokens = p.seqs.capacity < width ? p.seqs.capacity : width;
  int cluster = 1;
  while (cluster < atomk::kv4_evict_cfg::kMaxCluster && rows * cluster * 2 <= dev->sm_count &&
         tokens >= int64_t(2048) * cluster * 2)
    cluster *= 2;
  if (rows * cluster > INT32_MAX) return ATOM_ERR_SHAPE;
  // Where they are more than the GPU holds of the larger CTAs at once, CTAs of half
  // the size, which it holds twice as many of (64 sequences of 2048 tokens, 8 heads, with the
  // gather of what stays: 113 us with the larger, 108 with the smaller).
  const bool few_threads = rows > 2 * static_cast<int64_t>(dev->sm_count);
  void (*const fn)(atomk::Kv4Evict, int) =
      few_threads ? atomk::kv4_evict_kernel<atomk::kv4_evict_cfg::kFewThreads>
                  : atomk::kv4_evict_kernel<atomk::kv4_evict_cfg::kThreads>;
  if (!dev->kv4_evict_attr.load(std::memory_order_acquire)) {
    for (const void *f : {reinterpret_cast<const void *>(
                              atomk::kv4_evict_kernel<atomk::kv4_evict_cfg::kFewThreads>),
                          reinterpret_cast<const void *>(
                              atomk::kv4_evict_kernel<atomk::kv4_evict_cfg::kThreads>)})
      if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               atomk::kv4_evict_cfg::kKeys * 4 + 16) != cudaSuccess)
        return ATOM_ERR_CUDA;
    dev->kv4_evict_attr.store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster), 1, 1);
  cfg.blockDim = dim3(few_threads ? atomk::kv4_evict_cfg::kFewThreads
                                  : atomk::kv4_evict_cfg::kThreads, 1, 1);
  // room for the keys of a CTA's share; a share that does not fit is read again
  // in every pass
  const int64_t keys = tokens / cluster + 2 * atomk::kv4_evict_cfg::kRun;
  cfg.dynamicSmemBytes = keys > atomk::kv4_evict_cfg::kKeys
                             ? 0
                             : static_cast<size_t>((keys * 4 + 15) / 16 * 16);
  p.keys = keys > atomk::kv4_evict_cfg::kKeys ? 0 : static_cast<int>(keys);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p, cluster) == cudaSuccess ? ATOM_OK : ATOM_ERR_CUDA;
}

}  // extern "C"
