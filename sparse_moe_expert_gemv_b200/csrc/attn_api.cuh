// attn_api.cuh -- host side of the attention calls of include/moe.h (part of
// moe_api.cu's translation unit).
#pragma once

namespace {

constexpr int kAtGridPerSm = 2;  // resident blocks of attn_kernel

// The arguments every call over a batch shares.
moe_status attn_check(moe_ctx *c, const moe_kv_batch *b, const char *who) {
  if (!c->attn.ready) return fail(c, MOE_ERR_STATE, "%s: moe_attn_configure comes first", who);
  int dev = -1;
  CUDA_TRY(c, cudaGetDevice(&dev));
  if (dev != c->device)
    return fail(c, MOE_ERR_INVALID_ARG, "%s: the current device is %d, the context's %d", who, dev, c->device);
  if (!b) return MOE_OK;
  const moe_ctx::Attn &a = c->attn;
  if (!b->k || !b->v || !b->page_table || !b->row_off || !b->kv_len || b->n_pages < 1 || b->n_seqs < 1 ||
      b->max_pages < 1 || b->n_rows < 0 || !aligned16(b->k) || !aligned16(b->v))
    return fail(c, MOE_ERR_INVALID_ARG, "%s: bad batch (pages=%d seqs=%d max_pages=%d rows=%d)", who, b->n_pages,
                b->n_seqs, b->max_pages, b->n_rows);
  if ((b->k_scale || b->v_scale) && a.cache != MOE_KV_E4M3)
    return fail(c, MOE_ERR_INVALID_ARG, "%s: scales belong to an e4m3 cache", who);
  if ((long long)b->n_pages * a.n_kv * a.page > 0x7fffffffLL || (long long)b->max_pages * a.page > 0x7fffffffLL)
    return fail(c, MOE_ERR_NOT_SUPPORTED, "%s: more than 2^31 - 1 cache rows or positions", who);
  return MOE_OK;
}

// Rows are read in 16-byte (q of the attention) or 8-byte pieces.
bool rows_ok(const void *p, long long stride, long long width, int align) {
  return p && ((uintptr_t)p & (align - 1)) == 0 && stride >= width && stride % (align / 2) == 0;
}

moe_status rope_check(moe_ctx *c, const moe_qk_norm *norm, const moe_rope *rope, const char *who) {
  if (norm && (!(norm->eps >= 0.f) || norm->eps > 1e30f || !aligned16(norm->q_gamma) || !aligned16(norm->k_gamma)))
    return fail(c, MOE_ERR_INVALID_ARG, "%s: bad norm", who);
  if (rope && (!rope->inv_freq || ((uintptr_t)rope->inv_freq & 7) || rope->rot_dim < 8 || rope->rot_dim % 8 ||
               rope->rot_dim > c->attn.dim || (rope->interleaved != 0 && rope->interleaved != 1)))
    return fail(c, MOE_ERR_INVALID_ARG, "%s: bad rotation (rot_dim a multiple of 8, at most head_dim)", who);
  return MOE_OK;
}

template <int D, int CACHE, bool INTER>
cudaError_t launch_kv_rows_as(moe_ctx *c, cudaStream_t s, const KvRowsParams &p) {
  // A warp per row and four rows a block once that gives every other SM a
  // block (8192 rows of 16 + 4 heads of 128: 18.2 us, 19.0 us with eight rows
  // a block, 33.9 us with two of them on eight warps); below, one row a block,
  // its heads over eight warps (8 windows of 4 rows: 3.3 us, with four warps a
  // row 3.6 us).
  if (2 * p.n_rows >= kKvRows * c->n_sm)
    return launch(kv_rows_kernel<D, CACHE, kKvRows, INTER>, dim3((p.n_rows + kKvRows - 1) / kKvRows), dim3(kv_threads(kKvRows)), 0,
                  s, p);
  return launch(kv_rows_kernel<D, CACHE, 1, INTER>, dim3(p.n_rows), dim3(kv_threads(1)), 0, s, p);
}
template <int D, int CACHE>
cudaError_t launch_kv_rows(moe_ctx *c, cudaStream_t s, const KvRowsParams &p, bool inter) {
  return inter ? launch_kv_rows_as<D, CACHE, true>(c, s, p) : launch_kv_rows_as<D, CACHE, false>(c, s, p);
}

moe_status kv_rows(moe_ctx *c, cudaStream_t s, KvRowsParams &p, const moe_qk_norm *norm, const moe_rope *rope,
                   int cache) {
  p.n_q = c->attn.n_q;
  p.n_kv = c->attn.n_kv;
  p.page = c->attn.page;
  p.status = c->attn.status;
  if (norm) {
    p.norm = 1;
    p.q_gamma = norm->q_gamma;
    p.k_gamma = norm->k_gamma;
    p.eps = norm->eps;
  }
  if (rope) {
    p.inv_freq = rope->inv_freq;
    p.rot = rope->rot_dim;
  }
  const bool in = rope && rope->interleaved;
  cudaError_t e;
  if (c->attn.dim == 128)
    e = cache == 0 ? launch_kv_rows<128, 0>(c, s, p, in)
                   : cache == 1 ? launch_kv_rows<128, 1>(c, s, p, in) : launch_kv_rows<128, 2>(c, s, p, in);
  else
    e = cache == 0 ? launch_kv_rows<64, 0>(c, s, p, in)
                   : cache == 1 ? launch_kv_rows<64, 1>(c, s, p, in) : launch_kv_rows<64, 2>(c, s, p, in);
  CUDA_TRY(c, e);
  return MOE_OK;
}

// 2-D map of a paged cache seen as [n_pages * n_kv * page][D]: boxes of one
// page's keys (at most a tile's) x one swizzle row.
bool encode_cache_map(CUtensorMap *map, const moe_ctx::Attn &a, const void *base, int n_pages, int box_keys,
                      bool swizzle = true) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const bool fp8 = a.cache == MOE_KV_E4M3;
  const int row_bytes = a.dim * (fp8 ? 1 : 2), line = row_bytes < 128 ? row_bytes : 128;
  const cuuint64_t dims[2] = {(cuuint64_t)a.dim, (cuuint64_t)n_pages * a.n_kv * a.page};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)(fp8 ? line : line / 2), (cuuint32_t)box_keys};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
                      : line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FP8, int MT>
cudaError_t setup_attn(int *blocks) {
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<D, FP8, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       AttnCfg<D, FP8>::SMEM);
  int n = 0;
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_kernel<D, FP8, MT>, kAtThreads,
                                                      AttnCfg<D, FP8>::SMEM);
  if (n < *blocks) *blocks = n;
  return e;
}
template <int D, bool FP8>
cudaError_t setup_attn_all(int *blocks) {
  cudaError_t e = setup_attn<D, FP8, 1>(blocks);
  if (e == cudaSuccess) e = setup_attn<D, FP8, 2>(blocks);
  if (e == cudaSuccess) e = setup_attn<D, FP8, 4>(blocks);
  return e;
}

template <int D, bool FP8>
cudaError_t setup_attn_prefill() {
  return cudaFuncSetAttribute(attn_prefill_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              AttnPfCfg<D, FP8>::SMEM);
}

template <int D, bool FP8, int MT>
cudaError_t launch_attn_mt(moe_ctx *c, cudaStream_t s, const CUtensorMap &km, const CUtensorMap &vm,
                           const AttnParams &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c->attn.grid);
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = AttnCfg<D, FP8>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_kernel<D, FP8, MT>, km, vm, p);
}
template <int D, bool FP8>
cudaError_t launch_attn(moe_ctx *c, cudaStream_t s, const CUtensorMap &km, const CUtensorMap &vm,
                        const AttnParams &p, int rows) {
  if (rows <= 16) return launch_attn_mt<D, FP8, 1>(c, s, km, vm, p);
  if (rows <= 32) return launch_attn_mt<D, FP8, 2>(c, s, km, vm, p);
  return launch_attn_mt<D, FP8, 4>(c, s, km, vm, p);
}

// 3-D map of the query rows [n_rows][n_q][D]: boxes of 64 columns x `pack`
// heads x 128 / pack rows, so a box is 128 tile rows.
bool encode_q_map(CUtensorMap *map, const moe_ctx::Attn &a, const void *q, int n_rows, long long q_stride, int pack) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)a.dim, (cuuint64_t)a.n_q, (cuuint64_t)n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)a.dim * 2, (cuuint64_t)q_stride * 2};
  const cuuint32_t box[3] = {64u, (cuuint32_t)pack, (cuuint32_t)(128 / pack)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FP8>
cudaError_t launch_attn_prefill(cudaStream_t s, int grid, const CUtensorMap &qm, const CUtensorMap &km,
                                const CUtensorMap &vm, const AttnPfParams &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(AttnPfCfg<D, FP8>::THREADS);
  cfg.dynamicSmemBytes = AttnPfCfg<D, FP8>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_prefill_kernel<D, FP8>, qm, km, vm, p);
}

// The tensor-core kernel.
moe_status attend_chunk(moe_ctx *c, const moe_kv_batch *b, const void *q, int64_t q_stride, float scale, int window,
                        int n_sink, void *out, int64_t out_stride, cudaStream_t s, const char *who) {
  const moe_ctx::Attn &a = c->attn;
  AttnPfParams p{};
  p.out = (uint16_t *)out;
  p.out_stride = out_stride;
  p.page_table = b->page_table;
  p.row_off = b->row_off;
  p.kv_len = b->kv_len;
  p.scale_log2 = scale * 1.44269504088896340736f;
  p.window = window;
  p.n_sink = n_sink;
  p.n_rows = b->n_rows;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.group = a.n_q / a.n_kv;
  while (p.pack_shift < 7 && p.group % (2 << p.pack_shift) == 0) ++p.pack_shift;
  p.pack = 1 << p.pack_shift;
  p.n_pages = b->n_pages;
  p.n_seqs = b->n_seqs;
  p.max_pages = b->max_pages;
  p.page = a.page;
  while ((1 << p.page_shift) < a.page) ++p.page_shift;
  p.status = a.status;
  p.k_scale = b->k_scale;
  p.v_scale = b->v_scale;
  const bool fp8 = a.cache == MOE_KV_E4M3;  // its tiles are converted on the way: no swizzle
  CUtensorMap qm, km, vm;
  const int box = a.page < kApTile ? a.page : kApTile;
  if (!encode_q_map(&qm, a, q, b->n_rows, q_stride, p.pack) || !encode_cache_map(&km, a, b->k, b->n_pages, box, !fp8) ||
      !encode_cache_map(&vm, a, b->v, b->n_pages, box, !fp8))
    return fail(c, MOE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  // the row blocks of all sequences are at most this many, and their parts at
  // most one wave more (the rest leave at once); the workspace has room for a
  // part of 256 rows an SM
  p.n_sm = (int)std::min<long long>(c->n_sm, (long long)a.grid * 2 * kAtMaxRows / kApRows);
  const long long blocks = (long long)b->n_rows / (kApRows / p.pack) + b->n_seqs;
  const long long grid = blocks * (a.n_q / p.pack) + p.n_sm;
  if (grid > 0x7fffffffLL) return fail(c, MOE_ERR_NOT_SUPPORTED, "%s: %lld blocks", who, grid);
  p.ws = a.ws;
  p.arrived = a.arrived;
  cudaError_t e;
  if (a.dim == 128)
    e = fp8 ? launch_attn_prefill<128, true>(s, (int)grid, qm, km, vm, p)
            : launch_attn_prefill<128, false>(s, (int)grid, qm, km, vm, p);
  else
    e = fp8 ? launch_attn_prefill<64, true>(s, (int)grid, qm, km, vm, p)
            : launch_attn_prefill<64, false>(s, (int)grid, qm, km, vm, p);
  CUDA_TRY(c, e);
  return MOE_OK;
}

moe_status attend(moe_ctx *c, const moe_kv_batch *b, const void *q, int64_t q_stride, int max_T, float scale,
                  int window, int n_sink, void *out, int64_t out_stride, void *stream, const char *who) {
  moe_status st = attn_check(c, b, who);
  if (st != MOE_OK) return st;
  if (!b) return fail(c, MOE_ERR_INVALID_ARG, "%s: no batch", who);
  const moe_ctx::Attn &a = c->attn;
  const long long width = (long long)a.n_q * a.dim;
  if (max_T < 1 || !(scale > 0.f) || scale > 1e30f || window < 0 || n_sink < 0)
    return fail(c, MOE_ERR_INVALID_ARG, "%s: bad arguments (max_T=%d scale=%g window=%d n_sink=%d)", who, max_T,
                scale, window, n_sink);
  if (b->n_rows == 0) return MOE_OK;
  if (!rows_ok(q, q_stride, width, 16) || !rows_ok(out, out_stride, width, 16))
    return fail(c, MOE_ERR_INVALID_ARG, "%s: q and out rows are 16-byte aligned, at least n_q * head_dim apart", who);
  c->last_stream = (cudaStream_t)stream;
  // More rows of a KV head than one row block of the window kernel: 33 rows of
  // 16 heads over 2 KV heads behind 16384 keys take 45 us in the chunk kernel,
  // 64 us there; 128 rows 49 us and 99 us.  (max_T is the caller's word; the
  // window kernel takes more rows than it says in further row blocks.)  With
  // more than 32 rows its four row tiles leave a warp no others to hide behind,
  // so a bf16 cache goes to the chunk kernel while its blocks fill at most half
  // of the SMs: 8 windows of 64 rows over 8000 keys 48 us against 65 us; but 64
  // windows over up to 4096 keys 71 us against 57 us, and e4m3 tiles, converted
  // there, 26 us against 23 us for 16 windows of 40 rows over 1000 keys.
  const long long kv_rows = (long long)max_T * (a.n_q / a.n_kv);
  const long long chunk_blocks = ((long long)b->n_rows * a.n_q / kApRows / a.n_kv + b->n_seqs) * a.n_kv;
  if (kv_rows > kAtMaxRows || (kv_rows > 32 && a.cache == MOE_KV_BF16 && 2 * chunk_blocks <= c->n_sm))
    return attend_chunk(c, b, q, q_stride, scale, window, n_sink, out, out_stride, (cudaStream_t)stream, who);
  CUtensorMap km, vm;
  const int box = a.page < kAtTile ? a.page : kAtTile;
  if (!encode_cache_map(&km, a, b->k, b->n_pages, box) || !encode_cache_map(&vm, a, b->v, b->n_pages, box))
    return fail(c, MOE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  AttnParams p{};
  p.q = (const uint16_t *)q;
  p.out = (uint16_t *)out;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.page_table = b->page_table;
  p.row_off = b->row_off;
  p.kv_len = b->kv_len;
  p.k_scale = b->k_scale;
  p.v_scale = b->v_scale;
  p.scale_log2 = scale * 1.44269504088896340736f;
  p.window = window;
  p.n_sink = n_sink;
  p.n_rows = b->n_rows;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.group = a.n_q / a.n_kv;
  p.n_pages = b->n_pages;
  p.n_seqs = b->n_seqs;
  p.max_pages = b->max_pages;
  p.page = a.page;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page) ++p.page_shift;
  p.min_units = 4;
  p.ws = a.ws;
  p.arrived = a.arrived;
  p.status = a.status;
  cudaStream_t s = (cudaStream_t)stream;
  const int rows = (int)std::min<long long>((long long)std::min(max_T, b->n_rows) * p.group, kAtMaxRows);
  const bool fp8 = a.cache == MOE_KV_E4M3;
  cudaError_t e;
  if (a.dim == 128)
    e = fp8 ? launch_attn<128, true>(c, s, km, vm, p, rows) : launch_attn<128, false>(c, s, km, vm, p, rows);
  else
    e = fp8 ? launch_attn<64, true>(c, s, km, vm, p, rows) : launch_attn<64, false>(c, s, km, vm, p, rows);
  CUDA_TRY(c, e);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_attn_configure(moe_ctx *c, int n_q, int n_kv, int head_dim, int page_size, int cache_type) {
  if (!c) return MOE_ERR_INVALID_ARG;
  moe_ctx::Attn &a = c->attn;
  if (a.ready) return fail(c, MOE_ERR_STATE, "moe_attn_configure was called before");
  if (n_q < 1 || n_q > 1024 || n_kv < 1 || n_q % n_kv || page_size < 16 || page_size > 256 ||
      (page_size & (page_size - 1)) || (cache_type != MOE_KV_BF16 && cache_type != MOE_KV_E4M3))
    return fail(c, MOE_ERR_INVALID_ARG, "moe_attn_configure: bad geometry (n_q=%d n_kv=%d page_size=%d)", n_q, n_kv,
                page_size);
  if (head_dim != 64 && head_dim != 128)
    return fail(c, MOE_ERR_NOT_SUPPORTED, "moe_attn_configure: head_dim %d (64 and 128 are built)", head_dim);
  int dev = -1;
  CUDA_TRY(c, cudaGetDevice(&dev));
  if (dev != c->device)
    return fail(c, MOE_ERR_INVALID_ARG, "moe_attn_configure: the current device is %d, the context's %d", dev,
                c->device);
  const bool fp8 = cache_type == MOE_KV_E4M3;
  int blocks = kAtGridPerSm;
  cudaError_t e = head_dim == 128 ? (fp8 ? setup_attn_all<128, true>(&blocks) : setup_attn_all<128, false>(&blocks))
                                  : (fp8 ? setup_attn_all<64, true>(&blocks) : setup_attn_all<64, false>(&blocks));
  if (e == cudaSuccess)
    e = head_dim == 128 ? (fp8 ? setup_attn_prefill<128, true>() : setup_attn_prefill<128, false>())
                        : (fp8 ? setup_attn_prefill<64, true>() : setup_attn_prefill<64, false>());
  CUDA_TRY(c, e);
  if (blocks < 1) return fail(c, MOE_ERR_CUDA, "moe_attn_configure: the attention kernel does not fit this device");
  a.grid = c->n_sm * blocks;
  const size_t head = 256 + ((size_t)a.grid * sizeof(unsigned int) + 255) / 256 * 256;
  const size_t bytes = head + (size_t)a.grid * 2 * kAtMaxRows * (head_dim + 2) * sizeof(float);
  CUDA_TRY(c, cudaMalloc(&a.mem, bytes));
  e = cudaMemset(a.mem, 0, head);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // before any call on a non-blocking stream
  if (e != cudaSuccess) {
    dfree(a.mem);
    CUDA_TRY(c, e);
  }
  a.status = (int *)a.mem;
  a.arrived = (unsigned int *)(a.mem + 256);
  a.ws = (float *)(a.mem + head);
  a.n_q = n_q;
  a.n_kv = n_kv;
  a.dim = head_dim;
  a.page = page_size;
  a.cache = cache_type;
  a.ready = true;
  return MOE_OK;
}

moe_status moe_qk_norm_rope(moe_ctx *c, int n_rows, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                            const int32_t *pos, const moe_qk_norm *norm, const moe_rope *rope, void *q_out,
                            int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream) {
  if (!c) return MOE_ERR_INVALID_ARG;
  moe_status st = attn_check(c, nullptr, "moe_qk_norm_rope");
  if (st == MOE_OK) st = rope_check(c, norm, rope, "moe_qk_norm_rope");
  if (st != MOE_OK) return st;
  const moe_ctx::Attn &a = c->attn;
  const long long wq = (long long)a.n_q * a.dim, wk = (long long)a.n_kv * a.dim;
  if (n_rows < 0 || (rope && !pos) || (n_rows > 0 && (!rows_ok(q, q_stride, wq, 8) || !rows_ok(k, k_stride, wk, 8) ||
                                                      !rows_ok(q_out, q_out_stride, wq, 8) ||
                                                      !rows_ok(k_out, k_out_stride, wk, 8))))
    return fail(c, MOE_ERR_INVALID_ARG, "moe_qk_norm_rope: bad arguments (n_rows=%d)", n_rows);
  if (n_rows == 0) return MOE_OK;
  KvRowsParams p{};
  p.q = (const uint16_t *)q;
  p.k = (const uint16_t *)k;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out = (uint16_t *)q_out;
  p.k_out = (uint16_t *)k_out;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.pos = pos;
  p.n_rows = n_rows;
  c->last_stream = (cudaStream_t)stream;
  return kv_rows(c, (cudaStream_t)stream, p, norm, rope, 0);
}

moe_status moe_kv_append(moe_ctx *c, const moe_kv_batch *b, const void *q, int64_t q_stride, const void *k,
                         int64_t k_stride, const void *v, int64_t v_stride, const moe_qk_norm *norm,
                         const moe_rope *rope, void *q_out, int64_t q_out_stride, void *stream) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (!b) return fail(c, MOE_ERR_INVALID_ARG, "moe_kv_append: no batch");
  moe_status st = attn_check(c, b, "moe_kv_append");
  if (st == MOE_OK) st = rope_check(c, norm, rope, "moe_kv_append");
  if (st != MOE_OK) return st;
  const moe_ctx::Attn &a = c->attn;
  const long long wq = (long long)a.n_q * a.dim, wk = (long long)a.n_kv * a.dim;
  if (b->n_rows == 0) return MOE_OK;
  if (!rows_ok(k, k_stride, wk, 8) || !rows_ok(v, v_stride, wk, 8) || !q != !q_out ||
      (q && (!rows_ok(q, q_stride, wq, 8) || !rows_ok(q_out, q_out_stride, wq, 8))))
    return fail(c, MOE_ERR_INVALID_ARG, "moe_kv_append: bad rows");
  KvRowsParams p{};
  p.q = (const uint16_t *)q;
  p.k = (const uint16_t *)k;
  p.v = (const uint16_t *)v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = (uint16_t *)q_out;
  p.q_out_stride = q_out_stride;
  p.n_rows = b->n_rows;
  p.k_cache = (uint8_t *)b->k;
  p.v_cache = (uint8_t *)b->v;
  p.k_scale = b->k_scale;
  p.v_scale = b->v_scale;
  p.page_table = b->page_table;
  p.row_off = b->row_off;
  p.kv_len = b->kv_len;
  p.n_pages = b->n_pages;
  p.n_seqs = b->n_seqs;
  p.max_pages = b->max_pages;
  c->last_stream = (cudaStream_t)stream;
  return kv_rows(c, (cudaStream_t)stream, p, norm, rope, a.cache == MOE_KV_E4M3 ? 2 : 1);
}

moe_status moe_attn_forward(moe_ctx *c, const moe_kv_batch *b, const void *q, int64_t q_stride, int max_T,
                            float scale, int window, int n_sink, void *out, int64_t out_stride, void *stream) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (max_T > kDecMaxT)
    return fail(c, MOE_ERR_INVALID_ARG, "moe_attn_forward: max_T=%d, at most %d (moe_attn_prefill takes chunks)", max_T,
                kDecMaxT);
  return attend(c, b, q, q_stride, max_T, scale, window, n_sink, out, out_stride, stream, "moe_attn_forward");
}

moe_status moe_attn_prefill(moe_ctx *c, const moe_kv_batch *b, const void *q, int64_t q_stride, int max_T,
                            float scale, int window, int n_sink, void *out, int64_t out_stride, void *stream) {
  if (!c) return MOE_ERR_INVALID_ARG;
  return attend(c, b, q, q_stride, max_T, scale, window, n_sink, out, out_stride, stream, "moe_attn_prefill");
}

}  // extern "C"
