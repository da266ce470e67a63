// Entry points of a serving step around the attention (part of cpattn.cu's
// translation unit): plans and trims of the paged cache, norms and rotations of
// heads, and appending to the pages.  Contracts: include/cpattn.h.
#pragma once

namespace {

// CTAs of a plan or trim over `items` rows or pages at most: a cluster, so that
// they can wait for one another.
int plan_ctas(long long items) {
  return items <= cpattn::kPlanThreads ? 1 : cpattn::kPlanMaxCtas;
}

cpattn_status launch_plan(cpattn_ctx* ctx, void (*kernel)(cpattn::PagedPlanParams), int ctas,
                          size_t smem, cudaStream_t st, const cpattn::PagedPlanParams& p,
                          const char* what) {
  cudaLaunchAttribute attr[2];
  if (!ctx->plan_ready) {  // (the largest batches take a little more than 48 KB)
    for (const auto k : {cpattn::paged_plan_kernel, cpattn::paged_trim_kernel}) {
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 3 * 4 * CPATTN_MAX_PAGED_SEQS);
      if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaFuncSetAttribute(paged plan)");
    }
    ctx->plan_ready = true;
  }
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(cpattn::kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return cuda_fail(ctx, e, what);
  return after_launch(ctx, st, what);
}

// Rows of `heads` heads, `stride` elements apart, at `base`.
cpattn_status check_rows(cpattn_ctx* ctx, const char* name, const void* base, int64_t stride, int heads) {
  if (base == nullptr || !aligned16(base))
    return fail(ctx, CPATTN_E_INVALID, std::string(name) + ": must be 16-byte aligned and not NULL");
  if (stride < static_cast<int64_t>(heads) * ctx->cfg.head_dim || stride % 8 != 0)
    return fail(ctx, CPATTN_E_INVALID,
                std::string(name) + ": row stride below a row's heads, or no multiple of 8");
  return CPATTN_OK;
}

// What the dense and the appending form check alike.
cpattn_status check_norm_rope(cpattn_ctx* ctx, const cpattn_norm_rope_desc* d, int32_t num_rows,
                              const int32_t* positions, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, void* q_out, int64_t q_out_stride,
                              cpattn::NormRopeParams* p) {
  if (d == nullptr) return fail(ctx, CPATTN_E_INVALID, "norm_rope: the description must not be NULL");
  const cpattn_config& c = ctx->cfg;
  if (num_rows < 0) return fail(ctx, CPATTN_E_INVALID, "num_rows must be >= 0");
  if (d->rotary_dim < 0 || d->rotary_dim > c.head_dim || d->rotary_dim % 8 != 0)
    return fail(ctx, CPATTN_E_INVALID, "rotary_dim must be a multiple of 8 in [0, head_dim]");
  if (d->rotary_dim > 0 && (d->rope_steps == nullptr || (reinterpret_cast<uintptr_t>(d->rope_steps) & 7u) != 0))
    return fail(ctx, CPATTN_E_INVALID, "rope_steps: must be 8-byte aligned and not NULL");
  if (!(d->eps >= 0.f)) return fail(ctx, CPATTN_E_INVALID, "eps must be >= 0");
  if (!aligned4(d->q_weight) || !aligned4(d->k_weight))
    return fail(ctx, CPATTN_E_INVALID, "norm weights must be 4-byte aligned");
  if (positions == nullptr || !aligned4(positions))
    return fail(ctx, CPATTN_E_INVALID, "positions: must be 4-byte aligned and not NULL");
  cpattn_status s = check_rows(ctx, "q", q, q_stride, c.num_q_heads);
  if (s == CPATTN_OK) s = check_rows(ctx, "k", k, k_stride, c.num_kv_heads);
  if (s == CPATTN_OK) s = check_rows(ctx, "q_out", q_out, q_out_stride, c.num_q_heads);
  if (s != CPATTN_OK) return s;
  p->q = static_cast<const __nv_bfloat16*>(q);
  p->k = static_cast<const __nv_bfloat16*>(k);
  p->v = nullptr;
  p->q_out = static_cast<__nv_bfloat16*>(q_out);
  p->k_out = nullptr;
  p->q_weight = d->q_weight;
  p->k_weight = d->k_weight;
  p->steps = reinterpret_cast<const unsigned long long*>(d->rope_steps);
  p->positions = positions;
  p->slots = nullptr;
  p->q_stride = q_stride;
  p->k_stride = k_stride;
  p->v_stride = 0;
  p->q_out_stride = q_out_stride;
  p->k_out_stride = 0;
  p->status = ctx->d_status;
  p->eps = d->eps;
  p->scale = d->rope_scale;
  p->weight_f32 = d->weight_f32 != 0 ? 1 : 0;
  p->rows = num_rows;
  p->nq = c.num_q_heads;
  p->nkv = c.num_kv_heads;
  p->rot = d->rotary_dim;
  p->neighbours = d->interleaved != 0 ? 1 : 0;
  return CPATTN_OK;
}

cpattn_status launch_norm_rope(cpattn_ctx* ctx, void (*kernel)(cpattn::NormRopeParams), int format,
                               cpattn::NormRopeParams* p, cudaStream_t st, const char* what) {
  if (ctx->d_status == nullptr) return fail(ctx, CPATTN_E_CUDA, "no CUDA device");
  // Batches of one unit where whole ones leave less than a warp for every slot of
  // the GPU: few rows are a matter of latency.
  const bool append = format >= 0;
  const int per = 32 / (ctx->cfg.head_dim / 8);
  const int uq = (p->nq + per - 1) / per, uk = (p->nkv + per - 1) / per;
  constexpr int WARPS = cpattn::kNormThreads / 32;
  const long long room = static_cast<long long>(cpattn::kNormBlocks) * std::max(ctx->num_sms, 1);
  long long batches = 0;
  for (int batch : {cpattn::kNormBatch, 1}) {
    p->batch = batch;
    batches = static_cast<long long>(p->rows) *
              ((uq + batch - 1) / batch + (append ? 2 : 1) * ((uk + batch - 1) / batch));
    if (batches >= room * WARPS) break;
  }
  // Many rows: blocks of a row per warp, of which the SMs take the next as they end
  // one, or equal slices for resident blocks, which end apart.  A block's beginning
  // (weights, frequencies, a barrier) wants rows of 8 KB of Q and K, and 16 KB where K and
  // V are quantised, which balances the slices too.  Slices and in turn, us, by bytes of a row:
  //   dense   2560: 62.9, 89.2   5120: 76.8, 76.0   9216: 59.6, 50.6   17408: 124, 107
  //   bf16    2560: 80.4, 107    5120: 91.8, 91.2   9216: 67.8, 59.8   17408: 136, 113
  //   e4m3    5120: 87.9, 105    9216: 60.5, 62.2  17408: 136, 113     18432: 75.7, 65.4
  //   e2m1    5120: 97.7, 115    9216: 56.0, 63.9  17408: 135, 114     18432: 72.4, 63.4
  // (4 + 1 and 8 + 2 heads of 256, 32 + 4 of 128, 32 + 2 of 256, 64 + 8 of 128; 60000,
  // 40000, 17421, 20161, 10000 rows; 1024 B, 200000 rows of 1 + 1 of 256: 168, 269.)  Few
  // rows have to be spread (2000 rows, 32 + 4 of 128: in turn 11.4 us, slices 10.4).
  const int row_bytes = 2 * ctx->cfg.head_dim * (p->nq + p->nkv);
  const bool rows_in_turn = p->batch > 1 && row_bytes >= (format > 0 ? 16384 : 8192) &&
                            p->rows >= 2 * room * WARPS;
  const int grid = static_cast<int>(rows_in_turn ? (p->rows + WARPS - 1) / WARPS
                                                 : std::min<long long>((batches + WARPS - 1) / WARPS, room));
  const size_t smem = cpattn::norm_rope_smem(format);
  bool& ready = ctx->norm_ready[p->neighbours][format < 0 ? 0 : 1 + std::min<int>(format, 2)];
  if (!ready) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaFuncSetAttribute(norm_rope)");
    ready = true;
  }
  return launch_dependent(ctx, kernel, dim3(grid), cpattn::kNormThreads, smem, st, *p, what);
}

}  // namespace

extern "C" {

cpattn_status cpattn_rope_steps(const double* inv_freq, int32_t n, uint64_t* steps) {
  if (n < 0 || (n > 0 && (inv_freq == nullptr || steps == nullptr))) return CPATTN_E_INVALID;
  // 2^128 / (2 pi), upper and lower 64 bits.
  constexpr uint64_t hi = 0x28BE60DB9391054AULL, lo = 0x7F09D5F47D4D3770ULL;
  for (int32_t i = 0; i < n; ++i) {
    if (!(std::fabs(inv_freq[i]) <= 1048576.0)) return CPATTN_E_INVALID;  // (NaN too)
    int e = 0;
    const double f = std::frexp(std::fabs(inv_freq[i]), &e);              // f in [1/2, 1)
    const uint64_t m = static_cast<uint64_t>(std::ldexp(f, 53));          // |inv_freq| = m 2^(e - 53)
    // m (hi 2^64 + lo) 2^(e - 53 - 64): turns, times 2^64; e <= 21.
    const unsigned __int128 x = static_cast<unsigned __int128>(m) * hi +
                                ((static_cast<unsigned __int128>(m) * lo) >> 64);
    const int shift = 53 - e;                                             // >= 32
    uint64_t s = 0;
    if (shift <= 118) {
      const unsigned __int128 half = static_cast<unsigned __int128>(1) << (shift - 1);
      s = static_cast<uint64_t>((x + half) >> shift);
    }
    steps[i] = inv_freq[i] < 0 ? 0 - s : s;
  }
  return CPATTN_OK;
}

cpattn_status cpattn_norm_rope(cpattn_ctx* ctx, const cpattn_norm_rope_desc* desc, int32_t num_rows,
                               const int32_t* positions, const void* q, int64_t q_stride,
                               const void* k, int64_t k_stride, void* q_out, int64_t q_out_stride,
                               void* k_out, int64_t k_out_stride, void* stream) try {
  if (ctx == nullptr) return CPATTN_E_INVALID;
  cpattn::NormRopeParams p = {};
  cpattn_status s = check_norm_rope(ctx, desc, num_rows, positions, q, q_stride, k, k_stride, q_out,
                                    q_out_stride, &p);
  if (s == CPATTN_OK) s = check_rows(ctx, "k_out", k_out, k_out_stride, ctx->cfg.num_kv_heads);
  if (s == CPATTN_OK) s = check_device(ctx);
  if (s != CPATTN_OK) return s;
  if (num_rows == 0) return CPATTN_OK;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.k_out_stride = k_out_stride;
  const auto kernel =
      ctx->cfg.head_dim == 128
          ? (p.neighbours ? cpattn::norm_rope_kernel<128, true, -1> : cpattn::norm_rope_kernel<128, false, -1>)
          : (p.neighbours ? cpattn::norm_rope_kernel<256, true, -1> : cpattn::norm_rope_kernel<256, false, -1>);
  return launch_norm_rope(ctx, kernel, -1, &p, static_cast<cudaStream_t>(stream), "norm_rope launch");
} catch (...) {
  return CPATTN_E_NOMEM;
}

cpattn_status cpattn_norm_rope_write_kv(cpattn_ctx* ctx, const cpattn_norm_rope_desc* desc,
                                        const cpattn_pages* pages, int32_t num_rows,
                                        const int32_t* positions, const int32_t* slots,
                                        const void* q, int64_t q_stride, const void* k,
                                        int64_t k_stride, const void* v, int64_t v_stride,
                                        void* q_out, int64_t q_out_stride, void* stream) try {
  if (ctx == nullptr) return CPATTN_E_INVALID;
  cpattn::NormRopeParams p = {};
  cpattn_status s = check_pages(ctx, pages, 1, &p.pool);
  if (s == CPATTN_OK)
    s = check_norm_rope(ctx, desc, num_rows, positions, q, q_stride, k, k_stride, q_out, q_out_stride, &p);
  if (s == CPATTN_OK) s = check_rows(ctx, "v", v, v_stride, ctx->cfg.num_kv_heads);
  if (s != CPATTN_OK) return s;
  if (slots == nullptr || !aligned4(slots))
    return fail(ctx, CPATTN_E_INVALID, "slots: must be 4-byte aligned and not NULL");
  if (num_rows == 0) return CPATTN_OK;
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.v_stride = v_stride;
  p.slots = slots;
  const auto kernel =
      ctx->cfg.head_dim == 128
          ? (p.neighbours ? CPATTN_BY_FORMAT(cpattn::norm_rope_kernel, pages->format, 128, true)
                          : CPATTN_BY_FORMAT(cpattn::norm_rope_kernel, pages->format, 128, false))
          : (p.neighbours ? CPATTN_BY_FORMAT(cpattn::norm_rope_kernel, pages->format, 256, true)
                          : CPATTN_BY_FORMAT(cpattn::norm_rope_kernel, pages->format, 256, false));
  return launch_norm_rope(ctx, kernel, pages->format, &p, static_cast<cudaStream_t>(stream),
                          "norm_rope_write_kv launch");
} catch (...) {
  return CPATTN_E_NOMEM;
}

cpattn_status cpattn_paged_plan(cpattn_ctx* ctx, const cpattn_pages* pages, int32_t num_seqs,
                                int32_t num_rows, const int32_t* cache_lens,
                                const int32_t* new_lens, int32_t* free_pages, int32_t* free_count,
                                int32_t* lens, int32_t* row_starts, int32_t* positions,
                                int32_t* slots, void* stream) try {
  if (ctx == nullptr) return CPATTN_E_INVALID;
  cpattn::PagedPlanParams p = {};
  cpattn_status s = check_pages(ctx, pages, num_seqs, &p.pool);
  if (s != CPATTN_OK) return s;
  if (num_rows < 0) return fail(ctx, CPATTN_E_INVALID, "num_rows must be >= 0");
  for (const void* a : {static_cast<const void*>(cache_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(free_pages), static_cast<const void*>(free_count),
                        static_cast<const void*>(lens), static_cast<const void*>(row_starts)})
    if (a == nullptr || !aligned4(a))
      return fail(ctx, CPATTN_E_INVALID, "device arrays must be 4-byte aligned and not NULL");
  if (!aligned4(positions) || !aligned4(slots) ||
      (num_rows > 0 && (positions == nullptr || slots == nullptr)))
    return fail(ctx, CPATTN_E_INVALID, "positions, slots: must be 4-byte aligned and not NULL");
  if (ctx->d_status == nullptr) return fail(ctx, CPATTN_E_CUDA, "no CUDA device");
  p.table = const_cast<int*>(pages->block_table);
  p.cache_lens = cache_lens;
  p.new_lens = new_lens;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.lens = lens;
  p.row_starts = row_starts;
  p.positions = positions;
  p.slots = slots;
  p.status = ctx->d_status;
  p.num_seqs = num_seqs;
  p.rows = num_rows;
  return launch_plan(ctx, cpattn::paged_plan_kernel, plan_ctas(num_rows),
                     3 * sizeof(int) * static_cast<size_t>(num_seqs),
                     static_cast<cudaStream_t>(stream), p, "paged plan launch");
} catch (...) {
  return CPATTN_E_NOMEM;
}

cpattn_status cpattn_paged_trim(cpattn_ctx* ctx, const cpattn_pages* pages, int32_t num_seqs,
                                const int32_t* lens, const int32_t* keep, int32_t* free_pages,
                                int32_t* free_count, void* stream) try {
  if (ctx == nullptr) return CPATTN_E_INVALID;
  cpattn::PagedPlanParams p = {};
  cpattn_status s = check_pages(ctx, pages, num_seqs, &p.pool);
  if (s != CPATTN_OK) return s;
  for (const void* a : {static_cast<const void*>(lens), static_cast<const void*>(keep),
                        static_cast<const void*>(free_pages), static_cast<const void*>(free_count)})
    if (a == nullptr || !aligned4(a))
      return fail(ctx, CPATTN_E_INVALID, "device arrays must be 4-byte aligned and not NULL");
  if (ctx->d_status == nullptr) return fail(ctx, CPATTN_E_CUDA, "no CUDA device");
  p.table = const_cast<int*>(pages->block_table);
  p.lens = const_cast<int*>(lens);
  p.keep = keep;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.status = ctx->d_status;
  p.num_seqs = num_seqs;
  const long long most = std::min<long long>(static_cast<long long>(num_seqs) * pages->max_pages,
                                             pages->num_pages);
  return launch_plan(ctx, cpattn::paged_trim_kernel, plan_ctas(most),
                     2 * sizeof(int) * static_cast<size_t>(num_seqs),
                     static_cast<cudaStream_t>(stream), p, "paged trim launch");
} catch (...) {
  return CPATTN_E_NOMEM;
}

}  // extern "C"
