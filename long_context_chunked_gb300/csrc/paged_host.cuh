// Entry points of the paged KV cache (part of cpattn.cu's translation unit):
// argument checks and launches.  Contracts: include/cpattn.h.
#pragma once

namespace {

// Checks shared by the paged entry points; *out receives the device view.
cpattn_status check_pages(cpattn_ctx* ctx, const cpattn_pages* pages, int32_t num_seqs,
                          cpattn::PagedPool* out) {
  if (num_seqs < 1) return fail(ctx, CPATTN_E_INVALID, "num_seqs must be >= 1");
  if (num_seqs > CPATTN_MAX_PAGED_SEQS)
    return fail(ctx, CPATTN_E_UNSUPPORTED, "num_seqs exceeds CPATTN_MAX_PAGED_SEQS");
  if (pages == nullptr) return fail(ctx, CPATTN_E_INVALID, "pages must not be NULL");
  if (pages->format != CPATTN_PAGES_BF16 && pages->format != CPATTN_PAGES_E4M3)
    return fail(ctx, CPATTN_E_INVALID, "pages: unknown format");
  int shift = 4;
  while (shift < 8 && (1 << shift) != pages->page_size) ++shift;
  if ((1 << shift) != pages->page_size)
    return fail(ctx, CPATTN_E_UNSUPPORTED, "pages: page_size must be 16, 32, 64, 128 or 256");
  if (pages->num_pages < 1 || pages->max_pages < 1 || pages->table_stride < pages->max_pages)
    return fail(ctx, CPATTN_E_INVALID, "pages: num_pages, max_pages >= 1, table_stride >= max_pages");
  const long long nkv = ctx->cfg.num_kv_heads;
  if (static_cast<long long>(pages->num_pages) * pages->page_size * nkv >= (1LL << 31) ||
      static_cast<long long>(pages->max_pages) * pages->page_size >= (1LL << 31))
    return fail(ctx, CPATTN_E_UNSUPPORTED, "pages: pool rows or a sequence's capacity exceed 2^31");
  if (pages->k_pages == nullptr || pages->v_pages == nullptr || pages->block_table == nullptr)
    return fail(ctx, CPATTN_E_INVALID, "pages: pointers must not be NULL");
  if (!aligned16(pages->k_pages) || !aligned16(pages->v_pages) || !aligned4(pages->block_table))
    return fail(ctx, CPATTN_E_INVALID, "pages: pools 16-byte, table 4-byte aligned");
  if (pages->format == CPATTN_PAGES_E4M3 &&
      (pages->k_scales == nullptr || pages->v_scales == nullptr || !aligned16(pages->k_scales) ||
       !aligned16(pages->v_scales)))
    return fail(ctx, CPATTN_E_INVALID, "pages: e4m3 needs 16-byte aligned scales");
  out->k = pages->k_pages;
  out->v = pages->v_pages;
  out->k_scales = pages->k_scales;
  out->v_scales = pages->v_scales;
  out->table = pages->block_table;
  out->table_stride = pages->table_stride;
  out->num_pages = pages->num_pages;
  out->max_pages = pages->max_pages;
  out->page_shift = shift;
  out->nkv = ctx->cfg.num_kv_heads;
  return check_device(ctx);
}

// kv heads a warp of the paged copies takes of its rows (`units` of them): 4 or
// 2, which share the look-ups, where that leaves 16 warps per SM, else 1.
// (e4m3 write of 17421 tokens, 4 heads of 128: 16.4 us by 4 heads, 16.8 by 2, 18.3
// by 1, before launches overlapped.)
int heads_per_item(const cpattn_ctx* ctx, long long units) {
  const int nkv = ctx->cfg.num_kv_heads;
  for (int h = 4; h > 1; h /= 2)
    if (h <= nkv && units * ((nkv + h - 1) / h) >= 16LL * std::max(ctx->num_sms, 1)) return h;
  return 1;
}

int copy_grid(const cpattn_ctx* ctx, long long units, int hpi) {
  const long long items = units * ((ctx->cfg.num_kv_heads + hpi - 1) / hpi);
  return static_cast<int>(std::max(1LL, std::min<long long>((items + 7) / 8,
                                                            static_cast<long long>(ctx->num_sms) * 8)));
}

// Launch as a programmatic dependent of what is ahead on the stream: the launch
// overlaps its end, and the kernel waits for it before it touches memory.
template <class Params>
cpattn_status launch_dependent(cpattn_ctx* ctx, void (*kernel)(Params), dim3 grid, int threads,
                               size_t smem, cudaStream_t st, const Params& p, const char* what) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return cuda_fail(ctx, e, what);
  return after_launch(ctx, st, what);
}

template <int ROWS>
cpattn_status launch_paged_write(cpattn_ctx* ctx, const cpattn::PagedWriteParams& p, bool q8, int grid,
                                 cudaStream_t st) {
  const auto kernel = ctx->cfg.head_dim == 128 ? (q8 ? cpattn::paged_write_kernel<128, true, ROWS>
                                                     : cpattn::paged_write_kernel<128, false, ROWS>)
                                               : (q8 ? cpattn::paged_write_kernel<256, true, ROWS>
                                                     : cpattn::paged_write_kernel<256, false, ROWS>);
  return launch_dependent(ctx, kernel, dim3(grid), 256, 0, st, p, "paged write launch");
}

// CTAs of a decode launch: at most one per SM (and the join's table of pieces).
int decode_max_ctas(const cpattn_ctx* ctx) {
  return std::min(ctx->num_sms > 0 ? ctx->num_sms : 152, cpattn::kJoinPieces - 32);
}

// Workspace of a decode: O, then (m, l) of every worker's first and last row,
// then the rows that were cut.  It depends on neither the lengths nor the
// number of sequences.
struct DecodeWorkspace {
  uint64_t ml, cut, total;  // byte offsets
};
DecodeWorkspace decode_workspace(const cpattn_ctx* ctx) {
  // 8 workers per CTA, at most 16 rows per piece.
  const uint64_t workers = static_cast<uint64_t>(decode_max_ctas(ctx)) * 8;
  const uint64_t rows = 2 * workers * 16;
  DecodeWorkspace w;
  w.ml = cpattn::align256(rows * ctx->cfg.head_dim * sizeof(float));
  w.cut = w.ml + cpattn::align256(rows * sizeof(float2));
  w.total = w.cut + cpattn::align256(workers * sizeof(cpattn::DecodeCut));
  return w;
}

template <int HD, bool Q8, int NB>
cpattn_status launch_decode(cpattn_ctx* ctx, const cpattn_pages* pages,
                            cpattn::PagedDecodeParams* p, cudaStream_t st) {
  using Ly = cpattn::DecodeLayout<HD, Q8, NB>;
  static_assert(Ly::NW <= 8 && Ly::HEADS <= 16, "decode_workspace");
  bool& ready = ctx->decode_ready[HD == 256][Q8];
  if (!ready) {
    cudaError_t e = cudaFuncSetAttribute(cpattn::paged_decode_kernel<HD, Q8, NB>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Ly::SMEM_BYTES);
    // The join asks for the decode kernel's division of the SM's memory, so
    // that the SMs need not change it between the two.
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(cpattn::paged_join_kernel<HD>,
                               cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaFuncSetAttribute(paged decode)");
    ready = true;
  }
  const uint64_t rb = static_cast<uint64_t>(HD) * Ly::ESZ;
  const uint32_t box_rows = static_cast<uint32_t>(std::min(pages->page_size, Ly::WT));
  const CUtensorMapDataType type =
      Q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t rows = static_cast<uint64_t>(p->pool_rows);
  if (!encode3d(&p->tm_k, pages->k_pages, HD, 1, rows, rb, rb, Ly::BOXW, 1, box_rows, type) ||
      !encode3d(&p->tm_v, pages->v_pages, HD, 1, rows, rb, rb, Ly::BOXW, 1, box_rows, type))
    return fail(ctx, CPATTN_E_CUDA, "cuTensorMapEncodeTiled failed");
  // The lengths are known on the device only: the grid is sized for the most
  // tiles they can ask for, and a CTA without a tile leaves at once.
  const long long rows_all = static_cast<long long>(p->num_seqs) * p->pool.nkv * p->hblocks;
  const long long tiles =
      (static_cast<long long>(pages->max_pages) * pages->page_size + Ly::WT - 1) / Ly::WT;
  p->num_ctas = static_cast<int>(std::min<long long>(
      decode_max_ctas(ctx), (rows_all * std::min(tiles, 1LL << 20) + Ly::NW - 1) / Ly::NW));
  p->workers = Ly::NW;
  p->piece_rows = Ly::HEADS;
  p->by_row = rows_all <= p->num_ctas ? 1 : 0;
  if (ctx->bar_counts != nullptr) {
    if (ctx->bar_counts_bytes < static_cast<size_t>(p->num_ctas) * cpattn::kCountRecord * 4)
      return fail(ctx, CPATTN_E_INVALID, "barrier-count records smaller than the launch");
    p->bar_counts = ctx->bar_counts;
  }
  cpattn_status s = launch_dependent(ctx, cpattn::paged_decode_kernel<HD, Q8, NB>, dim3(p->num_ctas),
                                     Ly::THREADS, Ly::SMEM_BYTES, st, *p, "paged decode launch");
  // Rows of one tile are never cut, nor are few short ones (decode_slices).
  if (s != CPATTN_OK || tiles == 1 || (p->by_row && tiles <= cpattn::kBriefRounds * Ly::NW)) return s;
  // Few rows: one block per row and as many parts of its heads as fill the
  // GPU, each with the threads for many pieces.  Many rows have few pieces
  // each: four blocks per CTA of the decode share the rows that begin there.
  const int blocks = p->by_row ? static_cast<int>(rows_all) : p->num_ctas;
  const int parts = p->by_row ? std::min({std::max(1, ctx->num_sms / blocks), p->group, Ly::HEADS}) : 4;
  return launch_dependent(ctx, cpattn::paged_join_kernel<HD>, dim3(blocks, parts),
                          p->by_row ? cpattn::kJoinThreads : 256, 0, st, *p, "paged join launch");
}

}  // namespace

extern "C" {

cpattn_status cpattn_paged_write_kv(cpattn_ctx* ctx, const cpattn_pages* pages, int32_t num_seqs,
                                    int32_t num_rows, const int32_t* cache_lens,
                                    const int32_t* row_starts, const void* k_new,
                                    const void* v_new, void* stream) try {
  if (ctx == nullptr) return CPATTN_E_INVALID;
  cpattn::PagedWriteParams p;
  cpattn_status s = check_pages(ctx, pages, num_seqs, &p.pool);
  if (s != CPATTN_OK) return s;
  if (num_rows < 0) return fail(ctx, CPATTN_E_INVALID, "num_rows must be >= 0");
  if (row_starts == nullptr && num_rows != num_seqs)
    return fail(ctx, CPATTN_E_INVALID, "without row_starts, num_rows must equal num_seqs");
  if (num_rows == 0) return CPATTN_OK;
  if (cache_lens == nullptr || k_new == nullptr || v_new == nullptr)
    return fail(ctx, CPATTN_E_INVALID, "device pointers must not be NULL");
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(cache_lens) || !aligned4(row_starts))
    return fail(ctx, CPATTN_E_INVALID, "k_new, v_new 16-byte, integer arrays 4-byte aligned");
  if (ctx->d_status == nullptr) return fail(ctx, CPATTN_E_CUDA, "no CUDA device");
  p.k_new = static_cast<const uint4*>(k_new);
  p.v_new = static_cast<const uint4*>(v_new);
  p.cache_lens = cache_lens;
  p.row_starts = row_starts;
  p.status = ctx->d_status;
  p.num_seqs = num_seqs;
  p.rows = num_rows;
  // Four rows a warp where that leaves 16 warps per SM, else one (the same
  // write: 22.5 us by single rows, 19.7 by four).
  const int per = static_cast<long long>(num_rows) * ctx->cfg.num_kv_heads >=
                          4LL * 16 * std::max(ctx->num_sms, 1) ? 4 : 1;
  const long long units = (static_cast<long long>(num_rows) + per - 1) / per;
  p.heads_per_item = heads_per_item(ctx, units);
  const int grid = copy_grid(ctx, units, p.heads_per_item);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool q8 = pages->format == CPATTN_PAGES_E4M3;
  return per == 4 ? launch_paged_write<4>(ctx, p, q8, grid, st)
                  : launch_paged_write<1>(ctx, p, q8, grid, st);
} catch (...) {
  return CPATTN_E_NOMEM;
}

cpattn_status cpattn_paged_read_kv(cpattn_ctx* ctx, const cpattn_pages* pages, int32_t num_seqs,
                                   const int32_t* first, const int32_t* lens, void* k_cache,
                                   void* v_cache, void* stream) try {
  if (ctx == nullptr) return CPATTN_E_INVALID;
  cpattn::PagedReadParams p;
  cpattn_status s = check_pages(ctx, pages, num_seqs, &p.pool);
  if (s != CPATTN_OK) return s;
  if (lens == nullptr || k_cache == nullptr || v_cache == nullptr)
    return fail(ctx, CPATTN_E_INVALID, "device pointers must not be NULL");
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned4(lens) || !aligned4(first))
    return fail(ctx, CPATTN_E_INVALID, "caches 16-byte, integer arrays 4-byte aligned");
  const cpattn_config& c = ctx->cfg;
  const long long tokens = static_cast<long long>(num_seqs) * c.num_shards * c.shard_capacity;
  if (tokens * c.num_kv_heads >= (1LL << 31))
    return fail(ctx, CPATTN_E_UNSUPPORTED, "cache row count exceeds 2^31");
  if (ctx->d_status == nullptr) return fail(ctx, CPATTN_E_CUDA, "no CUDA device");
  p.first = first;
  p.lens = lens;
  p.k_cache = static_cast<uint4*>(k_cache);
  p.v_cache = static_cast<uint4*>(v_cache);
  p.status = ctx->d_status;
  p.num_seqs = num_seqs;
  p.P = c.num_shards;
  p.S = c.shard_capacity;
  p.v_f16 = c.v_cache_f16;
  // The most tokens the lengths can ask for (they are known on the device only).
  const long long most = std::min<long long>(
      tokens, static_cast<long long>(num_seqs) * pages->max_pages * pages->page_size);
  const long long runs = most / cpattn::kReadRun + num_seqs;
  p.heads_per_item = heads_per_item(ctx, runs);
  const int grid = copy_grid(ctx, runs, p.heads_per_item);
  const size_t smem = (static_cast<size_t>(num_seqs) + 1) * sizeof(int);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool q8 = pages->format == CPATTN_PAGES_E4M3;
  const auto kernel = c.head_dim == 128 ? (q8 ? cpattn::paged_read_kernel<128, true>
                                              : cpattn::paged_read_kernel<128, false>)
                                        : (q8 ? cpattn::paged_read_kernel<256, true>
                                              : cpattn::paged_read_kernel<256, false>);
  return launch_dependent(ctx, kernel, dim3(grid), 256, smem, st, p, "paged read launch");
} catch (...) {
  return CPATTN_E_NOMEM;
}

cpattn_status cpattn_paged_decode_workspace(const cpattn_ctx* ctx, int32_t num_seqs,
                                            uint64_t* bytes) {
  if (ctx == nullptr || bytes == nullptr || num_seqs < 1) return CPATTN_E_INVALID;
  if (num_seqs > CPATTN_MAX_PAGED_SEQS) return CPATTN_E_UNSUPPORTED;
  *bytes = decode_workspace(ctx).total;
  return CPATTN_OK;
}

cpattn_status cpattn_paged_decode(cpattn_ctx* ctx, const cpattn_pages* pages, int32_t num_seqs,
                                  const int32_t* lens, const void* q, void* out, float* lse,
                                  void* workspace, uint64_t workspace_bytes, void* stream) try {
  if (ctx == nullptr) return CPATTN_E_INVALID;
  cpattn::PagedDecodeParams p;
  cpattn_status s = check_pages(ctx, pages, num_seqs, &p.pool);
  if (s != CPATTN_OK) return s;
  if (lens == nullptr || q == nullptr || out == nullptr || workspace == nullptr)
    return fail(ctx, CPATTN_E_INVALID, "device pointers must not be NULL");
  if (!aligned16(q) || !aligned16(out) || !aligned4(lens) || !aligned4(lse) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(ctx, CPATTN_E_INVALID,
                "q, out 16-byte, lens, lse 4-byte, workspace 256-byte aligned");
  const DecodeWorkspace w = decode_workspace(ctx);
  if (workspace_bytes < w.total)
    return fail(ctx, CPATTN_E_INVALID, "workspace too small (cpattn_paged_decode_workspace)");
  if (ctx->d_status == nullptr) return fail(ctx, CPATTN_E_CUDA, "no CUDA device");
  const cpattn_config& c = ctx->cfg;
  char* ws = static_cast<char*>(workspace);
  p.lens = lens;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.ws_o = reinterpret_cast<float*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + w.ml);
  p.ws_cut = reinterpret_cast<cpattn::DecodeCut*>(ws + w.cut);
  p.status = ctx->d_status;
  p.timeout_ns = ctx->timeout_ns;
  p.debug_flags = ctx->debug_flags;
  p.bar_counts = nullptr;
  p.pool_rows = pages->num_pages * pages->page_size * c.num_kv_heads;
  p.num_seqs = num_seqs;
  p.nq = c.num_q_heads;
  p.group = c.num_q_heads / c.num_kv_heads;
  const bool one = p.group <= 8;
  p.hblocks = one ? 1 : (p.group + 15) / 16;
  p.scale_log2 = c.softmax_scale * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool q8 = pages->format == CPATTN_PAGES_E4M3;
  if (c.head_dim == 128) {
    if (one)
      return q8 ? launch_decode<128, true, 1>(ctx, pages, &p, st)
                : launch_decode<128, false, 1>(ctx, pages, &p, st);
    return q8 ? launch_decode<128, true, 2>(ctx, pages, &p, st)
              : launch_decode<128, false, 2>(ctx, pages, &p, st);
  }
  if (one)
    return q8 ? launch_decode<256, true, 1>(ctx, pages, &p, st)
              : launch_decode<256, false, 1>(ctx, pages, &p, st);
  return q8 ? launch_decode<256, true, 2>(ctx, pages, &p, st)
            : launch_decode<256, false, 2>(ctx, pages, &p, st);
} catch (...) {
  return CPATTN_E_NOMEM;
}

}  // extern "C"
