// paged_api.cuh — host side of the paged-cache calls (include/q1m.h, "Paged cache"): checks,
// scratch layout, tensor maps, launches. Included by q1m_api.cu, whose helpers it uses.
#pragma once

#include "paged.cuh"
#include "paged_attn.cuh"

namespace {

// Launch that may start before its predecessor in the stream has ended (grid_wait in the
// kernel orders what has to be ordered).
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

q1m_status check_heads(int batch, int hq, int hkv, int d) {
  if (batch < 0) return fail(Q1M_ERR_INVALID, "batch must be >= 0");
  if (batch > Q1M_MAX_PAGED_BATCH) return fail(Q1M_ERR_UNSUPPORTED, "batch %d exceeds %d", batch, Q1M_MAX_PAGED_BATCH);
  if (hq <= 0 || hkv <= 0 || hq % hkv != 0) return fail(Q1M_ERR_INVALID, "n_q_heads must be a positive multiple of n_kv_heads");
  if (hq > 4096) return fail(Q1M_ERR_UNSUPPORTED, "n_q_heads %d exceeds 4096", hq);
  if (d != 64 && d != 128) return fail(Q1M_ERR_UNSUPPORTED, "head_dim %d (64 or 128 supported)", d);
  return Q1M_OK;
}

// Entries of a table row.
int64_t table_width(const q1m_paged_cache* c) { return c->table_width > 0 ? c->table_width : c->table_stride; }

q1m_status check_cache(const q1m_paged_cache* c, int batch, int hq, const q1m_params* p, const float* table) {
  if (!c) return fail(Q1M_ERR_INVALID, "cache is NULL");
  Q1M_TRY(check_heads(batch, hq, c->n_kv_heads, c->head_dim));
  q1m_params q{};
  if (p) q = *p;
  q.vs_vertical = q.vs_slash = 0;
  q.equal_cost_chunks = 0;
  q.prefill_chunk = 128;           // the paged calls use neither the budgets nor the chunking
  Q1M_TRY(check_shape(1, hq, c->n_kv_heads, c->head_dim, p ? &q : nullptr));
  if (!c->k_pages || !c->v_pages || (!c->page_table && batch > 0) || !table) return fail(Q1M_ERR_INVALID, "NULL pointer");
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(Q1M_ERR_UNSUPPORTED, "page_size %d (16, 32, 64 or 128 supported)", c->page_size);
  if (c->n_pages <= 0 || c->table_stride <= 0) return fail(Q1M_ERR_INVALID, "n_pages and table_stride must be positive");
  if (c->table_width < 0 || c->table_width > c->table_stride)
    return fail(Q1M_ERR_INVALID, "table_width %d is not in 0 .. table_stride", c->table_width);
  if (c->n_pages >= (int64_t)1 << 31 || c->n_pages * c->n_kv_heads * c->page_size >= (int64_t)1 << 31)
    return fail(Q1M_ERR_UNSUPPORTED, "n_pages * n_kv_heads * page_size too large");
  // the tiles of 32 keys of all sequences are counted in 32 bits
  const int64_t most = (int64_t)1 << 30;
  const int64_t width = table_width(c), keys = width < most / c->page_size ? width * c->page_size : most;
  if (batch * keys >= (int64_t)1 << 35) return fail(Q1M_ERR_UNSUPPORTED, "batch * table_width * page_size too large");
  if ((reinterpret_cast<uintptr_t>(c->k_pages) | reinterpret_cast<uintptr_t>(c->v_pages) | reinterpret_cast<uintptr_t>(table)) & 15)
    return fail(Q1M_ERR_INVALID, "pages and table must be 16-byte aligned");
  return Q1M_OK;
}

q1m_status check_rows(const void* x, int64_t stride, int64_t width, const char* name) {
  if (!x) return fail(Q1M_ERR_INVALID, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(x) & 15) return fail(Q1M_ERR_INVALID, "%s must be 16-byte aligned", name);
  if (stride < width || stride % 8) return fail(Q1M_ERR_INVALID, "%s_stride must be a multiple of 8 and at least a row", name);
  return Q1M_OK;
}

q1m_status check_window(int64_t window, int64_t sinks, int32_t* w, int32_t* s) {
  if (window < 0 || sinks < 0) return fail(Q1M_ERR_INVALID, "window and sinks must be >= 0");
  const int64_t most = (int64_t)1 << 30;
  *w = (int32_t)(window < most ? window : most);
  *s = (int32_t)(sinks < most ? sinks : most);
  return Q1M_OK;
}

q1m_status check_out(const void* out, const void* scratch, size_t have, size_t need) {
  if (!out || !scratch) return fail(Q1M_ERR_INVALID, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(out) & 15) return fail(Q1M_ERR_INVALID, "out must be 16-byte aligned");
  if (have < need) return fail(Q1M_ERR_WORKSPACE, "scratch too small: %zu of %zu bytes", have, need);
  if (reinterpret_cast<uintptr_t>(scratch) & 255) return fail(Q1M_ERR_INVALID, "scratch must be 256-byte aligned");
  return Q1M_OK;
}

PagedCacheArgs cache_args(const q1m_paged_cache* c) {
  PagedCacheArgs a{};
  a.page_table = c->page_table;
  a.table_stride = c->table_stride;
  a.n_pages = (int32_t)c->n_pages;
  a.page_log2 = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  a.hkv = c->n_kv_heads;
  const int64_t width = table_width(c), held = width < PG_MAX_LEN ? width * c->page_size : PG_MAX_LEN;
  a.max_len = (int32_t)(held < PG_MAX_LEN ? held : PG_MAX_LEN);
  return a;
}

q1m_status page_maps(const q1m_paged_cache* c, uint32_t box_rows, CUtensorMap* mk, CUtensorMap* mv) {
  const uint64_t rows = (uint64_t)c->n_pages * c->n_kv_heads * c->page_size;
  Q1M_TRY(make_map(mk, c->k_pages, c->head_dim, rows, 64, box_rows));
  return make_map(mv, c->v_pages, c->head_dim, rows, 64, box_rows);
}

// The pages as (64-dim half, row, 64 dims), so that one copy brings whole rows, half by half.
q1m_status page_map_halves(CUtensorMap* m, const void* base, const q1m_paged_cache* c, uint32_t box_rows) {
  auto enc = tmap_encode();
  if (!enc) return fail(Q1M_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint32_t halves = (cuuint32_t)c->head_dim / 64;
  const cuuint64_t rows = (cuuint64_t)c->n_pages * c->n_kv_heads * c->page_size;
  cuuint64_t dims[3] = {64, rows, halves};
  cuuint64_t strides[2] = {(cuuint64_t)c->head_dim * 2, 128};
  cuuint32_t box[3] = {64, box_rows, halves};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(Q1M_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return Q1M_OK;
}

int paged_ctas(const Dev& dev) { return dev.sms < PG_MAX_CTAS ? dev.sms : PG_MAX_CTAS; }

// ---- decode ---------------------------------------------------------------------------------
struct PagedDecodeScratch {
  size_t o_part, lse_part, cut, pairs, o_whole, lse_whole, o_prefix, lse_prefix, total;
  int rows, n_rt, n_split, last_split, prefix_tiles;
};

// The key ranges that the row tiles of a shared prefix are cut into: the counts with which the
// pieces (one per range, row tile and KV head) take the least time on 148 SMs, a piece costing
// its key tiles plus about three tiles' time for its queries and results. A last row tile that
// uses both slots in turn (`light`) takes half the time a key tile and gets half the ranges.
void prefix_split(int64_t tiles, int64_t hkv, int64_t n_rt, bool light, int* n_split, int* last_split) {
  const int64_t sms = 148;
  int64_t best_cost = -1;
  for (int64_t ns = 1; ns <= tiles; ++ns) {
    const int64_t last = light ? (ns + 1) / 2 : ns;
    const int64_t items = hkv * ((n_rt - 1) * ns + last);
    if (items > 4 * sms && best_cost >= 0) break;
    int64_t each = n_rt > 1 ? 2 * ((tiles + ns - 1) / ns) : 0;     // half tiles
    const int64_t of_last = (light ? 1 : 2) * ((tiles + last - 1) / last);
    if (of_last > each) each = of_last;
    const int64_t cost = ((items + sms - 1) / sms) * (each + 6);
    if (best_cost < 0 || cost < best_cost) { best_cost = cost; *n_split = (int)ns; *last_split = (int)last; }
  }
}

PagedDecodeScratch decode_scratch(int batch, int hq, int hkv, int d, int64_t prefix_len, bool prec) {
  PagedDecodeScratch L{};
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t o = off; off = align_up(off + bytes); return o; };
  L.o_part = take((size_t)2 * PG_MAX_CTAS * 8 * d * 4);
  L.lse_part = take((size_t)2 * PG_MAX_CTAS * 8 * 4);
  L.cut = take((size_t)PG_MAX_CTAS * sizeof(int4));
  L.prefix_tiles = (int)(prefix_len / 128);
  if (L.prefix_tiles > 0) {
    L.rows = pa_rows(prec);
    L.n_rt = (int)(((int64_t)batch * (hq / hkv) + L.rows - 1) / L.rows);
    const bool light = !prec && (int64_t)batch * (hq / hkv) - (int64_t)(L.n_rt - 1) * L.rows <= 128;
    prefix_split(L.prefix_tiles, hkv, L.n_rt, light, &L.n_split, &L.last_split);
    L.pairs = take((size_t)batch * hkv * sizeof(int2));
    L.o_whole = take((size_t)batch * hq * d * 4);
    L.lse_whole = take((size_t)batch * hq * 4);
    const size_t rows = (size_t)L.n_rt * hkv * L.n_split * L.rows;
    L.o_prefix = take(rows * d * 4);
    L.lse_prefix = take(rows * 4);
  }
  L.total = off;
  return L;
}

template <int D>
q1m_status run_paged_attn(const PagedAttnArgs& a, const q1m_paged_cache* c, bool prec, int ctas, bool after, cudaStream_t st) {
  CUtensorMap mk, mv;
  Q1M_TRY(page_maps(c, (uint32_t)c->page_size, &mk, &mv));
  const size_t smem = sizeof(PaSmem<D>) + 1024;
  auto kernel = prec ? paged_attn_kernel<D, true> : paged_attn_kernel<D, false>;
  Q1M_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  if (after) Q1M_CUDA(launch_after(kernel, dim3(ctas), PA_THREADS, smem, st, mk, mv, a));
  else kernel<<<ctas, PA_THREADS, smem, st>>>(mk, mv, a);
  Q1M_LAUNCHED();
  return Q1M_OK;
}

template <typename T, typename TO, int D>
q1m_status run_paged_decode(const PagedDecodeArgs& a, const q1m_paged_cache* c, int ctas, cudaStream_t st) {
  CUtensorMap mk, mv;
  const uint32_t box_rows = (uint32_t)(c->page_size < PD_TILE ? c->page_size : PD_TILE);
  Q1M_TRY(page_map_halves(&mk, c->k_pages, c, box_rows));
  Q1M_TRY(page_map_halves(&mv, c->v_pages, c, box_rows));
  const size_t smem = sizeof(PdSmem<D>) + 1024;
  auto kernel = paged_decode_kernel<T, TO, D>;
  Q1M_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  kernel<<<ctas, PD_THREADS, smem, st>>>(mk, mv, a);
  Q1M_LAUNCHED();
  return Q1M_OK;
}

template <typename T, typename TO>
q1m_status run_paged_decode(const PagedDecodeArgs& a, const q1m_paged_cache* c, int ctas, cudaStream_t st) {
  return c->head_dim == 128 ? run_paged_decode<T, TO, 128>(a, c, ctas, st) : run_paged_decode<T, TO, 64>(a, c, ctas, st);
}

q1m_status paged_decode(const void* q, int64_t q_stride, const int32_t* seq_len, int batch, int32_t window,
                        int32_t sinks, const int32_t* prefix_table, int64_t prefix_len,
                        const q1m_paged_cache* c, int hq, const q1m_params* p, const float* table, void* out,
                        float* lse, void* scratch, cudaStream_t st) {
  Dev dev;
  Q1M_TRY(device_info(&dev));
  const bool prec = p->out_dtype == Q1M_F32;
  const int d = c->head_dim, ctas = paged_ctas(dev);
  const PagedDecodeScratch SL = decode_scratch(batch, hq, c->n_kv_heads, d, prefix_len, prec);
  PagedDecodeArgs a{};
  a.c = cache_args(c);
  a.q = q; a.q_stride = q_stride; a.seq_len = seq_len;
  a.batch = batch; a.hq = hq; a.G = hq / c->n_kv_heads;
  a.window = window; a.sinks = sinks;
  a.first_key = SL.prefix_tiles * 128;
  a.L = (int32_t)(p->dca_chunk - p->local_window);
  a.chunk = (int32_t)p->dca_chunk;
  a.scale = view_scale(p, d);
  a.table = reinterpret_cast<const float2*>(table);
  a.out = out; a.lse = lse;
  a.o_part = at<float>(scratch, SL.o_part);
  a.lse_part = at<float>(scratch, SL.lse_part);
  a.cut = at<int4>(scratch, SL.cut);
  PagedMergeArgs m{};
  if (SL.prefix_tiles > 0) {
    a.pairs = at<int2>(scratch, SL.pairs);
    a.o_whole = at<float>(scratch, SL.o_whole);
    a.lse_whole = at<float>(scratch, SL.lse_whole);
    m.n_prefix = SL.n_split;
    m.n_last = SL.last_split;
    m.n_rt = SL.n_rt;
    m.o_prefix = at<float>(scratch, SL.o_prefix);
    m.lse_prefix = at<float>(scratch, SL.lse_prefix);
    m.prefix_rows = SL.rows;
  }
  m.d = a;
  // The sequences' own keys come first: where they are few, most CTAs have none and make way for
  // the prefix's (8 sequences of 1 .. 511 keys behind 262,144 shared ones: 126 us with the prefix
  // first).
  if (p->in_dtype == Q1M_BF16)
    Q1M_TRY((prec ? run_paged_decode<__nv_bfloat16, float> : run_paged_decode<__nv_bfloat16, __nv_bfloat16>)(a, c, ctas, st));
  else
    Q1M_TRY((prec ? run_paged_decode<float, float> : run_paged_decode<float, __nv_bfloat16>)(a, c, ctas, st));
  if (SL.prefix_tiles > 0) {
    PagedAttnArgs t{};
    t.c = a.c;
    t.c.page_table = prefix_table;
    t.c.table_stride = prefix_len / c->page_size;
    t.q = q; t.q_stride = q_stride; t.n_tokens = batch;
    t.q_f32 = p->in_dtype == Q1M_F32;
    t.seq_len = seq_len;
    t.batch = batch; t.hq = hq; t.G = a.G;
    t.L = a.L; t.chunk = a.chunk; t.scale = a.scale; t.table = a.table;
    t.v_pages = c->v_pages;
    t.o_part = at<float>(scratch, SL.o_prefix);
    t.lse_part = at<float>(scratch, SL.lse_prefix);
    t.n_split = SL.n_split; t.last_split = SL.last_split; t.n_rt = SL.n_rt; t.prefix_tiles = SL.prefix_tiles;
    const int64_t items = (int64_t)c->n_kv_heads * (SL.n_split * (SL.n_rt - 1) + SL.last_split);
    const int grid = items < ctas ? (int)items : ctas;
    if (d == 128) Q1M_TRY(run_paged_attn<128>(t, c, prec, grid, true, st));
    else Q1M_TRY(run_paged_attn<64>(t, c, prec, grid, true, st));
  }
  const dim3 rows((unsigned)(a.pairs ? batch * hq : (ctas - 1) * a.G));
  if (prec) Q1M_CUDA(launch_after(d == 128 ? paged_merge_kernel<float, 128> : paged_merge_kernel<float, 64>, rows, 128, 0, st, m));
  else Q1M_CUDA(launch_after(d == 128 ? paged_merge_kernel<__nv_bfloat16, 128> : paged_merge_kernel<__nv_bfloat16, 64>, rows, 128, 0, st, m));
  Q1M_LAUNCHED();
  return Q1M_OK;
}

// ---- prefill --------------------------------------------------------------------------------
struct PagedPrefillScratch {
  size_t cut, o_part, lse_part, total;
};

PagedPrefillScratch prefill_scratch(int d, bool prec) {
  PagedPrefillScratch L{};
  const int rows = pa_rows(prec);
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t o = off; off = align_up(off + bytes); return o; };
  L.cut = take((size_t)PG_MAX_CTAS * sizeof(PagedRowCut));
  L.o_part = take((size_t)2 * PG_MAX_CTAS * rows * d * 4);
  L.lse_part = take((size_t)2 * PG_MAX_CTAS * rows * 4);
  L.total = off;
  return L;
}

q1m_status check_tokens(int64_t n_tokens, int batch, int hq, int hkv) {
  if (n_tokens < 0) return fail(Q1M_ERR_INVALID, "n_tokens must be >= 0");
  if (n_tokens >= (int64_t)1 << 30 || n_tokens * (hq / hkv) + (int64_t)256 * batch >= (int64_t)1 << 31)
    return fail(Q1M_ERR_UNSUPPORTED, "n_tokens too large");
  return Q1M_OK;
}

}  // namespace

extern "C" {

q1m_status q1m_paged_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int64_t n_tokens,
                            const int32_t* cu_tokens, const int32_t* seq_len, int batch,
                            const q1m_paged_cache* c, const q1m_params* p, const float* table, void* stream) {
  Q1M_TRY(check_cache(c, batch, c ? c->n_kv_heads : 1, p, table));
  Q1M_TRY(check_tokens(n_tokens, batch, 1, 1));
  if (!cu_tokens && n_tokens != batch) return fail(Q1M_ERR_INVALID, "without cu_tokens n_tokens is batch");
  if (n_tokens == 0 || batch == 0) return Q1M_OK;
  if (!seq_len) return fail(Q1M_ERR_INVALID, "seq_len is NULL");
  const int64_t width = (int64_t)c->n_kv_heads * c->head_dim;
  Q1M_TRY(check_rows(k, k_stride, width, "k"));
  Q1M_TRY(check_rows(v, v_stride, width, "v"));
  Dev dev;
  Q1M_TRY(device_info(&dev));
  PagedAppendArgs a{};
  a.c = cache_args(c);
  a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride;
  a.n_tokens = n_tokens; a.cu = cu_tokens; a.seq_len = seq_len; a.batch = batch;
  a.d = c->head_dim;
  a.L = (int32_t)(p->dca_chunk - p->local_window);
  a.table = reinterpret_cast<const float2*>(table);
  a.k_pages = c->k_pages; a.v_pages = c->v_pages;
  const int units = c->n_kv_heads * (c->head_dim / 16);
  // A block takes one item a thread while that leaves SMs idle, and up to four: the chain from
  // token to page is paid once a block.
  const int once = units >= PG_APPEND_THREADS ? 1 : PG_APPEND_THREADS / units;
  int64_t turns = n_tokens / ((int64_t)once * dev.sms * 4);
  turns = turns < 1 ? 1 : (turns > 4 ? 4 : turns);
  const int per_block = (int)(once * turns < PG_APPEND_TOKENS ? once * turns : PG_APPEND_TOKENS);
  const int grid = (int)((n_tokens + per_block - 1) / per_block);
  if (p->in_dtype == Q1M_BF16)
    paged_append_kernel<__nv_bfloat16><<<grid, PG_APPEND_THREADS, 0, S(stream)>>>(a, units, per_block);
  else
    paged_append_kernel<float><<<grid, PG_APPEND_THREADS, 0, S(stream)>>>(a, units, per_block);
  Q1M_LAUNCHED();
  return Q1M_OK;
}

size_t q1m_paged_decode_scratch_bytes(int batch, int hq, int hkv, int d) {
  if (check_heads(batch, hq, hkv, d) != Q1M_OK || hq / hkv > 8) return 0;
  return decode_scratch(batch, hq, hkv, d, 0, false).total;
}

q1m_status q1m_paged_decode(const void* q, int64_t q_stride, const int32_t* seq_len, int batch, int64_t window,
                            int64_t sinks, const q1m_paged_cache* c, int hq, const q1m_params* p,
                            const float* table, void* out, float* lse, void* scratch, size_t scratch_bytes,
                            void* stream) {
  Q1M_TRY(check_cache(c, batch, hq, p, table));
  if (hq / c->n_kv_heads > 8) return fail(Q1M_ERR_UNSUPPORTED, "decode supports at most 8 Q heads per KV head");
  int32_t w, s;
  Q1M_TRY(check_window(window, sinks, &w, &s));
  if (batch == 0) return Q1M_OK;
  if (!seq_len) return fail(Q1M_ERR_INVALID, "seq_len is NULL");
  Q1M_TRY(check_rows(q, q_stride, (int64_t)hq * c->head_dim, "q"));
  Q1M_TRY(check_out(out, scratch, scratch_bytes, q1m_paged_decode_scratch_bytes(batch, hq, c->n_kv_heads, c->head_dim)));
  return paged_decode(q, q_stride, seq_len, batch, w, s, nullptr, 0, c, hq, p, table, out, lse, scratch, S(stream));
}

size_t q1m_shared_prefix_decode_scratch_bytes(int batch, int64_t prefix_len, int hq, int hkv, int d,
                                              const q1m_params* p) {
  if (!p || check_heads(batch, hq, hkv, d) != Q1M_OK || hq / hkv > 8 || prefix_len < 128 || prefix_len > PG_MAX_LEN) return 0;
  return decode_scratch(batch, hq, hkv, d, prefix_len, p->out_dtype == Q1M_F32).total;
}

q1m_status q1m_shared_prefix_decode(const void* q, int64_t q_stride, const int32_t* seq_len, int batch,
                                    const int32_t* prefix_table, int64_t prefix_len, const q1m_paged_cache* c,
                                    int hq, const q1m_params* p, const float* table, void* out, float* lse,
                                    void* scratch, size_t scratch_bytes, void* stream) {
  Q1M_TRY(check_cache(c, batch, hq, p, table));
  if (hq / c->n_kv_heads > 8) return fail(Q1M_ERR_UNSUPPORTED, "decode supports at most 8 Q heads per KV head");
  if (prefix_len < 128 || prefix_len % c->page_size) return fail(Q1M_ERR_INVALID, "prefix_len must be a multiple of page_size and at least 128");
  if (prefix_len > PG_MAX_LEN) return fail(Q1M_ERR_UNSUPPORTED, "prefix_len too large");
  if (batch == 0) return Q1M_OK;
  if (!seq_len || !prefix_table) return fail(Q1M_ERR_INVALID, "NULL pointer");
  Q1M_TRY(check_rows(q, q_stride, (int64_t)hq * c->head_dim, "q"));
  Q1M_TRY(check_out(out, scratch, scratch_bytes,
                    q1m_shared_prefix_decode_scratch_bytes(batch, prefix_len, hq, c->n_kv_heads, c->head_dim, p)));
  return paged_decode(q, q_stride, seq_len, batch, 0, 0, prefix_table, prefix_len, c, hq, p, table, out, lse,
                      scratch, S(stream));
}

size_t q1m_paged_prefill_scratch_bytes(int64_t n_tokens, int batch, int hq, int hkv, int d, const q1m_params* p) {
  if (!p || check_heads(batch, hq, hkv, d) != Q1M_OK || check_tokens(n_tokens, batch, hq, hkv) != Q1M_OK) return 0;
  return prefill_scratch(d, p->out_dtype == Q1M_F32).total;
}

q1m_status q1m_paged_prefill(const void* q, int64_t q_stride, int64_t n_tokens, const int32_t* cu_tokens,
                             const int32_t* seq_len, int batch, int64_t window, int64_t sinks,
                             const q1m_paged_cache* c, int hq, const q1m_params* p, const float* table, void* out,
                             float* lse, void* scratch, size_t scratch_bytes, void* stream) {
  Q1M_TRY(check_cache(c, batch, hq, p, table));
  Q1M_TRY(check_tokens(n_tokens, batch, hq, c->n_kv_heads));
  PagedAttnArgs a{};
  Q1M_TRY(check_window(window, sinks, &a.window, &a.sinks));
  if (n_tokens == 0 || batch == 0) return Q1M_OK;
  if (!cu_tokens || !seq_len) return fail(Q1M_ERR_INVALID, "NULL pointer");
  Q1M_TRY(check_rows(q, q_stride, (int64_t)hq * c->head_dim, "q"));
  Q1M_TRY(check_out(out, scratch, scratch_bytes,
                    q1m_paged_prefill_scratch_bytes(n_tokens, batch, hq, c->n_kv_heads, c->head_dim, p)));
  Dev dev;
  Q1M_TRY(device_info(&dev));
  const bool prec = p->out_dtype == Q1M_F32;
  const int d = c->head_dim, ctas = paged_ctas(dev);
  const PagedPrefillScratch SL = prefill_scratch(d, prec);
  a.c = cache_args(c);
  a.q = q; a.q_stride = q_stride; a.n_tokens = n_tokens;
  a.q_f32 = p->in_dtype == Q1M_F32;
  a.cu = cu_tokens; a.seq_len = seq_len; a.batch = batch;
  a.hq = hq; a.G = hq / c->n_kv_heads;
  a.L = (int32_t)(p->dca_chunk - p->local_window);
  a.chunk = (int32_t)p->dca_chunk;
  a.scale = view_scale(p, d);
  a.table = reinterpret_cast<const float2*>(table);
  a.v_pages = c->v_pages;
  a.out = out; a.lse = lse;
  a.o_part = at<float>(scratch, SL.o_part);
  a.lse_part = at<float>(scratch, SL.lse_part);
  a.cut = at<PagedRowCut>(scratch, SL.cut);
  cudaStream_t st = S(stream);
  if (d == 128) Q1M_TRY(run_paged_attn<128>(a, c, prec, ctas, false, st));
  else Q1M_TRY(run_paged_attn<64>(a, c, prec, ctas, false, st));
  const dim3 grid(ctas - 1, pa_rows(prec) / 8);
  if (d == 128) Q1M_CUDA(prec ? launch_after(paged_attn_merge_kernel<128, true>, grid, 256, 0, st, a)
                              : launch_after(paged_attn_merge_kernel<128, false>, grid, 256, 0, st, a));
  else Q1M_CUDA(prec ? launch_after(paged_attn_merge_kernel<64, true>, grid, 256, 0, st, a)
                     : launch_after(paged_attn_merge_kernel<64, false>, grid, 256, 0, st, a));
  Q1M_LAUNCHED();
  return Q1M_OK;
}

}  // extern "C"
