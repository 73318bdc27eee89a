// Host side of the span attention and paged attention entry points (declared in
// fa.h; included by fa_ops.cu; uses the checks of fa_lib.cu).
#pragma once

namespace {

// what a key/value cache in pages has to be
struct PageShape {
  int num_pages, page_size, width;
  long long capacity() const { return (long long)width * page_size; }
  fa_status check() const {
    if (num_pages < 1 || page_size < 1 || width < 1) return FA_ERR_INVALID_ARG;
    if (page_size < 16 || (page_size & (page_size - 1))) return FA_ERR_UNSUPPORTED;
    return capacity() > 0x7fffff00LL ? FA_ERR_INVALID_ARG : FA_OK;
  }
  int shift() const {
    int s = 0;
    while (1 << s < page_size) ++s;
    return s;
  }
};

// strides: of sizes greater than one positive, of the others not used
fa_status check_pages(const fa_pages* r, const PageShape& s, int Hkv) {
  if (!r || !r->ptr) return FA_ERR_INVALID_ARG;
  const struct {
    long long stride;
    int size;
  } dims[3] = {{r->page, s.num_pages}, {r->head, Hkv}, {r->token, s.page_size}};
  for (const auto& x : dims)
    if (x.size > 1 && (x.stride < 1 || x.stride >= 1ll << 38)) return FA_ERR_INVALID_ARG;
  for (const auto& x : dims)
    if (x.size > 1 && x.stride % 8) return FA_ERR_MISALIGNED;
  return aligned16(r->ptr) ? FA_OK : FA_ERR_MISALIGNED;
}

fa_status check_span_args(float scale, float cap, int window, int causal) {
  fa_status st = check_scale(scale, causal);
  if (st != FA_OK) return st;
  if (!std::isfinite(cap) || cap < 0.f || window < 0) return FA_ERR_INVALID_ARG;
  if (cap > 0.f && !std::isfinite(2.f * scale / cap)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_span_shape(int B, int H, int Hkv, int N, int d) {
  int R;
  const fa_status st = check_cross_shape(B, H, Hkv, N, N, d, &R);
  return st == FA_OK ? check_shape(B, H, N, d) : st;
}

fa::PageRows page_rows(const fa_pages* r) {
  return {static_cast<__nv_bfloat16*>(r->ptr), r->page, r->head, r->token};
}

}  // namespace

extern "C" {

size_t fa_span_fwd_workspace_bytes(int B, int H, int Hkv, int N, int d) {
  return check_span_shape(B, H, Hkv, N, d) == FA_OK ? 256 : 0;
}

fa_status fa_span_fwd(const void* q, const void* k, const void* v, const int* key_begin, const int* key_end,
                      const float* slopes, void* o, float* lse, void* workspace, size_t ws_bytes, int B, int H, int Hkv,
                      int N, int d, float scale, float cap, int window, int causal, cudaStream_t stream) {
  if (!q || !k || !v || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  fa_status st = check_span_shape(B, H, Hkv, N, d);
  if (st != FA_OK) return st;
  if ((st = check_span_args(scale, cap, window, causal)) != FA_OK) return st;
  if (ws_bytes < fa_span_fwd_workspace_bytes(B, H, Hkv, N, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, o, lse, workspace}) || !all_aligned({key_begin, key_end, slopes}, 4))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k, v, o, lse, workspace})) != FA_OK) return st;
  if ((st = check_device_ptrs_given({key_begin, key_end, slopes})) != FA_OK) return st;
  fa::SpanRowsParams p{};
  p.view = {key_begin, key_end, nullptr, nullptr, nullptr, 0, 0, N, N, causal, window};
  p.score = {scale, cap, cap > 0.f ? 1.f / cap : 0.f, slopes};
  p.q = static_cast<const __nv_bfloat16*>(q), p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v), p.out = static_cast<__nv_bfloat16*>(o);
  p.lse = lse, p.B = B, p.H = H, p.Hkv = Hkv;
  d == 128 ? fa::span_rows_fwd<128><<<152 * 8, 256, 0, stream>>>(p) : fa::span_rows_fwd<64><<<152 * 8, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_span_bwd_workspace_bytes(int B, int H, int Hkv, int N, int d) {
  return check_span_shape(B, H, Hkv, N, d) == FA_OK ? 256 : 0;
}

fa_status fa_span_bwd(const void* q, const void* k, const void* v, const int* key_begin, const int* key_end,
                      const float* slopes, const void* o, const void* dout, const float* lse, void* dq, void* dk,
                      void* dv, void* workspace, size_t ws_bytes, int B, int H, int Hkv, int N, int d, float scale,
                      float cap, int window, int causal, cudaStream_t stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return FA_ERR_INVALID_ARG;
  fa_status st = check_span_shape(B, H, Hkv, N, d);
  if (st != FA_OK) return st;
  if ((st = check_span_args(scale, cap, window, causal)) != FA_OK) return st;
  if (ws_bytes < fa_span_bwd_workspace_bytes(B, H, Hkv, N, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, o, dout, lse, dq, dk, dv, workspace}) || !all_aligned({key_begin, key_end, slopes}, 4))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k, v, o, dout, lse, dq, dk, dv, workspace})) != FA_OK) return st;
  if ((st = check_device_ptrs_given({key_begin, key_end, slopes})) != FA_OK) return st;
  fa::SpanRowsParams p{};
  p.view = {key_begin, key_end, nullptr, nullptr, nullptr, 0, 0, N, N, causal, window};
  p.score = {scale, cap, cap > 0.f ? 1.f / cap : 0.f, slopes};
  p.q = static_cast<const __nv_bfloat16*>(q), p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v), p.o = static_cast<const __nv_bfloat16*>(o);
  p.dout = static_cast<const __nv_bfloat16*>(dout), p.lse = const_cast<float*>(lse);
  p.dq = static_cast<__nv_bfloat16*>(dq), p.dk = static_cast<__nv_bfloat16*>(dk), p.dv = static_cast<__nv_bfloat16*>(dv);
  p.B = B, p.H = H, p.Hkv = Hkv;
  d == 128 ? fa::span_rows_bwd<128><<<152 * 8, 256, 0, stream>>>(p) : fa::span_rows_bwd<64><<<152 * 8, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_paged_fwd_workspace_bytes(int B, int H, int Hkv, int T, int C, int d) {
  int R;
  return check_cross_shape(B, H, Hkv, T, C, d, &R) == FA_OK ? 256 : 0;
}

fa_status fa_paged_fwd(const void* q, const fa_pages* k_pages, const fa_pages* v_pages, const int* page_table,
                       const int* cache_lens, const int* chunk_lens, const float* slopes, void* o, float* lse,
                       void* workspace, size_t ws_bytes, int B, int H, int Hkv, int T, int d, int num_pages,
                       int page_size, int table_width, float scale, float cap, int window, cudaStream_t stream) {
  if (!q || !page_table || !cache_lens || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  const PageShape pages{num_pages, page_size, table_width};
  fa_status st = pages.check();
  if (st != FA_OK) return st;
  int R;
  if ((st = check_cross_shape(B, H, Hkv, T, (int)pages.capacity(), d, &R)) != FA_OK) return st;
  if ((st = check_span_args(scale, cap, window, 1)) != FA_OK) return st;
  if (ws_bytes < fa_paged_fwd_workspace_bytes(B, H, Hkv, T, (int)pages.capacity(), d)) return FA_ERR_INVALID_ARG;
  for (const fa_pages* r : {k_pages, v_pages})
    if ((st = check_pages(r, pages, Hkv)) != FA_OK) return st;
  if (!all_aligned16({q, o, lse, workspace}) || !all_aligned({page_table, cache_lens, chunk_lens, slopes}, 4))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k_pages->ptr, v_pages->ptr, page_table, cache_lens, o, lse, workspace})) != FA_OK)
    return st;
  if ((st = check_device_ptrs_given({chunk_lens, slopes})) != FA_OK) return st;
  fa::SpanRowsParams p{};
  p.view = {nullptr, nullptr, cache_lens, chunk_lens, page_table, table_width, pages.shift(), T,
            (int)pages.capacity(), 1, window};
  p.score = {scale, cap, cap > 0.f ? 1.f / cap : 0.f, slopes};
  p.q = static_cast<const __nv_bfloat16*>(q), p.out = static_cast<__nv_bfloat16*>(o);
  p.kp = page_rows(k_pages), p.vp = page_rows(v_pages);
  p.lse = lse, p.B = B, p.H = H, p.Hkv = Hkv, p.pages = num_pages;
  d == 128 ? fa::span_rows_fwd<128><<<152 * 8, 256, 0, stream>>>(p) : fa::span_rows_fwd<64><<<152 * 8, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_span_fwd_packed(const fa_span_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_span_fwd(a->q, a->k, a->v, a->key_begin, a->key_end, a->slopes, a->o, a->lse, a->workspace, a->ws_bytes,
                     a->B, a->H, a->Hkv, a->N, a->d, a->scale, a->cap, a->window, a->causal, a->stream);
}

fa_status fa_span_bwd_packed(const fa_span_bwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_span_bwd(a->q, a->k, a->v, a->key_begin, a->key_end, a->slopes, a->o, a->dout, a->lse, a->dq, a->dk, a->dv,
                     a->workspace, a->ws_bytes, a->B, a->H, a->Hkv, a->N, a->d, a->scale, a->cap, a->window, a->causal,
                     a->stream);
}

fa_status fa_paged_fwd_packed(const fa_paged_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_paged_fwd(a->q, &a->k_pages, &a->v_pages, a->page_table, a->cache_lens, a->chunk_lens, a->slopes, a->o,
                      a->lse, a->workspace, a->ws_bytes, a->B, a->H, a->Hkv, a->T, a->d, a->num_pages, a->page_size,
                      a->table_width, a->scale, a->cap, a->window, a->stream);
}

}  // extern "C"
