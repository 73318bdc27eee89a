// Host side of the cross attention, draft tree and rotation entry points
// (declared in fa.h; included by fa_ops.cu; uses the checks of fa_lib.cu).
#pragma once

namespace {

// shape checks of the cross attention entry points; `R` receives the query
// rows per key/value head
fa_status check_cross_shape(int B, int H, int Hkv, int Nq, int Nk, int d, int* R) {
  if (B < 1 || H < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || d < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  const long long rows = (long long)(H / Hkv) * Nq;
  if (rows > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  fa_status st = check_shape(B, Hkv, (int)rows, d);
  if (st == FA_OK) st = check_shape(B, Hkv, Nk, d);
  *R = (int)rows;
  return st;
}

bool all_aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  return true;
}

fa::CrossView cross_view(int H, int Hkv, int Nq, int Nk) {
  fa::CrossView v{};
  v.Nk = Nk;
  v.Nq = Nq;
  v.R = H / Hkv * Nq;
  v.Hkv = Hkv;
  return v;
}

fa_status run_cross_fwd(const fa::CrossFwdParams& p, int d, cudaStream_t stream) {
  const long long blocks = ((long long)p.B * p.view.Hkv * p.view.R + 7) / 8;
  if (blocks > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  if (d == 128)
    fa::fa_cross_fwd_kernel<128><<<(unsigned)blocks, 256, 0, stream>>>(p);
  else
    fa::fa_cross_fwd_kernel<64><<<(unsigned)blocks, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t cross_fwd_workspace(int B, int H, int Hkv, int Nq, int Nk, int d) {
  int R;
  return check_cross_shape(B, H, Hkv, Nq, Nk, d, &R) == FA_OK ? 256 : 0;
}

}  // namespace

extern "C" {

size_t fa_cross_fwd_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d) {
  return cross_fwd_workspace(B, H, Hkv, Nq, Nk, d);
}

fa_status fa_cross_fwd(const void* q, const void* k, const void* v, const int* key_lens, void* o, float* lse,
                       void* workspace, size_t ws_bytes, int B, int H, int Hkv, int Nq, int Nk, int d, float scale,
                       cudaStream_t stream) {
  if (!q || !k || !v || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  int R;
  fa_status st = check_cross_shape(B, H, Hkv, Nq, Nk, d, &R);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale, 0)) != FA_OK) return st;
  if (ws_bytes < cross_fwd_workspace(B, H, Hkv, Nq, Nk, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, key_lens, o, lse, workspace})) return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k, v, o, lse, workspace})) != FA_OK) return st;
  if (key_lens && (st = check_device_ptrs({key_lens})) != FA_OK) return st;
  fa::CrossFwdParams p{};
  p.view = cross_view(H, Hkv, Nq, Nk);
  p.view.lens = key_lens;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.B = B;
  p.scale = scale;
  return run_cross_fwd(p, d, stream);
}

size_t fa_cross_bwd_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d) {
  int R;
  if (check_cross_shape(B, H, Hkv, Nq, Nk, d, &R) != FA_OK) return 0;
  return (size_t)B * Hkv * R * sizeof(float);
}

fa_status fa_cross_bwd(const void* q, const void* k, const void* v, const int* key_lens, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, void* workspace,
                       size_t ws_bytes, int B, int H, int Hkv, int Nq, int Nk, int d, float scale,
                       cudaStream_t stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return FA_ERR_INVALID_ARG;
  int R;
  fa_status st = check_cross_shape(B, H, Hkv, Nq, Nk, d, &R);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale, 0)) != FA_OK) return st;
  if (ws_bytes < fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, key_lens, o, dout, lse, dq, dk, dv, workspace})) return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k, v, o, dout, lse, dq, dk, dv, workspace})) != FA_OK) return st;
  if (key_lens && (st = check_device_ptrs({key_lens})) != FA_OK) return st;
  fa::CrossBwdParams p{};
  p.view = cross_view(H, Hkv, Nq, Nk);
  p.view.lens = key_lens;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.o = static_cast<const __nv_bfloat16*>(o);
  p.dout = static_cast<const __nv_bfloat16*>(dout);
  p.lse = lse;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.delta = static_cast<float*>(workspace);
  p.B = B;
  p.scale = scale;
  const long long rows = ((long long)B * Hkv * R + 7) / 8, keys = ((long long)B * Hkv * Nk + 7) / 8;
  if (rows > 0x7fffffffLL || keys > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  if (d == 128) {
    fa::fa_cross_dq_kernel<128><<<(unsigned)rows, 256, 0, stream>>>(p);
    fa::fa_cross_dkv_kernel<128><<<(unsigned)keys, 256, 0, stream>>>(p);
  } else {
    fa::fa_cross_dq_kernel<64><<<(unsigned)rows, 256, 0, stream>>>(p);
    fa::fa_cross_dkv_kernel<64><<<(unsigned)keys, 256, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_tree_fwd_workspace_bytes(int B, int H, int Hkv, int T, int C, int d) {
  return cross_fwd_workspace(B, H, Hkv, T, C, d);
}

fa_status fa_tree_fwd(const void* q, const void* k_cache, const void* v_cache, const int* cache_lens,
                      const int* draft_lens, const unsigned long long* draft_masks, void* o, float* lse,
                      void* workspace, size_t ws_bytes, int B, int H, int Hkv, int T, int C, int d, float scale,
                      cudaStream_t stream) {
  if (!q || !k_cache || !v_cache || !cache_lens || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  int R;
  fa_status st = check_cross_shape(B, H, Hkv, T, C, d, &R);
  if (st != FA_OK) return st;
  if (draft_masks && T > 64) return FA_ERR_UNSUPPORTED;
  if ((st = check_scale(scale, 0)) != FA_OK) return st;
  if (ws_bytes < cross_fwd_workspace(B, H, Hkv, T, C, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k_cache, v_cache, cache_lens, draft_lens, draft_masks, o, lse, workspace}))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k_cache, v_cache, cache_lens, o, lse, workspace})) != FA_OK) return st;
  if (draft_lens && (st = check_device_ptrs({draft_lens})) != FA_OK) return st;
  if (draft_masks && (st = check_device_ptrs({draft_masks})) != FA_OK) return st;
  fa::CrossFwdParams p{};
  p.view = cross_view(H, Hkv, T, C);
  p.view.lens = cache_lens;
  p.view.drafts = draft_lens;
  p.view.masks = draft_masks;
  p.view.T = T;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k_cache);
  p.v = static_cast<const __nv_bfloat16*>(v_cache);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.B = B;
  p.scale = scale;
  return run_cross_fwd(p, d, stream);
}

}  // extern "C"
