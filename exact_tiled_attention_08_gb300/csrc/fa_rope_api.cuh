// Host side of the head norm and rotation entry points (declared in fa.h;
// included by fa_ops.cu; uses the checks of fa_lib.cu).
#pragma once

#include <algorithm>

namespace {

constexpr int kRopeFwdCtas = 152 * fa::kRopeFwdPerSm;
constexpr int kRopeBwdCtas = 152 * fa::kRopeBwdPerSm;  // CTAs of the backward, each with a row of weight gradient sums

fa_status check_rows(const fa_rows& r) {
  if (!aligned16(r.ptr) || r.batch % 8 || r.token % 8 || r.head % 8) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// written rows: no two of them may share memory
bool rows_disjoint(const fa_rows& r, int B, int N, int heads, int d) {
  struct Dim {
    long long stride, size;
  } dim[3] = {{r.batch, B}, {r.token, N}, {r.head, heads}};
  std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  long long extent = d;
  for (const Dim& x : dim) {
    if (x.size == 1) continue;
    if (x.stride < extent) return false;
    extent = x.stride * (x.size - 1) + extent;
  }
  return true;
}

fa::RopeRows rope_rows(const fa_rows* r) {
  fa::RopeRows x{};
  if (r && r->ptr) x = {static_cast<const __nv_bfloat16*>(r->ptr), r->batch, r->token, r->head};
  return x;
}

bool present(const fa_rows* r) { return r && r->ptr; }

// checks that the forward and the backward share
fa_status check_rope(const double* inv_freq, int B, int N, int H, int Hkv, int d, int rotary_dim, int norm, float eps,
                     float factor, int interleaved) {
  if (H < 1 || Hkv < 1) return FA_ERR_INVALID_ARG;
  fa_status st = check_shape(B, H, N, d);
  if (st == FA_OK) st = check_shape(B, Hkv, N, d);
  if (st != FA_OK) return st;
  if ((long long)H + 2LL * Hkv > 0x3fffffffLL || (long long)B * N > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > d) return FA_ERR_INVALID_ARG;
  if (rotary_dim % 16) return FA_ERR_UNSUPPORTED;
  if (rotary_dim > 0 && !inv_freq) return FA_ERR_INVALID_ARG;
  if ((norm != 0 && norm != 1) || (interleaved != 0 && interleaved != 1)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(factor) || (norm && (!std::isfinite(eps) || eps < 0.f))) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Warps' units of work: a warp's tokens times some heads.  The heads of a unit
// share the token's angles and one start of the ring, about four rows' time; the
// device holds `warps` warps at once, and the split that ends soonest is taken.
// (Measured, heads per unit: forward at 16384 tokens of 32 + 8 + 8 heads 8: 82 us,
// 16: 66 us, 24, with q and k in one unit: 71 us; backward at 8004 tokens 12, with q and k
// in one unit: 62 us, 16: 51 us.)
void rope_units(fa::RopeParams& p, int d, long long warps, bool q, bool k, bool v) {
  const long long per_warp = 32 / (d / 8), groups = ((p.tokens + per_warp - 1) / per_warp + 7) / 8 * 8;
  const int most = std::max(q ? p.H : 0, p.Hkv * ((k ? 1 : 0) + (v ? 1 : 0)));
  double best = 0;
  for (int step = 1; step <= most; ++step) {
    fa::RopeSplit s{};
    s.q_units = q ? (p.H + step - 1) / step : 0;
    s.q_step = q ? (p.H + s.q_units - 1) / s.q_units : 0;
    s.both = k && v && 2 * p.Hkv <= step;
    const int n = (p.Hkv + step - 1) / step;
    s.kv_step = (p.Hkv + n - 1) / n;
    s.k_units = k && !s.both ? n : 0;
    s.v_units = v && !s.both ? n : 0;
    s.steps = s.q_units + s.k_units + s.v_units + s.both;
    const long long units = groups * s.steps;
    const double turns = (double)((units + warps - 1) / warps);
    const double cost = turns * (std::max(s.q_step, s.both ? 2 * p.Hkv : s.kv_step) + 4);
    if (step == 1 || cost < best) {
      best = cost;
      p.split = s;
      p.units = units;
    }
    if (step >= 256) break;  // (more heads in a unit share nothing more worth having)
  }
}

template <int D, bool kNorm, class Params>
void launch_rope_fwd(const Params& p, unsigned grid, int interleaved, cudaStream_t stream) {
  if (interleaved)
    fa::fa_rope_fwd_kernel<D, true, kNorm, Params><<<grid, fa::kRopeThreads, 0, stream>>>(p);
  else
    fa::fa_rope_fwd_kernel<D, false, kNorm, Params><<<grid, fa::kRopeThreads, 0, stream>>>(p);
}

template <class Params>
fa_status run_rope_fwd(Params& p, int d, bool q, bool k, bool v, int interleaved, cudaStream_t stream) {
  rope_units(p, d, kRopeFwdCtas * 8LL, q, k, v);
  const unsigned grid = (unsigned)std::min<long long>((p.units + 7) / 8, kRopeFwdCtas);
  if (d == 128)
    p.norm ? launch_rope_fwd<128, true>(p, grid, interleaved, stream)
           : launch_rope_fwd<128, false>(p, grid, interleaved, stream);
  else
    p.norm ? launch_rope_fwd<64, true>(p, grid, interleaved, stream)
           : launch_rope_fwd<64, false>(p, grid, interleaved, stream);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool kNorm>
void launch_rope_bwd(const fa::RopeParams& p, unsigned grid, int interleaved, cudaStream_t stream) {
  constexpr int smem = fa::kRopeBwdSmemBytes<kNorm>;
  // (a failure to set the size shows in the launch)
  if (interleaved) {
    set_smem(fa::fa_rope_bwd_kernel<D, true, kNorm>, smem);
    fa::fa_rope_bwd_kernel<D, true, kNorm><<<grid, fa::kRopeThreads, smem, stream>>>(p);
  } else {
    set_smem(fa::fa_rope_bwd_kernel<D, false, kNorm>, smem);
    fa::fa_rope_bwd_kernel<D, false, kNorm><<<grid, fa::kRopeThreads, smem, stream>>>(p);
  }
}

}  // namespace

extern "C" {

fa_status fa_rope_fwd(const fa_rows* q, const fa_rows* k, const fa_rows* v, const float* q_weight,
                      const float* k_weight, const double* inv_freq, const int* positions, const int* starts,
                      void* q_out, void* k_out, void* v_out, int B, int N, int H, int Hkv, int C, int d,
                      int rotary_dim, int norm, float eps, float factor, int interleaved, cudaStream_t stream) {
  if (present(q) != (q_out != nullptr) || present(k) != (k_out != nullptr) || present(v) != (v_out != nullptr))
    return FA_ERR_INVALID_ARG;
  if (!q_out && !k_out && !v_out) return FA_ERR_INVALID_ARG;
  fa_status st = check_rope(inv_freq, B, N, H, Hkv, d, rotary_dim, norm, eps, factor, interleaved);
  if (st != FA_OK) return st;
  if (C < N) return FA_ERR_INVALID_ARG;
  for (const fa_rows* r : {q, k, v})
    if (present(r) && (st = check_rows(*r)) != FA_OK) return st;
  if (!all_aligned16({q_weight, k_weight, q_out, k_out, v_out}) || !all_aligned({positions, starts}, 4) ||
      !all_aligned({inv_freq}, 8))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs_given({q ? q->ptr : nullptr, k ? k->ptr : nullptr, v ? v->ptr : nullptr, q_weight,
                                     k_weight, inv_freq, positions, starts, q_out, k_out, v_out})) != FA_OK)
    return st;
  fa::RopeParams p{};
  p.q = rope_rows(q);
  p.k = rope_rows(k);
  p.v = rope_rows(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.starts = starts;
  p.N = N;
  p.H = H;
  p.Hkv = Hkv;
  p.C = C;
  p.rot = rotary_dim;
  p.tokens = (long long)B * N;
  p.eps = eps;
  p.factor = factor;
  p.norm = norm;
  return run_rope_fwd(p, d, q_out, k_out, v_out, interleaved, stream);
}

fa_status fa_rope_paged_fwd(const fa_rows* q, const fa_rows* k, const fa_rows* v, const float* q_weight,
                            const float* k_weight, const double* inv_freq, const int* positions,
                            const int* page_table, const int* cache_lens, const int* chunk_lens, void* q_out,
                            const fa_pages* k_pages, const fa_pages* v_pages, int B, int N, int H, int Hkv, int d,
                            int num_pages, int page_size, int table_width, int rotary_dim, int norm, float eps,
                            float factor, int interleaved, cudaStream_t stream) {
  const bool to_k = k_pages && k_pages->ptr, to_v = v_pages && v_pages->ptr;
  if (present(q) != (q_out != nullptr) || present(k) != to_k || present(v) != to_v) return FA_ERR_INVALID_ARG;
  if (!q_out && !to_k && !to_v) return FA_ERR_INVALID_ARG;
  fa_status st = check_rope(inv_freq, B, N, H, Hkv, d, rotary_dim, norm, eps, factor, interleaved);
  if (st != FA_OK) return st;
  const PageShape pages{num_pages, page_size, table_width};
  if (to_k || to_v) {
    if (!page_table || !cache_lens) return FA_ERR_INVALID_ARG;
    if ((st = pages.check()) != FA_OK) return st;
  }
  for (const fa_pages* r : {k_pages, v_pages}) {
    if (!r || !r->ptr) continue;
    if ((st = check_pages(r, pages, Hkv)) != FA_OK) return st;
    if (!rows_disjoint({r->ptr, r->page, r->token, r->head}, num_pages, page_size, Hkv, d)) return FA_ERR_INVALID_ARG;
  }
  for (const fa_rows* r : {q, k, v})
    if (present(r) && (st = check_rows(*r)) != FA_OK) return st;
  if (!all_aligned16({q_weight, k_weight, q_out}) ||
      !all_aligned({positions, page_table, cache_lens, chunk_lens}, 4) || !all_aligned({inv_freq}, 8))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs_given({q ? q->ptr : nullptr, k ? k->ptr : nullptr, v ? v->ptr : nullptr, q_weight,
                                     k_weight, inv_freq, positions, page_table, cache_lens, chunk_lens, q_out,
                                     to_k ? k_pages->ptr : nullptr, to_v ? v_pages->ptr : nullptr})) != FA_OK)
    return st;
  fa::RopePagedParams p{};
  p.q = rope_rows(q);
  p.k = rope_rows(k);
  p.v = rope_rows(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.starts = cache_lens;
  p.N = N;
  p.H = H;
  p.Hkv = Hkv;
  p.C = 0x7fffffff;
  p.rot = rotary_dim;
  p.tokens = (long long)B * N;
  p.eps = eps;
  p.factor = factor;
  p.norm = norm;
  p.chunks = chunk_lens;
  if (to_k || to_v) {
    if (to_k) p.k_pages = page_rows(k_pages);
    if (to_v) p.v_pages = page_rows(v_pages);
    p.C = (int)pages.capacity();
    p.table = page_table;
    p.width = table_width;
    p.page_shift = pages.shift();
    p.pages = num_pages;
  }
  return run_rope_fwd(p, d, q_out, to_k, to_v, interleaved, stream);
}

size_t fa_rope_bwd_workspace_bytes(int B, int H, int Hkv, int N, int d) {
  if (check_shape(B, H, N, d) != FA_OK || check_shape(B, Hkv, N, d) != FA_OK) return 0;
  return (size_t)kRopeBwdCtas * 2 * d * sizeof(float);
}

fa_status fa_rope_bwd(const fa_rows* q, const fa_rows* k, const float* q_weight, const float* k_weight,
                      const double* inv_freq, const int* positions, const void* dq_out, const void* dk_out,
                      const void* dv_out, const fa_rows* dq, const fa_rows* dk, const fa_rows* dv, float* dq_weight,
                      float* dk_weight, void* workspace, size_t ws_bytes, int B, int N, int H, int Hkv, int d,
                      int rotary_dim, int norm, float eps, float factor, int interleaved, cudaStream_t stream) {
  if (present(dq) != (dq_out != nullptr) || present(dk) != (dk_out != nullptr) || present(dv) != (dv_out != nullptr))
    return FA_ERR_INVALID_ARG;
  if (!dq_out && !dk_out && !dv_out) return FA_ERR_INVALID_ARG;
  fa_status st = check_rope(inv_freq, B, N, H, Hkv, d, rotary_dim, norm, eps, factor, interleaved);
  if (st != FA_OK) return st;
  const bool need_q = norm && dq_out, need_k = norm && dk_out;
  if ((need_q && !present(q)) || (need_k && !present(k))) return FA_ERR_INVALID_ARG;
  // a weight has a gradient only where the norm runs on its rows
  if ((dq_weight && !need_q) || (dk_weight && !need_k)) return FA_ERR_INVALID_ARG;
  const bool weights = dq_weight || dk_weight;
  if (weights && (!workspace || ws_bytes < fa_rope_bwd_workspace_bytes(B, H, Hkv, N, d))) return FA_ERR_INVALID_ARG;
  if ((need_q && (st = check_rows(*q)) != FA_OK) || (need_k && (st = check_rows(*k)) != FA_OK)) return st;
  for (const fa_rows* r : {dq, dk, dv}) {
    if (!present(r)) continue;
    if ((st = check_rows(*r)) != FA_OK) return st;
    if (!rows_disjoint(*r, B, N, r == dq ? H : Hkv, d)) return FA_ERR_INVALID_ARG;
  }
  if (!all_aligned16({q_weight, k_weight, dq_out, dk_out, dv_out, dq_weight, dk_weight,
                      weights ? workspace : nullptr}) ||
      !all_aligned({positions}, 4) || !all_aligned({inv_freq}, 8))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs_given({need_q ? q->ptr : nullptr, need_k ? k->ptr : nullptr, q_weight, k_weight,
                                     inv_freq, positions, dq_out, dk_out, dv_out, dq ? dq->ptr : nullptr,
                                     dk ? dk->ptr : nullptr, dv ? dv->ptr : nullptr, dq_weight, dk_weight,
                                     weights ? workspace : nullptr})) != FA_OK)
    return st;
  fa::RopeParams p{};
  if (need_q) p.q = rope_rows(q);
  if (need_k) p.k = rope_rows(k);
  p.dq = rope_rows(dq);
  p.dk = rope_rows(dk);
  p.dv = rope_rows(dv);
  p.q_out = static_cast<__nv_bfloat16*>(const_cast<void*>(dq_out));
  p.k_out = static_cast<__nv_bfloat16*>(const_cast<void*>(dk_out));
  p.v_out = static_cast<__nv_bfloat16*>(const_cast<void*>(dv_out));
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.partials = weights ? static_cast<float*>(workspace) : nullptr;
  p.N = N;
  p.H = H;
  p.Hkv = Hkv;
  p.C = N;
  p.rot = rotary_dim;
  p.tokens = (long long)B * N;
  p.eps = eps;
  p.factor = factor;
  p.norm = norm;
  rope_units(p, d, kRopeBwdCtas * 8LL, dq_out, dk_out, dv_out);
  const unsigned grid = (unsigned)std::min<long long>((p.units + 7) / 8, kRopeBwdCtas);
  if (d == 128)
    norm ? launch_rope_bwd<128, true>(p, grid, interleaved, stream) : launch_rope_bwd<128, false>(p, grid, interleaved, stream);
  else
    norm ? launch_rope_bwd<64, true>(p, grid, interleaved, stream) : launch_rope_bwd<64, false>(p, grid, interleaved, stream);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (weights) {
    if (launch_early(fa::fa_rope_dw_kernel, dim3((unsigned)(2 * d / 32)), 1024, 0, stream, p.partials, (int)grid, d,
                     dq_weight, dk_weight) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return FA_OK;
}

fa_status fa_rope_fwd_packed(const fa_rope_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_rope_fwd(&a->q, &a->k, &a->v, a->q_weight, a->k_weight, a->inv_freq, a->positions, a->starts, a->q_out,
                     a->k_out, a->v_out, a->B, a->N, a->H, a->Hkv, a->C, a->d, a->rotary_dim, a->norm, a->eps,
                     a->factor, a->interleaved, a->stream);
}

fa_status fa_rope_paged_fwd_packed(const fa_rope_paged_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_rope_paged_fwd(&a->q, &a->k, &a->v, a->q_weight, a->k_weight, a->inv_freq, a->positions, a->page_table,
                           a->cache_lens, a->chunk_lens, a->q_out, &a->k_pages, &a->v_pages, a->B, a->N, a->H, a->Hkv,
                           a->d, a->num_pages, a->page_size, a->table_width, a->rotary_dim, a->norm, a->eps, a->factor,
                           a->interleaved, a->stream);
}

fa_status fa_rope_bwd_packed(const fa_rope_bwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_rope_bwd(&a->q, &a->k, a->q_weight, a->k_weight, a->inv_freq, a->positions, a->dq_out, a->dk_out, a->dv_out,
                     &a->dq, &a->dk, &a->dv, a->dq_weight, a->dk_weight, a->workspace, a->ws_bytes, a->B, a->N, a->H,
                     a->Hkv, a->d, a->rotary_dim, a->norm, a->eps, a->factor, a->interleaved, a->stream);
}

}  // extern "C"
