// The span operators one row per warp: every lane holds d / 32 values of a row.
// Slow and plain; what the tiled kernels are checked against.
#pragma once

#include <math_constants.h>

#include "fa_span.cuh"

namespace fa {

// one pair's score, and d score / d (scale q k)
struct SpanScore {
  float scale, cap, inv_cap;  // cap 0: none
  const float* slopes;        // [H] or nullptr
  __device__ __forceinline__ float operator()(float qk, float slope, int far, float* bent) const {
    float s = qk * scale;
    *bent = 1.f;
    if (cap > 0.f) {
      const float t = tanhf(s * inv_cap);
      *bent = 1.f - t * t;
      s = t * cap;
    }
    return s - slope * (float)far;
  }
};

struct SpanRowsParams {
  SpanView view;
  SpanScore score;
  const __nv_bfloat16 *q, *k, *v, *o, *dout;
  PageRows kp, vp;
  float* lse;
  __nv_bfloat16 *out, *dq, *dk, *dv;
  int B, H, Hkv, pages;
};

template <int D>
__device__ __forceinline__ void rows_load(const __nv_bfloat16* row, float (&x)[D / 32]) {
  for (int e = 0; e < D / 32; ++e) x[e] = __bfloat162float(row[(threadIdx.x & 31) + 32 * e]);
}
template <int D>
__device__ __forceinline__ float rows_dot(const float (&x)[D / 32], const float (&y)[D / 32]) {
  float s = 0.f;
  for (int e = 0; e < D / 32; ++e) s = fmaf(x[e], y[e], s);
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int D>
__device__ __forceinline__ bool rows_key(const SpanRowsParams& p, const PageRows& pg, const __nv_bfloat16* flat, int b,
                                         int j, int key, float (&x)[D / 32]) {
  if (!p.view.table) {
    rows_load<D>(flat + (((long long)b * p.Hkv + j) * p.view.N + key) * D, x);
    return true;
  }
  const int page = p.view.table[(long long)b * p.view.width + (key >> p.view.page_shift)];
  if (page < 0 || page >= p.pages) {
    for (int e = 0; e < D / 32; ++e) x[e] = 0.f;
    return true;
  }
  rows_load<D>(pg.ptr + page * pg.page + j * pg.head + (key & ((1 << p.view.page_shift) - 1)) * pg.token, x);
  return true;
}

template <int D>
__global__ void __launch_bounds__(256) span_rows_fwd(const SpanRowsParams p) {
  const int N = p.view.N, lane = threadIdx.x & 31;
  for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < (long long)p.B * p.H * N;
       row += (long long)gridDim.x * 8) {
    const int i = row % N, h = row / N % p.H, b = row / N / p.H, j = h / (p.H / p.Hkv);
    const int len = p.view.len(b), pos = len + i;
    if (i >= p.view.rows(b, len)) continue;
    int lo, hi;
    p.view.span(b, i, pos, lo, hi);
    float q[D / 32], x[D / 32], o[D / 32] = {};
    rows_load<D>(p.q + row * D, q);
    float m = -CUDART_INF_F, l = 0.f;
    for (int key = lo; key < hi; ++key) {
      rows_key<D>(p, p.kp, p.k, b, j, key, x);
      float bent;
      const float s = p.score(rows_dot<D>(q, x), p.score.slopes ? p.score.slopes[h] : 0.f, abs(pos - key), &bent);
      const float mx = fmaxf(m, s);
      if (mx == -CUDART_INF_F) continue;
      const float a = expf(m - mx), w = expf(s - mx);
      rows_key<D>(p, p.vp, p.v, b, j, key, x);
      for (int e = 0; e < D / 32; ++e) o[e] = o[e] * a + w * x[e];
      l = l * a + w;
      m = mx;
    }
    for (int e = 0; e < D / 32; ++e) p.out[row * D + lane + 32 * e] = __float2bfloat16(l > 0.f ? o[e] / l : 0.f);
    if (lane == 0) p.lse[row] = l > 0.f ? m + logf(l) : -CUDART_INF_F;
  }
}

template <int D>
__device__ __forceinline__ void rows_pair(const SpanRowsParams& p, const float (&q)[D / 32], const float (&k)[D / 32],
                                          const float (&v)[D / 32], const float (&g)[D / 32], float lse, float delta,
                                          int h, int far, float& w, float& ds) {
  float bent;
  const float s = p.score(rows_dot<D>(q, k), p.score.slopes ? p.score.slopes[h] : 0.f, far, &bent);
  w = expf(s - lse);
  ds = w * (rows_dot<D>(g, v) - delta) * bent * p.score.scale;
}

template <int D>
__global__ void __launch_bounds__(256) span_rows_bwd(const SpanRowsParams p) {
  const int N = p.view.N, lane = threadIdx.x & 31, G = p.H / p.Hkv;
  const long long rows = (long long)p.B * p.H * N, keys = (long long)p.B * p.Hkv * N;
  float q[D / 32], k[D / 32], v[D / 32], g[D / 32], o[D / 32], w, ds;
  for (long long at = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); at < rows + keys; at += (long long)gridDim.x * 8) {
    float a[D / 32] = {}, c[D / 32] = {};
    if (at < rows) {
      const int i = at % N, h = at / N % p.H, b = at / N / p.H;
      int lo, hi;
      p.view.span(b, i, i, lo, hi);
      rows_load<D>(p.q + at * D, q);
      rows_load<D>(p.dout + at * D, g);
      rows_load<D>(p.o + at * D, o);
      const float delta = rows_dot<D>(g, o), lse = p.lse[at];
      for (int key = lo; key < hi && lse != -CUDART_INF_F; ++key) {
        rows_key<D>(p, p.kp, p.k, b, h / G, key, k);
        rows_key<D>(p, p.vp, p.v, b, h / G, key, v);
        rows_pair<D>(p, q, k, v, g, lse, delta, h, abs(i - key), w, ds);
        for (int e = 0; e < D / 32; ++e) a[e] = fmaf(ds, k[e], a[e]);
      }
      for (int e = 0; e < D / 32; ++e) p.dq[at * D + lane + 32 * e] = __float2bfloat16(a[e]);
      continue;
    }
    const long long kr = at - rows;
    const int key = kr % N, j = kr / N % p.Hkv, b = kr / N / p.Hkv;
    rows_load<D>(p.k + kr * D, k);
    rows_load<D>(p.v + kr * D, v);
    for (int h = j * G; h < j * G + G; ++h)
      for (int i = 0; i < N; ++i) {
        const long long row = ((long long)b * p.H + h) * N + i;
        int lo, hi;
        p.view.span(b, i, i, lo, hi);
        const float lse = p.lse[row];
        if (key < lo || key >= hi || lse == -CUDART_INF_F) continue;
        rows_load<D>(p.q + row * D, q);
        rows_load<D>(p.dout + row * D, g);
        rows_load<D>(p.o + row * D, o);
        rows_pair<D>(p, q, k, v, g, lse, rows_dot<D>(g, o), h, abs(i - key), w, ds);
        for (int e = 0; e < D / 32; ++e) a[e] = fmaf(ds, q[e], a[e]), c[e] = fmaf(w, g[e], c[e]);
      }
    for (int e = 0; e < D / 32; ++e) {
      p.dk[kr * D + lane + 32 * e] = __float2bfloat16(a[e]);
      p.dv[kr * D + lane + 32 * e] = __float2bfloat16(c[e]);
    }
  }
}

}  // namespace fa
