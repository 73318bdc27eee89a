// Attention whose keys have another length than the queries: a key length per
// request, key/value heads shared by groups of query heads, and (over a
// cache) drafted tokens behind the request's own that see each other by a mask.
//
// The G = H / Hkv query heads that share a key/value head lie next to one
// another in [B][H][Nq][d], so their rows are one run of G Nq query rows
// against one set of keys: everything below works on [B Hkv][R = G Nq][d].
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "sm103_ptx.cuh"

namespace fa {

// What the rows see.  Keys [0, len) of the request are visible to every row;
// with drafts, key len + t is visible to the row of token n when t < drafts
// and bit t of masks[b][n] is set (without masks: t <= n), and the rows of
// tokens n >= drafts are not written.
struct CrossView {
  const int* lens;                    // [B] or nullptr: all Nk keys
  const int* drafts;                  // [B] or nullptr: T
  const unsigned long long* masks;    // [B][T] or nullptr
  int T;                              // drafted tokens per request; 0: cross attention
  int Nk;                             // key rows per (request, head) in memory
  int Nq;                             // query rows per head
  int R;                              // query rows per key/value head (G Nq)
  int Hkv;
  __device__ __forceinline__ int len(int b) const {
    return lens ? min(max(__ldg(lens + b), 0), Nk) : (T ? max(Nk - T, 0) : Nk);
  }
  // drafts of request b that have a key row
  __device__ __forceinline__ int drafted(int b, int len) const {
    return T ? min(min(max(drafts ? __ldg(drafts + b) : T, 0), T), Nk - len) : 0;
  }
  __device__ __forceinline__ bool sees(int b, int n, int t) const {
    return masks ? ((__ldg(masks + (long long)b * T + n) >> t) & 1) : t <= n;
  }
};

struct CrossBwdParams {
  CrossView view;
  const __nv_bfloat16 *q, *k, *v, *o, *dout;
  const float* lse;
  __nv_bfloat16 *dq, *dk, *dv;
  float* delta;
  int B;
  float scale;
};

template <int D>
struct LaneRow {
  static constexpr int E = D / 32;
  float x[E];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int lane) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __bfloat162float(row[lane * E + i]);
  }
  __device__ __forceinline__ float dot(const LaneRow& o) const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(x[i], o.x[i], s);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    return s;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, int lane, float f) const {
#pragma unroll
    for (int i = 0; i < E; ++i) row[lane * E + i] = __float2bfloat16(x[i] * f);
  }
};

// one warp per query row: dQ, and delta for the pass over the keys
template <int D>
__global__ void __launch_bounds__(256) fa_cross_dq_kernel(const CrossBwdParams p) {
  const CrossView& v = p.view;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= (long long)p.B * v.Hkv * v.R) return;
  const long long bk = row / v.R;
  const int len = v.len((int)(bk / v.Hkv));
  LaneRow<D> q, o, go, k, x, acc{};
  q.load(p.q + row * D, lane);
  o.load(p.o + row * D, lane);
  go.load(p.dout + row * D, lane);
  const float delta = go.dot(o), lse = p.lse[row];
  if (lane == 0) p.delta[row] = delta;
  for (int j = 0; j < len; ++j) {
    k.load(p.k + (bk * v.Nk + j) * D, lane);
    x.load(p.v + (bk * v.Nk + j) * D, lane);
    const float ds = __expf(q.dot(k) * p.scale - lse) * (go.dot(x) - delta);
#pragma unroll
    for (int i = 0; i < LaneRow<D>::E; ++i) acc.x[i] = fmaf(ds, k.x[i], acc.x[i]);
  }
  acc.store(p.dq + row * D, lane, p.scale);
}

// one warp per key row: dK and dV
template <int D>
__global__ void __launch_bounds__(256) fa_cross_dkv_kernel(const CrossBwdParams p) {
  const CrossView& v = p.view;
  const long long key = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (key >= (long long)p.B * v.Hkv * v.Nk) return;
  const long long bk = key / v.Nk;
  LaneRow<D> q, go, k, x, dk{}, dv{};
  if (key - bk * v.Nk < v.len((int)(bk / v.Hkv))) {
    k.load(p.k + key * D, lane);
    x.load(p.v + key * D, lane);
    for (long long row = bk * v.R; row < (bk + 1) * v.R; ++row) {
      q.load(p.q + row * D, lane);
      go.load(p.dout + row * D, lane);
      const float pr = __expf(q.dot(k) * p.scale - p.lse[row]);
      const float ds = pr * (go.dot(x) - p.delta[row]);
#pragma unroll
      for (int i = 0; i < LaneRow<D>::E; ++i) {
        dk.x[i] = fmaf(ds, q.x[i], dk.x[i]);
        dv.x[i] = fmaf(pr, go.x[i], dv.x[i]);
      }
    }
  }
  dk.store(p.dk + key * D, lane, p.scale);
  dv.store(p.dv + key * D, lane, 1.f);
}

}  // namespace fa
