// Attention in which each query sees the keys of one span: self-attention with a
// causal mask, a window, packed documents or prefixes (fa_span_fwd, fa_span_bwd),
// and a chunk of new tokens over a cache in pages (fa_paged_fwd).
//
// Query i at position p_i sees the keys j with lo_i <= j < hi_i; the scores are
//   s_ij = cap tanh(scale q_i k_j / cap) - slope_h |p_i - j|
// (without a cap scale q_i k_j, without slopes no second term).
#pragma once

#include <cuda_bf16.h>

#include "fa_cross.cuh"

namespace fa {

// PAGED: keys in pages; else in [B][Hkv][N][d].  (The kernels are compiled for each of the two: what the other
// form needs costs instruction fetches.  N=8192 H=32/8 d=128 causal, one request, capped: 560 and 496 us
// when it was tried, 479 now.)
template <bool PAGED>
struct SpanView {
  const int *begin, *end;      // [B][N] or nullptr: 0 and C
  const int *lens, *chunks;    // pages: tokens before the chunk [B]; new tokens [B], or nullptr: N
  const int* table;            // pages: [B][width] page numbers
  int width, page_shift;       // pages: entries per request; log2 of a page's rows
  int N;                       // query rows per head
  int C;                       // keys: N, or width pages
  int causal, window;          // j <= p_i; |p_i - j| < window (0: any)
  __device__ __forceinline__ int len(int b) const { return PAGED ? min(max(lens[b], 0), C) : 0; }
  // query rows of request b that exist
  __device__ __forceinline__ int rows(int b, int len) const {
    return PAGED ? min(min(max(chunks ? chunks[b] : N, 0), N), C - len) : N;
  }
  // the keys that query i of request b sees (pos: its position); lo >= hi: none
  __device__ __forceinline__ void span(int b, int i, int pos, int& lo, int& hi) const {
    lo = !PAGED && begin ? min(max(begin[(long long)b * N + i], 0), C) : 0;
    hi = !PAGED && end ? min(max(end[(long long)b * N + i], 0), C) : C;
    clip(pos, pos, lo, hi);
  }
  // what is left of [lo, hi) for queries at positions p0 .. p1
  __device__ __forceinline__ void clip(int p0, int p1, int& lo, int& hi) const {
    if (PAGED || causal) hi = min(hi, p1 + 1);
    if (window) {
      lo = max(lo, p0 - window + 1);
      if (!PAGED) hi = (int)min((long long)hi, (long long)p1 + window);
    }
  }
};

// Rows of a cache in pages: token t of a page and head at ptr + page * page + head * head + t * token.
struct PageRows {
  __nv_bfloat16* ptr;
  long long page, head, token;  // strides in elements
};

// The keys that the rows of a tile of 128 see between them, [lo, hi), and where all of
// its rows see all keys: blocks from lo_cut on that end at hi_cut at the latest.
struct SpanTile {
  int lo, hi, lo_cut, hi_cut;
  __device__ __forceinline__ bool empty() const { return lo >= hi; }
};

// Query rows come in units: a query head's, or (pages) those of the heads that share a
// key/value head.  A tile has whole tokens, row r is head r % heads of its token r / heads, so
// that a request's new tokens fill as few tiles as they can, whatever the others bring.
template <bool PAGED>
struct SpanRows {
  SpanView<PAGED> view;
  const int4* bounds;  // [B][tiles] SpanTile, or nullptr: the mask is a formula of the position
  int unit_heads, tile_tokens;  // pages: heads of a unit; tokens of a tile
  int tiles;           // tiles of a unit's N tokens
  int units, kv_div;   // units of a request; of a key/value head
  __device__ __forceinline__ int heads() const { return PAGED ? unit_heads : 1; }
  __device__ __forceinline__ int tokens() const { return PAGED ? tile_tokens : 128; }
  // row of [B][H][N]
  __device__ __forceinline__ size_t row(int b, int u, int head, int token) const {
    return (((size_t)b * units + u) * heads() + head) * view.N + token;
  }
  __device__ __forceinline__ SpanTile tile(int b, int t) const {
    if (!PAGED && bounds) {
      const int4 x = bounds[(long long)b * tiles + t];
      return {x.x, x.y, x.z, x.w};
    }
    const int len = view.len(b), t0 = t * tokens(), t1 = min(t0 + tokens(), view.rows(b, len)) - 1;
    if (t0 > t1) return {0, 0, 0x7fffffff, 0};
    SpanTile s{0, view.C, 0, view.C};
    view.clip(len + t0, len + t1, s.lo, s.hi);
    int other = view.C;
    view.clip(len + t1, len + t1, s.lo_cut, other);
    other = 0;
    view.clip(len + t0, len + t0, other, s.hi_cut);
    return s;
  }
};

// The bounds of one tile from its rows' spans, by 128 threads (row: there is one).
__device__ __forceinline__ int4 span_tile_reduce(int lo, int hi, bool row, int4* scratch) {
  const bool live = row && lo < hi;
  const int4 x = make_int4(__reduce_min_sync(0xffffffffu, live ? lo : 0x7fffffff), __reduce_max_sync(0xffffffffu, live ? hi : 0),
                           __reduce_max_sync(0xffffffffu, row ? (live ? lo : 0x7fffffff) : 0),
                           __reduce_min_sync(0xffffffffu, row ? (live ? hi : 0) : 0x7fffffff));
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
  __syncthreads();
  int4 s = scratch[0];
  for (int w = 1; w < 4; ++w) {
    const int4 y = scratch[w];
    s = make_int4(min(s.x, y.x), max(s.y, y.y), max(s.z, y.z), min(s.w, y.w));
  }
  if (s.x >= s.y) s.x = s.y = 0;
  return s;
}

// Bounds of all tiles where the spans are given by row: a block of 128 threads per tile.
__global__ void __launch_bounds__(128) fa_span_bounds_kernel(const SpanView<false> v, int tiles, int4* bounds) {
  __shared__ int4 scratch[4];
  grid_wait();
  grid_trigger();
  const int b = blockIdx.x / tiles, i = (blockIdx.x - b * tiles) * 128 + threadIdx.x;
  int lo = 0, hi = 0;
  if (i < v.N) v.span(b, i, i, lo, hi);
  const int4 s = span_tile_reduce(lo, hi, i < v.N, scratch);
  if (threadIdx.x == 0) bounds[blockIdx.x] = s;
}

// The cap in log2 units: cap log2(e) tanh(x), x = scale q k / cap.
//
// Within |x| <= 0.6 it is x G(x^2) with the minimax polynomial of tanh(sqrt u) / sqrt u on
// [0, 0.36] (degree 4, by Remez exchange on the relative error: 7.3e-8), in powers of the product q k
// itself; beyond it 1 - 2 / (1 + e^2x), whose absolute error (2^-22) is what counts there.
// A warp takes the polynomial where all of its products of a block allow it.
//
// With caps of 30 and more it asks for less: no product above 0.6, and a row's largest not below
// -0.2.  Products below -0.6, where the polynomial goes its own way downwards (to the
// ninth power), then weigh less than e^-(0.53 - 0.2) 30 = 5e-5 in their row, and their weights'
// errors, e^-(tanh|x| - 0.2) 30 times 30 |x G(x^2) - tanh x|, are below 1e-8 everywhere.  And a product of
// -10 gives a weight of 0 beside such a largest one, so that it stands for a key that is not seen.
struct SpanCap {
  float mul;     // 2 log2(e) scale / cap
  float small;   // products up to there take the polynomial: 0.6 cap / scale
  float low;     // the lowest largest one: -0.2 cap / scale
  float hidden;  // -10 cap / scale; 0: a cap below 30, or coefficients that fp32 does not hold
  float top;     // cap log2(e)
  float d[5];    // q k (d[0] + d[1] (q k)^2 + ...)
};

// score / product of small products
__device__ __forceinline__ float2 span_cap_small(float2 s, const SpanCap& c) {
  const float2 u = __fmul2_rn(s, s);
  float2 g = __ffma2_rn(u, make_float2(c.d[4], c.d[4]), make_float2(c.d[3], c.d[3]));
#pragma unroll
  for (int i = 2; i >= 0; --i) g = __ffma2_rn(u, g, make_float2(c.d[i], c.d[i]));
  return g;
}

// 32 products of one row, in place
__device__ __forceinline__ void span_cap32_small(uint32_t (&s)[32], const SpanCap& c) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
    const float2 y = __fmul2_rn(x, span_cap_small(x, c));
    s[2 * i] = __float_as_uint(y.x);
    s[2 * i + 1] = __float_as_uint(y.y);
  }
}
__device__ __forceinline__ void span_cap32(uint32_t (&s)[32], const SpanCap& c) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float e = ex2_approx(__uint_as_float(s[i]) * c.mul);
    s[i] = __float_as_uint(fmaf(-2.f * c.top, rcp_approx(e + 1.f), c.top));
  }
}

__device__ __forceinline__ float absmax3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// the largest magnitude of 32 n products: eight running maxima
template <int n>
__device__ __forceinline__ float span_absmax(const uint32_t (&x)[n][32]) {
  float m[8];
#pragma unroll
  for (int a = 0; a < 8; ++a) m[a] = fabsf(__uint_as_float(x[0][a]));
#pragma unroll
  for (int i = 8; i + 16 <= 32 * n; i += 16)
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      const int e = i + 2 * a;
      m[a] = absmax3(m[a], __uint_as_float(x[e >> 5][e & 31]), __uint_as_float(x[(e + 1) >> 5][(e + 1) & 31]));
    }
  // (8 mod 16: the last eight)
#pragma unroll
  for (int a = 0; a < 8; ++a) m[a] = fmaxf(m[a], fabsf(__uint_as_float(x[n - 1][24 + a])));
  return fmaxf(max3(m[0], m[1], m[2]), max3(max3(m[3], m[4], m[5]), m[6], m[7]));
}

}  // namespace fa
