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

struct SpanView {
  const int *begin, *end;      // [B][N] or nullptr: 0 and C
  const int *lens, *chunks;    // pages: tokens before the chunk [B]; new tokens [B], or nullptr: N
  const int* table;            // pages: [B][width] page numbers, or nullptr: keys in [B][Hkv][N][d]
  int width, page_shift;       // pages: entries per request; log2 of a page's rows
  int N;                       // query rows per head
  int C;                       // keys: N, or width pages
  int causal, window;          // j <= p_i; |p_i - j| < window (0: any)
  __device__ __forceinline__ int len(int b) const { return table ? min(max(lens[b], 0), C) : 0; }
  // query rows of request b that exist
  __device__ __forceinline__ int rows(int b, int len) const {
    return table ? min(min(max(chunks ? chunks[b] : N, 0), N), C - len) : N;
  }
  // the keys that query i of request b sees (pos: its position); lo >= hi: none
  __device__ __forceinline__ void span(int b, int i, int pos, int& lo, int& hi) const {
    lo = begin ? max(begin[(long long)b * N + i], 0) : 0;
    hi = end ? min(end[(long long)b * N + i], C) : C;
    clip(pos, pos, lo, hi);
  }
  // what is left of [lo, hi) for queries at positions p0 .. p1
  __device__ __forceinline__ void clip(int p0, int p1, int& lo, int& hi) const {
    if (causal) hi = min(hi, p1 + 1);
    if (window) {
      lo = max(lo, p0 - window + 1);
      hi = (int)min((long long)hi, (long long)p1 + window);
    }
  }
};

// Rows of a cache in pages: token t of a page and head at ptr + page * page + head * head + t * token.
struct PageRows {
  __nv_bfloat16* ptr;
  long long page, head, token;  // strides in elements
};

// one pair's score in log2 units, and d score / d (scale q k)
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

}  // namespace fa
