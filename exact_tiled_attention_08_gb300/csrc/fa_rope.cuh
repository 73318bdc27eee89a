// Head norm and rotation of queries and keys, forward and backward.
//
// Forward, for each token and each query or key head (a row x of d values):
//   x^ = x / sqrt(mean(x^2) + eps),  u = w o x^        (or u = x without the norm)
//   y  = f R(pos) u on the first `rot` values, u beyond them
// where R turns each pair (a, b) of values by the angle pos * freq_i:
//   (a cos - b sin, a sin + b cos),
// pairs (i, i + rot / 2) ("half") or (2 i, 2 i + 1) ("interleaved").  Rows are
// read where a projection left them (token-major, any strides) and written
// head-major, as the attention kernels read them; value rows are moved along.
// Backward: g = f R^T dy, dw = sum g o x^, dx = (w o g - x^ mean(w o g o x^)) / rms.
//
// Angles.  A position may be far (millions), where pos * freq in fp32 has lost
// its fraction.  freq / 2 pi is kept as a 64-bit binary fraction of a turn;
// the 64-bit product with the position wraps by whole turns, so its upper
// 32 bits are the angle to 2^-32 of a turn at any 32-bit position.
//
// Both are bound by memory: a row is read once and written once.  A lane holds
// 8 values (16 bytes), D / 8 lanes a row, so a warp moves 32 * 16 bytes per
// access; the cosines and sines of a token are computed once per warp and used
// for `head_step` heads.  Statistics and rotation are fp32, rounded once.
#pragma once

#include <cuda_bf16.h>

#include "sm103_ptx.cuh"

namespace fa {

struct RopeRows {
  const __nv_bfloat16* ptr;  // nullptr: no such rows
  long long batch, token, head;  // strides in elements
};

struct RopeParams {
  RopeRows q, k, v;               // token-major rows: forward inputs; backward: q, k inputs (v unused)
  RopeRows dq, dk, dv;            // backward: token-major gradients, written
  __nv_bfloat16 *q_out, *k_out, *v_out;  // head-major [B][H][N][d], [B][Hkv][C][d]; backward: read
  const float *q_weight, *k_weight;      // [d] or nullptr (ones)
  const double* inv_freq;                // [rot / 2]
  const int* positions;                  // [B][N] or nullptr
  const int* starts;                     // [B] or nullptr (0)
  float* partials;                       // backward: [gridDim.x][2][d] sums of the weight gradients
  int N, H, Hkv, C, rot;
  long long tokens;     // B * N
  int head_step;        // heads handled by one unit of work
  int head_groups;      // ceil((H + Hkv + Hkv) / head_step)
  long long units;      // token groups * head_groups
  float eps, factor;
  int norm;
};

// a token's 8 values from and to bf16
__device__ __forceinline__ void rope_unpack(const uint4& a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 rope_pack(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// freq / 2 pi as a binary fraction of a turn (whole turns dropped)
__device__ __forceinline__ unsigned long long rope_turns(double freq) {
  const double t = freq * 0.15915494309189533576888;
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of pos * freq, times f
__device__ __forceinline__ void rope_angle(unsigned long long turns, int pos, float f, float& c, float& s) {
  const unsigned long long a = turns * (unsigned long long)(long long)pos;
  const float half_turns = (float)(int)(a >> 32) * 4.656612873077393e-10f;  // * 2^-31
  sincospif(half_turns, &s, &c);
  c *= f;
  s *= f;
}

// The rotation of a lane's 8 values.  kInterleaved: 4 pairs of its own;
// otherwise 8 values whose partners another lane holds (`peer`), the sine
// carrying the sign of this lane's half.
template <bool kInterleaved>
struct RopeTurn {
  static constexpr int kAngles = kInterleaved ? 4 : 8;
  float c[kAngles], s[kAngles];
  int peer;     // lane of the partner values
  bool active;  // the lane's values are in the rotated part

  __device__ __forceinline__ void setup(const unsigned long long* turns, int rot, int sub, int lane, int pos, float f) {
    const int half = rot >> 4;  // lanes of half the rotated part
    active = 8 * sub < rot;
    peer = lane;
    if (!active) return;
    if (kInterleaved) {
#pragma unroll
      for (int i = 0; i < kAngles; ++i) rope_angle(turns[4 * sub + i], pos, f, c[i], s[i]);
    } else {
      const bool low = sub < half;
      peer = low ? lane + half : lane - half;
      const int first = 8 * (low ? sub : sub - half);
#pragma unroll
      for (int i = 0; i < kAngles; ++i) {
        rope_angle(turns[first + i], pos, f, c[i], s[i]);
        if (low) s[i] = -s[i];
      }
    }
  }
  // every lane of the warp takes part
  template <bool kBack>
  __device__ __forceinline__ void apply(float (&x)[8]) const {
    if (kInterleaved) {
      if (!active) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1], sn = kBack ? -s[i % kAngles] : s[i % kAngles];
        x[2 * i] = fmaf(a, c[i % kAngles], -b * sn);
        x[2 * i + 1] = fmaf(a, sn, b * c[i % kAngles]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[i], peer);
        if (active) x[i] = fmaf(x[i], c[i % kAngles], kBack ? -(y * s[i % kAngles]) : y * s[i % kAngles]);
      }
    }
  }
};

template <int kLanes>
__device__ __forceinline__ float rope_row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kRopeThreads = 256;

// the 8 weights of a lane (ones without a weight)
__device__ __forceinline__ void rope_weights(const float* w, int sub, float (&out)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = w ? __ldg(w + 8 * sub + i) : 1.f;
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_fwd_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8, kTokens = 32 / kLanes;  // lanes per row, tokens per warp
  __shared__ unsigned long long turns[64];
  for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads) turns[i] = rope_turns(p.inv_freq[i]);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes, mine = lane / kLanes;
  const long long token_groups = (p.tokens + kTokens * (kRopeThreads / 32) - 1) / (kTokens * (kRopeThreads / 32));
  for (long long unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
    const long long group = unit % token_groups;
    const int h0 = (int)(unit / token_groups) * p.head_step;
    const int h1 = min(h0 + p.head_step, p.H + 2 * p.Hkv);
    const long long token = (group * (kRopeThreads / 32) + warp) * kTokens + mine;
    const bool valid = token < p.tokens;
    const int b = valid ? (int)(token / p.N) : 0;
    const int n = valid ? (int)(token - (long long)b * p.N) : 0;
    const int start = p.starts ? __ldg(p.starts + b) : 0;
    const int pos = p.positions ? __ldg(p.positions + (valid ? token : 0)) : start + n;
    const long long row = (long long)start + n;  // row of this token in k_out and v_out
    const bool stored = valid && row >= 0 && row < p.C;
    RopeTurn<kInterleaved> turn;
    turn.setup(turns, p.rot, sub, lane, pos, p.factor);
    for (int h = h0; h < h1; ++h) {
      const int kind = h < p.H ? 0 : (h < p.H + p.Hkv ? 1 : 2);
      const int head = kind == 0 ? h : (kind == 1 ? h - p.H : h - p.H - p.Hkv);
      const RopeRows& in = kind == 0 ? p.q : (kind == 1 ? p.k : p.v);
      if (!in.ptr) continue;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (valid)
        raw = __ldg(reinterpret_cast<const uint4*>(in.ptr + b * in.batch + n * in.token + head * in.head) + sub);
      if (kind < 2) {
        float x[8];
        rope_unpack(raw, x);
        if (p.norm) {
          float ss = 0.f, w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
          const float r = rsqrtf(rope_row_sum<kLanes>(ss) * (1.f / D) + p.eps);
          rope_weights(kind ? p.k_weight : p.q_weight, sub, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
        }
        turn.template apply<false>(x);
        raw = rope_pack(x);
      }
      if (kind == 0) {
        if (valid) reinterpret_cast<uint4*>(p.q_out + (((long long)b * p.H + head) * p.N + n) * D)[sub] = raw;
      } else if (stored) {
        __nv_bfloat16* out = kind == 1 ? p.k_out : p.v_out;
        reinterpret_cast<uint4*>(out + (((long long)b * p.Hkv + head) * p.C + row) * D)[sub] = raw;
      }
    }
  }
}

// Backward.  The weight gradients are summed in registers over a CTA's rows,
// over its warps in a fixed order, and over the CTAs by fa_rope_dw_kernel, so
// they are the same from run to run.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_bwd_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8, kTokens = 32 / kLanes;
  __shared__ unsigned long long turns[64];
  __shared__ float sums[kRopeThreads / 32][2][D];
  for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads) turns[i] = rope_turns(p.inv_freq[i]);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes, mine = lane / kLanes;
  const long long token_groups = (p.tokens + kTokens * (kRopeThreads / 32) - 1) / (kTokens * (kRopeThreads / 32));
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  for (long long unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
    const long long group = unit % token_groups;
    const int h0 = (int)(unit / token_groups) * p.head_step;
    const int h1 = min(h0 + p.head_step, p.H + 2 * p.Hkv);
    const long long token = (group * (kRopeThreads / 32) + warp) * kTokens + mine;
    const bool valid = token < p.tokens;
    const int b = valid ? (int)(token / p.N) : 0;
    const int n = valid ? (int)(token - (long long)b * p.N) : 0;
    const int pos = p.positions ? __ldg(p.positions + (valid ? token : 0)) : n;
    RopeTurn<kInterleaved> turn;
    turn.setup(turns, p.rot, sub, lane, pos, p.factor);
    for (int h = h0; h < h1; ++h) {
      const int kind = h < p.H ? 0 : (h < p.H + p.Hkv ? 1 : 2);
      const int head = kind == 0 ? h : (kind == 1 ? h - p.H : h - p.H - p.Hkv);
      const RopeRows& out = kind == 0 ? p.dq : (kind == 1 ? p.dk : p.dv);
      if (!out.ptr) continue;
      const __nv_bfloat16* dy = kind == 0 ? p.q_out : (kind == 1 ? p.k_out : p.v_out);
      const int heads = kind == 0 ? p.H : p.Hkv;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (valid) raw = __ldg(reinterpret_cast<const uint4*>(dy + (((long long)b * heads + head) * p.N + n) * D) + sub);
      if (kind < 2) {
        float g[8];
        rope_unpack(raw, g);
        turn.template apply<true>(g);
        if (p.norm) {
          const RopeRows& in = kind ? p.k : p.q;
          uint4 xraw = make_uint4(0, 0, 0, 0);
          if (valid)
            xraw = __ldg(reinterpret_cast<const uint4*>(in.ptr + b * in.batch + n * in.token + head * in.head) + sub);
          float x[8], w[8];
          rope_unpack(xraw, x);
          rope_weights(kind ? p.k_weight : p.q_weight, sub, w);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
          const float r = rsqrtf(rope_row_sum<kLanes>(ss) * (1.f / D) + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] *= r;
            const float gx = valid ? g[i] * x[i] : 0.f;
            if (kind) dw[1][i] += gx; else dw[0][i] += gx;
            g[i] *= w[i];
            dot = fmaf(g[i], x[i], dot);
          }
          dot = rope_row_sum<kLanes>(dot) * (1.f / D);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = r * fmaf(-x[i], dot, g[i]);
        }
        raw = rope_pack(g);
      }
      if (valid)
        reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(out.ptr) + b * out.batch + n * out.token +
                                 head * out.head)[sub] = raw;
    }
  }
  if (!p.partials) return;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = dw[t][i];
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (mine == 0) sums[warp][t][8 * sub + i] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
    float v = 0.f;
    for (int w = 0; w < kRopeThreads / 32; ++w) v += (&sums[w][0][0])[i];
    p.partials[(long long)blockIdx.x * 2 * D + i] = v;
  }
}

// dw[t][i] = sum over the CTAs of partials[cta][t][i], in CTA order; one warp
// per output value.
__global__ void __launch_bounds__(256)
    fa_rope_dw_kernel(const float* __restrict__ partials, int ctas, int d, float* __restrict__ dq_weight,
                      float* __restrict__ dk_weight) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= 2 * d) return;
  float v = 0.f;
  for (int c = lane; c < ctas; c += 32) v += partials[(long long)c * 2 * d + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  float* out = i < d ? dq_weight : dk_weight;
  if (lane == 0 && out) out[i < d ? i : i - d] = v;
}

}  // namespace fa
