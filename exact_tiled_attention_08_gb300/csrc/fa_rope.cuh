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
// its fraction.  freq / 2 pi, an fp64 product, is kept as a 64-bit binary fraction
// of a turn; the 64-bit product with the position wraps by whole turns, and its
// upper 32 bits become the fp32 angle.  In radians an angle is off by at most
// 2^-52 |pos freq| (freq / 2 pi: the product's and the constant's rounding) and
// 2^-23 (the fp32 half-turns, up to 2^-26 of a turn, and the bits cut off): 2^-22 at two
// million and freq = 1, 2^-20 at the last 32-bit position; bf16's half step is 2^-8.
//
// Both are bound by memory: a row is read once and written once.  A lane holds
// 8 values of a row, D / 8 lanes a row; it holds whole pairs (in the half layout
// 4 values of each half), so that the rotation needs no other lane, and keeps 4
// cosines and sines for the heads of its token.  A warp has the rows of the
// next kRopeStages - 1 heads on their way.  Statistics and rotation are fp32,
// rounded once.  Measured, with the norm: 16384 tokens of 48 heads of 128 in 69 us
// (5.8 TB/s), backward at 8004 tokens in 55 us (5.1 TB/s); a copy reaches
// 6.8 TB/s.  (Packed arithmetic, a quarter fewer instructions, left the forward
// as it was: what is left is how rows of many heads lie in memory.)
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "fa_cross.cuh"
#include "fa_span.cuh"
#include "sm103_ptx.cuh"

namespace fa {

struct RopeRows {
  const __nv_bfloat16* ptr;  // nullptr: no such rows
  long long batch, token, head;  // strides in elements
};

// A token's heads, q, k and v counted on, in units that do not mix q with the
// others: q_units of q_step heads, then k and v in one unit, or each in units
// of kv_step.
struct RopeSplit {
  int steps;             // units per token group
  int q_units, q_step;
  int k_units, v_units;  // (0: left out, or both in one unit)
  int kv_step;
  int both;              // 1: one unit of all key and value heads
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
  RopeSplit split;      // how a token's heads are divided into units of work
  long long units;      // warps' units of work: token groups (rounded up to whole CTAs) * split.steps
  float eps, factor;
  int norm;
};

// Pages (their tokens' first positions in starts, C = width pages; table nullptr: queries alone).
struct RopePagedParams : RopeParams {
  PageRows k_pages, v_pages;
  const int *table, *chunks;  // [B][width]; [B] or nullptr: N new tokens
  int width, page_shift, pages;
};

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

// A lane's 8 values of a row as four pairs to be turned, (a, b): those of the
// halves, elements e0 + i and e1 + i, or neighbours.  Two pairs side by side, so
// that the arithmetic is packed (two fp32 operations an instruction).
template <bool kInterleaved>
struct RopeLane {
  float2 a[2], b[2];

  // element i (0 .. 7: e0 .. e0 + 3, e1 .. e1 + 3)
  __device__ __forceinline__ float& at(int i) {
    if (kInterleaved) {
      float2& v = (i & 1) ? b[i >> 2] : a[i >> 2];
      return (i >> 1) & 1 ? v.y : v.x;
    }
    float2& v = i < 4 ? a[(i >> 1) & 1] : b[(i >> 1) & 1];
    return i & 1 ? v.y : v.x;
  }
  __device__ __forceinline__ void load(const uint8_t* row, int e0, int e1) {
    const uint2 lo = *reinterpret_cast<const uint2*>(row + 2 * e0), hi = *reinterpret_cast<const uint2*>(row + 2 * e1);
    const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at(2 * i) = __uint_as_float(w[i] << 16);
      at(2 * i + 1) = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, int e0, int e1) {
    *reinterpret_cast<uint2*>(row + e0) = make_uint2(pack_bf16x2(at(0), at(1)), pack_bf16x2(at(2), at(3)));
    *reinterpret_cast<uint2*>(row + e1) = make_uint2(pack_bf16x2(at(4), at(5)), pack_bf16x2(at(6), at(7)));
  }
  // the weights of these elements (ones without a weight)
  __device__ __forceinline__ void weights(const float* w, int e0, int e1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) at(i) = w ? __ldg(w + (i < 4 ? e0 : e1) + (i & 3)) : 1.f;
  }
  __device__ __forceinline__ void scale(const RopeLane& w) {
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = __fmul2_rn(a[i], w.a[i]), b[i] = __fmul2_rn(b[i], w.b[i]);
  }
  __device__ __forceinline__ void scale(float f) {
    const float2 f2 = make_float2(f, f);
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = __fmul2_rn(a[i], f2), b[i] = __fmul2_rn(b[i], f2);
  }
  // this lane's part of sum x o y
  __device__ __forceinline__ float dot(const RopeLane& y) const {
    float2 s = __fmul2_rn(a[0], y.a[0]);
    s = __ffma2_rn(a[1], y.a[1], s);
    s = __ffma2_rn(b[0], y.b[0], s);
    s = __ffma2_rn(b[1], y.b[1], s);
    return s.x + s.y;
  }
  // this += x o y
  __device__ __forceinline__ void add_product(const RopeLane& x, const RopeLane& y) {
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = __ffma2_rn(x.a[i], y.a[i], a[i]), b[i] = __ffma2_rn(x.b[i], y.b[i], b[i]);
  }
  // this += f x
  __device__ __forceinline__ void add(float f, const RopeLane& x) {
    const float2 f2 = make_float2(f, f);
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = __ffma2_rn(x.a[i], f2, a[i]), b[i] = __ffma2_rn(x.b[i], f2, b[i]);
  }
};

// Rows on their way to a warp: a ring of kRopeStages in shared memory, one row of
// each of the warp's tokens per stage (32 lanes x 16 bytes), filled with
// cp.async, so that what is in flight takes no registers.
constexpr int kRopeStages = 8;

__device__ __forceinline__ void rope_copy(uint32_t smem, const void* row, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(row), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void rope_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the last kRopeStages - 1 groups of this warp have landed
__device__ __forceinline__ void rope_landed() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kRopeStages - 1) : "memory");
  __syncwarp();
}

// The rotation of a lane's values for one token.
template <bool kInterleaved>
struct RopeTurn {
  float2 c[2], s[2];
  bool active;  // the lane's values are in the rotated part

  // a lane's elements: e0 .. e0 + 3 and e1 .. e1 + 3
  static __device__ __forceinline__ void place(int rot, int sub, int& e0, int& e1) {
    const bool pairs = !kInterleaved && 8 * sub < rot;
    e0 = pairs ? 4 * sub : 8 * sub;
    e1 = pairs ? (rot >> 1) + 4 * sub : 8 * sub + 4;
  }
  __device__ __forceinline__ void setup(const unsigned long long* turns, int rot, int sub, int pos, float f) {
    active = 8 * sub < rot;
    if (!active) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rope_angle(turns[4 * sub + 2 * i], pos, f, c[i].x, s[i].x);
      rope_angle(turns[4 * sub + 2 * i + 1], pos, f, c[i].y, s[i].y);
    }
  }
  template <bool kBack>
  __device__ __forceinline__ void apply(RopeLane<kInterleaved>& v) const {
    if (!active) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 n = make_float2(-s[i].x, -s[i].y);
      const float2 a = __ffma2_rn(v.b[i], kBack ? s[i] : n, __fmul2_rn(v.a[i], c[i]));
      v.b[i] = __ffma2_rn(v.a[i], kBack ? n : s[i], __fmul2_rn(v.b[i], c[i]));
      v.a[i] = a;
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
// CTAs held by an SM.  More of them are slower, although they would fit: the
// rows of more heads and tokens are then open in memory at once (forward with
// 16384 tokens of 48 heads: 3 take 70 us, 4 74 us, 5 94 us).
constexpr int kRopeFwdPerSm = 3, kRopeBwdPerSm = 2;

// A warp's tokens in a unit of work, one per D / 8 lanes.
struct RopeToken {
  int b, n, sub;
  long long token;
  bool valid;
  int h0, h1;  // heads of q, k and v, counted on
};
template <int D>
__device__ __forceinline__ RopeToken rope_token(const RopeParams& p, long long unit) {
  constexpr int kLanes = D / 8, kTokens = 32 / kLanes;
  // a CTA's warps take neighbouring tokens and the same heads, neighbouring CTAs
  // the other heads of these tokens
  constexpr int kWarps = kRopeThreads / 32;
  const int steps = p.split.steps;
  const int lane = threadIdx.x & 31;
  const long long cta = unit / kWarps;
  RopeToken t;
  int step = (int)(cta % steps);
  t.token = (cta / steps * kWarps + unit % kWarps) * kTokens + lane / kLanes;
  t.sub = lane % kLanes;
  t.valid = t.token < p.tokens;
  t.b = t.valid ? (int)(t.token / p.N) : 0;
  t.n = t.valid ? (int)(t.token - (long long)t.b * p.N) : 0;
  if (step < p.split.q_units) {
    t.h0 = step * p.split.q_step;
    t.h1 = min(t.h0 + p.split.q_step, p.H);
  } else if (p.split.both) {
    t.h0 = p.H;
    t.h1 = p.H + 2 * p.Hkv;
  } else {
    step -= p.split.q_units;
    const bool v = step >= p.split.k_units;
    if (v) step -= p.split.k_units;
    const int first = p.H + (v ? p.Hkv : 0);
    t.h0 = first + step * p.split.kv_step;
    t.h1 = min(t.h0 + p.split.kv_step, first + p.Hkv);
  }
  return t;
}

// Heads [h0, h1) of one of q, k, v: norm, rotation and store.  (Each of the three
// has a loop of its own with running addresses: one loop over all heads that
// looks up where a head's row is takes 86 instead of 70 us, its ring not
// emptying in between notwithstanding.)
template <int D, bool kInterleaved, bool kNorm, bool kTurn>
__device__ __forceinline__ void rope_fwd_heads(const RopeTurn<kInterleaved>& turn, uint8_t* ring,
                                               const __nv_bfloat16* in, long long in_head, __nv_bfloat16* out,
                                               long long out_head, int h0, int h1, int e0, int e1, bool valid,
                                               bool stored, const float* weight, float eps) {
  constexpr int kLanes = D / 8;
  if (h0 >= h1) return;
  const int lane = threadIdx.x & 31;
  const uint8_t* mine = ring + (lane / kLanes) * (2 * D);  // this token's row of a stage
  const uint32_t dst = smem_u32(ring) + lane * 16;
  const __nv_bfloat16* src = in + 8 * (lane % kLanes) + h0 * in_head;
  out += h0 * out_head;
  RopeLane<kInterleaved> w;
  if (kNorm) w.weights(weight, e0, e1);
  int left = h1 - h0;  // rows to fetch
#pragma unroll
  for (int i = 0; i < kRopeStages - 1; ++i) {
    if (left > 0) rope_copy(dst + i * 512, src, valid);
    rope_commit();
    src += in_head;
    --left;
  }
  int stage = 0;
  for (int n = h1 - h0; n > 0; --n) {
    __syncwarp();  // the stage filled next has been read
    if (left > 0) rope_copy(dst + ((stage + kRopeStages - 1) % kRopeStages) * 512, src, valid);
    rope_commit();
    src += in_head;
    --left;
    rope_landed();
    RopeLane<kInterleaved> v;
    v.load(mine + stage * 512, e0, e1);
    stage = (stage + 1) % kRopeStages;
    if (kNorm) {
      const float r = rsqrtf(rope_row_sum<kLanes>(v.dot(v)) * (1.f / D) + eps);
      v.scale(w);
      v.scale(r);
    }
    if (kTurn) turn.template apply<false>(v);
    if (stored) v.store(out, e0, e1);
    out += out_head;
  }
  __syncwarp();  // the ring has been read
}

// Params: RopePagedParams where keys and values go to the pages of a cache, else RopeParams.  (Kernels of their
// own, so that contiguous caches keep their addresses and registers: 16384 tokens of 48 heads of 128 with
// the norm 69 us, 78 where addresses of pages are kept through the queries.)
template <int D, bool kInterleaved, bool kNorm, class Params>
__global__ void __launch_bounds__(kRopeThreads, kRopeFwdPerSm) fa_rope_fwd_kernel(const Params p) {
  constexpr bool kPaged = std::is_same<Params, RopePagedParams>::value;
  __shared__ unsigned long long turns[64];
  __shared__ __align__(16) uint8_t rings[kRopeThreads / 32][kRopeStages * 512];
  uint8_t* ring = rings[threadIdx.x >> 5];
  for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads) turns[i] = rope_turns(p.inv_freq[i]);
  __syncthreads();
  for (long long unit = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); unit < p.units;
       unit += (long long)gridDim.x * (kRopeThreads / 32)) {
    const RopeToken t = rope_token<D>(p, unit);
    int start = p.starts ? __ldg(p.starts + t.b) : 0;
    bool here = t.valid;  // a token of the chunk
    if constexpr (kPaged) {
      start = min(max(start, 0), p.C);
      here = here && t.n < min(p.chunks ? __ldg(p.chunks + t.b) : p.N, p.C - start);
      if (!__any_sync(0xffffffffu, here)) continue;  // (padding is not read)
    }
    const int pos = p.positions ? __ldg(p.positions + (t.valid ? t.token : 0)) : start + t.n;
    const long long row = (long long)start + t.n;  // row of this token in k_out and v_out
    bool stored = here && row >= 0 && row < p.C;
    int page = 0;
    if constexpr (kPaged) {
      if (stored && p.table) page = __ldg(p.table + (long long)t.b * p.width + (row >> p.page_shift));
      stored = stored && page >= 0 && page < p.pages;
      if (!stored) page = 0;
    }
    int e0, e1;
    RopeTurn<kInterleaved>::place(p.rot, t.sub, e0, e1);
    RopeTurn<kInterleaved> turn;
    if (t.h0 < p.H + p.Hkv) turn.setup(turns, p.rot, t.sub, pos, p.factor);
    auto in = [&](const RopeRows& r) { return r.ptr + t.b * r.batch + t.n * r.token; };
    if (p.q.ptr && t.h0 < p.H)
      rope_fwd_heads<D, kInterleaved, kNorm, true>(turn, ring, in(p.q), p.q.head,
                                                   p.q_out + ((long long)t.b * p.H * p.N + t.n) * D,
                                                   (long long)p.N * D, t.h0, min(t.h1, p.H), e0, e1,
                                                   kPaged ? here : t.valid, here, p.q_weight, p.eps);
    // where the row of the first key/value head goes, and how far the next one's is
    __nv_bfloat16 *k_to, *v_to;
    long long k_next = (long long)p.C * D, v_next = k_next;
    if constexpr (kPaged) {
      const long long in_page = row & ((1 << p.page_shift) - 1);
      k_to = p.k_pages.ptr + page * p.k_pages.page + in_page * p.k_pages.token;
      v_to = p.v_pages.ptr + page * p.v_pages.page + in_page * p.v_pages.token;
      k_next = p.k_pages.head;
      v_next = p.v_pages.head;
    } else {
      const long long cache = ((long long)t.b * p.Hkv * p.C + row) * D;
      k_to = p.k_out + cache;
      v_to = p.v_out + cache;
    }
    if (p.k.ptr)
      rope_fwd_heads<D, kInterleaved, kNorm, true>(turn, ring, in(p.k), p.k.head, k_to, k_next, max(t.h0 - p.H, 0),
                                                   min(t.h1 - p.H, p.Hkv), e0, e1, kPaged ? here : t.valid, stored,
                                                   p.k_weight, p.eps);
    if (p.v.ptr)
      rope_fwd_heads<D, kInterleaved, false, false>(turn, ring, in(p.v), p.v.head, v_to, v_next,
                                                    max(t.h0 - p.H - p.Hkv, 0), t.h1 - p.H - p.Hkv, e0, e1,
                                                    kPaged ? here : t.valid, stored, nullptr, 0.f);
  }
}

// heads [h0, h1) of one of q, k, v, backwards: dw gathers g o x^ of its rows
template <int D, bool kInterleaved, bool kNorm, bool kTurn>
__device__ __forceinline__ void rope_bwd_heads(const RopeTurn<kInterleaved>& turn, uint8_t* ring,
                                               const __nv_bfloat16* dy, long long dy_head, const __nv_bfloat16* in,
                                               long long in_head, __nv_bfloat16* out, long long out_head, int h0,
                                               int h1, int e0, int e1, bool valid, const float* weight, float eps,
                                               RopeLane<kInterleaved>& dw) {
  constexpr int kLanes = D / 8;
  if (h0 >= h1) return;
  const int lane = threadIdx.x & 31;
  const uint8_t* mine = ring + (lane / kLanes) * (2 * D);
  const uint32_t dst = smem_u32(ring) + lane * 16;
  const __nv_bfloat16* src = dy + 8 * (lane % kLanes) + h0 * dy_head;
  const __nv_bfloat16* xsrc = kNorm ? in + 8 * (lane % kLanes) + h0 * in_head : nullptr;
  out += h0 * out_head;
  int left = h1 - h0;  // rows to fetch
  auto fetch = [&](int stage) {
    if (left > 0) {
      rope_copy(dst + stage * 512, src, valid);
      if (kNorm) rope_copy(dst + (kRopeStages + stage) * 512, xsrc, valid);
    }
    rope_commit();
    src += dy_head;
    if (kNorm) xsrc += in_head;
    --left;
  };
  RopeLane<kInterleaved> w;
  if (kNorm) w.weights(weight, e0, e1);
#pragma unroll
  for (int i = 0; i < kRopeStages - 1; ++i) fetch(i);
  int stage = 0;
  for (int n = h1 - h0; n > 0; --n) {
    __syncwarp();  // the stage filled next has been read
    fetch((stage + kRopeStages - 1) % kRopeStages);
    rope_landed();
    RopeLane<kInterleaved> g;
    g.load(mine + stage * 512, e0, e1);
    if (kTurn) turn.template apply<true>(g);
    if (kNorm) {
      RopeLane<kInterleaved> x;  // (of a token that is not there: zeros, which add nothing)
      x.load(mine + (kRopeStages + stage) * 512, e0, e1);
      const float r = rsqrtf(rope_row_sum<kLanes>(x.dot(x)) * (1.f / D) + eps);
      x.scale(valid ? r : 0.f);  // x^
      dw.add_product(g, x);
      g.scale(w);
      const float mean = rope_row_sum<kLanes>(g.dot(x)) * (1.f / D);  // of w g x^
      g.add(-mean, x);
      g.scale(r);
    }
    stage = (stage + 1) % kRopeStages;
    if (valid) g.store(out, e0, e1);
    out += out_head;
  }
  __syncwarp();  // the ring has been read
}

template <bool kNorm>
constexpr int kRopeBwdSmemBytes = kRopeThreads / 32 * (kNorm ? 2 : 1) * kRopeStages * 512;
static_assert(kRopeBwdSmemBytes<true> >= kRopeThreads / 32 * 2 * 128 * 4, "the warps' sums take the rings' place");

// Backward.  The weight gradients are summed in registers over a warp's rows,
// over a CTA's warps in a fixed order, and over the CTAs by fa_rope_dw_kernel,
// so they are the same from run to run.
template <int D, bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, kRopeBwdPerSm) fa_rope_bwd_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;
  __shared__ unsigned long long turns[64];
  extern __shared__ __align__(16) uint8_t rope_smem[];  // the warps' rings; at the end their sums [warp][2][D]
  for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads) turns[i] = rope_turns(p.inv_freq[i]);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = rope_smem + warp * (kRopeBwdSmemBytes<kNorm> / (kRopeThreads / 32));
  RopeLane<kInterleaved> dw[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0].at(i) = dw[1].at(i) = 0.f;
  int e0, e1;
  RopeTurn<kInterleaved>::place(p.rot, lane % kLanes, e0, e1);
  for (long long unit = (long long)blockIdx.x * (kRopeThreads / 32) + warp; unit < p.units;
       unit += (long long)gridDim.x * (kRopeThreads / 32)) {
    const RopeToken t = rope_token<D>(p, unit);
    const int pos = p.positions ? __ldg(p.positions + (t.valid ? t.token : 0)) : t.n;
    RopeTurn<kInterleaved> turn;
    if (t.h0 < p.H + p.Hkv) turn.setup(turns, p.rot, t.sub, pos, p.factor);
    auto at = [&](const RopeRows& r) { return const_cast<__nv_bfloat16*>(r.ptr) + t.b * r.batch + t.n * r.token; };
    const long long next = (long long)p.N * D, kv = ((long long)t.b * p.Hkv * p.N + t.n) * D;
    if (p.dq.ptr && t.h0 < p.H)
      rope_bwd_heads<D, kInterleaved, kNorm, true>(turn, ring, p.q_out + ((long long)t.b * p.H * p.N + t.n) * D, next,
                                                   at(p.q), p.q.head, at(p.dq), p.dq.head, t.h0, min(t.h1, p.H), e0,
                                                   e1, t.valid, p.q_weight, p.eps, dw[0]);
    if (p.dk.ptr)
      rope_bwd_heads<D, kInterleaved, kNorm, true>(turn, ring, p.k_out + kv, next, at(p.k), p.k.head, at(p.dk), p.dk.head,
                                                   max(t.h0 - p.H, 0), min(t.h1 - p.H, p.Hkv), e0, e1, t.valid,
                                                   p.k_weight, p.eps, dw[1]);
    if (p.dv.ptr)
      rope_bwd_heads<D, kInterleaved, false, false>(turn, ring, p.v_out + kv, next, nullptr, 0, at(p.dv), p.dv.head,
                                                    max(t.h0 - p.H - p.Hkv, 0), t.h1 - p.H - p.Hkv, e0, e1, t.valid,
                                                    nullptr, 0.f, dw[1]);
  }
  if constexpr (kNorm) {
    grid_trigger();  // the next kernel adds the CTAs' sums
    if (!p.partials) return;
    __syncthreads();
    float* sums = reinterpret_cast<float*>(rope_smem);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = dw[t].at(i);
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < kLanes) sums[(warp * 2 + t) * D + (i < 4 ? e0 : e1) + (i & 3)] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
    float v = 0.f;
    for (int w = 0; w < kRopeThreads / 32; ++w) v += sums[w * 2 * D + i];
    p.partials[(long long)blockIdx.x * 2 * D + i] = v;
  }
  }
}

// dw[t][i] = sum over the CTAs of partials[cta][t][i]: a block per 32 values,
// its warps over the CTAs, then over the warps in order.
__global__ void __launch_bounds__(1024)
    fa_rope_dw_kernel(const float* partials, int ctas, int d, float* dq_weight, float* dk_weight) {
  __shared__ float sums[32][32];
  grid_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * 32 + lane;
  float v = 0.f;
#pragma unroll 4
  for (int c = warp; c < ctas; c += 32) v += partials[(long long)c * 2 * d + i];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) v += sums[w][lane];
  float* out = i < d ? dq_weight : dk_weight;
  if (out) out[i < d ? i : i - d] = v;
}

}  // namespace fa
