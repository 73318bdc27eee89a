// Backward of attention to spans of keys (fa_span_bwd).
//
// The per-block arithmetic, roles and barriers are those of fa_bwd_kernel with
// the atomic dQ: a CTA keeps K_j and V_j (128 keys) and streams query blocks past
// them; dQ goes to an fp32 accumulator by TMA reduces.  What differs:
//
// Work.  An item is a key block of a request and key/value head; it meets, for each of the
// G query heads that share the head, the query blocks from the first to the last that has
// a row which sees one of its keys, so dK and dV are summed over the group in tensor memory.
// Items cost what they have of them (a causal mask: from 1 to all).  fa_span_plan_kernel lists them, the
// longest of a request first, and cuts those that are longer than a CTA's share of
// everything into runs, whose sums fa_span_bwd_post_kernel adds in order; the CTAs draw runs by
// a ticket when they are about to need one.
//
// Masks.  A block that all of the query block's rows see whole takes none.  In others a lane
// takes one query's span as bits of the warp's 32 keys, and the warp transposes them to
// a thread's (one key's) bits of 32 queries; P and so dS are zero outside them.
//
// Scores as in the forward: P = 2^(s log2e - LSE log2e) with the capped and biased score
// s, and dS = P o (dP - delta) o (1 - tanh^2); P (1 - tanh^2) is what is kept
// between the two halves of the elementwise step.
//
// Measured on a GB300 (two requests, H=32/8 N=8192 d=128, causal): 2.28 ms, 1204 TFLOP/s (fa_bwd at H=32: 2.18),
// capped 2.71 ms, capped and with slopes 2.95; 25 packed documents of one request, capped, 421 us, of which the
// main kernel takes 340.
// The elementwise warps bound it.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "fa_cross_bwd.cuh"
#include "fa_span.cuh"
#include "fa_span_fwd.cuh"

namespace fa {

// A unit of work: blocks [f0, f1) of the G cnt query blocks (head by head, cnt of them from
// block i0 on) of a key block.
struct SpanRun {
  int jb, i0, cnt, f0, f1;
  int part, slot;  // slot < 0: the item is whole; else its sums go to slot + part Hkv + head
  int pad;
};

struct SpanBwdPlan {
  int ticket;     // the next unit
  int units;      // of all requests
  int cut;        // entries (request and key block) that are cut
  int pad;
};

constexpr int kSpanBwdSlots = 608;  // runs of cut items
constexpr int kSpanBwdSegs = 2;

struct SpanBwdParams {
  SpanRows<false> rows;           // (tiles of the query heads; bounds always given)
  const int *lo, *hi;      // [B][npad] spans of the queries
  SpanBwdPlan* plan;
  SpanRun* runs;           // [entries + kSpanBwdSlots], request by request
  int* first;              // [B + 1] a request's first run
  int2* hulls;             // [entries]
  int* order;              // [entries] a request's key blocks, the longest first
  int4* cuts;              // [kSpanBwdSlots / 2] entries that are cut: request, key block, slot, parts
  float* sums;             // [slot][dK, dV][128][d], fp32, unscaled
  __nv_bfloat16 *dk, *dv;
  __nv_bfloat16* dq;       // one key block: written directly (scaled, bf16); else nullptr
  int B, H, Hkv, N, nb;    // nb: blocks of N
  float scale_log2;        // scale * log2(e)
  float scale;
  SpanCap cap;
  const float* slopes;
  uint64_t wait_limit_ns;
  int debug_stall;
  int out_align32;
};

// Per row of each request and query head, padded to whole 128-row blocks: -delta, delta = sum dO O
// (0 behind the rows) and -LSE log2(e) (-inf behind them, and for rows without keys, so that
// P = 0 there; negated here, not 128 times in the main kernel's loop); the dQ accumulator, if
// there is one, is zeroed.  The blocks behind
// these write the queries' spans and their tiles' bounds (128 rows a block).
template <int D>
__global__ void __launch_bounds__(256)
    fa_span_bwd_prep_kernel(const __nv_bfloat16* o, const __nv_bfloat16* dout, const float* lse, float* delta_pad,
                            float* lse2_pad, float* dq_acc, const SpanView<false> v, int* lo_pad, int* hi_pad, int4* bounds,
                            int B, int npad, long long padded_rows) {
  constexpr int kThreadsPerRow = D / 8, kRows = 256 / kThreadsPerRow;
  __shared__ int4 scratch[8];  // (of the first four warps, and what the others leave)
  const int sub = threadIdx.x % kThreadsPerRow;
  const int N = v.N, tiles = npad / 128, row_blocks = gridDim.x - (B * tiles + 1) / 2;
  grid_wait();
  grid_trigger();
  if ((int)blockIdx.x >= row_blocks) {
    // two tiles, one after the other
    for (int half = 0; half < 2; ++half) {
      const int k = 2 * (blockIdx.x - row_blocks) + half;
      if (k >= B * tiles) return;
      const int b = k / tiles, i = (k - b * tiles) * 128 + (int)threadIdx.x;
      int lo = 0, hi = 0;
      if (threadIdx.x < 128) {
        if (i < N) v.span(b, i, i, lo, hi);
        lo_pad[(long long)b * npad + i] = lo;
        hi_pad[(long long)b * npad + i] = hi;
      }
      const int4 s = span_tile_reduce(lo, hi, threadIdx.x < 128 && i < N, scratch);
      if (threadIdx.x == 0) bounds[k] = s;
      __syncthreads();
    }
    return;
  }
  for (long long prow = (long long)blockIdx.x * kRows + threadIdx.x / kThreadsPerRow;
       prow - threadIdx.x / kThreadsPerRow < padded_rows; prow += (long long)row_blocks * kRows) {
    const long long bh = prow / npad;
    const int n = (int)(prow - bh * npad);
    const bool in_range = prow < padded_rows, valid = in_range && n < N;
    const long long row = bh * N + n;
    float s = 0.f;
    if (valid) {
      const uint4 a = reinterpret_cast<const uint4*>(o + row * D)[sub];
      const uint4 g = reinterpret_cast<const uint4*>(dout + row * D)[sub];
      const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a);
      const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = __bfloat1622float2(a2[i]), y = __bfloat1622float2(g2[i]);
        s = fmaf(x.x, y.x, s);
        s = fmaf(x.y, y.y, s);
      }
      if (dq_acc) {
        float4* z = reinterpret_cast<float4*>(dq_acc + row * D) + 2 * sub;
        z[0] = z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int off = kThreadsPerRow / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (in_range && sub == 0) {
      const float l = valid ? lse[row] : -CUDART_INF_F;
      delta_pad[prow] = valid ? -s : 0.f;
      lse2_pad[prow] = l == -CUDART_INF_F ? -CUDART_INF_F : l * -1.4426950408889634f;
    }
  }
}

// The query blocks of a key block: from the first to the last that sees one of its keys
// (none: the first, whose pairs are all masked, so that zeros are written).  By one warp.
__device__ __forceinline__ int2 span_bwd_hull(const SpanBwdParams& p, int b, int jb) {
  const SpanView<false>& v = p.rows.view;
  const int lane = threadIdx.x & 31;
  if (!v.begin && !v.end) {
    int i0 = 0, i1 = p.nb;
    if (v.causal) i0 = jb;
    if (v.window) {
      i1 = (int)min((long long)p.nb, ((long long)jb * 128 + 127 + v.window - 1) / 128 + 1);
      if (!v.causal) i0 = (int)max(0ll, ((long long)jb * 128 - v.window + 1) / 128);
    }
    return make_int2(i0, i1);
  }
  const int4* bounds = p.rows.bounds + (long long)b * p.nb;
  int first = p.nb, last = -1;
#pragma unroll 2
  for (int i = lane; i < p.nb; i += 32) {
    const int4 x = bounds[i];
    if (x.x < (jb + 1) * 128 && x.y > jb * 128) {
      first = min(first, i);
      last = i;
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  return last < 0 ? make_int2(0, 1) : make_int2(first, last + 1);
}

// Items longer than half of a CTA's share of everything are cut into runs of about that
// (so at most kSpanBwdSlots runs come of it), but none shorter than kSpanBwdRun blocks.
// (Measured, cutting only where an item is longer than a whole share: 25 packed documents,
// N=8192 H=32/8 d=128, 390 and 372 us; equal where nothing is that long.)
constexpr int kSpanBwdRun = 4;

// One CTA: hulls and costs, the cut length, and the runs in the order of the entries.  With spans by row it
// looks at all of a request's blocks for each of them, twice: 7 us at 64 blocks, and it grows with their square
// (documents of 512 tokens, H=8/1 d=128: N=131072 0.13 of 1.04 ms, N=524288 1.8 of 5.4 ms).
__global__ void __launch_bounds__(1024) fa_span_plan_kernel(const __grid_constant__ SpanBwdParams p) {
  __shared__ long long work_of[32];
  __shared__ int runs_of[32], cut_of[32], slots_of[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = p.B * p.nb, G = p.H / p.Hkv, chunk = (E + 1023) / 1024, e0 = min(E, tid * chunk), e1 = min(E, e0 + chunk);
  grid_wait();
  for (int e = warp; e < E; e += 32) {
    const int b = e / p.nb;
    const int2 h = span_bwd_hull(p, b, e - b * p.nb);
    if (lane == 0) p.hulls[e] = h;
  }
  __syncthreads();
  // each request's key blocks by falling cost (a formula's fall with the key block already)
  const bool sorted = p.rows.view.begin || p.rows.view.end;
  for (int e = sorted ? tid : E; e < E; e += 1024) {
    const int b = e / p.nb, jb = e - b * p.nb;
    const int2 mine = p.hulls[e], *all = p.hulls + (long long)b * p.nb;
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < p.nb; ++i) {
      const int more = (all[i].y - all[i].x) - (mine.y - mine.x);
      rank += more > 0 || (more == 0 && i < jb) ? 1 : 0;
    }
    p.order[(long long)b * p.nb + rank] = jb;
  }
  __syncthreads();
  auto block_of = [&](int e, int b) { return sorted ? p.order[e] : e - b * p.nb; };
  long long work = 0;
  for (int e = e0; e < e1; ++e) {
    const int2 h = p.hulls[e];
    work += h.y - h.x;
  }
  auto sum = [&](long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  auto upto = [&](int x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int add = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += add;
    }
    return x;
  };
  work = sum(work);
  if (lane == 0) work_of[warp] = work;
  __syncthreads();
  work = sum(work_of[lane]) * G * p.Hkv;
  const int length = (int)min((long long)0x7fffffff, max((long long)kSpanBwdRun, (2 * work + kSpanBwdSlots - 1) / kSpanBwdSlots));
  auto parts = [&](int cost) { return cost > length ? (cost + length - 1) / length : 1; };
  // this thread's runs, cut entries and their runs, and those of all before it
  int runs = 0, cut = 0, slots = 0;
  for (int e = e0; e < e1; ++e) {
    const int b = e / p.nb;
    const int2 h = p.hulls[(long long)b * p.nb + block_of(e, b)];
    const int n = parts((h.y - h.x) * G);
    runs += n;
    if (n > 1) ++cut, slots += n;
  }
  int at = upto(runs) - runs, cut_at = upto(cut) - cut, slot = upto(slots) - slots;
  if (lane == 31) runs_of[warp] = at + runs, cut_of[warp] = cut_at + cut, slots_of[warp] = slot + slots;
  __syncthreads();
  const int all_runs = upto(runs_of[lane]), all_cut = upto(cut_of[lane]), all_slots = upto(slots_of[lane]);
  if (warp > 0) {
    at += __shfl_sync(0xffffffffu, all_runs, warp - 1);
    cut_at += __shfl_sync(0xffffffffu, all_cut, warp - 1);
    slot += __shfl_sync(0xffffffffu, all_slots, warp - 1);
  }
  for (int e = e0; e < e1; ++e) {
    const int b = e / p.nb, jb = block_of(e, b);
    const int2 h = p.hulls[(long long)b * p.nb + jb];
    const int cost = (h.y - h.x) * G, n = parts(cost);
    if (e == b * p.nb) p.first[b] = at;
    for (int i = 0; i < n; ++i)
      p.runs[at + i] = SpanRun{jb, h.x, h.y - h.x, cross_bwd_cut(i, n, cost), cross_bwd_cut(i + 1, n, cost), i,
                               n > 1 ? slot * p.Hkv : -1, 0};
    at += n;
    if (n > 1) {
      p.cuts[cut_at++] = make_int4(b, jb, slot * p.Hkv, n);
      slot += n;
    }
  }
  if (tid == 31) {
    p.first[p.B] = all_runs;
    *p.plan = SpanBwdPlan{0, all_runs * p.Hkv, all_cut, 0};
  }
}

// a drawn unit, as the other warps read it
struct SpanBwdSeg {
  int b, kvh, jb, i0, cnt, n;  // n: blocks
  int head, i;                 // of the first block: head of the group, query block
  int slot;
  int end;                     // no more units
};

// Unit k: requests one after another, in a request run by run, of all key/value heads.  (Groups of
// heads, which keep fewer query rows in use at a time, are slower: N=4096 H=32 d=128, two requests,
// causal, 713 us, in groups of 18 heads 727, of 4 781.)
__device__ __forceinline__ bool span_bwd_unit(const SpanBwdParams& p, int k, SpanBwdSeg& s) {
  if (k >= p.plan->units) return false;
  const int run = k / p.Hkv;
  int b = 0, top = p.B;  // first[b] <= run < first[b + 1]
  while (top - b > 1) {
    const int mid = (b + top) >> 1;
    if (p.first[mid] <= run) b = mid;
    else top = mid;
  }
  s.b = b;
  s.kvh = k - run * p.Hkv;
  const SpanRun x = p.runs[run];
  s.jb = x.jb, s.i0 = x.i0, s.cnt = x.cnt, s.n = x.f1 - x.f0;
  s.head = x.f0 / x.cnt;
  s.i = x.i0 + x.f0 - s.head * x.cnt;
  s.slot = x.slot < 0 ? -1 : x.slot + x.part * p.Hkv + s.kvh;
  s.end = 0;
  return true;
}

struct SpanBwdBarriers {
  BwdBarriers b;
  uint64_t seg_full[kSpanBwdSegs], seg_empty[kSpanBwdSegs];
  SpanBwdSeg seg[kSpanBwdSegs];
  int cut[4];  // of the query block in each statistics entry: some pair of the block is hidden
};
constexpr int kSpanBwdReaders = 15;  // issuers, the dO producer, four reducer and eight elementwise warps
static_assert(sizeof(SpanBwdBarriers) <= 768, "barriers overflow their shared-memory slot");
template <int D>
constexpr int kSpanBwdSmemBytes = BwdCfg<D, true>::kSmemBytes - 256 + 768;
static_assert(kSpanBwdSmemBytes<128> <= 227 * 1024, "shared memory budget");

enum : int { kSiteSpanBwdSeg = 80, kSiteSpanBwdSegFree };

__device__ __forceinline__ bool span_bwd_segment(SpanBwdBarriers* bar, int n, const WaitCtx& ctx, SpanBwdSeg& t) {
  const int s = n % kSpanBwdSegs;
  if (!span_wait(&bar->seg_full[s], (n / kSpanBwdSegs) & 1, ctx, kSiteSpanBwdSeg)) return false;
  t = bar->seg[s];
  return !t.end;
}

// bit q of lane k's result: bit k of lane q's value
__device__ __forceinline__ uint32_t span_transpose(uint32_t v, int lane) {
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const uint32_t m = j == 16 ? 0x0000ffffu : j == 8 ? 0x00ff00ffu : j == 4 ? 0x0f0f0f0fu : j == 2 ? 0x33333333u : 0x55555555u;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, v, j);
    v = lane & j ? (v & ~m) | ((y >> j) & m) : (v & m) | ((y << j) & ~m);
  }
  return v;
}

// Blocks seen in part, by one warp, 32 queries at a time: hidden products become -inf in tensor
// memory (with a cap their tanh is -1, its derivative 0), and with a cap hidden
// probabilities 0 behind that (with a bias too those that are kept for dS).  (Small code away from the loop: masks unrolled into it
// cost a block that is seen in part more than twice another's time.)
__device__ __forceinline__ void span_bwd_hide_s(uint32_t at, const uint32_t (&seen)[2]) {
#pragma unroll 1
  for (int ch = 0; ch < 2; ++ch) {
    const uint32_t bits = ch ? seen[1] : seen[0];
    if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
    uint32_t x[32];
    tmem_ld32(at + 32 * ch, x);
    tmem_wait_ld();
    reg_fence32(x);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((bits >> e) & 1u)) x[e] = __float_as_uint(-CUDART_INF_F);
    tmem_st32(at + 32 * ch, x);
  }
  tmem_wait_st();
}
// (P of query groups 2 ch and 2 ch + 1: over the first 8 of their 16 columns)
__device__ __forceinline__ void span_bwd_hide_p(uint32_t at, const uint32_t (&seen)[2]) {
  tmem_wait_st();
#pragma unroll 1
  for (int ch = 0; ch < 2; ++ch) {
    const uint32_t bits = ch ? seen[1] : seen[0];
    uint32_t x[32];
    tmem_ld32(at + 32 * ch, x);
    tmem_wait_ld();
    reg_fence32(x);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      uint32_t& pair = x[(e >> 3) * 16 + (e & 7)];
      pair &= ((bits >> (2 * e)) & 1u ? 0x0000ffffu : 0u) | ((bits >> (2 * e + 1)) & 1u ? 0xffff0000u : 0u);
    }
    tmem_st8(at + 32 * ch, x);
    tmem_st8(at + 32 * ch + 16, x + 16);
  }
}

// the block after (head, i)
__device__ __forceinline__ void span_bwd_step(const SpanBwdSeg& t, int& head, int& i) {
  if (++i == t.i0 + t.cnt) i = t.i0, ++head;
}

template <int D, int MOD>
__global__ void __launch_bounds__(512, 1)
    fa_span_bwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                       const __grid_constant__ CUtensorMap map_lse2, const __grid_constant__ CUtensorMap map_delta,
                       const __grid_constant__ CUtensorMap map_dq, const __grid_constant__ SpanBwdParams p) {
  using C = BwdCfg<D, true>;
  using R = BwdRegs<D, true>;
  static_assert(R::kLaunch == C::kLaunchRegs, "register split of the launch budget");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    // the 128-byte-swizzled tiles need 1024-byte alignment: report, do nothing
    grid_wait();
    if (threadIdx.x == 0) atomicCAS(&g_fa_device_status, 0u, kStatusBadSmem);
    return;
  }
  uint8_t* smem = smem_raw;
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTileBytes;
  uint8_t* sRing = smem + 2 * C::kTileBytes;
  uint8_t* sDS = sRing + C::kSlots * C::kTileBytes;
  uint8_t* sStage = sDS + C::kDsBytes;
  // query block g: entry g % kStatEntries = -LSE*log2e [128], -delta [128]
  uint8_t* sStat = sStage + C::kStageBytes;
  SpanBwdBarriers* xbar = reinterpret_cast<SpanBwdBarriers*>(sStat + C::kStatEntries * C::kStatBytes);
  BwdBarriers* bar = &xbar->b;
  static_assert(C::kStatEntries <= 4, "a cut flag for each entry");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.H / p.Hkv;

  if (tid == 0) {
    mbar_init(&bar->kv_full, 1);
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bar->ring_full[s], 1);
      mbar_init(&bar->ring_empty[s], 1);
    }
    mbar_init(&bar->s_full, 1);
    mbar_init(&bar->dp_full, 1);
    mbar_init(&bar->p_done, 256);
    mbar_init(&bar->ew_done, 256);
    mbar_init(&bar->dv_done, 1);
    mbar_init(&bar->dq_full, 1);
    mbar_init(&bar->dq_free, 128);
    mbar_init(&bar->dk_done, 1);
    mbar_init(&bar->acc_done, 1);
    mbar_init(&bar->drain[0], 1);
    mbar_init(&bar->drain[1], 1);
    mbar_init(&bar->never, 1);
    for (int s = 0; s < kSpanBwdSegs; ++s) {
      mbar_init(&xbar->seg_full[s], 1);
      mbar_init(&xbar->seg_empty[s], kSpanBwdReaders);
    }
    bar->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(&bar->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 13 && lane == 0) {
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
    tma_prefetch_map(&map_do);
    tma_prefetch_map(&map_lse2);
    tma_prefetch_map(&map_delta);
    tma_prefetch_map(&map_dq);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_wait();
  grid_trigger();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtx ctx{&bar->abort_flag, p.wait_limit_ns};
  SpanBwdSeg t;
  // (a segment's copy is in registers: its place is free)
  auto next_segment = [&](int n) { return span_bwd_segment(xbar, n, ctx, t); };
  auto taken = [&](int n) { mbar_arrive(&xbar->seg_empty[n % kSpanBwdSegs]); };
  if (warp >= 12) {
    setmaxnreg_dec<R::kMisc>();
    if (warp == 13) {
      // ---------------------------------------------------------------- units, and TMA of K, V and the Q tiles
      // g counts query blocks over all of the CTA's units
      if (lane == 0) {
        int g = 0, kv_loads = 0;
        bool ok = true;
        int ticket = atomicAdd(&p.plan->ticket, 1);
#pragma unroll 1
        for (int w = 0; ok; ++w) {
          const bool more = span_bwd_unit(p, ticket, t);
          if (!more) t.end = 1;
          const int place = w % kSpanBwdSegs;
          if (!span_wait(&xbar->seg_empty[place], ((w / kSpanBwdSegs) & 1) ^ 1, ctx, kSiteSpanBwdSegFree)) break;
          xbar->seg[place] = t;
          mbar_arrive(&xbar->seg_full[place]);
          if (!more) break;
          ticket = atomicAdd(&p.plan->ticket, 1);  // (the next one is on its way meanwhile)
          // K and V of the item, once the previous item's last products
          // (acc_done) have read the old ones
          if (w > 0 && !span_wait(&bar->acc_done, (w - 1) & 1, ctx, kSiteBwdProducer)) break;
          mbar_arrive_expect_tx(&bar->kv_full, 2 * C::kTileBytes);
          const int bk = t.b * p.Hkv + t.kvh;
          for (int a = 0; a < C::kAtoms; ++a) {
            tma_load_3d(sK + a * 16384, &map_k, &bar->kv_full, a * 64, t.jb * 128, bk);
            tma_load_3d(sV + a * 16384, &map_v, &bar->kv_full, a * 64, t.jb * 128, bk);
          }
          ++kv_loads;
          int head = t.head, i = t.i;
          const int4* bounds = p.rows.bounds + (long long)t.b * p.nb;
          int4 tile = bounds[i];
#pragma unroll 1
          for (int it = 0; it < t.n; ++it, ++g) {
            const int at = i, bh = t.b * p.H + t.kvh * G + head;
            const bool cut = t.jb * 128 < tile.z || t.jb * 128 + 128 > tile.w;
            span_bwd_step(t, head, i);
            tile = bounds[i];
            const int s = g % C::kQSlots;
            if (!span_wait(&bar->ring_empty[s], ((g / C::kQSlots) & 1) ^ 1, ctx, kSiteBwdProducer)) {
              ok = false;
              break;
            }
            xbar->cut[g % C::kStatEntries] = cut;
            mbar_arrive_expect_tx(&bar->ring_full[s], C::kTileBytes + C::kStatBytes);
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_3d(sRing + s * C::kTileBytes + a * 16384, &map_q, &bar->ring_full[s], a * 64, at * 128, bh);
            uint8_t* st = sStat + (g % C::kStatEntries) * C::kStatBytes;
            tma_load_2d(st, &map_lse2, &bar->ring_full[s], at * 128, bh);
            tma_load_2d(st + 512, &map_delta, &bar->ring_full[s], at * 128, bh);
          }
        }
        // every load this warp started has landed before the CTA may end
        if (kv_loads > 0) wait_drain_inl(&bar->kv_full, (kv_loads - 1) & 1, kDrainLimitNs);
#pragma unroll 1
        for (int k = 0; k < C::kQSlots; ++k)
          if (g > k) wait_drain_inl(&bar->ring_full[k], ((g - 1 - k) / C::kQSlots) & 1, kDrainLimitNs);
      }
      __syncwarp();
    } else if (warp == 15) {
      // ---------------------------------------------------------------- TMA producer: the dO tiles
      if (lane == 0) {
        int g = 0;
        bool ok = true;
#pragma unroll 1
        for (int w = 0; ok && next_segment(w); ++w) {
          taken(w);
          int head = t.head, i = t.i;
#pragma unroll 1
          for (int it = 0; it < t.n; ++it, ++g) {
            const int s = C::kQSlots + g % C::kDoSlots;
            if (!span_wait(&bar->ring_empty[s], ((g / C::kDoSlots) & 1) ^ 1, ctx, kSiteBwdProducer)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bar->ring_full[s], C::kTileBytes);
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_3d(sRing + s * C::kTileBytes + a * 16384, &map_do, &bar->ring_full[s], a * 64, i * 128,
                          t.b * p.H + t.kvh * G + head);
            span_bwd_step(t, head, i);
          }
        }
#pragma unroll 1
        for (int k = 0; k < C::kDoSlots; ++k)
          if (g > k) wait_drain_inl(&bar->ring_full[C::kQSlots + k], ((g - 1 - k) / C::kDoSlots) & 1, kDrainLimitNs);
      }
      __syncwarp();
    } else if (warp == 12) {
      // ---------------------------------------------------------------- issuer A: S^T and dP^T
      if (lane == 0) {
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
        const uint32_t ring = smem_u32(sRing);
        const uint64_t kdesc = sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t vdesc = sdesc_sw128(smem_u32(sV), 16, 1024);
        const uint32_t tS = tmem + C::kSCol, tDP = tmem + C::kDpCol;
        bool ok = !(p.debug_stall && !span_wait(&bar->never, 0, ctx, kSiteStall));
        // S^T goes first: the first half of the elementwise step needs only
        // S^T, its columns are free as soon as dV of the previous block has
        // run, and dP^T waits for the reducers to take the previous dQ out of
        // its columns.
        int g = 0;
#pragma unroll 1
        for (int w = 0; ok && next_segment(w); ++w) {
          taken(w);
          ok = span_wait(&bar->kv_full, w & 1, ctx, kSiteBwdKV);
#pragma unroll 1
          for (int it = 0; ok && it < t.n; ++it, ++g) {
            // S^T = K Q_i^T, once dV has consumed the previous P^T held in
            // these columns
            const int sq = g % C::kQSlots, sd = C::kQSlots + g % C::kDoSlots;
            ok = span_wait(&bar->ring_full[sq], (g / C::kQSlots) & 1, ctx, kSiteBwdQ) &&
                 (g == 0 || span_wait(&bar->dv_done, (g - 1) & 1, ctx, kSiteBwdDvDone));
            if (!ok) break;
            tc_fence_after();
            const uint64_t qdesc = sdesc_sw128(ring + sq * C::kTileBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              mma_bf16_ss(tS, kdesc + off, qdesc + off, id_s, kk > 0 ? 1u : 0u);
            }
            mma_commit(&bar->s_full);
            // dP^T = V dO_i^T, once the reducers have taken the previous dQ
            // out of these columns
            ok = span_wait(&bar->ring_full[sd], (g / C::kDoSlots) & 1, ctx, kSiteBwdDo) &&
                 (g == 0 || span_wait(&bar->dq_free, (g - 1) & 1, ctx, kSiteBwdDqFree));
            if (!ok) break;
            tc_fence_after();
            const uint64_t dodesc = sdesc_sw128(ring + sd * C::kTileBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              mma_bf16_ss(tDP, vdesc + off, dodesc + off, id_s, kk > 0 ? 1u : 0u);
            }
            mma_commit(&bar->dp_full);
          }
        }
        mma_commit(&bar->drain[0]);
        wait_drain_inl(&bar->drain[0], 0, kDrainLimitNs);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- issuer B: dV, dQ and dK
      if (lane == 0) {
        constexpr uint32_t id_v = idesc_bf16_f32(128, D, false, true);  // dV (A = P^T in TMEM), dK
        constexpr uint32_t id_q = idesc_bf16_f32(128, D, true, true);   // dQ (A = dS, M-major)
        const uint32_t ring = smem_u32(sRing);
        const uint64_t kdesc_mn = sdesc_sw128(smem_u32(sK), 16384, 1024);
        const uint64_t dsdesc_k = sdesc_sw128(smem_u32(sDS), 16, 1024);
        const uint64_t dsdesc_mn = sdesc_sw128(smem_u32(sDS), 16384, 1024);
        const uint32_t tS = tmem + C::kSCol, tDP = tmem + C::kDpCol;
        const uint32_t tDK = tmem + C::kDkCol, tDV = tmem + C::kDvCol;
        bool ok = true;
        int g = 0;
#pragma unroll 1
        for (int w = 0; ok && next_segment(w); ++w) {
          taken(w);
#pragma unroll 1
          for (int it = 0; ok && it < t.n; ++it, ++g) {
            const int sq = g % C::kQSlots, sd = C::kQSlots + g % C::kDoSlots;
            // dV += P^T dO_i as soon as the elementwise warps have written P^T
            // (P^T of query group kk sits at S^T column 16 kk) and dP^T, which
            // also reads dO_i, is complete (so dO_i has landed, and its slot can
            // be released after dV); this frees the S^T columns for the next
            // block's scores
            ok = span_wait(&bar->dp_full, g & 1, ctx, kSiteBwdEw) && span_wait(&bar->p_done, g & 1, ctx, kSiteBwdEw);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dodesc_mn = sdesc_sw128(ring + sd * C::kTileBytes, 16384, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts(tDV, tS + kk * 16, dodesc_mn + (uint32_t)((kk * 2048) >> 4), id_v,
                          (it > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&bar->dv_done);
            mma_commit(&bar->ring_empty[sd]);
            // dQ_i = dS K (into the dP^T columns, read by now; the next dP^T
            // waits for the reducers to take it out), then dK += dS^T Q_i, once
            // dS^T is written
            if (!(ok = span_wait(&bar->ew_done, g & 1, ctx, kSiteBwdEw))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss(tDP, dsdesc_mn + (uint32_t)((kk * 2048) >> 4), kdesc_mn + (uint32_t)((kk * 2048) >> 4), id_q,
                          kk > 0 ? 1u : 0u);
            mma_commit(&bar->dq_full);
            const uint64_t qdesc_mn = sdesc_sw128(ring + sq * C::kTileBytes, 16384, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              mma_bf16_ss(tDK, dsdesc_k + off, qdesc_mn + (uint32_t)((kk * 2048) >> 4), id_v,
                          (it > 0 || kk > 0) ? 1u : 0u);
            }
            // Q_i has been read by S^T (long complete) and dK: release its slot;
            // the dS^T tile is free for the next elementwise step (dQ, issued
            // before dK, has read it too)
            mma_commit(&bar->ring_empty[sq]);
            mma_commit(&bar->dk_done);
          }
          // the item's dK and dV are complete, and its K and V read for the last time
          if (ok) mma_commit(&bar->acc_done);
        }
        mma_commit(&bar->drain[1]);
        wait_drain_inl(&bar->drain[1], 0, kDrainLimitNs);
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ reducers
    if constexpr (R::kRed > R::kLaunch)
      setmaxnreg_inc<R::kRed>();
    else if constexpr (R::kRed < R::kLaunch)
      setmaxnreg_dec<R::kRed>();
    const int q = warp & 3;
    const uint32_t tDQ = tmem + C::kDpCol + ((uint32_t)(q * 32) << 16);
    uint8_t* stage = sStage + q * 8192;  // two 4 KB tiles
    constexpr int kChunks = D / 32;      // 32-column chunks of a dQ row
    bool alive = true;
    int g = 0, r = 0;                    // r: tiles handed to the TMA so far
#pragma unroll 1
    for (int w = 0; alive && __all_sync(0xffffffffu, next_segment(w)); ++w) {
      __syncwarp();
      if (lane == 0) taken(w);
      int head = t.head, i = t.i;
#pragma unroll 1
      for (int it = 0; it < t.n; ++it, ++g) {
        if (!__all_sync(0xffffffffu, span_wait(&bar->dq_full, g & 1, ctx, kSiteBwdDq))) {
          alive = false;
          break;
        }
        tc_fence_after();
        uint32_t dqv[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) tmem_ld32(tDQ + 32 * c, dqv[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kChunks; ++c) reg_fence32(dqv[c]);
        // dQ_i is in registers: issuer A may overwrite these columns with dP^T
        tc_fence_before();
        mbar_arrive(&bar->dq_free);
        // thread = query row 32 q + lane.  Each 32 x 32 block goes to a stage
        // tile in the TMA's 128-byte-swizzled layout (row = lane, 16-byte chunk
        // j at position j ^ (row & 7)), and one TMA reduce adds the tile to the
        // accumulator (rows past N are not written).  The two tiles alternate:
        // before a tile is refilled, the reduce issued from it two chunks ago
        // must have read it.
        const int qrow0 = i * 128 + 32 * q, bh = t.b * p.H + t.kvh * G + head;
        span_bwd_step(t, head, i);
        if (p.dq) {
          __nv_bfloat16* row = p.dq + ((size_t)bh * p.N + qrow0 + lane) * D;
          if (qrow0 + lane < p.N) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              uint32_t w16[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                w16[e] = pack_bf16x2(__uint_as_float(dqv[c][2 * e]) * p.scale, __uint_as_float(dqv[c][2 * e + 1]) * p.scale);
              if (p.out_align32) {
                st_global_v8(row + 32 * c, w16);
                st_global_v8(row + 32 * c + 16, w16 + 8);
              } else {
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4)
                  reinterpret_cast<uint4*>(row + 32 * c)[v4] =
                      make_uint4(w16[4 * v4], w16[4 * v4 + 1], w16[4 * v4 + 2], w16[4 * v4 + 3]);
              }
            }
          }
          __syncwarp();  // the next tensor memory load is a whole warp's
          continue;
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c, ++r) {
          uint8_t* tile = stage + (r & 1) * 4096;
          if (r >= 2) {
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
          }
#pragma unroll
          for (int c16 = 0; c16 < 8; ++c16)
            *reinterpret_cast<uint4*>(tile + lane * 128 + ((c16 ^ (lane & 7)) << 4)) =
                make_uint4(dqv[c][4 * c16], dqv[c][4 * c16 + 1], dqv[c][4 * c16 + 2], dqv[c][4 * c16 + 3]);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            // (a tile wholly past N, in the last block of a head, is not sent;
            // its group is empty)
            if (qrow0 < p.N) tma_reduce_add_3d(&map_dq, tile, 32 * c, qrow0, bh);
            tma_store_commit();
          }
        }
      }
    }
    // every reduce has completed (and read its tile) before the CTA ends
    if (lane == 0) tma_store_wait_all();
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ elementwise
    setmaxnreg_inc<R::kWork>();
    const int grp = warp >> 2;  // warpgroup: query columns [64 grp, 64 grp + 64)
    const int wq = warp & 3;
    const int r = wq * 32 + lane;  // key row
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + C::kSCol + lane_off;
    const uint32_t tDP = tmem + C::kDpCol + lane_off;
    uint8_t* ds_row = sDS + grp * 16384 + r * 128;
    bool alive = true;
    int g = 0;
#pragma unroll 1
    for (int w = 0; alive && __all_sync(0xffffffffu, next_segment(w)); ++w) {
      __syncwarp();
      if (lane == 0) taken(w);
      int head = t.head, i = t.i;
      const int key = t.jb * 128 + r;
#pragma unroll 1
      for (int it = 0; alive && it < t.n; ++it, ++g) {
        const float* stat = reinterpret_cast<const float*>(sStat + (g % C::kStatEntries) * C::kStatBytes);
        const int q0 = i * 128 + 64 * grp;
        [[maybe_unused]] float slope2 = 0.f;
        if constexpr (MOD & 1) slope2 = p.slopes[t.kvh * G + head] * 1.4426950408889634f;
        span_bwd_step(t, head, i);
        // the pairs that are seen, of this thread's key (a bit per query), while the scores are
        // formed (the cut flag is a plain store before the Q tile's arrival)
        if (!__all_sync(0xffffffffu, span_wait(&bar->ring_full[g % C::kQSlots], (g / C::kQSlots) & 1, ctx, kSiteBwdS))) {
          alive = false;
          break;
        }
        const bool cut = xbar->cut[g % C::kStatEntries];
        uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
        if (__builtin_expect(cut, 0)) {
          // a lane's query's bits of the warp's keys, transposed
          const long long at = (long long)t.b * p.nb * 128 + q0 + lane;
          const int key0 = key - lane;
#pragma unroll
          for (int ch = 0; ch < 2; ++ch)
            seen[ch] = span_transpose(span_bits(p.lo[at + 32 * ch] - key0, p.hi[at + 32 * ch] - key0), lane);
        }
        // ---- phase 1: P^T = 2^(S^T c - L log2e) into TMEM, the fp32 values kept
        // in registers; issuer B starts dV as soon as all of P^T is written
        if (!__all_sync(0xffffffffu, span_wait(&bar->s_full, g & 1, ctx, kSiteBwdS))) {
          alive = false;
          break;
        }
        tc_fence_after();
        if (__builtin_expect(cut, 0)) span_bwd_hide_s(tS + 64 * grp, seen);
        float2 pf[2][16];
        {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const int qc = 64 * grp + 32 * ch;  // first query column of this chunk
            uint32_t sv[32];
            tmem_ld32(tS + qc, sv);
            tmem_wait_ld();
            reg_fence32(sv);
            [[maybe_unused]] const float rel = (float)(q0 + 32 * ch - key);  // of the chunk's first query
            uint32_t pk[16];
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
              // four queries' -L*log2e (the same for every thread: a broadcast read)
              const float4 l4 = *reinterpret_cast<const float4*>(stat + qc + 4 * e4);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int e = 4 * e4 + 2 * h;  // two queries at a time (packed fp32x2 arithmetic)
                float2 nl = h ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
                const float2 s2 = make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                if constexpr (MOD & 1)
                  nl = make_float2(fmaf(-slope2, fabsf(rel + (float)e), nl.x), fmaf(-slope2, fabsf(rel + (float)(e + 1)), nl.y));
                float2 xs;
                [[maybe_unused]] float2 wt;
                if constexpr (MOD < 2) {
                  xs = __ffma2_rn(s2, make_float2(p.scale_log2, p.scale_log2), nl);
                } else {
                  // (the special-function unit is idle enough here: the forward's polynomial, with its
                  // test and its other path, takes as many instructions)
                  const float2 x = __fmul2_rn(s2, make_float2(p.cap.mul, p.cap.mul));
                  const float2 d = __fadd2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(1.f, 1.f));
                  const float2 tn = __ffma2_rn(make_float2(rcp_approx(d.x), rcp_approx(d.y)), make_float2(-2.f, -2.f),
                                               make_float2(1.f, 1.f));  // the tanh
                  xs = __ffma2_rn(tn, make_float2(p.cap.top, p.cap.top), nl);
                  wt = __ffma2_rn(make_float2(-tn.x, -tn.y), tn, make_float2(1.f, 1.f));
                }
                float2 pe = make_float2(ex2_approx(xs.x), ex2_approx(xs.y));
                pk[2 * e4 + h] = pack_bf16x2(pe.x, pe.y);
                if constexpr (MOD >= 2) pe = __fmul2_rn(pe, wt);
                pf[ch][e / 2] = pe;
              }
            }
            // P^T of query groups qc/16 and qc/16 + 1 over the first 8 of their own columns
            tmem_st8(tS + qc, pk);
            tmem_st8(tS + qc + 16, pk + 8);
          }
        }
        if (MOD >= 2 && __builtin_expect(cut, 0)) {
          span_bwd_hide_p(tS + 64 * grp, seen);
          // (Without a bias 2^(-cap - LSE) is at most 1, and times 1 - tanh^2 = 0.  With one a hidden key may be
          // so much nearer than those that the row sees (farther, if the slope is negative) that it is infinite.)
          if constexpr (MOD == 3) {
#pragma unroll
            for (int ch = 0; ch < 2; ++ch)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                if (!((seen[ch] >> (2 * e)) & 1u)) pf[ch][e].x = 0.f;
                if (!((seen[ch] >> (2 * e + 1)) & 1u)) pf[ch][e].y = 0.f;
              }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar->p_done);

        // ---- phase 2: dS^T = P^T o (dP^T - delta) into the shared dS^T tile,
        // once the previous block's dK and dQ have read it (dP^T of this block
        // was issued after the reducers took the previous dQ out of TMEM; dK,
        // which runs after dQ, reports on its own)
        bool ok2 = span_wait(&bar->dp_full, g & 1, ctx, kSiteBwdDp);
        if (g > 0) ok2 = ok2 && span_wait(&bar->dk_done, (g - 1) & 1, ctx, kSiteBwdDp);
        if (!__all_sync(0xffffffffu, ok2)) {
          alive = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          const int qc = 64 * grp + 32 * ch;
          uint32_t dp[32];
          tmem_ld32(tDP + qc, dp);
          tmem_wait_ld();
          reg_fence32(dp);
          uint32_t dk[16];
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 d4 = *reinterpret_cast<const float4*>(stat + 128 + qc + 4 * e4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = 4 * e4 + 2 * h;
              const float2 nd = h ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y);
              const float2 dpd = __fadd2_rn(make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), nd);
              const float2 dse = __fmul2_rn(pf[ch][e / 2], dpd);
              dk[2 * e4 + h] = pack_bf16x2(dse.x, dse.y);
            }
          }
          // dS^T row r, queries [qc, qc+32): 4 chunks of 16 B in the swizzled atom grp
#pragma unroll
          for (int c16 = 0; c16 < 4; ++c16) {
            const int chunk = ((qc & 63) >> 3) + c16;
            *reinterpret_cast<uint4*>(ds_row + ((chunk ^ (r & 7)) << 4)) =
                make_uint4(dk[4 * c16], dk[4 * c16 + 1], dk[4 * c16 + 2], dk[4 * c16 + 3]);
          }
        }
        fence_async_shared();
        tc_fence_before();
        mbar_arrive(&bar->ew_done);
      }
      // ---- epilogue: warpgroup 0 writes dK = scale dK_acc, warpgroup 1 writes
      // dV.  The next item's first dV and dK overwrite these columns only
      // after this warpgroup's next p_done arrival, which follows these reads.
      if (!alive || !__all_sync(0xffffffffu, span_wait(&bar->acc_done, w & 1, ctx, kSiteBwdAcc))) {
        alive = false;
        break;
      }
      {
        tc_fence_after();
        const uint32_t tAcc = tmem + (grp ? C::kDvCol : C::kDkCol) + lane_off;
        const float mul = grp ? 1.f : p.scale;  // dK = scale dS^T Q
        const int kg = t.jb * 128 + r;
        __nv_bfloat16* out = (grp ? p.dv : p.dk) + ((size_t)(t.b * p.Hkv + t.kvh) * p.N + kg) * D;
        float* sums = p.sums + (((size_t)(t.slot < 0 ? 0 : t.slot) * 2 + grp) * 128 + r) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(tAcc + 32 * c, v);
          tmem_wait_ld();
          reg_fence32(v);
          if (t.slot >= 0) {
#pragma unroll
            for (int v8 = 0; v8 < 4; ++v8) st_global_v8(sums + 32 * c + 8 * v8, v + 8 * v8);
          } else if (kg < p.N) {
            uint32_t w16[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w16[e] = pack_bf16x2(__uint_as_float(v[2 * e]) * mul, __uint_as_float(v[2 * e + 1]) * mul);
            if (p.out_align32) {
              // whole 32-byte sectors (a thread's row is contiguous)
              st_global_v8(out + 32 * c, w16);
              st_global_v8(out + 32 * c + 16, w16 + 8);
            } else {
              uint4* o4 = reinterpret_cast<uint4*>(out + 32 * c);
#pragma unroll
              for (int v4 = 0; v4 < 4; ++v4)
                o4[v4] = make_uint4(w16[4 * v4], w16[4 * v4 + 1], w16[4 * v4 + 2], w16[4 * v4 + 3]);
            }
          }
          __syncwarp();  // the next tensor memory load is a whole warp's
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// After the main kernel: the first 4 kSpanBwdSlots blocks write a quarter (32 rows) of dK or
// dV of a cut item, the sum of its runs in order; the others write dQ = scale *
// accumulator in bf16 (none where the main kernel wrote dQ).
template <int D>
__global__ void __launch_bounds__(256)
    fa_span_bwd_post_kernel(const __grid_constant__ SpanBwdParams p, const float* dq_acc, __nv_bfloat16* dq, long long n8) {
  grid_wait();
  constexpr int cut_blocks = 4 * kSpanBwdSlots;
  int x = blockIdx.x;
  if (x < cut_blocks) {
    const int item = x >> 3, grp = (x >> 2) & 1, quarter = x & 3;
    if (item >= p.plan->cut * p.Hkv) return;
    const int4 cut = p.cuts[item / p.Hkv];
    const int kvh = item % p.Hkv;
    const float mul = grp ? 1.f : p.scale;
    __nv_bfloat16* out = (grp ? p.dv : p.dk) + ((size_t)(cut.x * p.Hkv + kvh) * p.N + cut.y * 128) * D;
    for (int i = threadIdx.x; i < 32 * D / 4; i += 256) {
      const int row = quarter * 32 + i / (D / 4), col = i % (D / 4);
      if (cut.y * 128 + row >= p.N) break;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int part = 0; part < cut.w; ++part) {
        const size_t slot = cut.z + (size_t)part * p.Hkv + kvh;
        const float4 a = reinterpret_cast<const float4*>(p.sums + ((slot * 2 + grp) * 128 + row) * D)[col];
        sum.x += a.x;
        sum.y += a.y;
        sum.z += a.z;
        sum.w += a.w;
      }
      reinterpret_cast<uint2*>(out + (size_t)row * D)[col] =
          make_uint2(pack_bf16x2(sum.x * mul, sum.y * mul), pack_bf16x2(sum.z * mul, sum.w * mul));
    }
    return;
  }
  x -= cut_blocks;
  for (long long i = (long long)x * 256 + threadIdx.x; i < n8; i += (long long)(gridDim.x - cut_blocks) * 256) {
    const float4 a = reinterpret_cast<const float4*>(dq_acc)[2 * i];
    const float4 b = reinterpret_cast<const float4*>(dq_acc)[2 * i + 1];
    reinterpret_cast<uint4*>(dq)[i] =
        make_uint4(pack_bf16x2(a.x * p.scale, a.y * p.scale), pack_bf16x2(a.z * p.scale, a.w * p.scale),
                   pack_bf16x2(b.x * p.scale, b.y * p.scale), pack_bf16x2(b.z * p.scale, b.w * p.scale));
  }
}

}  // namespace fa
