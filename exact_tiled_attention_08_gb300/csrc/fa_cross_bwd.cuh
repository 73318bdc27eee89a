// Backward of cross attention (fa_cross_bwd).
//
// The per-block arithmetic, roles and barriers are those of fa_bwd_kernel with
// the atomic dQ: a CTA keeps K_j and V_j (128 keys) and streams the query
// blocks past them; dQ goes to an fp32 accumulator by TMA reduces.  The rows of
// the query heads that share a key/value head are one run of R rows, so dK and
// dV are summed over the group in tensor memory.  What differs:
//
// Work.  Items (key block j of a request and key/value head, blocks behind the
// request's keys left out) all cost n = ceil(R / 128) query blocks.  CTA c takes
// the items c, c + G, ... of the full rounds whole: the CTAs of a round sweep
// the same heads' query blocks together, so that Q, dO and the dQ accumulator
// are read from L2.  (Equal contiguous shares of all query blocks, as the
// forward cuts its keys, put the CTAs out of step: every tile would come from
// DRAM.)  The r = items mod G that remain are each cut into `parts` runs of
// query blocks, handed out run by run; a run leaves its sums of dK and dV in
// the workspace, and fa_cross_bwd_post_kernel adds an item's runs in order.
//
// Keys behind the request's length, in its last key block: P and dS are zero,
// and their rows of K (which may hold anything, and meet dS in dQ = dS K) are
// zeroed in shared memory by the reducer warps before the first product.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "fa_fwd.cuh"  // (fa_bwd.cuh uses its limits)
#include "fa_bwd.cuh"
#include "fa_cross.cuh"

namespace fa {

// How the items are handed out; written to the workspace for the post kernel.
struct CrossBwdPlan {
  int rounds;  // full rounds: rounds * G items, each whole
  int rest;    // items of the last round
  int parts;   // runs each of them is cut into (1: whole)
};

constexpr int kCrossBwdMaxCtas = 152;
constexpr int kCrossBwdTurns = 4;                                 // of runs that a CTA may take
constexpr int kCrossBwdSlots = kCrossBwdTurns * kCrossBwdMaxCtas;  // runs of cut items: rest * parts at most

struct CrossBwdParams {
  CrossView view;
  __nv_bfloat16 *dk, *dv;
  CrossBwdPlan* plan;
  float* runs;       // [run][dK, dV][128][d], fp32, unscaled
  int B;
  int nqb;           // query blocks per item
  float scale_log2;  // scale * log2(e)
  float scale;
  uint64_t wait_limit_ns;
  int debug_stall;
  int out_align32;   // dk, dv (and dq, where it is written directly) are 32-byte aligned
  // With at most one key block per request each query block meets one item:
  // its dQ is written here (scaled, bf16) instead of being added to the
  // accumulator.  nullptr: more key blocks.
  __nv_bfloat16* dq;
};

// A CTA's unit of work: query blocks [i0, i1) of a key block.
struct CrossBwdSeg {
  int bk;     // request and key/value head
  int jb;     // key block
  int valid;  // keys of the block (128 but in a request's last block)
  int i0, i1;
  int run;    // where its sums go, or -1: the item is whole
};

// key blocks of a request with `len` keys (direct dQ: one even without keys, so
// that its rows are written)
__device__ __forceinline__ int cross_bwd_blocks(int len, bool direct) { return direct ? 1 : (len + 127) >> 7; }

// item -> request, key/value head and key block; the items are walked upwards
// from the request that the last call stopped at
struct CrossBwdWalk {
  int k = 0;            // the CTA's next unit
  int b = 0, start = 0;  // a request and its first item
};

__device__ __forceinline__ void cross_bwd_item(const CrossView& v, bool direct, int item, CrossBwdWalk& at,
                                               CrossBwdSeg& s) {
  int nkb = (v.Nk + 127) >> 7, len = v.Nk;
  if (!v.lens) {
    at.b = item / (v.Hkv * nkb);
    at.start = at.b * v.Hkv * nkb;
  } else {
    if (item < at.start) at.b = at.start = 0;
    for (;;) {
      len = v.len(at.b);
      nkb = cross_bwd_blocks(len, direct);
      if (item < at.start + v.Hkv * nkb) break;
      at.start += v.Hkv * nkb;
      ++at.b;
    }
  }
  const int kvh = (item - at.start) / nkb;
  s.jb = item - at.start - kvh * nkb;
  s.bk = at.b * v.Hkv + kvh;
  s.valid = min(128, len - s.jb * 128);
}

// The first query block of run `part`: floor(part nqb / parts), in 32 bits (a long
// item's 2^24 blocks times its hundreds of runs do not fit them).
__host__ __device__ __forceinline__ int cross_bwd_cut(int part, int parts, int nqb) {
  const int each = nqb / parts;
  return part * each + part * (nqb - parts * each) / parts;
}

__device__ __forceinline__ bool cross_bwd_next(const CrossBwdParams& p, const CrossBwdPlan& plan, CrossBwdWalk& at,
                                               CrossBwdSeg& s) {
  const int k = at.k++, G = gridDim.x, c = blockIdx.x;
  int item;
  if (k < plan.rounds) {
    item = k * G + c;
    s.i0 = 0;
    s.i1 = p.nqb;
    s.run = -1;
  } else {
    const int u = (k - plan.rounds) * G + c;
    if (u >= plan.rest * plan.parts) return false;
    const int part = u / plan.rest;
    item = plan.rounds * G + (u - part * plan.rest);
    s.i0 = cross_bwd_cut(part, plan.parts, p.nqb);
    s.i1 = cross_bwd_cut(part + 1, plan.parts, p.nqb);
    s.run = plan.parts > 1 ? u : -1;
  }
  cross_bwd_item(p.view, p.dq != nullptr, item, at, s);
  return true;
}

// Rounds, and the number of runs that ends the last one soonest: parts runs of
// an item take ceil(rest parts / G) turns of ceil(n / parts) query blocks each
// and about two blocks' time to start and write.  (Measured, at most 16 runs and as
// many as there are CTAs: B=4 H=5/1 Nq=7058 Nk=69 d=64, four items of 276 query
// blocks, 67 and 57 us.)
__host__ __device__ inline CrossBwdPlan cross_bwd_split(int items, int nqb, int G) {
  CrossBwdPlan plan{items / G, items % G, 1};
  if (plan.rest == 0) return plan;
  int best = nqb + 2;  // whole: one turn
  for (int turns = 1; turns <= kCrossBwdTurns; ++turns) {
    // as many runs as `turns` turns of all CTAs take
    int parts = turns * G / plan.rest;
    if (parts > nqb) parts = nqb;
    const int cost = turns * ((nqb + parts - 1) / parts + 2);
    if (cost < best) {
      best = cost;
      plan.parts = parts;
    }
  }
  return plan;
}

template <int kThreads>
__device__ __forceinline__ void cross_bwd_plan(const CrossBwdParams& p, int* scratch, CrossBwdPlan* out) {
  const CrossView& v = p.view;
  int items = 0;
  if (!v.lens) {
    items = threadIdx.x == 0 ? p.B * ((v.Nk + 127) >> 7) : 0;
  } else {
    for (int b = threadIdx.x; b < p.B; b += kThreads) items += cross_bwd_blocks(v.len(b), p.dq != nullptr);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = items;
  __syncthreads();
  if (threadIdx.x == 0) {
    items = 0;
    for (int w = 0; w < kThreads / 32; ++w) items += scratch[w];
    items *= v.Hkv;
    const int G = gridDim.x;
    const CrossBwdPlan plan = cross_bwd_split(items, p.nqb, G);
    *out = plan;
    if (blockIdx.x == 0) *p.plan = plan;
  }
}

struct CrossBwdBarriers {
  BwdBarriers b;
  uint64_t k_clean;  // the rows of K behind the keys are zero (128 reducer threads)
  CrossBwdPlan plan;
};
static_assert(sizeof(CrossBwdBarriers) <= 512, "barriers overflow their shared-memory slot");

template <int D>
constexpr int kCrossBwdSmemBytes = BwdCfg<D, true>::kSmemBytes + 256;  // 512 bytes of barriers
static_assert(kCrossBwdSmemBytes<128> <= 227 * 1024, "shared memory budget");

enum : int { kSiteCrossBwdClean = 60 };

// Per row of each (request, key/value head), padded to whole 128-row blocks:
// delta = sum dO O (0 behind the rows) and LSE log2(e) (+inf behind them, and
// for rows without keys, so that P = 0 there); the dQ accumulator, if there is
// one, is zeroed.
template <int D>
__global__ void __launch_bounds__(256)
    fa_cross_bwd_prep_kernel(const __nv_bfloat16* o, const __nv_bfloat16* dout, const float* lse, float* delta_pad,
                             float* lse2_pad, float* dq_acc, int R, int Rpad, long long padded_rows) {
  constexpr int kThreadsPerRow = D / 8, kRows = 256 / kThreadsPerRow;
  const int sub = threadIdx.x % kThreadsPerRow;
  grid_wait();
  grid_trigger();
  for (long long prow = (long long)blockIdx.x * kRows + threadIdx.x / kThreadsPerRow;
       prow - threadIdx.x / kThreadsPerRow < padded_rows; prow += (long long)gridDim.x * kRows) {
    const long long bk = prow / Rpad;
    const int n = (int)(prow - bk * Rpad);
    const bool in_range = prow < padded_rows, valid = in_range && n < R;
    const long long row = bk * R + n;
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
      delta_pad[prow] = valid ? s : 0.f;
      lse2_pad[prow] = l == -CUDART_INF_F ? CUDART_INF_F : l * 1.4426950408889634f;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(512, 1)
    fa_cross_bwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                  const __grid_constant__ CUtensorMap map_lse2, const __grid_constant__ CUtensorMap map_delta,
                  const __grid_constant__ CUtensorMap map_dq, const CrossBwdParams p) {
  using C = BwdCfg<D, true>;
  using R = BwdRegs<D, true>;
  static_assert(R::kLaunch == C::kLaunchRegs, "register split of the launch budget");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    // the 128-byte-swizzled tiles need 1024-byte alignment: report, do nothing
    grid_wait();
    if (threadIdx.x == 0) {
      atomicCAS(&g_fa_device_status, 0u, kStatusBadSmem);
      if (blockIdx.x == 0) *p.plan = CrossBwdPlan{0, 0, 1};  // no runs for the post kernel to add
    }
    return;
  }
  uint8_t* smem = smem_raw;
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTileBytes;
  uint8_t* sRing = smem + 2 * C::kTileBytes;
  uint8_t* sDS = sRing + C::kSlots * C::kTileBytes;
  uint8_t* sStage = sDS + C::kDsBytes;
  // query block g: entry g % kStatEntries = LSE*log2e [128], delta [128]
  uint8_t* sStat = sStage + C::kStageBytes;
  CrossBwdBarriers* xbar = reinterpret_cast<CrossBwdBarriers*>(sStat + C::kStatEntries * C::kStatBytes);
  BwdBarriers* bar = &xbar->b;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

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
    mbar_init(&xbar->k_clean, 128);
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
  grid_wait();
  cross_bwd_plan<C::kThreads>(p, reinterpret_cast<int*>(sRing), &xbar->plan);
  fence_async_shared();  // the ring's first copies follow the plan's plain writes
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtx ctx{&bar->abort_flag, p.wait_limit_ns};
  grid_trigger();
  const CrossBwdPlan plan = xbar->plan;
  CrossBwdWalk at;  // every role walks the same segments
  CrossBwdSeg t;
  if (warp >= 12) {
    setmaxnreg_dec<R::kMisc>();
    if (warp == 13 || warp == 15) {
      // ---------------------------------------------------------------- TMA producers
      // warp 13: K and V of each item and the Q tiles (with the statistics),
      // warp 15: the dO tiles, so that neither queue waits on the other's
      // slot.  g counts query blocks over all of the CTA's items.
      if (lane == 0) {
        const bool q_side = warp == 13;
        const int nslot = q_side ? C::kQSlots : C::kDoSlots, slot0 = q_side ? 0 : C::kQSlots;
        int g = 0, w = 0, kv_loads = 0;
        bool ok = true;
        for (; ok && cross_bwd_next(p, plan, at, t); ++w) {
          if (q_side) {
            // K and V of the item, once the previous item's last products
            // (acc_done) have read the old ones
            if (w > 0 && !wait_bounded_inl(&bar->acc_done, (w - 1) & 1, ctx, kSiteBwdProducer)) break;
            mbar_arrive_expect_tx(&bar->kv_full, 2 * C::kTileBytes);
            for (int a = 0; a < C::kAtoms; ++a) {
              tma_load_3d(sK + a * 16384, &map_k, &bar->kv_full, a * 64, t.jb * 128, t.bk);
              tma_load_3d(sV + a * 16384, &map_v, &bar->kv_full, a * 64, t.jb * 128, t.bk);
            }
            ++kv_loads;
          }
          for (int it = 0; it < t.i1 - t.i0; ++it, ++g) {
            const int i = t.i0 + it;
            const int s = slot0 + g % nslot;
            if (!wait_bounded_inl(&bar->ring_empty[s], ((g / nslot) & 1) ^ 1, ctx, kSiteBwdProducer)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bar->ring_full[s], C::kTileBytes + (q_side ? C::kStatBytes : 0));
            const CUtensorMap* map = q_side ? &map_q : &map_do;
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_3d(sRing + s * C::kTileBytes + a * 16384, map, &bar->ring_full[s], a * 64, i * 128, t.bk);
            if (q_side) {
              uint8_t* st = sStat + (g % C::kStatEntries) * C::kStatBytes;
              tma_load_2d(st, &map_lse2, &bar->ring_full[s], i * 128, t.bk);
              tma_load_2d(st + 512, &map_delta, &bar->ring_full[s], i * 128, t.bk);
            }
          }
        }
        // every load this warp started has landed before the CTA may end
        if (kv_loads > 0) wait_drain_inl(&bar->kv_full, (kv_loads - 1) & 1, kDrainLimitNs);
        for (int k = 0; k < nslot; ++k) {
          if (g > k) {
            const int uses = (g - 1 - k) / nslot + 1;
            wait_drain_inl(&bar->ring_full[slot0 + k], (uses - 1) & 1, kDrainLimitNs);
          }
        }
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
        bool ok = !(p.debug_stall && !wait_bounded_inl(&bar->never, 0, ctx, kSiteStall));
        // S^T goes first: the first half of the elementwise step needs only
        // S^T, its columns are free as soon as dV of the previous block has
        // run, and dP^T waits for the reducers to take the previous dQ out of
        // its columns.
        // g counts query blocks over all of the CTA's items, w the items.
        int g = 0, w = 0, cleaned = 0;
        for (; ok && cross_bwd_next(p, plan, at, t); ++w) {
          ok = wait_bounded_inl(&bar->kv_full, w & 1, ctx, kSiteBwdKV);
          if (ok && t.valid < 128 && t.jb * 128 + t.valid < p.view.Nk) {
            ok = wait_bounded_inl(&xbar->k_clean, cleaned & 1, ctx, kSiteCrossBwdClean);
            ++cleaned;
          }
          for (int it = 0; ok && it < t.i1 - t.i0; ++it, ++g) {
#pragma unroll
            for (int step = 0; step < 2; ++step) {
              if (step == 0) {
                // S^T = K Q_i^T, once dV has consumed the previous P^T held in
                // these columns
                const int sq = g % C::kQSlots;
                if (!wait_bounded_inl(&bar->ring_full[sq], (g / C::kQSlots) & 1, ctx, kSiteBwdQ)) {
                  ok = false;
                  break;
                }
                if (g > 0 && !wait_bounded_inl(&bar->dv_done, (g - 1) & 1, ctx, kSiteBwdDvDone)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                const uint64_t qdesc = sdesc_sw128(ring + sq * C::kTileBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                  mma_bf16_ss(tS, kdesc + off, qdesc + off, id_s, kk > 0 ? 1u : 0u);
                }
                mma_commit(&bar->s_full);
              } else {
                // dP^T = V dO_i^T, once the reducers have taken the previous dQ
                // out of these columns
                const int sd = C::kQSlots + g % C::kDoSlots;
                if (!wait_bounded_inl(&bar->ring_full[sd], (g / C::kDoSlots) & 1, ctx, kSiteBwdDo)) {
                  ok = false;
                  break;
                }
                if (g > 0 && !wait_bounded_inl(&bar->dq_free, (g - 1) & 1, ctx, kSiteBwdDqFree)) {
                  ok = false;
                  break;
                }
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
          }
        }
        mma_commit(&bar->drain[0]);
        wait_drain_inl(&bar->drain[0], 0, kDrainLimitNs);
      }
      __syncwarp();
    } else if (warp == 14) {
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
        while (ok && cross_bwd_next(p, plan, at, t)) {
          for (int it = 0; ok && it < t.i1 - t.i0; ++it, ++g) {
            const int sq = g % C::kQSlots, sd = C::kQSlots + g % C::kDoSlots;
            // dV += P^T dO_i as soon as the elementwise warps have written P^T
            // (P^T of query group kk sits at S^T column 16 kk) and dP^T, which
            // also reads dO_i, is complete (so dO_i has landed, and its slot can
            // be released after dV); this frees the S^T columns for the next
            // block's scores
            ok = wait_bounded_inl(&bar->dp_full, g & 1, ctx, kSiteBwdEw) &&
                 wait_bounded_inl(&bar->p_done, g & 1, ctx, kSiteBwdEw);
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
            if (!(ok = wait_bounded_inl(&bar->ew_done, g & 1, ctx, kSiteBwdEw))) break;
            tc_fence_after();
            // (fully unrolled: the MMAs are issued back to back; in a loop, a
            // 32-cycle MMA at d = 64 outruns its issue.  The issuing warps get
            // 88 registers for the unrolled descriptors.)
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
    int g = 0, w = 0, r = 0;             // r: tiles handed to the TMA so far
    for (; alive && cross_bwd_next(p, plan, at, t); ++w) {
      if (t.valid < 128 && t.jb * 128 + t.valid < p.view.Nk) {
        // rows of K behind the keys (past Nk the TMA has filled zeros)
        if (!__all_sync(0xffffffffu, wait_bounded_inl(&bar->kv_full, w & 1, ctx, kSiteCrossBwdClean))) {
          alive = false;
          break;
        }
        for (int a = 0; a < C::kAtoms; ++a)
          for (int c = t.valid * 8 + q * 32 + lane; c < 128 * 8; c += 128)
            *reinterpret_cast<uint4*>(sK + a * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
        fence_async_shared();
        mbar_arrive(&xbar->k_clean);
      }
      for (int it = 0; it < t.i1 - t.i0; ++it, ++g) {
        if (!__all_sync(0xffffffffu, wait_bounded_inl(&bar->dq_full, g & 1, ctx, kSiteBwdDq))) {
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
        // accumulator (rows past R are not written).  The two tiles alternate:
        // before a tile is refilled, the reduce issued from it two chunks ago
        // must have read it.
        const int qrow0 = (t.i0 + it) * 128 + 32 * q;
        if (p.dq) {
          __nv_bfloat16* row = p.dq + ((size_t)t.bk * p.view.R + qrow0 + lane) * D;
          if (qrow0 + lane < p.view.R) {
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
            // (a tile wholly past R, in the last block of a head, is not sent;
            // its group is empty)
            if (qrow0 < p.view.R) tma_reduce_add_3d(&map_dq, tile, 32 * c, qrow0, t.bk);
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
    const float sl2 = p.scale_log2;
    uint8_t* ds_row = sDS + grp * 16384 + r * 128;
    bool alive = true;
    int g = 0, w = 0;
    for (; alive && cross_bwd_next(p, plan, at, t); ++w) {
      for (int it = 0; alive && it < t.i1 - t.i0; ++it, ++g) {
        const float* stat = reinterpret_cast<const float*>(sStat + (g % C::kStatEntries) * C::kStatBytes);
        // ---- phase 1: P^T = 2^(S^T c - L log2e) into TMEM, the fp32 values kept
        // in registers; issuer B starts dV as soon as all of P^T is written
        if (!__all_sync(0xffffffffu, wait_bounded_inl(&bar->s_full, g & 1, ctx, kSiteBwdS))) {
          alive = false;
          break;
        }
        tc_fence_after();
        const bool cut = t.valid < 128, dead = r >= t.valid;  // this thread's key is behind the request's
        const float2 c2 = make_float2(sl2, sl2);
        float2 pf[2][16];
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          const int qc = 64 * grp + 32 * ch;  // first query column of this chunk
          uint32_t sv[32];
          tmem_ld32(tS + qc, sv);
          tmem_wait_ld();
          reg_fence32(sv);
          uint32_t pk[16];
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            // four queries' L*log2e (the same for every thread: a broadcast read)
            const float4 l4 = *reinterpret_cast<const float4*>(stat + qc + 4 * e4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = 4 * e4 + 2 * h;  // two queries at a time (packed fp32x2 arithmetic)
              const float2 nl = h ? make_float2(-l4.z, -l4.w) : make_float2(-l4.x, -l4.y);
              const float2 xs = __ffma2_rn(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, nl);
              float2 pe = make_float2(ex2_approx(xs.x), ex2_approx(xs.y));
              if (cut && dead) pe = make_float2(0.f, 0.f);
              pf[ch][e / 2] = pe;
              pk[2 * e4 + h] = pack_bf16x2(pe.x, pe.y);
            }
          }
          // P^T of query groups qc/16 and qc/16 + 1 over the first 8 of their own columns
          tmem_st8(tS + qc, pk);
          tmem_st8(tS + qc + 16, pk + 8);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar->p_done);

        // ---- phase 2: dS^T = P^T o (dP^T - delta) into the shared dS^T tile,
        // once the previous block's dK and dQ have read it (dP^T of this block
        // was issued after the reducers took the previous dQ out of TMEM; dK,
        // which runs after dQ, reports on its own)
        bool ok2 = wait_bounded_inl(&bar->dp_full, g & 1, ctx, kSiteBwdDp);
        if (g > 0) ok2 = ok2 && wait_bounded_inl(&bar->dk_done, (g - 1) & 1, ctx, kSiteBwdDp);
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
              const float2 nd = h ? make_float2(-d4.z, -d4.w) : make_float2(-d4.x, -d4.y);
              const float2 dpd = __fadd2_rn(make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), nd);
              const float2 dse = __fmul2_rn(pf[ch][e / 2], dpd);
              dk[2 * e4 + h] = cut && dead ? 0u : pack_bf16x2(dse.x, dse.y);
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
      if (!alive || !__all_sync(0xffffffffu, wait_bounded_inl(&bar->acc_done, w & 1, ctx, kSiteBwdAcc))) {
        alive = false;
        break;
      }
      {
        tc_fence_after();
        const uint32_t tAcc = tmem + (grp ? C::kDvCol : C::kDkCol) + lane_off;
        const float mul = grp ? 1.f : p.scale;  // dK = scale dS^T Q
        const int kg = t.jb * 128 + r;
        __nv_bfloat16* out = (grp ? p.dv : p.dk) + ((size_t)t.bk * p.view.Nk + kg) * D;
        float* run = p.runs + (((size_t)(t.run < 0 ? 0 : t.run) * 2 + grp) * 128 + r) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(tAcc + 32 * c, v);
          tmem_wait_ld();
          reg_fence32(v);
          if (t.run >= 0) {
#pragma unroll
            for (int v8 = 0; v8 < 4; ++v8) st_global_v8(run + 32 * c + 8 * v8, v + 8 * v8);
          } else if (kg < p.view.Nk) {
            uint32_t w16[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w16[e] = r >= t.valid ? 0u
                                    : pack_bf16x2(__uint_as_float(v[2 * e]) * mul, __uint_as_float(v[2 * e + 1]) * mul);
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
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// After the main kernel: block x of the first 8 G writes a quarter (32 rows) of
// dK or dV of a cut item, the sum of its runs in order; the next B Hkv blocks
// zero dK and dV in the key blocks behind a request's keys; the others write
// dQ = scale * accumulator in bf16 (none where the main kernel wrote dQ).
struct CrossBwdPostParams {
  CrossBwdParams p;
  const float* dq_acc;
  __nv_bfloat16* dq;
  long long n8;  // eighths of dQ's values
  int ctas;      // of the main kernel
};

template <int D>
__global__ void __launch_bounds__(256) fa_cross_bwd_post_kernel(const CrossBwdPostParams q) {
  const CrossBwdParams& p = q.p;
  const CrossView& v = p.view;
  grid_wait();  // (no grid_trigger: a next call's first blocks would take the place of this one's)
  const int cut_blocks = 8 * q.ctas, zero_blocks = v.lens && !p.dq ? p.B * v.Hkv : 0;
  int x = blockIdx.x;
  if (x < cut_blocks) {
    const CrossBwdPlan plan = *p.plan;
    const int rest = x >> 3, grp = (x >> 2) & 1, quarter = x & 3;
    if (plan.parts == 1 || rest >= plan.rest) return;
    CrossBwdWalk at;
    CrossBwdSeg s;
    cross_bwd_item(v, p.dq != nullptr, plan.rounds * q.ctas + rest, at, s);
    const float mul = grp ? 1.f : p.scale;
    __nv_bfloat16* out = (grp ? p.dv : p.dk) + ((size_t)s.bk * v.Nk + s.jb * 128) * D;
    for (int i = threadIdx.x; i < 32 * D / 4; i += 256) {
      const int row = quarter * 32 + i / (D / 4), col = i % (D / 4);
      if (s.jb * 128 + row >= v.Nk) break;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < s.valid) {
#pragma unroll 4
        for (int part = 0; part < plan.parts; ++part) {
          const size_t run = (size_t)part * plan.rest + rest;
          const float4 a = reinterpret_cast<const float4*>(p.runs + ((run * 2 + grp) * 128 + row) * D)[col];
          sum.x += a.x;
          sum.y += a.y;
          sum.z += a.z;
          sum.w += a.w;
        }
      }
      reinterpret_cast<uint2*>(out + (size_t)row * D)[col] =
          make_uint2(pack_bf16x2(sum.x * mul, sum.y * mul), pack_bf16x2(sum.z * mul, sum.w * mul));
    }
    return;
  }
  x -= cut_blocks;
  if (x < zero_blocks) {
    const int first = ((v.len(x / v.Hkv) + 127) >> 7) * 128;
    if (first >= v.Nk) return;
    const size_t at = ((size_t)x * v.Nk + first) * D / 8, n = (size_t)(v.Nk - first) * D / 8;
    for (size_t i = threadIdx.x; i < n; i += 256) {
      reinterpret_cast<uint4*>(p.dk)[at + i] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(p.dv)[at + i] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  x -= zero_blocks;
  for (long long i = (long long)x * 256 + threadIdx.x; i < q.n8;
       i += (long long)(gridDim.x - cut_blocks - zero_blocks) * 256) {
    const float4 a = reinterpret_cast<const float4*>(q.dq_acc)[2 * i];
    const float4 b = reinterpret_cast<const float4*>(q.dq_acc)[2 * i + 1];
    reinterpret_cast<uint4*>(q.dq)[i] =
        make_uint4(pack_bf16x2(a.x * p.scale, a.y * p.scale), pack_bf16x2(a.z * p.scale, a.w * p.scale),
                   pack_bf16x2(b.x * p.scale, b.y * p.scale), pack_bf16x2(b.z * p.scale, b.w * p.scale));
  }
}

}  // namespace fa
