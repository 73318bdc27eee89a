// Forward of attention to spans of keys in pages, for units of at most 16 rows: a token, or
// a few, of the query heads that share a key/value head.
//
// What fa_span_fwd_kernel does for 128 rows would be empty rows here, and its
// exponentials (128 keys of 128 rows a block) take longer than the block's 64 KB of keys
// and values need from memory.  So the products are turned around: S^T = K Q^T has
// the keys on the tensor memory's lanes and 16 columns of rows, a thread holds one
// key's 16 scores, and O^T += V^T P^T has the d channels on the lanes.  P goes to
// shared memory as [row][key], where it is the B operand.
//
// The maximum of a row is over lanes now.  The four warps keep one reference per row in
// shared memory and move it only when a score rises above it by more than the
// threshold (one vote a block; exact maxima over the block then): P stays below 2^8, and O and
// the sums are scaled to the new reference.  Sums are kept per thread and added up at the end of
// a segment.
//
// Items, shares, parts, masks and pages are those of fa_span_fwd_kernel.  A few items
// (CLUSTER): 2, 4 or 8 CTAs of a cluster share an item's key blocks and join their parts
// through one another's shared memory, without the second kernel.
//
// What bounds it is memory, as far as there are blocks enough: the ring holds three K and
// three V tiles at d = 128.  Measured on a GB300: 16 requests of 300 to 8100 tokens, H=32/8 d=128, a token
// each, 60 us (4.5 TB/s with start and join), capped or not, pages of 16 or 64; fa_span_fwd_kernel
// takes 66 us with pages of 64, capped 82.  (With 32 columns it was slower than that kernel: 76 and 67 us.)
#pragma once

#include "fa_span_fwd.cuh"

namespace fa {

constexpr int kFewRows = 16;

template <int D>
struct FewCfg {
  static constexpr int R = kFewRows;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kAtoms = D / 64;
  static constexpr int kThreads = 256;  // four softmax warps, one that loads K, the issuing one, one that loads V
  static constexpr int kKSlots = D == 128 ? 3 : 6, kVSlots = kKSlots, kSlots = kKSlots + kVSlots;
  static __device__ __forceinline__ int slot(int kv, int g) { return kv ? kKSlots + g % kVSlots : g % kKSlots; }
  static __device__ __forceinline__ int use(int kv, int g) { return g / (kv ? kVSlots : kKSlots); }
  static constexpr int kQAtom = R * 128, kQBytes = kAtoms * kQAtom;  // atoms of 64 columns
  static constexpr int kPAtom = R * 128, kPBytes = 2 * kPAtom;       // atoms of 64 keys
  static constexpr uint32_t kTmemCols = 128;                         // S^T of two blocks, O^T
  static constexpr uint32_t kOCol = 2 * R;
  static_assert(3 * R <= kTmemCols, "tensor memory budget");
  static constexpr int kStatBytes = 1024;
  static constexpr int kScheduleBytes = 1536;
  // (16 KB behind the ring: with d = 64 the V^T operand's upper 64 rows are whatever lies there)
  static constexpr int kTail = 2 * kQBytes + 2 * kPBytes + kStatBytes + kScheduleBytes + 1024;
  static constexpr int kSmemBytes = kSlots * kTileBytes + (kTail > 16384 ? kTail : 16384);
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(R * (D + 4) * 4 <= kSlots * kTileBytes, "a cluster's parts take the ring's place");
};

// as SpanBarriers, with what this kernel has
struct FewBarriers {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[12], kv_empty[12];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t drain;
  uint64_t never;
  uint64_t seg_full[kSpanSegs], seg_empty[kSpanSegs];
  SpanSeg seg[kSpanSegs];
  SpanPlace place;
  long long total, end;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr int kFewSegReaders = 6;  // the issuer, the warp that loads V and the softmax warps
static_assert(sizeof(FewBarriers) <= 1024, "barriers overflow their shared-memory slot");

// Of the segment's rows, in shared memory.
struct FewRows {
  int lo[kFewRows], hi[kFewRows];
  float slope2[kFewRows];
  float rel[2][kFewRows];  // positions from the first key of a block and of the one that follows
  float ref[kFewRows];     // the reference (log2 units), -inf: no key so far
  float part[4][kFewRows];  // of each warp: maxima, sums
  float inv[kFewRows];     // at the end: 1 / sum
  char* out[kFewRows];     // at the end: where the row goes, or nullptr
  float lse[kFewRows];     // CLUSTER: this CTA's part
};
static_assert(sizeof(FewRows) <= 1024, "statistics overflow their shared-memory slot");
static_assert(offsetof(FewRows, slope2) % 16 == 0 && offsetof(FewRows, rel) % 16 == 0 && offsetof(FewRows, ref) % 16 == 0,
              "read four rows at a time");

// the four softmax warps: a barrier, and one that says whether any thread of them has x
__device__ __forceinline__ void few_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool few_any(bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)x)
      : "memory");
  return any != 0;
}

// lane q's (q < 16) sum of l[q] over the warp
__device__ __forceinline__ float few_sum(float (&l)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 8; h > 0; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? l[i] : l[i + h], keep = up ? l[i + h] : l[i];
      l[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  return l[0] + __shfl_xor_sync(0xffffffffu, l[0], 16);
}

__device__ __forceinline__ void few_tmem_ld(uint32_t at, uint32_t (&x)[16]) {
  tmem_ld16(at, x);
  tmem_wait_ld();
  reg_fence16(x);
}
__device__ __forceinline__ void few_tmem_st(uint32_t at, const uint32_t (&x)[16]) {
  tmem_st16(at, x);
  tmem_wait_st();
}

// floats in the order of integers
__device__ __forceinline__ int few_order(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float few_order(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// The share of a cluster's item, by one thread.
__device__ __forceinline__ void span_cluster_share(const SpanFwdParams<true>& p, SpanPlace* place) {
  const int k = blockIdx.x / p.cluster, rank = blockIdx.x - k * p.cluster, e = k / p.rows.units;
  const int n = SpanItem<false, true>(p, e).n, j0 = rank * n / p.cluster, j1 = (rank + 1) * n / p.cluster;
  *place = SpanPlace{e, k - e * p.rows.units, j0 + kCrossStart, j1 - j0, kSpanShares};
}

template <int D, bool CLUSTER>
__global__ void __launch_bounds__(256, 1)
    fa_span_few_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ SpanFwdParams<true> p) {
  using C = FewCfg<D>;
  constexpr int R = kFewRows;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    // the 128-byte-swizzled tiles need 1024-byte alignment: report, do nothing
    grid_wait();
    if (threadIdx.x == 0) {
      atomicCAS(&g_fa_device_status, 0u, kStatusBadSmem);
      if (!CLUSTER) p.meta[blockIdx.x].split = 0;
    }
    return;
  }
  uint8_t* sKV = smem_raw;
  uint8_t* sQ = sKV + C::kSlots * C::kTileBytes;
  uint8_t* sP = sQ + 2 * C::kQBytes;
  FewRows* rows = reinterpret_cast<FewRows*>(sP + 2 * C::kPBytes);
  uint8_t* sSchedule = reinterpret_cast<uint8_t*>(rows) + C::kStatBytes;
  FewBarriers* bar = reinterpret_cast<FewBarriers*>(sSchedule + C::kScheduleBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const SpanView<true>& v = p.rows.view;

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar->q_full[t], 1);
      mbar_init(&bar->q_empty[t], 1);
      mbar_init(&bar->s_full[t], 1);
      mbar_init(&bar->s_free[t], 128);
      mbar_init(&bar->p_full[t], 128);
      mbar_init(&bar->pv_done[t], 1);
    }
#pragma unroll 1
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bar->kv_full[s], 1);
      mbar_init(&bar->kv_empty[s], 1);
    }
    for (int s = 0; s < kSpanSegs; ++s) {
      mbar_init(&bar->seg_full[s], 1);
      mbar_init(&bar->seg_empty[s], kFewSegReaders);
    }
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->never, 1);
    bar->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&bar->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  grid_wait();
  if (CLUSTER) {
    if (tid < R) rows->lse[tid] = -CUDART_INF_F;  // no part so far
    if (tid == 0) span_cluster_share(p, &bar->place);
  } else {
    span_schedule<false, C::kThreads>(p, sSchedule, &bar->place, &bar->total, &bar->end);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_trigger();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtx ctx{&bar->abort_flag, p.wait_limit_ns};

  if (warp == 4 || warp == 6) {
    // ------------------------------------------------------------------ segments and TMA
    span_load_warp<C, false, false, C::kQBytes, C::kQAtom>(p, warp == 6, &map_q, &map_k, &map_v, bar, nullptr, sQ, sKV, ctx,
                                                           [](const SpanSeg&) {});
  } else if (warp == 5) {
    // ------------------------------------------------------------------ issuer: S^T of a block ahead of its neighbour's O^T
    if (lane == 0) {
      const uint32_t sq = smem_u32(sQ), skv = smem_u32(sKV), sp = smem_u32(sP);
      constexpr uint32_t id_s = idesc_bf16_f32(128, R, false, false);
      constexpr uint32_t id_pv = idesc_bf16_f32(128, R, true, false);  // (d = 64: the upper 64 rows of V^T are not used)
      int g = 0;  // blocks over all segments
      const SpanSeg* at;
      bool ok = !(p.debug_stall && !span_wait(&bar->never, 0, ctx, kSiteStall));
#pragma unroll 1
      for (int n = 0; ok && span_segment(bar, n, ctx, at); ++n) {
        const int blocks = at->j1 - at->j0;
        mbar_arrive(&bar->seg_empty[n % kSpanSegs]);
        if (!(ok = span_wait(&bar->q_full[n & 1], (n >> 1) & 1, ctx, kSiteCrossQ))) break;
        const uint64_t qdesc = sdesc_sw128(sq + (n & 1) * C::kQBytes, 16, 1024);
#pragma unroll 1
        for (int i = 0; ok && i <= blocks; ++i) {
          if (i < blocks) {
            const int k = g + i, ks = C::slot(0, k), buf = k & 1;
            ok = span_wait(&bar->kv_full[ks], C::use(0, k) & 1, ctx, kSiteCrossK) &&
                 (k < 2 || span_wait(&bar->s_free[buf], ((k >> 1) - 1) & 1, ctx, kSiteCrossSFree));
            if (!ok) break;
            tc_fence_after();
            const uint64_t kdesc = sdesc_sw128(skv + ks * C::kTileBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ss(tmem + buf * R, kdesc + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                          qdesc + (uint32_t)(((kk >> 2) * C::kQAtom + (kk & 3) * 32) >> 4), id_s, kk > 0 ? 1u : 0u);
            mma_commit(&bar->s_full[buf]);
            mma_commit(&bar->kv_empty[ks]);
            if (i == blocks - 1) mma_commit(&bar->q_empty[n & 1]);  // the segment's queries have been read
          }
          if (i > 0) {
            const int k = g + i - 1, vs = C::slot(1, k), buf = k & 1;
            ok = span_wait(&bar->kv_full[vs], C::use(1, k) & 1, ctx, kSiteCrossV) &&
                 span_wait(&bar->p_full[buf], (k >> 1) & 1, ctx, kSiteCrossP);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vdesc = sdesc_sw128(skv + vs * C::kTileBytes, 16384, 1024);
            const uint64_t pdesc = sdesc_sw128(sp + buf * C::kPBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss(tmem + C::kOCol, vdesc + (uint32_t)((kk * 2048) >> 4),
                          pdesc + (uint32_t)(((kk >> 2) * C::kPAtom + (kk & 3) * 32) >> 4), id_pv,
                          (i > 1 || kk > 0) ? 1u : 0u);
            mma_commit(&bar->pv_done[buf]);
            mma_commit(&bar->kv_empty[vs]);
          }
        }
        g += blocks;
      }
      mma_commit(&bar->drain);
      wait_drain_inl(&bar->drain, 0, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------------ softmax (thread: a key; a channel of O)
    // (The warps meet at barriers of their own: a wait that ran out is carried to the next one,
    // where all of them leave.)
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tO = tmem + C::kOCol + lane_off;
    // this key's place in a P buffer: row q at q * 128, 16-byte chunk (key / 8) ^ (q & 7) of its atom
    const uint32_t p_at = (uint32_t)((tid >> 6) * C::kPAtom + (tid & 7) * 2), p_chunk = (uint32_t)((tid & 63) >> 3);
    int g = 0;  // blocks over all segments
    bool bad = false;
    SpanMeta meta{};
    float* sPart = reinterpret_cast<float*>(sKV);  // CLUSTER: this CTA's part, rows of D + 4 floats
#pragma unroll 1
    for (int n = 0;; ++n) {
      const SpanSeg* seg;
      const bool got = span_segment(bar, n, ctx, seg);
      if (few_any(!got || bad)) {
        bad = bad || *ctx.abort_flag;
        break;
      }
      const int j0 = seg->j0, j1 = seg->j1, b = seg->b, u = seg->u, flags = seg->flags, seg_lo = seg->lo, seg_hi = seg->hi;
      const int lo_cut = seg->lo_cut[0], hi_cut = seg->hi_cut[0], rest = seg->rest;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->seg_empty[n % kSpanSegs]);
      const int len = v.len(b), fresh = v.rows(b, len);
      int pos = 0;  // of row `tid`
      if (tid < R) {
        int lo = 0, hi = 0;
        float slope2 = 0.f;
        const int tok = tid / p.rows.heads();
        if (tok < fresh) {
          pos = len + tok;
          v.span(b, tok, pos, lo, hi);
          if (p.slopes) slope2 = p.slopes[(u - tok) * p.rows.heads() + tid] * 1.4426950408889634f;
        }
        rows->lo[tid] = lo, rows->hi[tid] = hi, rows->slope2[tid] = slope2;
        rows->rel[g & 1][tid] = (float)(pos - (j1 - 1) * 128);
        rows->ref[tid] = -CUDART_INF_F;
      }
      float l[R];
#pragma unroll
      for (int q = 0; q < R; ++q) l[q] = 0.f;
      few_sync();
#pragma unroll 1
      for (int j = j1 - 1; j >= j0; --j, ++g) {
        const int buf = g & 1, key = j * 128 + tid;
        bad = bad || !__all_sync(0xffffffffu, span_wait(&bar->s_full[buf], (g >> 1) & 1, ctx, kSiteCrossS));
        tc_fence_after();
        uint32_t x[R];
        few_tmem_ld(tmem + buf * R + lane_off, x);
        tc_fence_before();
        mbar_arrive(&bar->s_free[buf]);
        // scores in log2 units
        if (p.cap.top > 0.f) {
#pragma unroll
          for (int q = 0; q < R; ++q)
            x[q] = __float_as_uint(
                fmaf(-2.f * p.cap.top, rcp_approx(ex2_approx(__uint_as_float(x[q]) * p.cap.mul) + 1.f), p.cap.top));
        } else {
#pragma unroll
          for (int q = 0; q < R; ++q) x[q] = __float_as_uint(__uint_as_float(x[q]) * p.scale_log2);
        }
        if (p.slopes) {
          if (tid < R) rows->rel[buf ^ 1][tid] = (float)(pos - j * 128 + 128);  // (a barrier before it is read)
#pragma unroll
          for (int q4 = 0; q4 < R; q4 += 4) {
            const float4 rel = *reinterpret_cast<const float4*>(rows->rel[buf] + q4);
            const float4 slope2 = *reinterpret_cast<const float4*>(rows->slope2 + q4);
            x[q4] = __float_as_uint(fmaf(-slope2.x, fabsf(rel.x - (float)tid), __uint_as_float(x[q4])));
            x[q4 + 1] = __float_as_uint(fmaf(-slope2.y, fabsf(rel.y - (float)tid), __uint_as_float(x[q4 + 1])));
            x[q4 + 2] = __float_as_uint(fmaf(-slope2.z, fabsf(rel.z - (float)tid), __uint_as_float(x[q4 + 2])));
            x[q4 + 3] = __float_as_uint(fmaf(-slope2.w, fabsf(rel.w - (float)tid), __uint_as_float(x[q4 + 3])));
          }
        }
        if (j * 128 < lo_cut || j * 128 + 128 > hi_cut) {
#pragma unroll
          for (int q = 0; q < R; ++q)
            if (key < rows->lo[q] || key >= rows->hi[q]) x[q] = __float_as_uint(-CUDART_INF_F);
        }
        // (rows that there are not have queries of zeros, or anything: nothing of theirs is written)
        bool rise = false;
#pragma unroll
        for (int q = 0; q < R; q += 4) {
          const float4 ref = *reinterpret_cast<const float4*>(rows->ref + q);
          rise = rise || __uint_as_float(x[q]) > ref.x + kRescaleThresholdLog2 ||
                 __uint_as_float(x[q + 1]) > ref.y + kRescaleThresholdLog2 ||
                 __uint_as_float(x[q + 2]) > ref.z + kRescaleThresholdLog2 ||
                 __uint_as_float(x[q + 3]) > ref.w + kRescaleThresholdLog2;
        }
        if (few_any(rise || bad)) {
          if (few_any(bad)) {
            bad = true;
            break;
          }
          // the block's maxima, and the references' rise
#pragma unroll
          for (int q = 0; q < R; ++q) {
            const int most = __reduce_max_sync(0xffffffffu, few_order(__uint_as_float(x[q])));
            if (lane == q) rows->part[warp][q] = few_order(most);
          }
          few_sync();
          const bool again = j < j1 - 1;
          if (again) bad = !__all_sync(0xffffffffu, span_wait(&bar->pv_done[buf ^ 1], ((g - 1) >> 1) & 1, ctx, kSiteCrossPv));
          tc_fence_after();
          uint32_t o[R];
          if (again) few_tmem_ld(tO, o);
#pragma unroll
          for (int q = 0; q < R; ++q) {
            const float was = rows->ref[q];
            const float now = fmaxf(was, fmaxf(fmaxf(rows->part[0][q], rows->part[1][q]), fmaxf(rows->part[2][q], rows->part[3][q])));
            const float alpha = was == now ? 1.f : ex2_approx(was - now);
            l[q] *= alpha;
            if (again) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
          }
          if (again) few_tmem_st(tO, o);
          few_sync();
          if (tid < R)
            rows->ref[tid] = fmaxf(rows->ref[tid], fmaxf(fmaxf(rows->part[0][tid], rows->part[1][tid]),
                                                         fmaxf(rows->part[2][tid], rows->part[3][tid])));
          few_sync();
        }
        // P, once the product before the last one has read its buffer
        if (g >= 2) bad = bad || !__all_sync(0xffffffffu, span_wait(&bar->pv_done[buf], ((g >> 1) - 1) & 1, ctx, kSiteCrossPv));
        uint8_t* pb = sP + buf * C::kPBytes;
#pragma unroll
        for (int q4 = 0; q4 < R; q4 += 4) {
          const float4 r4 = *reinterpret_cast<const float4*>(rows->ref + q4);
          const float ref[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int q = q4 + i;
            // (a reference that is finite for a row without keys so far: every P is 2^-inf = 0)
            const float w = ex2_approx(__uint_as_float(x[q]) - fmaxf(ref[i], -3.402823466e38f));
            l[q] += w;
            *reinterpret_cast<__nv_bfloat16*>(pb + p_at + q * 128 + ((p_chunk ^ (q & 7)) << 4)) = __float2bfloat16(w);
          }
        }
        // rows of V that nobody sees may hold anything: this key's
        const bool unseen = key < seg_lo || key >= seg_hi;
        if (seg_lo > j * 128 || seg_hi < j * 128 + 128) {
          bad = bad || !__all_sync(0xffffffffu, span_wait(&bar->kv_full[C::slot(1, g)], C::use(1, g) & 1, ctx, kSiteCrossTail));
          if (unseen)
            for (int c = 0; c < C::kAtoms * 8; ++c)
              *reinterpret_cast<uint4*>(sKV + C::slot(1, g) * C::kTileBytes + (c >> 3) * 16384 + tid * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
        tc_fence_before();
        mbar_arrive(&bar->p_full[buf]);
      }
      if (few_any(bad)) {
        bad = true;
        break;
      }
      bad = !__all_sync(0xffffffffu, span_wait(&bar->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, ctx, kSiteCrossPv));
      tc_fence_after();
      // ---- end of the segment: sums over the keys, a thread per row for its statistics and a channel
      // per thread for its values.  (With the statistics in an unrolled loop over the rows, of code that
      // runs once per segment, a row of a segment took 0.6 us of instruction fetches.)
      const float sums = few_sum(l);
      if (lane < R) rows->part[warp][lane] = sums;
      uint32_t o[R];
      few_tmem_ld(tO, o);
      if (few_any(bad)) {
        bad = true;
        break;
      }
      const bool first = flags & kSegFirst, whole = first && (flags & kSegLast);
      if (tid < R) {
        const float sum = rows->part[0][tid] + rows->part[1][tid] + rows->part[2][tid] + rows->part[3][tid];
        const float lse2 = sum == 0.f ? -CUDART_INF_F : rows->ref[tid] + log2f(sum);
        const int tok = tid / p.rows.heads();
        rows->inv[tid] = sum == 0.f ? 0.f : 1.f / sum;
        char* out = nullptr;
        if (CLUSTER) {
          rows->lse[tid] = lse2;
        } else if (tok < fresh) {
          if (whole) {
            const size_t grow = p.rows.row(b, u, tid - tok * p.rows.heads(), tok);
            out = reinterpret_cast<char*>(p.o + grow * D);
            p.lse[grow] = lse2 * 0.6931471805599453f;
          } else {
            const size_t prow = ((size_t)2 * blockIdx.x + (first ? 1 : 0)) * p.part_rows + tid;
            out = reinterpret_cast<char*>(p.part_o + prow * D);
            p.part_lse[prow] = lse2;
          }
        }
        rows->out[tid] = out;
      }
      few_sync();
      if (tid < D) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          const float value = __uint_as_float(o[q]) * rows->inv[q];
          if (CLUSTER) {
            sPart[q * (D + 4) + tid] = value;
          } else if (char* out = rows->out[q]) {
            if (whole)
              reinterpret_cast<__nv_bfloat16*>(out)[tid] = __float2bfloat16(value);
            else
              reinterpret_cast<float*>(out)[tid] = value;
          }
        }
      }
      if ((flags & (kSegFirst | kSegLast)) == kSegFirst) {
        // (the CTA's last segment: the item's other blocks follow its share)
        meta.split = 1;
        meta.b = b;
        meta.u = u;
        meta.token0 = 0;
        meta.last = bar->end + rest;
        meta.total = bar->total;
      }
    }
    if (bad) meta.split = 0;
    if (!CLUSTER && tid == 0) p.meta[blockIdx.x] = meta;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if constexpr (CLUSTER) {
    // every CTA of the cluster writes every p.cluster-th row, a warp per row
    cluster_sync();
    constexpr int E = D / 32, kMost = 8;
    const int ctas = p.cluster, item = blockIdx.x / ctas, b = item / p.rows.units;
    const int fresh = v.rows(b, v.len(b));
    const float* parts = reinterpret_cast<const float*>(sKV) + lane * E;
    for (int row = (int)cluster_ctarank() + ctas * warp; row < p.rows.heads() * fresh; row += ctas * (C::kThreads / 32)) {
      float l[kMost], o[kMost][E], mx = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < ctas) {
          l[i] = cluster_load(&rows->lse[row], i);
          cluster_load<E>(parts + row * (D + 4), i, o[i]);
        }
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < ctas) mx = fmaxf(mx, l[i]);
      const float ref = fmaxf(mx, -3.402823466e38f);
      float sum = 0.f, acc[E];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < ctas && l[i] != -CUDART_INF_F) {  // (a part without keys may not have been written)
          const float wt = ex2_approx(l[i] - ref);
          sum += wt;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, o[i][e], acc[e]);
        }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int tok = row / p.rows.heads();
      const size_t grow = p.rows.row(b, item - b * p.rows.units, row - tok * p.rows.heads(), tok);
      uint32_t* orow = reinterpret_cast<uint32_t*>(p.o + grow * D) + lane * (E / 2);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) orow[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      if (lane == 0) p.lse[grow] = (sum == 0.f ? -CUDART_INF_F : ref + log2f(sum)) * 0.6931471805599453f;
    }
    cluster_sync();  // the others have read this CTA's part
  }
}

}  // namespace fa
