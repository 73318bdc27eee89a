// Forward kernel of attention to spans of keys, over contiguous keys (fa_span_fwd) or
// a cache in pages (fa_paged_fwd).
//
// The arithmetic, the roles and the pipeline are those of fa_cross_fwd_kernel (TMA
// fills a ring of K and V tiles, one thread issues S = Q K^T, one O += P V, two softmax
// warpgroups hold a row of scores per thread; two row tiles per item, PAIR, or one
// whose key blocks go to the warpgroups in turn, ALT).  Up to 16 rows of a unit over
// pages go to fa_span_few_kernel.  What differs:
//
// Work.  An item is a tile (pair) of query rows of a unit (SpanRows) with the blocks of
// 128 keys that any of its rows sees; items cost what they have of them.  Where enough of them
// are there, the CTAs take whole items (the longest first, or head by head); otherwise even
// shares of all items' blocks, and fa_span_combine_kernel joins the items that shares cut.
// Within an item each row tile takes only the blocks that it sees something of, from the last
// to the first: where a bias grows with the distance the largest scores come first, and the
// running maximum stays (from the first to the last it rises in every block: H=32/8 N=8192
// d=128, two requests, causal, with slopes, 1022 and 951 us).
//
// Measured on a GB300 (two requests, H=32/8 N=8192 d=128, causal): 703 us, 1565 TFLOP/s, with slopes 742 us,
// with a window of 1024 237 us; one request capped at 50 479 us, at 20 (where blocks on the diagonal take the
// exponential) 528 us; 2048 new tokens of two requests over 2000 and 16000 in pages of 64 457 us, 1470 TFLOP/s.
// These are loops over the same tensors; with others from call to call the last takes 487 us, 1380 TFLOP/s.
// The softmax warps bound it (tensor cores 56 % busy, DRAM idle).
//
// Scores.  Blocks that some row sees in part are masked by the row's own span; the cap
// (MOD 2 and 3) and the bias (MOD 1 and 3) change the scores in registers, before the maximum.
//
// Pages.  A tile of 128 keys is 128 / page_size boxes, one per lane of the loading
// warp, from where the page table says; pages that no row sees, and those outside the
// pool, are asked for at a coordinate outside the tensor, which the TMA fills with zeros
// without reading.
//
// Keys of an item's first and last block that none of its rows sees may hold
// anything: their scores become -inf and the warp that loads V zeroes their rows of it.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include <type_traits>

#include "fa_cross_fwd.cuh"
#include "fa_span.cuh"

namespace fa {

struct SpanMeta {     // of each CTA, for the combine kernel
  int split;          // its last item goes on in the next CTA
  int b, u, token0;   // that item
  long long last;     // the place behind the item's last block
  long long total;    // places of the sequence
};

template <bool PAGED>
struct SpanFwdParams {
  SpanRows<PAGED> rows;
  __nv_bfloat16* o;
  float* lse;
  SpanMeta* meta;    // [grid]
  float* part_lse;   // [2 grid][part_rows], base 2
  float* part_o;     // [2 grid][part_rows][d]
  int part_rows;     // rows of a part: 256 (PAIR) or a unit's (ALT)
  int q_bytes;       // of a row tile's queries
  int B;
  int row_tiles;     // row tiles (PAIR: pairs of them) per unit
  int cluster;       // fa_span_few_kernel: CTAs per item, joined in a cluster (1: none)
  int pages;         // pages in the pool
  float scale_log2;  // without a cap
  SpanCap cap;
  const float* slopes;  // [H] or nullptr
  uint64_t wait_limit_ns;
  int debug_stall;
  int o_align32;
};

// A CTA's work: whole items, one of each round of G ranks (rank k G + c in even rounds k, k G +
// G - 1 - c in odd ones, so that what the first gets more of evens out), or a share of places.
enum : int { kSpanShares, kSpanSorted, kSpanByHead, kSpanByEntry };
struct SpanPlace {
  int e, u;   // shares: entry (request and row tile) and unit of it; whole: e is the rank
  int j;      // shares: place in the item; whole: the round
  int left;   // places or items from there on
  int mode;   // kSpanShares: places; how ranks are numbered otherwise
};
__device__ __forceinline__ long long span_rank(int round, int G, int c) {
  return (long long)round * G + (round & 1 ? G - 1 - c : c);
}

// A run of key blocks of one item; blocks are counted from key 0.  The loading warp works the
// segments out and leaves them in shared memory, where the other warps read them.  (Each warp
// working them out for itself takes 20 KB more of code, and the loops of the kernel no
// longer fit the instruction cache.)
enum : int { kSegFirst = 1, kSegLast = 2, kSegTwo = 4, kSegDirtyFront = 8, kSegDirtyBack = 16, kSegEnd = 32 };
struct SpanSeg {
  int b, u, token0;
  int flags;           // the item's first and last block are in it; PAIR: there is a second row tile;
                       // rows of V in block j0 and j1 - 1 that nobody sees; no more segments
  int j0, j1, rest;    // blocks; the item's blocks behind them
  int lo, hi;          // keys that the item's rows see
  int a0[2], a1[2];    // PAIR: the blocks of each row tile
  int lo_cut[2], hi_cut[2];  // of each row tile: see SpanTile
};
constexpr int kSpanSegs = 4;  // segments in shared memory
enum : int { kSiteSpanSeg = 70, kSiteSpanSegFree };

template <bool PAIR, bool PAGED>
struct SpanItem {
  SpanTile t[PAIR ? 2 : 1];
  int lo, hi, base;  // keys seen; first block
  int n;             // number of blocks: none without tokens, else at least one, so that rows without keys are written
  int token0;
  bool two;          // there are tokens in the second tile
  __device__ __forceinline__ SpanItem(const SpanFwdParams<PAGED>& p, int e) {
    const int b = e / p.row_tiles, rt = p.row_tiles - 1 - (e - b * p.row_tiles);
    t[0] = p.rows.tile(b, PAIR ? 2 * rt : rt);
    lo = t[0].lo, hi = t[0].hi;
    if constexpr (PAIR) {
      t[1] = 2 * rt + 1 < p.rows.tiles ? p.rows.tile(b, 2 * rt + 1) : SpanTile{0, 0, 0x7fffffff, 0};
      if (t[0].empty()) lo = t[1].lo, hi = t[1].hi;
      else if (!t[1].empty()) lo = min(lo, t[1].lo), hi = max(hi, t[1].hi);
    }
    base = lo >> 7;
    const int there = p.rows.view.rows(b, p.rows.view.len(b));
    token0 = (PAIR ? 2 * rt : rt) * p.rows.tokens();
    two = PAIR && token0 + p.rows.tokens() < there;
    n = token0 < there ? max(((hi + 127) >> 7) - base, 1) : 0;
  }
  __device__ __forceinline__ int places() const { return n > 0 ? n + kCrossStart : 0; }
};

// The next segment.  Ranks are numbered by entry (with `order`: entries by falling cost), all
// units of one after another, or head by head (all row tiles of a unit one after another, whose
// keys the CTAs of a round then share in L2).  Places beside an item's blocks as in fa_cross_fwd.cuh.
template <bool PAIR, bool PAGED>
__device__ __forceinline__ bool span_next(const SpanFwdParams<PAGED>& p, const uint16_t* order, SpanPlace& at, SpanSeg& s) {
  const int U = p.rows.units;
  while (at.left > 0) {
    int e = at.e;
    s.u = at.u;
    if (at.mode == kSpanByHead) {
      const int head = at.e / p.row_tiles, b = head / U;
      s.u = head - b * U;
      e = b * p.row_tiles + (at.e - head * p.row_tiles);
    } else if (at.mode != kSpanShares) {
      e = at.e / U;
      s.u = at.e - e * U;
      if (PAIR && at.mode == kSpanSorted) e = order[e];
    }
    const SpanItem<PAIR, PAGED> item(p, e);
    s.b = e / p.row_tiles;
    s.token0 = item.token0;
    s.lo = item.lo, s.hi = item.hi;
    const int end_block = item.base + item.n;
    if (at.mode != kSpanShares) {
      s.j0 = item.base, s.j1 = end_block;
      --at.left;
      at.e = (int)span_rank(++at.j, gridDim.x, blockIdx.x);
      if (item.n == 0) continue;
    } else if (item.n == 0) {
      ++at.e;  // (the entry's units all)
      continue;
    } else {
      const int places = item.places(), end = min(places, at.j + min(at.left, places));
      s.j0 = item.base + max(at.j - kCrossStart, 0);
      s.j1 = item.base + end - kCrossStart;
      at.left -= end - at.j;
      at.j = end;
      if (end == places) {
        at.j = 0;
        if (++at.u == U) at.u = 0, ++at.e;
      }
      if (s.j1 <= item.base) continue;  // only places before the item's blocks
    }
    s.rest = end_block - s.j1;
    s.flags = (s.j0 == item.base ? kSegFirst : 0) | (s.rest == 0 ? kSegLast : 0) |
              (item.two ? kSegTwo : 0);
    // (past the keys of a contiguous tensor the TMA has filled zeros)
    const int filled = PAGED ? s.j1 * 128 : min(p.rows.view.C, s.j1 * 128);
    if (s.lo > s.j0 * 128 || (s.j1 == s.j0 + 1 && s.hi < filled)) s.flags |= kSegDirtyFront;
    if (s.hi < filled || (s.j1 == s.j0 + 1 && s.lo > s.j0 * 128)) s.flags |= kSegDirtyBack;
#pragma unroll
    for (int t = 0; t < (PAIR ? 2 : 1); ++t) {
      s.lo_cut[t] = item.t[t].lo_cut, s.hi_cut[t] = item.t[t].hi_cut;
      s.a0[t] = max(s.j0, item.t[t].lo >> 7);
      s.a1[t] = min(s.j1, (item.t[t].hi + 127) >> 7);
      // a tile that sees nothing here takes one block, whose keys are all masked
      if (s.a0[t] >= s.a1[t]) s.a0[t] = s.j0, s.a1[t] = s.j0 + 1;
    }
    return true;
  }
  return false;
}

// the row tiles (bits) that take block j
template <bool PAIR>
__device__ __forceinline__ int span_active(const SpanSeg& s, int j) {
  if (!PAIR) return 1 << ((s.j1 - 1 - j) & 1);
  return (j >= s.a0[0] && j < s.a1[0] ? 1 : 0) | (s.flags & kSegTwo && j >= s.a0[1] && j < s.a1[1] ? 2 : 0);
}

// whether block j of the segment has rows of V that no row of the item sees
__device__ __forceinline__ bool span_dirty(const SpanSeg& s, int j) {
  return (s.flags & kSegDirtyFront && j == s.j0) || (s.flags & kSegDirtyBack && j == s.j1 - 1);
}

// How the CTAs divide the items, by all T threads.  `scratch` (kMergeBytes of shared memory)
// keeps the order of the entries with PAIR.  More than kSpanRounds items a CTA even out: they
// go whole, head by head but where a causal mask alone makes the last row tiles the longest.  Fewer: the slowest CTA's items are added up for each way of
// numbering them, and the items go whole where that ends no later than even shares and the
// join of what they cut.
constexpr int kSpanRounds = 32;
template <bool PAIR, int T, bool PAGED>
__device__ __forceinline__ void span_schedule(const SpanFwdParams<PAGED>& p, void* scratch, SpanPlace* place, long long* all,
                                              long long* share_end) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = p.B * p.row_tiles, U = p.rows.units, G = gridDim.x, c = blockIdx.x;
  const long long count = (long long)E * U;
  auto whole = [&](int mode) {
    const int rounds = (int)(count / G);
    if (tid == 0) *place = SpanPlace{c, 0, 0, rounds + (span_rank(rounds, G, c) < count ? 1 : 0), mode};
  };
  if (count > (long long)kSpanRounds * G) {
    const SpanView<PAGED>& v = p.rows.view;
    whole(PAIR && (v.window || !v.causal || v.begin) ? kSpanByHead : kSpanByEntry);
    return;
  }
  uint16_t* order = static_cast<uint16_t*>(scratch);                   // [T]
  int* sums = reinterpret_cast<int*>(order + T);                       // [160] places of each CTA's whole items
  long long* part = reinterpret_cast<long long*>(sums + 160);          // [T / 32]
  static_assert(kCrossMaxCtas <= 160 && T >= 160 && T % 64 == 0 && T * 2 + 160 * 4 + T / 4 <= CrossCfg<128>::kMergeBytes, "a sum for each CTA");
  if (tid == 0) *place = SpanPlace{0, 0, 0, 0, kSpanShares};
  const int chunk = (E + T - 1) / T, e0 = min(E, tid * chunk), e1 = min(E, e0 + chunk);
  const bool sorted = PAIR && E <= T;  // a thread per entry
  int one = 0, place_of = tid;         // (sorted) the entry's cost and its place in the order
  long long mine = 0, upto = 0, total = 0, start = 0, end = 0;
  int lead[2] = {0, 0};
  // Passes over this thread's entries: their places; with whole items, the CTAs' places by
  // entry (by falling cost) and head by head; with shares, where this CTA's begins.
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    if (pass == 1 || pass == 2) {
      if (tid < 160) sums[tid] = 0;
      __syncthreads();
    }
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      const int n = sorted && pass > 0 ? one : SpanItem<PAIR, PAGED>(p, e).places();
      if (pass == 0) {
        mine += n;
        one = n;
      } else if (pass < 3) {
        if (n == 0) continue;
        const int b = e / p.row_tiles, at = sorted ? place_of : e;
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const int k = pass == 2 ? (b * U + u) * p.row_tiles + (e - b * p.row_tiles) : at * U + u;
          const int round = k / G, i = k - round * G;
          atomicAdd(&sums[round & 1 ? G - 1 - i : i], n);
        }
      } else {
        if (start < upto + (long long)n * U) {
          const long long off = start - upto;
          const int u = (int)(off / n);
          *place = SpanPlace{e, u, (int)(off - (long long)u * n), (int)(end - start), kSpanShares};
          break;
        }
        upto += (long long)n * U;
      }
    }
    if (pass == 0) {
      if (sorted) {
        int* costs = static_cast<int*>(scratch);
        if (tid < E) costs[tid] = one;
        __syncthreads();
        place_of = 0;
#pragma unroll 1
        for (int e = 0; e < E; ++e) {
          const int n = costs[e];
          place_of += n > one || (n == one && e < tid) ? 1 : 0;
        }
        __syncthreads();
        if (tid < E) order[place_of] = (uint16_t)tid;
      }
      upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long add = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += add;
      }
      if (lane == 31) part[warp] = upto;
    } else if (pass < 3) {
      __syncthreads();
      int most = 0;
      for (int i = lane; i < G; i += 32) most = max(most, sums[i]);
      most = __reduce_max_sync(0xffffffffu, most);
      __syncthreads();
      lead[pass - 1] = most;
      if (PAIR && pass == 1) continue;
      long long before = 0;
#pragma unroll 1
      for (int w = 0; w < T / 32; ++w) {
        if (w == warp) before = total;
        total += part[w];
      }
      total *= U;
      // (head by head where that is as even to 3 %)
      const bool by_head = PAIR && lead[1] * 32LL <= lead[0] * 33LL;
      const long long slowest = by_head ? lead[1] : lead[0];
      if ((slowest - kCrossCut) * G <= total || slowest * G <= total + total / 16) {
        whole(by_head ? kSpanByHead : sorted ? kSpanSorted : kSpanByEntry);
        return;
      }
      const long long g = min((long long)G, total);
      if (c >= g) return;
      start = c * total / g, end = (c + 1) * total / g;
      if (tid == 0) *all = total, *share_end = end;
      const long long at = (before + upto - mine) * U;
      if (start < at || start >= (before + upto) * U) return;
      upto = at;
      pass = 2;
    }
  }
}

// (as CrossBarriers, and the segments)
struct SpanBarriers {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[12], kv_empty[12];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t v_ask, v_clean;
  uint64_t merge_ready, merge_free;
  uint64_t drain[2];
  uint64_t never;
  uint64_t seg_full[kSpanSegs], seg_empty[kSpanSegs];  // (read by the issuers, the warp that loads V and eight softmax warps)
  SpanSeg seg[kSpanSegs];
  SpanPlace place;
  long long total, end;  // places of the sequence; end of the CTA's share
  uint32_t tmem_base;
  int abort_flag;
};
constexpr int kSpanSegReaders = 11;
static_assert(sizeof(SpanBarriers) <= 1024, "barriers overflow their shared-memory slot");

// wait_bounded_inl in a third of its code
__device__ __forceinline__ bool span_wait(uint64_t* bar, uint32_t parity, const WaitCtx& ctx, int site) {
  uint64_t since = 0;
#pragma unroll 1
  for (int n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if (n & 31) continue;
    if (*ctx.abort_flag) return false;
    const uint64_t now = global_timer_ns();
    if (since == 0) since = now;
    if (now - since > ctx.limit_ns) {
      atomicCAS(&g_fa_device_status, 0u, kStatusTimeout | ((unsigned)(site & 0xff) << 8));
      *ctx.abort_flag = 1;
      __threadfence_block();
      return false;
    }
  }
}

// The n-th segment; false: there are no more (or the wait ran out).
template <class Bar>
__device__ __forceinline__ bool span_segment(Bar* bar, int n, const WaitCtx& ctx, const SpanSeg*& w) {
  const int s = n % kSpanSegs;
  if (!span_wait(&bar->seg_full[s], (n / kSpanSegs) & 1, ctx, kSiteSpanSeg)) return false;
  w = &bar->seg[s];
  return !(w->flags & kSegEnd);
}

// A tile of 128 keys as TMA boxes, a lane per page.
template <bool PAGED>
struct SpanBoxes {
  int lane, shift, rows, count;
  uint8_t* ring;
  __device__ __forceinline__ SpanBoxes(const SpanFwdParams<PAGED>& p, uint8_t* sKV) {
    lane = threadIdx.x & 31;
    shift = p.rows.view.page_shift;
    rows = PAGED ? min(1 << shift, 128) : 128;
    count = 128 / rows;
    ring = sKV;
  }
  // the page of this lane's part of block j, or -1: nothing there that a row sees
  __device__ __forceinline__ int page(const SpanFwdParams<PAGED>& p, const SpanSeg& w, int j) const {
    if (!PAGED) return w.b;
    if (lane >= count) return -1;
    const int key = j * 128 + lane * rows;
    if (key >= w.hi || key + rows <= w.lo) return -1;
    const int page = p.rows.view.table[(long long)w.b * p.rows.view.width + (key >> shift)];
    return page >= 0 && page < p.pages ? page : -1;
  }
  // block j's K (kv = 0) or V tile as the g-th of its kind; false: the wait for its slot ran out
  template <class C, class Bar>
  __device__ __forceinline__ bool load(const CUtensorMap* map, Bar* bar, int kv, int g, const SpanSeg& w, int j, int kvh,
                                       int page, const WaitCtx& ctx) const {
    const int slot = C::slot(kv, g);
    if (!__all_sync(0xffffffffu, span_wait(&bar->kv_empty[slot], (C::use(kv, g) & 1) ^ 1, ctx, kSiteCrossKvEmpty)))
      return false;
    if (lane == 0) mbar_arrive_expect_tx(&bar->kv_full[slot], C::kTileBytes);
    __syncwarp();
    if (lane < count) {
      const int row = !PAGED ? j * 128 : count > 1 ? 0 : (j * 128) & ((1 << shift) - 1);
      for (int a = 0; a < C::kAtoms; ++a)
        tma_load_4d(ring + slot * C::kTileBytes + a * 16384 + lane * rows * 128, map, &bar->kv_full[slot], a * 64, row, kvh, page);
    }
    return true;
  }
};

// Rows of V that nobody sees, of the tile loaded as the `tile`-th; -1: none are waiting.
struct SpanUnseen {
  int tile, segment;
  int from, to;  // rows [from, to) are seen
};

// The two loading warps, in one piece of code.  The first works out the segments, publishes them, and fills
// Q's two buffers (QBYTES each, atoms of 64 columns QATOM bytes apart) and the K tiles of the ring.  The V
// tiles are the second's with pages, else the first's as well.  (A box costs the warp that asks for it some
// 50 cycles: with pages of 16 tokens one warp for both takes longer over a block than the rest of the
// kernel, 594 instead of 466 us for 2048 tokens of two requests over 2000 and 16000, H=32/8 d=128; with
// one box a tile the two are equal.)  CLEAN: the second zeroes rows of V that nobody sees, when
// the warp that issues P V has come to their block and is asking.  It puts that off, to load on, but not
// until it waits for something that only comes after that block: its tile's slot, or a segment that is
// published when the block's is done with.  `done` is called with every segment of the second.  False: a
// wait ran out.
template <class C, bool PAIR, bool CLEAN, int QBYTES, int QATOM, bool PAGED, class Bar, class Done>
__device__ __forceinline__ bool span_load_warp(const SpanFwdParams<PAGED>& p, bool second, const CUtensorMap* map_q,
                                               const CUtensorMap* map_k, const CUtensorMap* map_v, Bar* bar, const uint16_t* order, uint8_t* sQ,
                                               uint8_t* sKV, const WaitCtx& ctx, Done done) {
  const int lane = threadIdx.x & 31;
  SpanPlace at = bar->place;
  SpanSeg w{};
  const SpanBoxes<PAGED> boxes(p, sKV);
  const int kv0 = second ? PAGED ? 1 : 2 : 0, kv1 = second || !PAGED ? 2 : 1;  // what this warp loads
  int g = 0, loads = 0, segments = 0, nq = 0;  // blocks, tiles, segments, Q loads
  bool ok = true;
  SpanUnseen unseen{-1, 0, 0, 0};
  int cleaned = 0;
  auto load_q = [&](int qs) {
    if (lane == 0) {
      const int tiles = w.flags & kSegTwo ? 2 : 1;
      mbar_arrive_expect_tx(&bar->q_full[qs], tiles * p.q_bytes);
      for (int t = 0; t < tiles; ++t)
        for (int a = 0; a < C::kAtoms; ++a)
          tma_load_4d(sQ + (PAIR ? t : qs) * QBYTES + a * QATOM, map_q, &bar->q_full[qs], a * 64, 0,
                      w.token0 + p.rows.tokens() * t, w.b * p.rows.units + w.u);
    }
    __syncwarp();
    ++nq;
  };
  auto clean = [&] {
    if constexpr (CLEAN) {
      if (!__all_sync(0xffffffffu, span_wait(&bar->v_ask, cleaned & 1, ctx, kSiteCrossTail))) return false;
      ++cleaned;
      uint8_t* tile = sKV + C::slot(1, unseen.tile) * C::kTileBytes;
      const int from = unseen.from, to = unseen.to, chunks = (from + 128 - to) * 8;  // of 16 bytes of an atom
      for (int i = lane; i < C::kAtoms * chunks; i += 32) {
        const int a = i >= chunks ? 1 : 0, k = i - a * chunks, c = k < from * 8 ? k : k - from * 8 + to * 8;
        *reinterpret_cast<uint4*>(tile + a * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->v_clean);
      unseen.tile = -1;
    }
    return true;
  };
#pragma unroll 1
  while (ok) {
    const int s = segments % kSpanSegs;
    if (!second) {
      const bool more = span_next<PAIR>(p, order, at, w);
      if (!more) w.flags = kSegEnd;
      // the segment for the other warps, once they have done with the one in its place
      ok = __all_sync(0xffffffffu, span_wait(&bar->seg_empty[s], ((segments / kSpanSegs) & 1) ^ 1, ctx, kSiteSpanSegFree));
      if (!ok) break;
      if (lane == 0) {
        bar->seg[s] = w;
        mbar_arrive(&bar->seg_full[s]);
      }
      __syncwarp();
      if (!more) break;
      // a later segment's first key block needs only ring slots: it goes out
      // before the queries, whose buffer an earlier segment may still be reading
      if (segments == 0) load_q(0);
    } else {
      const SpanSeg* seg;
      if (unseen.tile >= 0 && (!PAGED || segments - unseen.segment > 1) && !(ok = clean())) break;
      if (!__all_sync(0xffffffffu, span_segment(bar, segments, ctx, seg))) {
        ok = !*ctx.abort_flag;
        break;
      }
      w = *seg;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->seg_empty[s]);
    }
    const int kvh = w.u / p.rows.kv_div;
    int page = boxes.page(p, w, w.j1 - 1);
#pragma unroll 1
    for (int j = w.j1 - 1; ok && j >= w.j0; --j) {
      const int next = j > w.j0 ? boxes.page(p, w, j - 1) : 0;  // (asked for a block ahead)
      const bool dirty = CLEAN && second && span_dirty(w, j);
      if (unseen.tile >= 0 && (dirty || !PAGED || g - unseen.tile >= C::kVSlots) && !(ok = clean())) break;
#pragma unroll 1
      for (int kv = kv0; kv < kv1; ++kv) {
        if (!(ok = boxes.template load<C>(kv ? map_v : map_k, bar, kv, g, w, j, kvh, page, ctx))) break;
        ++loads;
      }
      if (!ok) break;
      if (dirty) {
        const int from = max(w.lo - j * 128, 0);
        unseen = {g, segments, from, max(min(w.hi - j * 128, 128), from)};
      }
      ++g;
      page = next;
      if (!second && j == w.j1 - 1 && segments > 0) {
        const int qs = PAIR ? 0 : segments & 1, use = PAIR ? segments : segments >> 1;
        if (use > 0) ok = __all_sync(0xffffffffu, span_wait(&bar->q_empty[qs], (use - 1) & 1, ctx, kSiteCrossQEmpty));
        if (ok) load_q(qs);
      }
    }
    ++segments;
    if (second) done(w);
  }
  if (ok && unseen.tile >= 0) ok = clean();
  // every copy this warp started must land before the CTA can exit
  if (lane == 0) {
    if (!second)
      for (int s = 0; s < (PAIR ? 1 : 2); ++s) {
        const int uses = PAIR ? nq : (nq + 1 - s) >> 1;
        if (uses > 0) wait_drain_inl(&bar->q_full[s], (uses - 1) & 1, kDrainLimitNs);
      }
#pragma unroll 1
    for (int s = 0; s < C::kSlots; ++s) {
      // loads into slot s
      const bool vslot = s >= C::kKSlots;
      const int n = PAGED ? (vslot == second ? loads : 0) : vslot ? loads >> 1 : (loads + 1) >> 1;
      const int first = vslot ? s - C::kKSlots : s;
      if (n > first) wait_drain_inl(&bar->kv_full[s], C::use(vslot, n - 1 - first) & 1, kDrainLimitNs);
    }
  }
  __syncwarp();
  return ok;
}

// multiplies a block's scores with mul and adds a bias of -slope2 |rel - c| to that of key c
// (log2 units); rel: the row's position from the block's first key
__device__ __forceinline__ void span_bias(uint32_t (&s)[4][32], float mul, float slope2, int rel, bool causal) {
  const float relf = (float)rel;
  if (causal || __all_sync(0xffffffffu, rel >= 127 || rel <= 0)) {
    // all keys (with a causal mask: all that are seen) on one side of the row: a line
    // g c - g rel, as a value for each eight keys and offsets within them
    const float g = causal || rel > 0 ? slope2 : -slope2, base = -g * relf;
    const float2 mul2 = make_float2(mul, mul);
    float2 off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = make_float2(g * (float)(2 * i), g * (float)(2 * i + 1));
#pragma unroll
    for (int c8 = 0; c8 < 16; ++c8) {
      const float at = fmaf(g, (float)(8 * c8), base);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t* e = &s[c8 >> 2][8 * (c8 & 3) + 2 * i];
        const float2 x = __ffma2_rn(make_float2(__uint_as_float(e[0]), __uint_as_float(e[1])), mul2,
                                    __fadd2_rn(off[i], make_float2(at, at)));
        e[0] = __float_as_uint(x.x);
        e[1] = __float_as_uint(x.y);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i)
        s[c][i] = __float_as_uint(fmaf(-slope2, fabsf(relf - (float)(32 * c + i)), __uint_as_float(s[c][i]) * mul));
  }
}

// 32 keys' bits of those in [from, to)
__device__ __forceinline__ uint32_t span_bits(int from, int to) {
  const uint32_t below = to >= 32 ? 0xffffffffu : to <= 0 ? 0u : (1u << to) - 1u;
  const uint32_t before = from >= 32 ? 0xffffffffu : from <= 0 ? 0u : (1u << from) - 1u;
  return below & ~before;
}

// PAIR: two row tiles per item.  MOD: 0 plain scores, 1 with a bias, 2 capped, 3 both.
template <int D, int MOD, bool PAIR, bool PAGED>
__global__ void __launch_bounds__(384, 1)
    fa_span_fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ SpanFwdParams<PAGED> p) {
  using C = CrossCfg<D>;
  // The issuing threads' loops over the two row tiles: one copy of the products where the kernel's loops
  // together outgrow the instruction cache (H=32/8 N=8192 d=128, two requests, causal, with slopes: 743 us, and
  // 785 with two copies; one request capped 479 and 566), else two (plain scores 701 us, and 735 with one copy;
  // H=16 N=2048 d=64, four requests, 59 and 66 us).
  constexpr int kIssueUnroll = D == 64 || MOD == 0 ? 2 : 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    // the 128-byte-swizzled tiles need 1024-byte alignment: report, do nothing
    grid_wait();
    if (threadIdx.x == 0) {
      atomicCAS(&g_fa_device_status, 0u, kStatusBadSmem);
      p.meta[blockIdx.x].split = 0;
    }
    return;
  }
  uint8_t* smem = smem_raw;
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * C::kTileBytes;
  float* sMerge = reinterpret_cast<float*>(sKV + C::kSlots * C::kTileBytes);  // [3][128]
  SpanBarriers* bar = reinterpret_cast<SpanBarriers*>(reinterpret_cast<uint8_t*>(sMerge) + C::kMergeBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const SpanView<PAGED>& v = p.rows.view;

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar->q_full[t], 1);
      mbar_init(&bar->q_empty[t], 1);
      mbar_init(&bar->s_full[t], 1);
      mbar_init(&bar->s_free[t], 128);
      mbar_init(&bar->p_full[t], 128);
      mbar_init(&bar->pv_done[t], 1);
      mbar_init(&bar->drain[t], 1);
    }
#pragma unroll 1
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bar->kv_full[s], 1);
      mbar_init(&bar->kv_empty[s], 1);
    }
    for (int s = 0; s < kSpanSegs; ++s) {
      mbar_init(&bar->seg_full[s], 1);
      mbar_init(&bar->seg_empty[s], kSpanSegReaders);
    }
    mbar_init(&bar->v_clean, 1);
    mbar_init(&bar->v_ask, 1);
    mbar_init(&bar->merge_ready, 128);
    mbar_init(&bar->merge_free, 128);
    mbar_init(&bar->never, 1);
    bar->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&bar->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  grid_wait();
  span_schedule<PAIR, C::kThreads>(p, sMerge, &bar->place, &bar->total, &bar->end);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_trigger();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtx ctx{&bar->abort_flag, p.wait_limit_ns};
  if (warp >= 8) {
    setmaxnreg_dec<C::kMiscRegs>();
    if (warp == 9 || warp == 11) {
      // ------------------------------------------------------------------ segments and TMA
      const bool second = warp == 11;
      SpanMeta meta{};
      const bool ok = span_load_warp<C, PAIR, true, C::kTileBytes, 16384>(
          p, second, &map_q, &map_k, &map_v, bar, reinterpret_cast<const uint16_t*>(sMerge), sQ, sKV, ctx,
          [&](const SpanSeg& w) {
            if ((w.flags & (kSegFirst | kSegLast)) == kSegFirst) {
              // (the CTA's last segment: the item's other blocks follow its share)
              meta.split = 1;
              meta.b = w.b;
              meta.u = w.u;
              meta.token0 = w.token0;
              meta.last = bar->end + w.rest;
              meta.total = bar->total;
            }
          });
      if (!ok) meta.split = 0;
      if (second && lane == 0) p.meta[blockIdx.x] = meta;
      __syncwarp();
    } else if (warp == 8) {
      // ------------------------------------------------------------------ S issuer
      // g counts key blocks over all segments
      if (lane == 0) {
        const uint32_t sq = smem_u32(sQ), skv = smem_u32(sKV);
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
        int s_uses[2] = {0, 0}, g = 0, nq = 0;
        const SpanSeg* at;
        bool ok = !(p.debug_stall && !span_wait(&bar->never, 0, ctx, kSiteStall));
#pragma unroll 1
        while (ok && span_segment(bar, nq, ctx, at)) {
          const SpanSeg w = *at;
          mbar_arrive(&bar->seg_empty[nq % kSpanSegs]);
          const int qs = PAIR ? 0 : nq & 1, use = PAIR ? nq : nq >> 1;
          if (!span_wait(&bar->q_full[qs], use & 1, ctx, kSiteCrossQ)) break;
          ++nq;
#pragma unroll 1
          for (int j = w.j1 - 1; ok && j >= w.j0; --j, ++g) {
            const int ks = C::slot(0, g);
            if (!(ok = span_wait(&bar->kv_full[ks], C::use(0, g) & 1, ctx, kSiteCrossK))) break;
            const uint64_t kdesc = sdesc_sw128(skv + ks * C::kTileBytes, 16, 1024);
            const int active = span_active<PAIR>(w, j);
#pragma unroll kIssueUnroll
            for (int t = 0; t < 2; ++t) {
              if (active >> t & 1) {
                const int sb = C::kDualS ? t : 0;
                int& uses = sb ? s_uses[1] : s_uses[0];
                if (uses > 0 && !span_wait(&bar->s_free[sb], (uses - 1) & 1, ctx, kSiteCrossSFree)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                const uint64_t qd = sdesc_sw128(sq + (PAIR ? t : qs) * C::kTileBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                  mma_bf16_ss(tmem + (sb ? C::kSCol1 : C::kSCol), qd + off, kdesc + off, id_s, kk > 0 ? 1u : 0u);
                }
                mma_commit(&bar->s_full[t]);
                ++uses;
              }
            }
            if (!ok) break;
            mma_commit(&bar->kv_empty[ks]);
          }
          if (!ok) break;
          mma_commit(&bar->q_empty[qs]);  // the segment's queries have been read
        }
        mma_commit(&bar->drain[0]);
        wait_drain_inl(&bar->drain[0], 0, kDrainLimitNs);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ P V issuer
      // O_t += P_t(j) V_j once the softmax of tile t wrote P_t(j)
      if (lane == 0) {
        const uint32_t skv = smem_u32(sKV);
        constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
        int g = 0, cleaned = 0;
        int pv_uses[2] = {0, 0};
        bool ok = true;
        const SpanSeg* at;
#pragma unroll 1
        for (int n = 0; ok && span_segment(bar, n, ctx, at); ++n) {
          const SpanSeg w = *at;
          mbar_arrive(&bar->seg_empty[n % kSpanSegs]);
#pragma unroll 1
          for (int j = w.j1 - 1; ok && j >= w.j0; --j, ++g) {
            const int vs = C::slot(1, g);
            if (!(ok = span_wait(&bar->kv_full[vs], C::use(1, g) & 1, ctx, kSiteCrossV))) break;
            // rows that nobody sees: the warp that loads V zeroes them while P is being formed
            const bool dirty = span_dirty(w, j);
            if (dirty) mbar_arrive(&bar->v_ask);
            const uint64_t vdesc = sdesc_sw128(skv + vs * C::kTileBytes, 16384, 1024);
            const int active = span_active<PAIR>(w, j);
            bool clean = !dirty;
#pragma unroll kIssueUnroll
            for (int t = 0; t < 2; ++t) {
              if (active >> t & 1) {
                int& uses = t ? pv_uses[1] : pv_uses[0];
                if (!span_wait(&bar->p_full[t], uses & 1, ctx, kSiteCrossP) ||
                    (!clean && !span_wait(&bar->v_clean, cleaned & 1, ctx, kSiteCrossClean))) {
                  ok = false;
                  break;
                }
                clean = true;
                tc_fence_after();
                const bool add = j + 1 < (PAIR ? (t ? w.a1[1] : w.a1[0]) : w.j1 - 1);  // not the tile's first product
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_bf16_ts(tmem + (t ? C::kOCol1 : C::kOCol0), tmem + (t ? C::kPCol1 : C::kPCol0) + kk * 8,
                              vdesc + (uint32_t)((kk * 2048) >> 4), id_pv, (add || kk > 0) ? 1u : 0u);
                mma_commit(&bar->pv_done[t]);
                ++uses;
              }
            }
            if (ok && !clean) ok = span_wait(&bar->v_clean, cleaned & 1, ctx, kSiteCrossClean);
            if (!ok) break;
            cleaned += dirty ? 1 : 0;
            mma_commit(&bar->kv_empty[vs]);
          }
        }
        mma_commit(&bar->drain[1]);
        wait_drain_inl(&bar->drain[1], 0, kDrainLimitNs);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<C::kSoftRegs>();
    // ------------------------------------------------------------------ softmax warpgroups
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + ((C::kDualS && t) ? C::kSCol1 : C::kSCol) + lane_off;
    const uint32_t tP = tmem + (t ? C::kPCol1 : C::kPCol0) + lane_off;
    const uint32_t tO = tmem + (t ? C::kOCol1 : C::kOCol0) + lane_off;
    const float cj = MOD == 0 ? p.scale_log2 : 1.f;  // (with MOD the scores are in log2 units)
    int uses = 0;    // blocks this tile has processed over all segments
    int merges = 0;  // ALT: segments whose two accumulators were joined
    bool alive = true;
#pragma unroll 1
    for (int n = 0; alive; ++n) {
      const SpanSeg* seg;
      if (!__all_sync(0xffffffffu, span_segment(bar, n, ctx, seg))) break;
      const volatile SpanSeg& w = *seg;  // (read where it is needed, not kept in registers)
      auto release = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->seg_empty[n % kSpanSegs]);
      };
      // nothing for this tile
      if (PAIR ? (t == 1 && !(w.flags & kSegTwo)) : (t == 1 && w.j1 - w.j0 < 2)) {
        release();
        continue;
      }
      int row_lo, row_hi, pos;
      float slope2 = 0.f;
      bool there = true;  // the row is written
      const int jfirst = (PAIR ? w.a1[t] : w.j1 - t) - 1, jend = PAIR ? w.a0[t] : w.j0;
      const int lo_cut = w.lo_cut[PAIR ? t : 0], hi_cut = w.hi_cut[PAIR ? t : 0];  // blocks that all rows see whole
      {
        const int b = w.b, i = r / p.rows.heads(), token = w.token0 + (PAIR ? p.rows.tokens() * t : 0) + i;
        const int tok = min(token, v.N - 1), len = v.len(b);
        pos = len + tok;
        v.span(b, tok, pos, row_lo, row_hi);
        if (MOD >= 2) there = i < p.rows.tokens() && token < v.rows(b, len);
        if (MOD & 1) slope2 = p.slopes[w.u * p.rows.heads() + r - i * p.rows.heads()] * 1.4426950408889634f;
      }
      float m = -CUDART_INF_F;  // exponent reference (log2 units), a stale running max
      // l: sum of the fp32 probabilities; lcorr: the rounding errors of each
      // block's largest one, so that l + lcorr normalises O (see fa_fwd_kernel)
      float l = 0.f, lcorr = 0.f;
      for (int j = jfirst; j >= jend; j -= PAIR ? 1 : 2, ++uses) {
        if (!__all_sync(0xffffffffu, span_wait(&bar->s_full[t], uses & 1, ctx, kSiteCrossS))) {
          alive = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[4][32];
        float mx_a = 0.f;
        if constexpr (C::kDualS && MOD == 0) {  // two halves: the first's maximum is taken while the second loads
          tmem_ld32(tS, sr[0]);
          tmem_ld32(tS + 32, sr[1]);
          tmem_wait_ld();
          reg_fence32(sr[0]);
          reg_fence32(sr[1]);
          tmem_ld32(tS + 64, sr[2]);
          tmem_ld32(tS + 96, sr[3]);
          mx_a = cross_max64(sr[0], sr[1]);
          tmem_wait_ld();
          reg_fence32(sr[2]);
          reg_fence32(sr[3]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, sr[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) reg_fence32(sr[c]);
        }
        // the scores are in registers: the next scores may now overwrite S
        tc_fence_before();
        mbar_arrive(&bar->s_free[C::kDualS ? t : 0]);

        const int kbase = j * 128;
        const bool cut = kbase < lo_cut || kbase + 128 > hi_cut;
        auto hide = [&](float value) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t bits = span_bits(row_lo - kbase - 32 * c, row_hi - kbase - 32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((bits >> i) & 1u)) sr[c][i] = __float_as_uint(value);
          }
        };
        auto row_max = [&] { return fmaxf(cross_max64(sr[0], sr[1]), cross_max64(sr[2], sr[3])); };
        // MOD 2 and 3: small products are capped by the polynomial, in MOD 2 inside the exponent's
        // argument below; others in place.  What is not seen has no say in it.
        // (That the row sees nothing of the block is asked of its span, not of the maximum: products that it
        // sees may lie below the one that stands for hidden keys, all of them.)
        bool fused = false;
        bool none = false;
        float mx = 0.f;
        if constexpr (MOD >= 2) {
          bool small;
          if (MOD == 2 && p.cap.hidden < 0.f) {
            if (__builtin_expect(cut, 0)) {
              hide(p.cap.hidden);
              none = max(row_lo, kbase) >= min(row_hi, kbase + 128);
            }
            mx = row_max();
            small = mx <= p.cap.small && (mx >= p.cap.low || none);
          } else {
            mx = row_max();
            small = !cut && span_absmax(sr) <= p.cap.small;
          }
          small = __all_sync(0xffffffffu, !there || small);
          fused = MOD == 2 && small;
          if (MOD == 3 && __builtin_expect(small, 1)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) span_cap32_small(sr[c], p.cap);
          } else if (__builtin_expect(!small, 0)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) span_cap32(sr[c], p.cap);
            if (cut) hide(-CUDART_INF_F);
            mx = row_max();
          }
          if constexpr (MOD == 3) {
            span_bias(sr, 1.f, slope2, pos - kbase, PAGED || v.causal);
            mx = row_max();
          }
        } else {
          if constexpr (MOD == 1) span_bias(sr, p.scale_log2, slope2, pos - kbase, PAGED || v.causal);
          if (__builtin_expect(cut, 0)) hide(-CUDART_INF_F);
          if constexpr (C::kDualS && MOD == 0)
            mx = fmaxf(cut ? cross_max64(sr[0], sr[1]) : mx_a, cross_max64(sr[2], sr[3]));
          else
            mx = row_max();
        }
        // mx cmx: the largest score; a row that sees nothing of the block has none
        const float cmx = MOD == 2 && fused ? span_cap_small(make_float2(mx, mx), p.cap).x : cj;
        if (MOD == 2 && none) mx = -CUDART_INF_F;
        const float m_new = fmaxf(m, mx * cmx);
        // conditional rescale: the reference moves only when the row maximum
        // rose by more than the threshold (always from -inf: no key so far)
        float alpha = 1.f;
        bool rescale_warp = false;
        if (j == jfirst) {
          m = m_new;
        } else {
          const bool need = (m_new - m) > kRescaleThresholdLog2;
          rescale_warp = __any_sync(0xffffffffu, need);
          if (need) {
            alpha = ex2_approx(m - m_new);
            m = m_new;
          }
        }
        // (finite for a row without keys so far, whose every P is 2^-inf, or of hidden products, = 0)
        const float ref = MOD == 2 ? (m == -CUDART_INF_F ? 0.f : m) : fmaxf(m, -3.402823466e38f);
        const float2 c2 = make_float2(cj, cj);
        const float2 mneg2 = make_float2(-ref, -ref);
        float2 acc[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) acc[a] = make_float2(0.f, 0.f);
        {
          const float pbm = ex2_approx(fmaf(mx, cmx, -ref));
          const float pbm_r = __uint_as_float(pack_bf16x2(pbm, 0.f) << 16);
          lcorr = lcorr * alpha + (pbm_r - pbm);
        }
        uint32_t pk[4][16];
        auto exponentials = [&](auto capped) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 s2 = make_float2(__uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1]));
              const float2 x = capped.value ? __ffma2_rn(s2, span_cap_small(s2, p.cap), mneg2)
                               : MOD == 0   ? __ffma2_rn(s2, c2, mneg2)
                                            : __fadd2_rn(s2, mneg2);
              const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
              pk[c][i] = pack_bf16x2(p0, p1);
              acc[i & 3] = __fadd2_rn(acc[i & 3], make_float2(p0, p1));
            }
          }
        };
        if (MOD == 2 && __builtin_expect(fused, 1))
          exponentials(std::true_type{});
        else
          exponentials(std::false_type{});
        const float2 accs = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        l = l * alpha + (accs.x + accs.y);
        // P_t and O_t are in use until the tile's previous product has completed
        // (a segment's first block: its predecessor's epilogue has waited for
        // it; ALT: O_1 also until warpgroup 0 has read it)
        if (j < jfirst) {
          if (!__all_sync(0xffffffffu, span_wait(&bar->pv_done[t], (uses - 1) & 1, ctx, kSiteCrossPv))) {
            alive = false;
            break;
          }
          tc_fence_after();
        } else if (!PAIR && t == 1 && merges > 0) {
          if (!__all_sync(0xffffffffu, span_wait(&bar->merge_free, (merges - 1) & 1, ctx, kSiteCrossMerge))) {
            alive = false;
            break;
          }
          tc_fence_after();
        }
        if (__builtin_expect(rescale_warp, 0)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(tO + 32 * c, ov);
            tmem_wait_ld();
            reg_fence32(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(tO + 32 * c, ov);
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(tP + 16 * c, pk[c]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar->p_full[t]);
      }
      if (!alive) break;
      if (!__all_sync(0xffffffffu, span_wait(&bar->pv_done[t], (uses - 1) & 1, ctx, kSiteCrossPv))) {
        alive = false;
        break;
      }
      tc_fence_after();
      // ---- end of the segment
      const int flags = w.flags;
      const bool seg_first = flags & kSegFirst, whole = seg_first && (flags & kSegLast);
      const bool join = !PAIR && w.j1 - w.j0 >= 2;
      float lo = l + lcorr, a0 = 1.f, a1 = 0.f;
      if (join) {
        if (t == 1) {
          sMerge[r] = m;
          sMerge[128 + r] = l;
          sMerge[256 + r] = lo;
          tc_fence_before();
          mbar_arrive(&bar->merge_ready);
          ++merges;
          release();
          continue;
        }
        if (!__all_sync(0xffffffffu, span_wait(&bar->merge_ready, merges & 1, ctx, kSiteCrossMerge))) {
          alive = false;
          break;
        }
        tc_fence_after();
        ++merges;
        const float m1 = sMerge[r], mm = fmaxf(m, m1), ref = mm == -CUDART_INF_F ? 0.f : mm;
        a0 = ex2_approx(m - ref);
        a1 = ex2_approx(m1 - ref);
        l = l * a0 + sMerge[128 + r] * a1;
        lo = lo * a0 + sMerge[256 + r] * a1;
        m = mm;
      }
      const float inv = lo == 0.f ? 0.f : 1.f / lo;
      a0 *= inv;
      a1 *= inv;
      const float lse2 = l == 0.f ? -CUDART_INF_F : m + log2f(l);
      const int of_tile = r / p.rows.heads(), token = w.token0 + (PAIR ? p.rows.tokens() * t : 0) + of_tile;
      const bool write = of_tile < p.rows.tokens() && token < v.rows(w.b, v.len(w.b));
      const size_t grow = p.rows.row(w.b, w.u, r - of_tile * p.rows.heads(), token);
      const size_t prow = ((size_t)2 * blockIdx.x + (seg_first ? 1 : 0)) * p.part_rows + (PAIR ? 128 * t : 0) + r;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32], ow[32];
        tmem_ld32(tO + 32 * c, ov);
        if (join) tmem_ld32(tmem + C::kOCol1 + lane_off + 32 * c, ow);
        tmem_wait_ld();
        reg_fence32(ov);
        if (join) {
          reg_fence32(ow);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            ov[i] = __float_as_uint(fmaf(__uint_as_float(ow[i]), a1, __uint_as_float(ov[i]) * a0));
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * a0);
        }
        if (join && c == D / 32 - 1) {
          tc_fence_before();
          mbar_arrive(&bar->merge_free);
        }
        if (write && whole) {
          __nv_bfloat16* orow = p.o + grow * D + 32 * c;
          uint32_t w16[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w16[e] = pack_bf16x2(__uint_as_float(ov[2 * e]), __uint_as_float(ov[2 * e + 1]));
          if (p.o_align32) {
            st_global_v8(orow, w16);
            st_global_v8(orow + 16, w16 + 8);
          } else {
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
              reinterpret_cast<uint4*>(orow)[v4] =
                  make_uint4(w16[4 * v4], w16[4 * v4 + 1], w16[4 * v4 + 2], w16[4 * v4 + 3]);
          }
        } else if (write) {
          float* prow_o = p.part_o + prow * D + 32 * c;
#pragma unroll
          for (int v8 = 0; v8 < 4; ++v8) st_global_v8(prow_o + 8 * v8, ov + 8 * v8);
        }
        __syncwarp();  // the next tensor memory load is a whole warp's
      }
      if (write) {
        if (whole)
          p.lse[grow] = lse2 * 0.6931471805599453f;
        else
          p.part_lse[prow] = lse2;
      }
      release();
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the parts of the items that share ends cut: block x takes the item that
// begins in CTA x's share and goes on behind it, kRows rows per warp.  O = sum of
// the parts' O weighted by 2^(their LSE - the largest), in CTA order.
template <int D, bool PAIR, bool PAGED>
__global__ void __launch_bounds__(256) fa_span_combine_kernel(const __grid_constant__ SpanFwdParams<PAGED> p) {
  constexpr int E = D / 32;
  constexpr int kRows = PAIR ? 4 : 1;  // rows of a warp
  constexpr int kBatch = 8;            // parts whose loads are in flight together
  grid_wait();
  grid_trigger();
  const SpanMeta meta = p.meta[blockIdx.x];
  if (!meta.split) return;
  const SpanView<PAGED>& v = p.rows.view;
  const int parts = (int)((meta.last * min((long long)gridDim.x, meta.total) - 1) / meta.total) - (int)blockIdx.x + 1;
  const int lane = threadIdx.x & 31, local0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kRows;
  const int fresh = v.rows(meta.b, v.len(meta.b));
  // part i: the last segment of CTA x, then the first of each CTA after it
  auto part = [&](int i) { return ((size_t)2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * p.part_rows + local0; };
  for (int r = 0; r < kRows; ++r) {
    const int local = local0 + r, second = PAIR ? local >> 7 : 0, of_tile = (local - second * 128) / p.rows.heads();
    const int token = meta.token0 + second * p.rows.tokens() + of_tile;
    if (local >= p.part_rows || of_tile >= p.rows.tokens() || token >= fresh) continue;
    const size_t grow = p.rows.row(meta.b, meta.u, local - second * 128 - of_tile * p.rows.heads(), token);
    float acc[E], sum = 0.f, ref = -CUDART_INF_F;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < parts; i0 += kBatch) {
      float l[kBatch], o[kBatch][E];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        l[u] = -CUDART_INF_F;
        if (i0 + u < parts) {
          l[u] = p.part_lse[part(i0 + u) + r];
          cross_join_load<E>(p.part_o + (part(i0 + u) + r) * D + lane * E, o[u]);
        }
      }
      float mx = ref;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) mx = fmaxf(mx, l[u]);
      // finite where no part so far has a key; `ref` stays -inf there, so that parts
      // of any low log-sum-exp count
      const float safe = fmaxf(mx, -3.402823466e38f);
      const float alpha = ex2_approx(ref - safe);
      ref = mx;
      sum *= alpha;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= alpha;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (i0 + u < parts) {
          const float wt = ex2_approx(l[u] - safe);
          sum += wt;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, o[u][e], acc[e]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t* orow = reinterpret_cast<uint32_t*>(p.o + grow * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) orow[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0) p.lse[grow] = (sum == 0.f ? -CUDART_INF_F : ref + log2f(sum)) * 0.6931471805599453f;
  }
}

}  // namespace fa
