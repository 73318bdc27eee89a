// Forward kernel for keys of another length than the queries: cross attention
// and attention over a cache (see CrossView in fa_cross.cuh).
//
// The arithmetic and the pipeline are those of fa_fwd_kernel: TMA fills a ring
// of K and V tiles, one thread issues S = Q K^T, one O += P V, and two softmax
// warpgroups hold a row of scores per thread.  What differs:
//
// Work.  The keys of every (request, key/value head, row tile) are cut into
// blocks of 128; all items' blocks, each item's after a place or two for what a
// segment costs at its ends, form one sequence, and CTA c of G takes the places
// [c Tot / G, (c + 1) Tot / G) of it: the CTAs' shares are even whatever the
// requests' lengths, and few rows over many keys use every SM.  An item that
// lies within one CTA's share is written directly; one cut by a share's end
// leaves a normalised fp32 O and a log-sum-exp per row and part (at most two
// parts per CTA) that fa_cross_combine_kernel joins in CTA order.
//
// The two softmax warpgroups.  With more than 128 rows per key/value head
// (PAIR) they take two row tiles that share each key block, as in
// fa_fwd_kernel.  With up to 128 rows (ALT) there is one row tile and they take
// its key blocks in turn, each with its own maximum, sum and accumulator; at
// the end warpgroup 0 joins the two, reading O_1 from the same TMEM lanes.
//
// A few items (CLUSTER, with ALT): 2, 4 or 8 CTAs of a cluster share an item's
// key blocks and join their parts through one another's shared memory, without
// parts in global memory and without the second kernel.
//
// Keys behind a request's length.  Their scores become -inf; their rows of V
// (which may hold anything, and 0 times NaN is NaN) are zeroed in shared
// memory by warp 11 before the last block's P V.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "fa_cross.cuh"
#include "fa_fwd.cuh"

namespace fa {

constexpr int kCrossMaxCtas = 152;  // the grid's bound: one CTA per SM

struct CrossMeta {   // of each CTA, for the combine kernel
  int split;         // its last item goes on in the next CTA
  int b, it;         // that item
  int fresh;         // drafted tokens of the request (TREE)
  long long last;    // the place behind the item's last block
  long long total;   // places of the sequence
};

struct CrossFwdParams {
  CrossView view;
  __nv_bfloat16* o;
  float* lse;
  CrossMeta* meta;       // [grid]
  float* part_lse;       // [2 grid][part_rows], base 2
  float* part_o;         // [2 grid][part_rows][d]
  int part_rows;         // rows of a part: 256 (PAIR) or R (ALT)
  int B;
  int row_tiles;         // row tiles (PAIR: pairs of them) per key/value head
  int cluster;           // CLUSTER: CTAs per item
  float scale_log2;
  uint64_t wait_limit_ns;
  int debug_stall;
  int o_align32;
};

// key blocks of a request: at least one, so that rows without keys are written
__device__ __forceinline__ int cross_blocks(int keys) { return keys > 128 ? (keys + 127) >> 7 : 1; }

// What a segment costs beyond its blocks (queries, first scores, epilogue), in
// blocks: each item takes kCrossStart places of the sequence before its blocks.
// (Measured, 2 and 4: eight requests of 24 drafts over caches of 600 to 8100
// tokens 43.0 and 41.6 us; the other shapes within 2 %.)
constexpr int kCrossStart = 4;

// What cutting items costs at the end (parts written, read and joined), in places.
// (Measured, 5, 9 and 13: B=4 H=32/8 Nq=Nk=1024 d=128 80.5, 74.4 and 74.4 us;
// B=1 H=8 Nq=1 Nk=1500 d=64 17.0, 16.0 and 16.7 us.)
constexpr int kCrossCut = 9;

// Whether the CTAs take whole items, ceil(items / ctas) at most: where that
// ends no later than even shares and the join of what they cut.
__host__ __device__ __forceinline__ bool cross_whole(int items, int ctas, int most, long long total) {
  const long long turns = ((unsigned)items + (unsigned)ctas - 1u) / (unsigned)ctas;
  return (turns * most - kCrossCut) * ctas <= total;
}

// Where all items cost the same and there are enough of them, CTA c takes the
// items c, c + G, ... of the full rounds: the CTAs of a round work on few heads
// together, whose keys they share through L2.  (In contiguous shares every head
// is read at the same time: B=2 H=32 Nq=Nk=4096 d=128 takes 390 instead of
// 364 us.)  The `rest` items of the last round: as single row tiles
// where these fit the CTAs, whole, or cut evenly.
enum : int { kCrossTailWhole, kCrossTailSingle, kCrossTailCut };
__host__ __device__ __forceinline__ int cross_tail(int rest, int ctas, int places, bool pair) {
  if (pair && rest > 0 && 2 * rest <= ctas) return kCrossTailSingle;
  return rest == 0 || (long long)(places - kCrossCut) * ctas <= (long long)rest * places ? kCrossTailWhole : kCrossTailCut;
}

// CTAs per item in a cluster (1: no clusters), for items of at most 128 rows: the
// largest size whose clusters of all items the device holds at once, where that
// ends no later than whole items or even shares and their join.  The join costs
// a place and one for each 32 rows in a cluster, 15 places with its kernel.  Where
// lengths may differ the host only knows that no item has more than `blocks`: clusters
// for few of them.
// (Measured at 33 numbers of items from 1 to 76, 256 to 32k keys, 1 and 128 rows: 0.8 %
// above the best of no clusters and of 2, 4 and 8 on average, 21 % at most.  Without
// and with clusters, d = 128, one row: 8 items, 2048 keys 19 and 15 us, 16k 31 and
// 31, 32k 44 and 50; 33 items, 2048 keys 24 and 19; 15 items, 8192 keys 29 and 25;
// 16, one more than the device holds clusters of 8, 31 and 38.)
struct CrossClusterFit {
  int clusters[3];  // of 8, 4 and 2 CTAs
};
inline int cross_cluster(long long items, int blocks, int rows, bool alike, int sms, const CrossClusterFit& fit) {
  for (int i = 0; i < 3; ++i) {
    const int ctas = 8 >> i;
    if (items > fit.clusters[i]) continue;
    if (!alike) return blocks > 1 && blocks <= 4 * ctas ? ctas : 1;
    const long long places = blocks + kCrossStart;
    long long apart = items * places / sms + 15;
    if (items <= sms && places < apart) apart = places;
    return blocks > 1 && (blocks + ctas - 1) / ctas + kCrossStart + 1 + rows / 32 <= apart ? ctas : 1;
  }
  return 1;
}

// A CTA's work: places of the sequence of items' places, one item after another
// or every step-th, and then, maybe, a second run of them.
struct CrossPlace {
  int b, it, j;    // request, item of it (head, row tile), place in the item
  int step;        // from one item to the next
  int single;      // PAIR: one row tile (0 or 1) of each item; -1: both
  int more;        // another run follows
  long long left;  // places of this run from there on
};

// A run of key blocks of one item.
struct CrossSeg {
  int b, it, j0, j1, n;
  int len, keys;  // the request's own keys; with its drafts
  int single;     // as in CrossPlace
  __device__ __forceinline__ bool first() const { return j0 == 0; }
  __device__ __forceinline__ bool last() const { return j1 == n; }
  // the last block's rows of V behind the keys hold anything (past Nk the TMA fills zeros)
  __device__ __forceinline__ bool dirty(const CrossView& v) const { return last() && keys < (n << 7) && keys < v.Nk; }
};

// The next segment of the CTA's work; `second`: the run after the first.
__device__ __forceinline__ bool cross_next(const CrossView& v, int items, const CrossPlace* second, CrossPlace& at,
                                           CrossSeg& s) {
  for (;;) {
    if (at.left <= 0) {
      if (!at.more) return false;
      at = *second;
      if (at.left <= 0) return false;
    }
    s.b = at.b;
    s.it = at.it;
    s.single = at.single;
    s.len = v.len(at.b);
    s.keys = s.len + v.drafted(at.b, s.len);
    s.n = cross_blocks(s.keys);
    const int end = (int)min((long long)s.n + kCrossStart, at.j + at.left);
    s.j0 = max(at.j - kCrossStart, 0);
    s.j1 = end - kCrossStart;
    at.left -= end - at.j;
    at.j = end;
    if (at.j == s.n + kCrossStart) {
      at.j = 0;
      at.it += at.step;
      if (at.it >= items) {
        const int over = at.step == 1 ? 1 : at.it / items;
        at.b += over;
        at.it -= over * items;
      }
    }
    if (s.j1 > 0) return true;  // (else only places before the item's blocks)
  }
}

// a b / c, in 32 bits where they hold the product (64-bit divisions take a
// quarter of a microsecond of the start)
__device__ __forceinline__ long long cross_share(int a, long long b, int c) {
  if (b < (1 << 23)) return (uint32_t)a * (uint32_t)b / (uint32_t)c;  // a <= 152
  return a * b / c;
}

// The work of CTA `cta` of at most `ctas`, by one warp.  (The numbers of places
// of all requests fit 32 bits, with the items' not: the shape checks bound them.)
template <bool PAIR>
__device__ __forceinline__ void cross_schedule(const CrossView& v, int B, int items, int cta, int ctas,
                                               CrossPlace* place, CrossPlace* second, long long* all,
                                               long long* share_end) {
  const int lane = threadIdx.x & 31;
  const int count = B * items;
  auto places = [&](int b) {
    const int len = v.len(b);
    return cross_blocks(len + v.drafted(b, len)) + kCrossStart;
  };
  // places of this lane's requests, and of all before them
  const int chunk = (B + 31) / 32, b0 = min(B, lane * chunk), b1 = min(B, b0 + chunk);
  int mine = 0, upto = 0, sum, most, least;
  const bool alike = B == 1 || !v.lens;
  if (alike) {
    most = least = places(0);
    sum = B * most;
  } else {
    most = 0, least = 0x7fffffff;
    for (int b = b0; b < b1; ++b) {
      const int n = places(b);
      mine += n;
      most = max(most, n);
      least = min(least, n);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int add = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += add;
    }
    sum = __shfl_sync(0xffffffffu, upto, 31);
  }
  const long long total = (long long)sum * items;
  CrossPlace x{0, 0, 0, 1, -1, 0, 0};
  // a share of `count` items from `item` on, all of `most` places
  auto share = [&](int item, long long of) {
    const int g = (int)min((long long)ctas, of);
    if (cta < g) {
      const long long start = cross_share(cta, of, g), end = cross_share(cta + 1, of, g);
      const int skip = start < (1ll << 31) ? (int)((uint32_t)start / (uint32_t)most) : (int)(start / most);
      item += skip;
      x.j = (int)(start - (long long)skip * most);
      x.left = end - start;
      if (lane == 0) {
        *all = of;
        *share_end = end;
      }
    }
    return item;
  };
  auto put = [&](CrossPlace* to, int item) {
    x.b = item / items;
    x.it = item - x.b * items;
    if (lane == 0) *to = x;
  };
  if (most == least && count >= ctas) {
    const int full = count / ctas, rest = count - full * ctas;
    const int tail = cross_tail(rest, ctas, most, PAIR);
    x.step = ctas;
    x.left = (long long)(full + (tail == kCrossTailWhole && cta < rest ? 1 : 0)) * most;
    x.more = tail != kCrossTailWhole;
    put(place, cta);
    if (tail == kCrossTailWhole) return;
    int item = full * ctas;
    x = {0, 0, 0, 1, -1, 0, 0};
    if (tail == kCrossTailSingle) {
      item += cta >> 1;
      x.single = cta & 1;
      const int row0 = (item % items % ((v.R + 255) / 256)) * 256 + 128 * x.single;
      if (cta < 2 * rest && row0 < v.R) x.left = most;
    } else {
      item = share(item, (long long)rest * most);
    }
    put(second, item);
    return;
  }
  if (alike) {
    int item = cta;
    if (cross_whole(count, ctas, most, total))
      x.left = cta < count ? most : 0;
    else
      item = share(0, total);
    put(place, item);
    return;
  }
  if (cross_whole(count, ctas, most, total)) {
    if (lane == 0) {
      int at = (int)((long long)cta * count / ctas), left = (int)((cta + 1LL) * count / ctas) - at;
      x.b = at / items;
      x.it = at - x.b * items;
      for (int b = x.b, it = x.it; left > 0; ++b, it = 0) {  // the places of those items
        const int take = min(left, items - it);
        x.left += (long long)take * places(b);
        left -= take;
      }
      *place = x;
    }
    return;
  }
  const int g = (int)min((long long)ctas, total);
  if (cta >= g) {
    if (lane == 0) *place = x;
    return;
  }
  const long long start = cross_share(cta, total, g), end = cross_share(cta + 1, total, g);
  if (lane == 0) {
    *all = total;
    *share_end = end;
  }
  long long at = (long long)(upto - mine) * items;
  if (start >= at && start < (long long)upto * items) {
    for (int b = b0; b < b1; ++b) {
      const int n = places(b);
      if (start < at + (long long)n * items) {
        const long long off = start - at;
        x.b = b;
        x.it = off < (1ll << 31) ? (int)((uint32_t)off / (uint32_t)n) : (int)(off / n);
        x.j = (int)(off - (long long)x.it * n);
        x.left = end - start;
        *place = x;
        break;
      }
      at += (long long)n * items;
    }
  }
}

// A segment's first row, and (PAIR) whether it has a second row tile.
template <bool PAIR>
__device__ __forceinline__ int cross_row0(const CrossSeg& w, int row_tiles) {
  return (w.it % row_tiles) * (PAIR ? 256 : 128) + (PAIR && w.single > 0 ? 128 : 0);
}
template <bool PAIR>
__device__ __forceinline__ bool cross_two(const CrossSeg& w, int row0, int R) {
  return PAIR && w.single < 0 && row0 + 128 < R;
}

template <int D>
struct CrossCfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kAtoms = D / 64;
  static constexpr int kThreads = 384;
  static constexpr int kLaunchRegs = 168;
  static constexpr uint32_t kSoftRegs = D == 64 ? 216 : 208;
  static constexpr uint32_t kMiscRegs = 3 * kLaunchRegs - 2 * kSoftRegs;
  static_assert(kSoftRegs % 8 == 0 && kMiscRegs % 8 == 0 && kMiscRegs >= 24 && kSoftRegs > kLaunchRegs,
                "2 kSoftRegs + kMiscRegs = the three warpgroups' launch budget");
  static constexpr bool kDualS = D == 64;
  static constexpr int kSlots = D == 128 ? 5 : 12;
  // Ring slot and use of key block g's K (kv = 0) or V tile (g counts over the
  // CTA's segments).  K and V have slots of their own (3 and 2 at d = 128), so that
  // each issuer waits for every tile that its slots take: a wait by parity cannot
  // take the phase before last for its own.
  static constexpr int kKSlots = (kSlots + 1) / 2, kVSlots = kSlots / 2;
  static __device__ __forceinline__ int slot(int kv, int g) { return kv ? kKSlots + g % kVSlots : g % kKSlots; }
  static __device__ __forceinline__ int use(int kv, int g) { return g / (kv ? kVSlots : kKSlots); }
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kSCol = 0, kPCol0 = 128, kPCol1 = 192, kOCol0 = 256, kOCol1 = 256 + D;
  static constexpr uint32_t kSCol1 = kDualS ? kOCol1 + D : kSCol;
  static_assert((kDualS ? kSCol1 + 128 : kOCol1 + D) <= kTmemCols, "tensor memory budget");
  static constexpr int kMergeBytes = 3 * 128 * 4;
  // (declared 1024-byte aligned, which is checked at run time)
  static constexpr int kSmemBytes = 2 * kTileBytes + kSlots * kTileBytes + kMergeBytes + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(128 * (D + 4) * 4 <= kSlots * kTileBytes, "a cluster's parts take the ring's place");
};

struct CrossBarriers {
  uint64_t q_full[2], q_empty[2];  // PAIR: both tiles by [0]; ALT: the segments' queries in turn
  uint64_t kv_full[12], kv_empty[12];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  // an item's last V tile has landed: warp 11 may zero its rows behind the
  // keys; they are zero.  (The P V issuer asks: warp 11 could not wait for the
  // tile's own barrier, whose phases go on while it waits for nothing.)
  uint64_t v_ask, v_clean;
  uint64_t merge_ready, merge_free;    // ALT: warpgroup 1's sums are in place; O_1 has been read
  uint64_t drain[2];
  uint64_t never;
  CrossPlace place, second;
  long long total, end;  // places of the sequence; end of the CTA's share
  int fresh;             // CLUSTER: drafted tokens of the item's request
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(CrossBarriers) <= 512, "barriers overflow their shared-memory slot");

// A softmax warp's place and segment, kept here while its registers hold scores.
struct CrossWarp {
  CrossPlace at;
  CrossSeg w;
};
static_assert(sizeof(CrossWarp) <= 64, "512 bytes for eight warps");

enum : int { kSiteCrossQEmpty = 40, kSiteCrossKvEmpty, kSiteCrossQ, kSiteCrossK, kSiteCrossSFree, kSiteCrossV,
             kSiteCrossClean, kSiteCrossP, kSiteCrossS, kSiteCrossPv, kSiteCrossMerge, kSiteCrossTail };

// the maximum of 64 scores: a tree of 3-input maxima
__device__ __forceinline__ float cross_max64(const uint32_t* x, const uint32_t* y) {
  float t1[22];
#pragma unroll
  for (int i = 0; i < 21; ++i) {
    const int e = 3 * i;
    t1[i] = max3(__uint_as_float(e < 32 ? x[e] : y[e - 32]), __uint_as_float(e + 1 < 32 ? x[e + 1] : y[e - 31]),
                 __uint_as_float(e + 2 < 32 ? x[e + 2] : y[e - 30]));
  }
  t1[21] = __uint_as_float(y[31]);
  float t2[8];
#pragma unroll
  for (int i = 0; i < 7; ++i) t2[i] = max3(t1[3 * i], t1[3 * i + 1], t1[3 * i + 2]);
  t2[7] = t1[21];
  return max3(max3(t2[0], t2[1], t2[2]), max3(t2[3], t2[4], t2[5]), fmaxf(t2[6], t2[7]));
}

// 32 bits of what a row sees, from key `rel` keys behind the request's own
__device__ __forceinline__ uint32_t cross_bits(unsigned long long mask, int rel) {
  if (rel <= -32) return 0xffffffffu;
  if (rel < 0) return ((1u << -rel) - 1u) | (uint32_t)(mask << -rel);
  return rel < 64 ? (uint32_t)(mask >> rel) : 0u;
}

// The share of a cluster's item, by one lane.
__device__ __forceinline__ void cross_cluster_share(const CrossView& v, int items, int ctas, CrossPlace* place,
                                                    int* fresh) {
  const int item = blockIdx.x / ctas, rank = blockIdx.x - item * ctas;
  const int b = item / items, len = v.len(b), drafted = v.drafted(b, len);
  const int n = cross_blocks(len + drafted), j0 = rank * n / ctas, j1 = (rank + 1) * n / ctas;
  *place = {b, item - b * items, j0 + kCrossStart, 1, -1, 0, j1 - j0};
  *fresh = drafted;
}

// fp32 values of shared memory of CTA `rank` of the cluster
__device__ __forceinline__ float cluster_load(const float* local, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(local), rank)));
  return v;
}
template <int E>
__device__ __forceinline__ void cluster_load(const float* local, uint32_t rank, float (&x)[E]) {
  const uint32_t at = mapa_shared(smem_u32(local), rank);
  if constexpr (E == 4)
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                 : "r"(at));
  else
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(at));
}

// TREE: drafted tokens behind the request's own.  PAIR: two row tiles per item.
// CLUSTER: a cluster of p.cluster CTAs per item (not with PAIR).
template <int D, bool TREE, bool PAIR, bool CLUSTER>
__global__ void __launch_bounds__(384, 1)
    fa_cross_fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const CrossFwdParams p) {
  using C = CrossCfg<D>;
  static_assert(!(PAIR && CLUSTER), "clusters take one row tile");
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
  uint8_t* smem = smem_raw;
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * C::kTileBytes;
  float* sMerge = reinterpret_cast<float*>(sKV + C::kSlots * C::kTileBytes);  // [3][128]
  CrossBarriers* bar = reinterpret_cast<CrossBarriers*>(reinterpret_cast<uint8_t*>(sMerge) + C::kMergeBytes);
  uint8_t* sWarps = reinterpret_cast<uint8_t*>(bar) + 512;  // CrossWarp of each softmax warp, 64 bytes apart
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CrossView& v = p.view;
  const int items = v.Hkv * p.row_tiles;

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
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bar->kv_full[s], 1);
      mbar_init(&bar->kv_empty[s], 1);
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
  if (CLUSTER) {
    if (tid < 128) sMerge[tid] = -CUDART_INF_F;  // no part so far
    if (warp == 10 && lane == 0) cross_cluster_share(v, items, p.cluster, &bar->place, &bar->fresh);
  } else if (warp == 10)
    cross_schedule<PAIR>(v, p.B, items, blockIdx.x, gridDim.x, &bar->place, &bar->second,
                         &bar->total, &bar->end);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_trigger();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtx ctx{&bar->abort_flag, p.wait_limit_ns};
  CrossPlace at = bar->place;  // every role walks the same segments
  CrossSeg w;

  if (warp >= 8) {
    setmaxnreg_dec<C::kMiscRegs>();
    if (warp == 9) {
      // ------------------------------------------------------------------ TMA producer
      if (lane == 0) {
        int loads = 0, nq = 0;  // K and V tiles, in turn
        bool ok = true;
        auto load_kv = [&](int j, int kv, int bk) -> bool {
          const int g = loads >> 1, s = C::slot(kv, g);
          const CUtensorMap* map = kv ? &map_v : &map_k;
          if (!wait_bounded_inl(&bar->kv_empty[s], (C::use(kv, g) & 1) ^ 1, ctx, kSiteCrossKvEmpty))
            return false;
          mbar_arrive_expect_tx(&bar->kv_full[s], C::kTileBytes);
          for (int a = 0; a < C::kAtoms; ++a)
            tma_load_3d(sKV + s * C::kTileBytes + a * 16384, map, &bar->kv_full[s], a * 64, j * 128, bk);
          ++loads;
          return true;
        };
        while (ok && cross_next(v, items, &bar->second, at, w)) {
          const int kvh = w.it / p.row_tiles;
          const int row0 = cross_row0<PAIR>(w, p.row_tiles);
          const int bk = w.b * v.Hkv + kvh;
          const int qs = PAIR ? 0 : nq & 1, use = PAIR ? nq : nq >> 1;
          const int tiles = cross_two<PAIR>(w, row0, v.R) ? 2 : 1;
          auto load_q = [&] {
            mbar_arrive_expect_tx(&bar->q_full[qs], tiles * C::kTileBytes);
            for (int t = 0; t < tiles; ++t)
              for (int a = 0; a < C::kAtoms; ++a)
                tma_load_3d(sQ + (PAIR ? t : qs) * C::kTileBytes + a * 16384, &map_q, &bar->q_full[qs], a * 64,
                            row0 + 128 * t, bk);
          };
          // a later segment's first key block needs only ring slots: it goes out
          // before the queries, whose buffer an earlier segment may still be reading
          if (nq == 0) load_q();
          ok = load_kv(w.j0, 0, bk) && load_kv(w.j0, 1, bk);
          if (!ok) break;
          if (nq > 0) {
            if (use > 0 && !(ok = wait_bounded_inl(&bar->q_empty[qs], (use - 1) & 1, ctx, kSiteCrossQEmpty))) break;
            load_q();
          }
          ++nq;
          for (int j = w.j0 + 1; ok && j < w.j1; ++j) ok = load_kv(j, 0, bk) && load_kv(j, 1, bk);
        }
        // every copy this thread started must land before the CTA can exit
        for (int s = 0; s < 2; ++s) {
          const int uses = PAIR ? (s ? 0 : nq) : (nq + 1 - s) >> 1;
          if (uses > 0) wait_drain_inl(&bar->q_full[s], (uses - 1) & 1, kDrainLimitNs);
        }
        for (int s = 0; s < C::kSlots; ++s) {
          // loads into slot s
          const bool vslot = s >= C::kKSlots;
          const int n = vslot ? loads >> 1 : (loads + 1) >> 1, first = vslot ? s - C::kKSlots : s;
          if (n > first) wait_drain_inl(&bar->kv_full[s], C::use(vslot, n - 1 - first) & 1, kDrainLimitNs);
        }
      }
      __syncwarp();
    } else if (warp == 8) {
      // ------------------------------------------------------------------ S issuer
      // g counts key blocks over all segments
      if (lane == 0) {
        const uint32_t sq = smem_u32(sQ), skv = smem_u32(sKV);
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
        int s_uses[2] = {0, 0}, g = 0, nq = 0;
        bool ok = !(p.debug_stall && !wait_bounded_inl(&bar->never, 0, ctx, kSiteStall));
        while (ok && cross_next(v, items, &bar->second, at, w)) {
          const int qs = PAIR ? 0 : nq & 1, use = PAIR ? nq : nq >> 1;
          if (!wait_bounded_inl(&bar->q_full[qs], use & 1, ctx, kSiteCrossQ)) break;
          ++nq;
          const bool two = cross_two<PAIR>(w, cross_row0<PAIR>(w, p.row_tiles), v.R);
          for (int j = w.j0; ok && j < w.j1; ++j, ++g) {
            const int ks = C::slot(0, g);
            if (!(ok = wait_bounded_inl(&bar->kv_full[ks], C::use(0, g) & 1, ctx, kSiteCrossK))) break;
            const uint64_t kdesc = sdesc_sw128(skv + ks * C::kTileBytes, 16, 1024);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (PAIR ? (t == 0 || two) : (((j - w.j0) & 1) == t)) {
                const int sb = C::kDualS ? t : 0;
                if (s_uses[sb] > 0 && !wait_bounded_inl(&bar->s_free[sb], (s_uses[sb] - 1) & 1, ctx, kSiteCrossSFree)) {
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
                ++s_uses[sb];
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
    } else if (warp == 10) {
      // ------------------------------------------------------------------ P V issuer
      // O_t += P_t(j) V_j once the softmax of tile t wrote P_t(j)
      if (lane == 0) {
        const uint32_t skv = smem_u32(sKV);
        constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
        int g = 0, cleaned = 0;
        int pv_uses[2] = {0, 0};
        bool ok = true;
        while (ok && cross_next(v, items, &bar->second, at, w)) {
          const bool two = cross_two<PAIR>(w, cross_row0<PAIR>(w, p.row_tiles), v.R);
          const bool dirty = w.dirty(v);
          for (int j = w.j0; ok && j < w.j1; ++j, ++g) {
            const int vs = C::slot(1, g);
            if (!(ok = wait_bounded_inl(&bar->kv_full[vs], C::use(1, g) & 1, ctx, kSiteCrossV))) break;
            bool clean = !(dirty && j == w.n - 1);
            if (!clean) mbar_arrive(&bar->v_ask);
            const uint64_t vdesc = sdesc_sw128(skv + vs * C::kTileBytes, 16384, 1024);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (PAIR ? (t == 0 || two) : (((j - w.j0) & 1) == t)) {
                if (!wait_bounded_inl(&bar->p_full[t], pv_uses[t] & 1, ctx, kSiteCrossP)) {
                  ok = false;
                  break;
                }
                if (!clean) {
                  if (!(ok = wait_bounded_inl(&bar->v_clean, cleaned & 1, ctx, kSiteCrossClean))) break;
                  ++cleaned;
                  clean = true;
                }
                tc_fence_after();
                const bool add = j > w.j0 + (PAIR ? 0 : 1);  // not the tile's first block of the segment
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_bf16_ts(tmem + (t ? C::kOCol1 : C::kOCol0), tmem + (t ? C::kPCol1 : C::kPCol0) + kk * 8,
                              vdesc + (uint32_t)((kk * 2048) >> 4), id_pv, (add || kk > 0) ? 1u : 0u);
                mma_commit(&bar->pv_done[t]);
                ++pv_uses[t];
              }
            }
            if (!ok) break;
            mma_commit(&bar->kv_empty[vs]);
          }
        }
        mma_commit(&bar->drain[1]);
        wait_drain_inl(&bar->drain[1], 0, kDrainLimitNs);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ warp 11: rows of V behind the keys
      int g = 0, cleaned = 0;
      bool ok = true;
      CrossMeta meta{};
      while (ok && cross_next(v, items, &bar->second, at, w)) {
        if (w.dirty(v)) {
          const int vs = C::slot(1, g + w.j1 - 1 - w.j0);
          ok = __all_sync(0xffffffffu, wait_bounded_inl(&bar->v_ask, cleaned & 1, ctx, kSiteCrossTail));
          if (!ok) break;
          ++cleaned;
          uint8_t* tile = sKV + vs * C::kTileBytes;
          const int row = w.keys - (w.n - 1) * 128;  // first row behind the keys
          for (int a = 0; a < C::kAtoms; ++a)
            for (int c = row * 8 + lane; c < 128 * 8; c += 32)
              *reinterpret_cast<uint4*>(tile + a * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->v_clean);
        }
        g += w.j1 - w.j0;
        if (w.first() && !w.last()) {
          // (the CTA's last segment: the item's other blocks follow its share)
          meta.split = 1;
          meta.b = w.b;
          meta.it = w.it;
          meta.fresh = w.keys - w.len;
          meta.last = bar->end + w.n - w.j1;
          meta.total = bar->total;
        }
      }
      if (!ok) meta.split = 0;
      if (!CLUSTER && lane == 0) p.meta[blockIdx.x] = meta;
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
    const float cj = p.scale_log2;
    int uses = 0;   // blocks this tile has processed over all segments
    int merges = 0;  // ALT: segments whose two accumulators were joined
    bool alive = true;
    // (volatile: read again after the segment's blocks, not kept in registers)
    volatile CrossWarp* mine = reinterpret_cast<volatile CrossWarp*>(sWarps + 64 * warp);
    auto store = [&] {
      __syncwarp();
      if (lane == 0) {
        mine->at.step = at.step, mine->at.single = at.single, mine->at.more = at.more;
        mine->at.b = at.b, mine->at.it = at.it, mine->at.j = at.j, mine->at.left = at.left;
        mine->w.b = w.b, mine->w.it = w.it, mine->w.j0 = w.j0, mine->w.j1 = w.j1, mine->w.n = w.n;
        mine->w.len = w.len, mine->w.keys = w.keys, mine->w.single = w.single;
      }
      __syncwarp();
    };
    auto load_place = [&] {
      at.step = mine->at.step, at.single = mine->at.single, at.more = mine->at.more;
      at.b = mine->at.b, at.it = mine->at.it, at.j = mine->at.j, at.left = mine->at.left;
    };
    auto load_seg = [&] {
      w.b = mine->w.b, w.it = mine->w.it, w.j0 = mine->w.j0, w.j1 = mine->w.j1, w.n = mine->w.n;
      w.len = mine->w.len, w.keys = mine->w.keys, w.single = mine->w.single;
    };
    store();
    // CLUSTER: this CTA's part of the item, in the ring's memory once the ring has
    // been read: rows of D + 4 floats (so that a warp's rows spread over the banks);
    // its log-sum-exps at sMerge
    float* sPart = reinterpret_cast<float*>(sKV);
    while (alive) {
      load_place();
      if (!cross_next(v, items, &bar->second, at, w)) break;
      store();
      int jfirst, j1, cut_from, last_key;
      unsigned long long mask = 0;  // TREE: what the row's token sees of the drafts
      {
        const int row0 = cross_row0<PAIR>(w, p.row_tiles) + (PAIR ? 128 * t : 0);
        // nothing for this tile
        if (PAIR ? (t == 1 && !cross_two<PAIR>(w, row0 - 128, v.R)) : (t == 1 && w.j1 - w.j0 < 2)) continue;
        jfirst = w.j0 + (PAIR ? 0 : t);
        j1 = w.j1;
        cut_from = (TREE ? w.len : w.keys) - 127;  // first key of a block that is not seen whole
        last_key = w.keys - 1;
        if constexpr (TREE) {
          const int tok = (row0 + r) % v.Nq;
          if (v.masks) {
            mask = v.masks[(long long)w.b * v.T + tok] &
                   (w.keys - w.len >= 64 ? ~0ull : (1ull << (w.keys - w.len)) - 1ull);
            last_key = w.len;  // (the drafts' first key, from which the mask counts)
          } else {
            last_key = min(last_key, w.len + tok);
          }
        }
      }
      float m = -CUDART_INF_F;  // exponent reference (log2 units), a stale running max
      // l: sum of the fp32 probabilities; lcorr: the rounding errors of each
      // block's largest one, so that l + lcorr normalises O (see fa_fwd_kernel)
      float l = 0.f, lcorr = 0.f;
      for (int j = jfirst; j < j1; j += PAIR ? 1 : 2, ++uses) {
        if (!__all_sync(0xffffffffu, wait_bounded_inl(&bar->s_full[t], uses & 1, ctx, kSiteCrossS))) {
          alive = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[4][32];
        float mx_a = 0.f;
        if constexpr (C::kDualS) {  // two halves: the first's maximum is taken while the second loads
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
        const bool cut = kbase >= cut_from;
        if (cut) {
          if (TREE && v.masks) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t bits = cross_bits(mask, kbase + 32 * c - last_key);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((bits >> i) & 1u)) sr[c][i] = __float_as_uint(-CUDART_INF_F);
            }
          } else {
            const int last = last_key - kbase;
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c > last) sr[c >> 5][c & 31] = __float_as_uint(-CUDART_INF_F);
          }
        }
        float mx;
        if constexpr (C::kDualS) {
          mx = fmaxf(cut ? cross_max64(sr[0], sr[1]) : mx_a, cross_max64(sr[2], sr[3]));
        } else {
          mx = fmaxf(cross_max64(sr[0], sr[1]), cross_max64(sr[2], sr[3]));
        }
        const float m_new = fmaxf(m, mx * cj);
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
        const float ref = fmaxf(m, -3.402823466e38f);  // (finite for a row without keys so far: every P is 2^-inf = 0)
        const float2 c2 = make_float2(cj, cj);
        const float2 mneg2 = make_float2(-ref, -ref);
        float2 acc[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) acc[a] = make_float2(0.f, 0.f);
        {
          const float pbm = ex2_approx(fmaf(mx, cj, -ref));
          const float pbm_r = __uint_as_float(pack_bf16x2(pbm, 0.f) << 16);
          lcorr = lcorr * alpha + (pbm_r - pbm);
        }
        uint32_t pk[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1])),
                                        c2, mneg2);
            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            pk[c][i] = pack_bf16x2(p0, p1);
            acc[i & 3] = __fadd2_rn(acc[i & 3], make_float2(p0, p1));
          }
        }
        const float2 accs = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        l = l * alpha + (accs.x + accs.y);
        // P_t and O_t are in use until the tile's previous product has completed
        // (a segment's first block: its predecessor's epilogue has waited for
        // it; ALT: O_1 also until warpgroup 0 has read it)
        if (j > jfirst) {
          if (!__all_sync(0xffffffffu, wait_bounded_inl(&bar->pv_done[t], (uses - 1) & 1, ctx, kSiteCrossPv))) {
            alive = false;
            break;
          }
          tc_fence_after();
        } else if (!PAIR && t == 1 && merges > 0) {
          if (!__all_sync(0xffffffffu, wait_bounded_inl(&bar->merge_free, (merges - 1) & 1, ctx, kSiteCrossMerge))) {
            alive = false;
            break;
          }
          tc_fence_after();
        }
        if (rescale_warp) {
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
      if (!__all_sync(0xffffffffu, wait_bounded_inl(&bar->pv_done[t], (uses - 1) & 1, ctx, kSiteCrossPv))) {
        alive = false;
        break;
      }
      tc_fence_after();
      // ---- end of the segment
      load_seg();
      const int row = cross_row0<PAIR>(w, p.row_tiles) + (PAIR ? 128 * t : 0) + r;
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
          continue;
        }
        if (!__all_sync(0xffffffffu, wait_bounded_inl(&bar->merge_ready, merges & 1, ctx, kSiteCrossMerge))) {
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
      const bool whole = w.first() && w.last();
      bool write = row < v.R;
      if (TREE) write = write && (row % v.Nq) < w.keys - w.len;
      const int kvh = w.it / p.row_tiles;
      const size_t grow = ((size_t)w.b * v.Hkv + kvh) * v.R + row;
      const size_t prow = ((size_t)2 * blockIdx.x + (w.first() ? 1 : 0)) * p.part_rows + (PAIR ? 128 * t : 0) + r;
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
        if (CLUSTER) {
          if (write)
#pragma unroll
            for (int v4 = 0; v4 < 8; ++v4)
              reinterpret_cast<uint4*>(sPart + r * (D + 4) + 32 * c)[v4] =
                  make_uint4(ov[4 * v4], ov[4 * v4 + 1], ov[4 * v4 + 2], ov[4 * v4 + 3]);
        } else if (write && whole) {
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
      if (CLUSTER) {
        sMerge[r] = write ? lse2 : -CUDART_INF_F;
      } else if (write) {
        if (whole)
          p.lse[grow] = lse2 * 0.6931471805599453f;
        else
          p.part_lse[prow] = lse2;
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if constexpr (CLUSTER) {
    // every CTA of the cluster writes every p.cluster-th row, a warp per row
    cluster_sync();
    constexpr int E = D / 32, kMost = 8;
    const int ctas = p.cluster, item = blockIdx.x / ctas, fresh = bar->fresh;
    const float* parts = reinterpret_cast<const float*>(sKV) + lane * E;
    for (int row = (int)cluster_ctarank() + ctas * warp; row < v.R; row += ctas * (C::kThreads / 32)) {
      if (TREE && row % v.Nq >= fresh) continue;
      float l[kMost], o[kMost][E], mx = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < ctas) {
          l[i] = cluster_load(sMerge + row, i);
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
        if (i < ctas && l[i] != -CUDART_INF_F) {  // (a part without keys was not written)
          const float wt = ex2_approx(l[i] - ref);
          sum += wt;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, o[i][e], acc[e]);
        }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const size_t grow = (size_t)item * v.R + row;  // (one row tile per key/value head)
      uint32_t* orow = reinterpret_cast<uint32_t*>(p.o + grow * D) + lane * (E / 2);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) orow[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      if (lane == 0) p.lse[grow] = (sum == 0.f ? -CUDART_INF_F : ref + log2f(sum)) * 0.6931471805599453f;
    }
    cluster_sync();  // the others have read this CTA's part
  }
}

// Joins the parts of the items that share ends cut: block x takes the item that
// begins in CTA x's share and goes on behind it, kRows rows per warp.  O = sum of
// the parts' O weighted by 2^(their LSE - the largest), in CTA order.
template <int E>
__device__ __forceinline__ void cross_join_load(const float* o, float (&x)[E]) {
  if constexpr (E == 4) {
    const float4 a = *reinterpret_cast<const float4*>(o);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  } else {
    const float2 a = *reinterpret_cast<const float2*>(o);
    x[0] = a.x, x[1] = a.y;
  }
}

template <int D, bool TREE, bool PAIR>
__global__ void __launch_bounds__(256) fa_cross_combine_kernel(const CrossFwdParams p) {
  constexpr int E = D / 32;
  constexpr int kRows = PAIR ? 4 : 1;  // rows of a warp (cut PAIR items have mostly two parts)
  grid_wait();
  grid_trigger();
  const CrossMeta meta = p.meta[blockIdx.x];
  if (!meta.split) return;
  const CrossView& v = p.view;
  const int parts = (int)((meta.last * min((long long)gridDim.x, meta.total) - 1) / meta.total) - (int)blockIdx.x + 1;
  const int lane = threadIdx.x & 31, local0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kRows;
  const int kvh = meta.it / p.row_tiles;
  const int row0 = (meta.it - kvh * p.row_tiles) * (PAIR ? 256 : 128) + local0;
  const int drafted = meta.fresh;
  const size_t grow0 = ((size_t)meta.b * v.Hkv + kvh) * v.R + row0;
  // part i: the last segment of CTA x, then the first of each CTA after it
  auto part = [&](int i) { return ((size_t)2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * p.part_rows + local0; };
  auto there = [&](int r) {
    return local0 + r < p.part_rows && row0 + r < v.R && (!TREE || (row0 + r) % v.Nq < drafted);
  };
  auto write = [&](int r, const float (&acc)[E], float sum, float ref) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t* orow = reinterpret_cast<uint32_t*>(p.o + (grow0 + r) * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) orow[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0) p.lse[grow0 + r] = (sum == 0.f ? -CUDART_INF_F : ref + log2f(sum)) * 0.6931471805599453f;
  };
  if (kRows > 1 && parts == 2) {
    float l[2][kRows], o[2][kRows][E];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (there(r))
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i][r] = p.part_lse[part(i) + r];
          cross_join_load<E>(p.part_o + (part(i) + r) * D + lane * E, o[i][r]);
        }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (!there(r)) continue;
      const float mx = fmaxf(l[0][r], l[1][r]), ref = mx == -CUDART_INF_F ? 0.f : mx;
      const float w0 = ex2_approx(l[0][r] - ref), w1 = ex2_approx(l[1][r] - ref);
      float acc[E];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w1, o[1][r][e], w0 * o[0][r][e]);
      write(r, acc, w0 + w1, ref);
    }
    return;
  }
  constexpr int kBatch = 8;  // parts whose loads are in flight together
  for (int r = 0; r < kRows; ++r) {
    if (!there(r)) continue;
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
    write(r, acc, sum, ref);
  }
}

}  // namespace fa
