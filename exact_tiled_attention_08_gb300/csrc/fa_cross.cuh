// Attention whose keys have another length than the queries: a key length per
// request, key/value heads shared by groups of query heads, and (over a
// cache) drafted tokens behind the request's own that see each other by a mask.
//
// The G = H / Hkv query heads that share a key/value head lie next to one
// another in [B][H][Nq][d], so their rows are one run of G Nq query rows
// against one set of keys: everything below works on [B Hkv][R = G Nq][d].
#pragma once

#include <cuda_bf16.h>

#include "sm103_ptx.cuh"

namespace fa {

// Programmatic dependent launch: a kernel launched with it may start before the
// kernel in front of it has ended.  grid_wait() returns once that one has
// ended and its writes are visible (at once without such a launch): nothing in
// global memory is read or written before it, and nothing that an earlier
// kernel may have written is read through the read-only path (__ldg).  grid_trigger() lets the next
// kernel start; all of a kernel's CTAs have to come by (or end) first.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
    return lens ? min(max(lens[b], 0), Nk) : (T ? max(Nk - T, 0) : Nk);
  }
  // drafts of request b that have a key row
  __device__ __forceinline__ int drafted(int b, int len) const {
    return T ? min(min(max(drafts ? drafts[b] : T, 0), T), Nk - len) : 0;
  }
};

}  // namespace fa
