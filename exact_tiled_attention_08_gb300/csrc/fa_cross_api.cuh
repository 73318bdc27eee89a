// Host side of the cross attention, draft tree and rotation entry points
// (declared in fa.h; included by fa_ops.cu; uses the checks of fa_lib.cu).
#pragma once

#include <algorithm>
#include <atomic>

namespace {

// shape checks of the cross attention entry points; `R` receives the query
// rows per key/value head
fa_status check_cross_shape(int B, int H, int Hkv, int Nq, int Nk, int d, int* R) {
  if (B < 1 || H < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || d < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  const long long rows = (long long)(H / Hkv) * Nq;
  // (rounded up to whole row tile pairs and blocks they still fit an int)
  if (rows > 0x7fffff00LL || Nk > 0x7fffff00) return FA_ERR_INVALID_ARG;
  fa_status st = check_shape(B, Hkv, (int)rows, d);
  if (st == FA_OK) st = check_shape(B, Hkv, Nk, d);
  // the forward counts the key blocks of all requests, with what each costs at
  // its start, in 32 bits
  if (st == FA_OK && ((Nk + 127LL) / 128 + fa::kCrossStart) * B * Hkv > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  *R = (int)rows;
  return st;
}

bool all_aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  return true;
}

// Launch with programmatic stream serialization: the kernel may start while the
// one in front of it ends (it calls grid_wait before it touches memory).
template <typename... Params, typename... Args>
cudaError_t launch_early_clusters(void (*kernel)(Params...), dim3 grid, int cluster, int threads, int smem,
                                  cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                         const Args&... args) {
  return launch_early_clusters(kernel, grid, 1, threads, smem, stream, args...);
}

// Whether `kernel` launches with `regs` registers per thread, asked once per
// device.  (The warpgroups re-divide the block's registers with setmaxnreg,
// which only works if the block really gets that many.)
template <typename Kernel>
bool has_launch_regs(Kernel kernel, int regs, int dev, std::atomic<unsigned long long>& known) {
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (known.load(std::memory_order_relaxed) & bit) return true;
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess || attr.numRegs != regs) return false;
  known.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// arrays of lengths, positions and masks: their element's alignment
bool all_aligned(std::initializer_list<const void*> ptrs, unsigned bytes) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) return false;
  return true;
}

fa_status check_device_ptrs_given(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs) {
    if (!p) continue;
    const fa_status st = check_device_ptrs({p});
    if (st != FA_OK) return st;
  }
  return FA_OK;
}

fa::CrossView cross_view(int H, int Hkv, int Nq, int Nk) {
  fa::CrossView v{};
  v.Nk = Nk;
  v.Nq = Nq;
  v.R = H / Hkv * Nq;
  v.Hkv = Hkv;
  return v;
}

// Grid and workspace of the forward: CTAs (at most one per SM, and one per
// place), and two parts per CTA where an item can be cut (more than one block).
struct CrossFwdPlan {
  int row_tiles, part_rows, ctas;
  bool pair, cuts;
  size_t lse_at, o_at, total;
  static CrossFwdPlan of(int B, int Hkv, int R, int Nk, int d) {
    CrossFwdPlan w;
    w.pair = R > 128;
    w.row_tiles = w.pair ? (R + 255) / 256 : 1;
    w.part_rows = w.pair ? 256 : R;
    const long long blocks = (long long)B * Hkv * w.row_tiles * ((Nk + 127LL) / 128 + fa::kCrossStart);
    w.ctas = (int)std::min<long long>(blocks, fa::kCrossMaxCtas);
    w.cuts = Nk > 128;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t rows = w.cuts ? (size_t)2 * w.ctas * w.part_rows : 0;
    w.lse_at = up(w.ctas * sizeof(fa::CrossMeta));
    w.o_at = w.lse_at + up(rows * sizeof(float));
    w.total = w.o_at + up(rows * d * sizeof(float)) + 256;  // (the base is brought to a 256-byte boundary)
    return w;
  }
};

// Clusters of 8, 4 and 2 CTAs of a kernel that the device holds at once (15, 36 and 76 on a
// GB300 whose 152 SMs are free, at a CTA per SM), asked once per device.
template <typename Kernel>
fa::CrossClusterFit cluster_fit(Kernel kernel, int threads, int smem, int dev, std::atomic<unsigned long long>* known) {
  fa::CrossClusterFit fit{};
  const unsigned long long was = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (was) {
    for (int i = 0; i < 3; ++i) fit.clusters[i] = (int)(was >> (16 * i) & 0xffff);
    return fit;
  }
  if (set_smem(kernel, smem) != cudaSuccess) return fit;
  unsigned long long found = 1ull << 63;
  for (int i = 0; i < 3; ++i) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 8u >> i;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((8u >> i) * fa::kCrossMaxCtas, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return fa::CrossClusterFit{};
    }
    fit.clusters[i] = std::min(n, 0xffff);
    found |= (unsigned long long)fit.clusters[i] << (16 * i);
  }
  if (dev < 64) known[dev].store(found, std::memory_order_relaxed);
  return fit;
}
template <int D, bool TREE>
fa::CrossClusterFit cross_cluster_fit(int dev) {
  using C = fa::CrossCfg<D>;
  static std::atomic<unsigned long long> known[64];  // by device: the three numbers and a bit that says so
  return cluster_fit(fa::fa_cross_fwd_kernel<D, TREE, false, true>, C::kThreads, C::kSmemBytes, dev, known);
}

template <int D, bool TREE>
fa_status launch_cross_clusters(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                const fa::CrossFwdParams& p, int items, cudaStream_t stream) {
  using C = fa::CrossCfg<D>;
  auto kernel = fa::fa_cross_fwd_kernel<D, TREE, false, true>;
  if (set_smem(kernel, C::kSmemBytes) != cudaSuccess) return FA_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  static std::atomic<unsigned long long> known{0};
  if (!has_launch_regs(kernel, C::kLaunchRegs, dev, known)) return FA_ERR_CUDA;
  return launch_early_clusters(kernel, dim3((unsigned)(items * p.cluster)), p.cluster, C::kThreads, C::kSmemBytes, stream,
                               mq, mk, mv, p) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

template <int D, bool TREE, bool PAIR>
fa_status launch_cross_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                           const fa::CrossFwdParams& p, const CrossFwdPlan& plan, cudaStream_t stream) {
  using C = fa::CrossCfg<D>;
  auto kernel = fa::fa_cross_fwd_kernel<D, TREE, PAIR, false>;
  if (set_smem(kernel, C::kSmemBytes) != cudaSuccess) return FA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return FA_ERR_CUDA;
  static std::atomic<unsigned long long> known{0};
  if (!has_launch_regs(kernel, C::kLaunchRegs, dev, known)) return FA_ERR_CUDA;
  const int grid = std::min(plan.ctas, sms);
  if (launch_early(kernel, dim3((unsigned)grid), C::kThreads, C::kSmemBytes, stream, mq, mk, mv, p) != cudaSuccess)
    return FA_ERR_CUDA;
  // without lengths the host knows whether the CTAs cut items
  bool cuts = plan.cuts;
  if (cuts && !p.view.lens) {
    const int most = (p.view.Nk + 127) / 128 + fa::kCrossStart;
    const long long items = (long long)p.B * p.view.Hkv * p.row_tiles;
    cuts = items >= grid ? fa::cross_tail((int)(items % grid), grid, most, PAIR) == fa::kCrossTailCut
                         : !fa::cross_whole((int)items, grid, most, items * most);
  }
  if (cuts) {
    const int per_block = PAIR ? 32 : 8;  // rows of a block
    const dim3 rows((unsigned)grid, (unsigned)((plan.part_rows + per_block - 1) / per_block));
    if (launch_early(fa::fa_cross_combine_kernel<D, TREE, PAIR>, rows, 256, 0, stream, p) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return FA_OK;
}

fa_status run_cross_fwd(const fa::CrossView& view, const void* q, const void* k, const void* v, void* o, float* lse,
                        void* workspace, int B, int d, float scale, cudaStream_t stream) {
  const CrossFwdPlan plan = CrossFwdPlan::of(B, view.Hkv, view.R, view.Nk, d);
  CUtensorMap mq, mk, mv;
  if (!encode_bhnd(&mq, q, B * view.Hkv, view.R, d) || !encode_bhnd(&mk, k, B * view.Hkv, view.Nk, d) ||
      !encode_bhnd(&mv, v, B * view.Hkv, view.Nk, d))
    return FA_ERR_CUDA;
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
  fa::CrossFwdParams p{};
  p.view = view;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.meta = reinterpret_cast<fa::CrossMeta*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + plan.lse_at);
  p.part_o = reinterpret_cast<float*>(ws + plan.o_at);
  p.part_rows = plan.part_rows;
  p.B = B;
  p.row_tiles = plan.row_tiles;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = wait_limit_ns();
  p.debug_stall = g_debug_stall.load();
  p.o_align32 = aligned32(o);
  const bool tree = view.T > 0;
  if (!plan.pair) {
    const long long items = (long long)B * view.Hkv;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
      return FA_ERR_CUDA;
    const fa::CrossClusterFit fit =
        d == 128 ? (tree ? cross_cluster_fit<128, true>(dev) : cross_cluster_fit<128, false>(dev))
                 : (tree ? cross_cluster_fit<64, true>(dev) : cross_cluster_fit<64, false>(dev));
    // One request of a length that only the device knows counts as half of what its cache
    // holds.  (H=32/8 d=128, one token, with and without clusters: 1000 tokens 15 and
    // 17 us, 8000 23 and 27, 16k 33 and 33, 32k 54 and 45; a 32k cache takes them, 64k not.)
    int blocks = (view.Nk + 127) / 128;
    if (B == 1 && view.lens && blocks > 2) blocks = (blocks + 1) / 2;
    p.cluster = fa::cross_cluster(items, blocks, view.R, B == 1 || !view.lens, std::min(sms, fa::kCrossMaxCtas), fit);
    if (p.cluster > 1) {
      if (d == 128)
        return tree ? launch_cross_clusters<128, true>(mq, mk, mv, p, (int)items, stream)
                    : launch_cross_clusters<128, false>(mq, mk, mv, p, (int)items, stream);
      return tree ? launch_cross_clusters<64, true>(mq, mk, mv, p, (int)items, stream)
                  : launch_cross_clusters<64, false>(mq, mk, mv, p, (int)items, stream);
    }
  }
  if (d == 128) {
    if (tree)
      return plan.pair ? launch_cross_fwd<128, true, true>(mq, mk, mv, p, plan, stream)
                       : launch_cross_fwd<128, true, false>(mq, mk, mv, p, plan, stream);
    return plan.pair ? launch_cross_fwd<128, false, true>(mq, mk, mv, p, plan, stream)
                     : launch_cross_fwd<128, false, false>(mq, mk, mv, p, plan, stream);
  }
  if (tree)
    return plan.pair ? launch_cross_fwd<64, true, true>(mq, mk, mv, p, plan, stream)
                     : launch_cross_fwd<64, true, false>(mq, mk, mv, p, plan, stream);
  return plan.pair ? launch_cross_fwd<64, false, true>(mq, mk, mv, p, plan, stream)
                   : launch_cross_fwd<64, false, false>(mq, mk, mv, p, plan, stream);
}

size_t cross_fwd_workspace(int B, int H, int Hkv, int Nq, int Nk, int d) {
  int R;
  if (check_cross_shape(B, H, Hkv, Nq, Nk, d, &R) != FA_OK) return 0;
  return CrossFwdPlan::of(B, Hkv, R, Nk, d).total;
}

// workspace of the backward: plan, dQ accumulator (more than one key block), delta and LSE log2(e) padded
// to whole blocks, runs of cut items
struct CrossBwdWorkspace {
  size_t dq_at, delta_at, lse_at, runs_at, total;
  static CrossBwdWorkspace of(int B, int Hkv, int R, int Nk, int d) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t bk = (size_t)B * Hkv, rpad = ((size_t)R + 127) / 128 * 128;
    CrossBwdWorkspace w;
    w.dq_at = up(sizeof(fa::CrossBwdPlan));
    w.delta_at = w.dq_at + (Nk > 128 ? up(bk * R * d * sizeof(float)) : 0);
    w.lse_at = w.delta_at + up(bk * rpad * sizeof(float));
    w.runs_at = w.lse_at + up(bk * rpad * sizeof(float));
    // (an item of one query block is never cut, and none into more runs than it has of them)
    const size_t blocks = bk * (((size_t)Nk + 127) / 128) * (rpad / 128);
    const size_t runs = R > 128 ? std::min<size_t>(fa::kCrossBwdSlots, blocks) : 0;
    w.total = w.runs_at + runs * 2 * 128 * d * sizeof(float) + 256;
    return w;
  }
};

template <int D>
fa_status run_cross_bwd(const fa::CrossView& view, const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv, void* workspace, int B,
                        float scale, cudaStream_t stream) {
  using C = fa::BwdCfg<D, true>;
  const int BK = B * view.Hkv, R = view.R, nqb = (R + 127) / 128, rpad = nqb * 128;
  // One key block per request at most: dQ is written where it is formed, without
  // the accumulator's zeroing, adding and casting (and mostly without the last
  // kernel).  Measured, with the accumulator and direct: B=8 H=16 Nq=4096 Nk=77
  // d=64 153 and 113 us; B=4 H=32/8 Nq=4096 Nk=128 d=128 299 and 174 us.
  const bool direct = view.Nk <= 128;
  const CrossBwdWorkspace w = CrossBwdWorkspace::of(B, view.Hkv, R, view.Nk, D);
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
  float* dq_acc = reinterpret_cast<float*>(ws + w.dq_at);
  float* delta = reinterpret_cast<float*>(ws + w.delta_at);
  float* lse2 = reinterpret_cast<float*>(ws + w.lse_at);
  CUtensorMap mq, mk, mv, mdo, ml, mdel, mdq;
  if (!encode_bhnd(&mq, q, BK, R, D) || !encode_bhnd(&mk, k, BK, view.Nk, D) || !encode_bhnd(&mv, v, BK, view.Nk, D) ||
      !encode_bhnd(&mdo, dout, BK, R, D) || !encode_f32_rows(&ml, lse2, BK, rpad, 128) ||
      !encode_f32_rows(&mdel, delta, BK, rpad, 128) || !encode_dq_acc(&mdq, dq_acc, BK, R, D))
    return FA_ERR_CUDA;
  auto kernel = fa::fa_cross_bwd_kernel<D>;
  if (set_smem(kernel, fa::kCrossBwdSmemBytes<D>) != cudaSuccess) return FA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return FA_ERR_CUDA;
  static std::atomic<unsigned long long> known{0};
  if (!has_launch_regs(kernel, C::kLaunchRegs, dev, known)) return FA_ERR_CUDA;
  const long long rows = (long long)BK * rpad, per_block = 256 / (D / 8);
  const long long prep = std::min((rows + per_block - 1) / per_block, 152LL * 16);
  if (launch_early(fa::fa_cross_bwd_prep_kernel<D>, dim3((unsigned)prep), 256, 0, stream,
                   static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dout), lse, delta, lse2,
                   direct ? static_cast<float*>(nullptr) : dq_acc, R, rpad, rows) != cudaSuccess)
    return FA_ERR_CUDA;
  fa::CrossBwdPostParams post{};
  fa::CrossBwdParams& p = post.p;
  p.view = view;
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.plan = reinterpret_cast<fa::CrossBwdPlan*>(ws);
  p.runs = reinterpret_cast<float*>(ws + w.runs_at);
  p.B = B;
  p.nqb = nqb;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.scale = scale;
  p.wait_limit_ns = wait_limit_ns();
  p.debug_stall = g_debug_stall.load();
  p.out_align32 = aligned32(dk) && aligned32(dv) && aligned32(dq);
  p.dq = direct ? static_cast<__nv_bfloat16*>(dq) : nullptr;
  // one CTA per SM, and no more than there are query blocks to hand out
  const long long blocks = (long long)BK * ((view.Nk + 127LL) / 128) * nqb;
  const int grid = (int)std::min<long long>(blocks, std::min(sms, fa::kCrossBwdMaxCtas));
  if (launch_early(kernel, dim3((unsigned)grid), C::kThreads, fa::kCrossBwdSmemBytes<D>, stream, mq, mk, mv, mdo, ml,
                   mdel, mdq, p) != cudaSuccess)
    return FA_ERR_CUDA;
  if (direct && fa::cross_bwd_split(BK, nqb, grid).parts == 1) return FA_OK;
  post.dq_acc = dq_acc;
  post.dq = static_cast<__nv_bfloat16*>(dq);
  post.n8 = (long long)BK * R * D / 8;
  post.ctas = grid;
  const long long convert = direct ? 0 : std::min((post.n8 + 255) / 256, 152LL * 16);
  const long long post_grid = 8LL * grid + (view.lens && !direct ? BK : 0) + convert;
  return launch_early(fa::fa_cross_bwd_post_kernel<D>, dim3((unsigned)post_grid), 256, 0, stream, post) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t fa_cross_fwd_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d) {
  return cross_fwd_workspace(B, H, Hkv, Nq, Nk, d);
}

fa_status fa_cross_fwd(const void* q, const void* k, const void* v, const int* key_lens, void* o, float* lse,
                       void* workspace, size_t ws_bytes, int B, int H, int Hkv, int Nq, int Nk, int d, float scale,
                       cudaStream_t stream) {
  if (!q || !k || !v || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  int R;
  fa_status st = check_cross_shape(B, H, Hkv, Nq, Nk, d, &R);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale, 0)) != FA_OK) return st;
  if (ws_bytes < cross_fwd_workspace(B, H, Hkv, Nq, Nk, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, o, lse, workspace}) || !all_aligned({key_lens}, 4)) return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k, v, o, lse, workspace})) != FA_OK) return st;
  if (key_lens && (st = check_device_ptrs({key_lens})) != FA_OK) return st;
  fa::CrossView view = cross_view(H, Hkv, Nq, Nk);
  view.lens = key_lens;
  return run_cross_fwd(view, q, k, v, o, lse, workspace, B, d, scale, stream);
}

size_t fa_cross_bwd_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d) {
  int R;
  if (check_cross_shape(B, H, Hkv, Nq, Nk, d, &R) != FA_OK) return 0;
  return CrossBwdWorkspace::of(B, Hkv, R, Nk, d).total;
}

fa_status fa_cross_bwd(const void* q, const void* k, const void* v, const int* key_lens, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, void* workspace,
                       size_t ws_bytes, int B, int H, int Hkv, int Nq, int Nk, int d, float scale,
                       cudaStream_t stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return FA_ERR_INVALID_ARG;
  int R;
  fa_status st = check_cross_shape(B, H, Hkv, Nq, Nk, d, &R);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale, 0)) != FA_OK) return st;
  if (ws_bytes < fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, o, dout, lse, dq, dk, dv, workspace}) || !all_aligned({key_lens}, 4))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k, v, o, dout, lse, dq, dk, dv, workspace})) != FA_OK) return st;
  if (key_lens && (st = check_device_ptrs({key_lens})) != FA_OK) return st;
  fa::CrossView view = cross_view(H, Hkv, Nq, Nk);
  view.lens = key_lens;
  if (d == 128)
    return run_cross_bwd<128>(view, q, k, v, o, dout, lse, dq, dk, dv, workspace, B, scale, stream);
  return run_cross_bwd<64>(view, q, k, v, o, dout, lse, dq, dk, dv, workspace, B, scale, stream);
}

size_t fa_tree_fwd_workspace_bytes(int B, int H, int Hkv, int T, int C, int d) {
  return cross_fwd_workspace(B, H, Hkv, T, C, d);
}

fa_status fa_tree_fwd(const void* q, const void* k_cache, const void* v_cache, const int* cache_lens,
                      const int* draft_lens, const unsigned long long* draft_masks, void* o, float* lse,
                      void* workspace, size_t ws_bytes, int B, int H, int Hkv, int T, int C, int d, float scale,
                      cudaStream_t stream) {
  if (!q || !k_cache || !v_cache || !cache_lens || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  int R;
  fa_status st = check_cross_shape(B, H, Hkv, T, C, d, &R);
  if (st != FA_OK) return st;
  if (draft_masks && T > 64) return FA_ERR_UNSUPPORTED;
  if ((st = check_scale(scale, 0)) != FA_OK) return st;
  if (ws_bytes < cross_fwd_workspace(B, H, Hkv, T, C, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k_cache, v_cache, o, lse, workspace}) || !all_aligned({cache_lens, draft_lens}, 4) ||
      !all_aligned({draft_masks}, 8))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k_cache, v_cache, cache_lens, o, lse, workspace})) != FA_OK) return st;
  if (draft_lens && (st = check_device_ptrs({draft_lens})) != FA_OK) return st;
  if (draft_masks && (st = check_device_ptrs({draft_masks})) != FA_OK) return st;
  fa::CrossView view = cross_view(H, Hkv, T, C);
  view.lens = cache_lens;
  view.drafts = draft_lens;
  view.masks = draft_masks;
  view.T = T;
  return run_cross_fwd(view, q, k_cache, v_cache, o, lse, workspace, B, d, scale, stream);
}

fa_status fa_cross_fwd_packed(const fa_cross_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_cross_fwd(a->q, a->k, a->v, a->key_lens, a->o, a->lse, a->workspace, a->ws_bytes, a->B, a->H, a->Hkv, a->Nq,
                      a->Nk, a->d, a->scale, a->stream);
}

fa_status fa_cross_bwd_packed(const fa_cross_bwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_cross_bwd(a->q, a->k, a->v, a->key_lens, a->o, a->dout, a->lse, a->dq, a->dk, a->dv, a->workspace,
                      a->ws_bytes, a->B, a->H, a->Hkv, a->Nq, a->Nk, a->d, a->scale, a->stream);
}

fa_status fa_tree_fwd_packed(const fa_tree_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_tree_fwd(a->q, a->k_cache, a->v_cache, a->cache_lens, a->draft_lens, a->draft_masks, a->o, a->lse,
                     a->workspace, a->ws_bytes, a->B, a->H, a->Hkv, a->T, a->C, a->d, a->scale, a->stream);
}

}  // extern "C"
