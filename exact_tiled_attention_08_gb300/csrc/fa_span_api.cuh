// Host side of the span attention and paged attention entry points (declared in
// fa.h; included by fa_ops.cu; uses the checks of fa_lib.cu).
#pragma once

namespace {

// what a key/value cache in pages has to be
struct PageShape {
  int num_pages, page_size, width;
  long long capacity() const { return (long long)width * page_size; }
  fa_status check() const {
    if (num_pages < 1 || page_size < 1 || width < 1) return FA_ERR_INVALID_ARG;
    if (page_size < 16 || (page_size & (page_size - 1))) return FA_ERR_UNSUPPORTED;
    return capacity() > 0x7fffff00LL ? FA_ERR_INVALID_ARG : FA_OK;
  }
  int shift() const {
    int s = 0;
    while (1 << s < page_size) ++s;
    return s;
  }
};

// strides: of sizes greater than one positive, of the others not used
fa_status check_pages(const fa_pages* r, const PageShape& s, int Hkv) {
  if (!r || !r->ptr) return FA_ERR_INVALID_ARG;
  const struct {
    long long stride;
    int size;
  } dims[3] = {{r->page, s.num_pages}, {r->head, Hkv}, {r->token, s.page_size}};
  for (const auto& x : dims)
    if (x.size > 1 && (x.stride < 1 || x.stride >= 1ll << 38)) return FA_ERR_INVALID_ARG;
  for (const auto& x : dims)
    if (x.size > 1 && x.stride % 8) return FA_ERR_MISALIGNED;
  return aligned16(r->ptr) ? FA_OK : FA_ERR_MISALIGNED;
}

// 1 - 2 / (1 + e^2x), which the backward, few rows and blocks with large products take, is off by 2^-21 of the
// cap however small the score (half of it from the rounding of 1 + e^2x and the two approximations at x = 0,
// all of it at -1).  Up to this cap that is at most 2^-7 of a score, a change of a weight by two of bf16's
// half steps.
constexpr float kMaxCap = 16384.f;

fa_status check_span_args(float scale, float cap, int window, int causal) {
  fa_status st = check_scale(scale, causal);
  if (st != FA_OK) return st;
  if (!(cap >= 0.f && cap <= kMaxCap) || window < 0) return FA_ERR_INVALID_ARG;
  if (cap > 0.f && (!std::isnormal(scale / cap) || !std::isfinite(4.f * scale / cap))) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_span_shape(int B, int H, int Hkv, int N, int d) {
  int R;
  const fa_status st = check_cross_shape(B, H, Hkv, N, N, d, &R);
  return st == FA_OK ? check_shape(B, H, N, d) : st;
}

fa::PageRows page_rows(const fa_pages* r) {
  return {static_cast<__nv_bfloat16*>(r->ptr), r->page, r->head, r->token};
}

// keys or values as a 4-D tensor (d, tokens, heads, pages) for boxes of 64 x box_rows,
// 128-byte swizzle; what lies outside reads as zero
bool encode_pages(CUtensorMap* map, const fa::PageRows& r, int tokens, int heads, int pages, int box_rows, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)tokens, (cuuint64_t)heads, (cuuint64_t)pages};
  // (the stride of a dimension of one is not used, but looked at)
  auto bytes = [&](long long stride, int size) { return (cuuint64_t)(size > 1 ? stride : d) * 2; };
  const cuuint64_t strides[3] = {bytes(r.token, tokens), bytes(r.head, heads), bytes(r.page, pages)};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r.ptr, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// tanh(sqrt u) / sqrt u on [0, 0.36]: minimax polynomial of degree 4 (Remez exchange), relative error 7.3e-8
constexpr double kTanhPoly[5] = {0.9999999268689591, -0.3333230997439495, 0.13310173657879062, -0.05210148011192052,
                                 0.015475427482730527};

fa::SpanCap span_cap(float scale, float cap) {
  fa::SpanCap c{};
  if (cap == 0.f) return c;
  const double x = (double)scale / cap, top = 1.4426950408889634 * cap;
  c.mul = (float)(2 * 1.4426950408889634 * x);
  c.top = (float)top;
  bool held = true;  // (where fp32 does not hold the coefficients no product is small)
  for (int i = 0; i < 5; ++i) {
    c.d[i] = (float)(top * kTanhPoly[i] * std::pow(x, 2 * i + 1));
    held = held && std::isnormal(c.d[i]);
  }
  c.small = held ? 0.6f * cap / scale : -1.f;
  c.low = -0.2f * cap / scale;
  c.hidden = held && cap >= 30.f && std::isfinite(10.f * cap / scale) ? -10.f * cap / scale : 0.f;
  return c;
}

// Heads of a unit of the heads that share a key/value head: a divisor of their number, the largest
// that leaves at most an eighth of the rows of a tile of 128 empty, or all rows in one tile.
int span_unit_heads(int group, int N) {
  for (int h = std::min(group, 128);; --h)
    if (group % h == 0 && ((long long)h * N <= 128 || 128 / h * h >= 112)) return h;
}

// queries as a 4-D tensor (d, heads of a unit, tokens, units) for boxes of 64 columns of a tile's rows
bool encode_units(CUtensorMap* map, const void* q, int units, int heads, int N, int tokens, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)N, (cuuint64_t)units};
  const cuuint64_t strides[3] = {(cuuint64_t)N * d * 2, (cuuint64_t)d * 2, (cuuint64_t)heads * N * d * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)heads, (cuuint32_t)tokens, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Grid and workspace of the forward, as CrossFwdPlan; with spans by row their tiles' bounds first.
struct SpanFwdPlan {
  bool few;  // the kernel for up to 16 rows of a unit
  int tokens, tiles, row_tiles, part_rows, ctas;
  bool pair, cuts;
  size_t meta_at, lse_at, o_at, total;
  static SpanFwdPlan of(int B, int H, int heads, int N, int C, int d, bool paged) {
    SpanFwdPlan w;
    const long long rows_all = (long long)heads * N;
    w.few = paged && rows_all <= fa::kFewRows;
    w.tokens = (w.few ? fa::kFewRows : 128) / heads;
    w.tiles = (N + w.tokens - 1) / w.tokens;
    w.pair = !paged || w.tiles > 1;  // (a tile of contiguous keys alone has but one block)
    w.row_tiles = w.pair ? (w.tiles + 1) / 2 : 1;
    w.part_rows = w.pair ? 256 : (int)rows_all;
    const long long blocks = (long long)B * (H / heads) * w.row_tiles * ((C + 127LL) / 128 + fa::kCrossStart);
    w.ctas = (int)std::min<long long>(blocks, fa::kCrossMaxCtas);
    w.cuts = C > 128;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t rows = w.cuts ? (size_t)2 * w.ctas * w.part_rows : 0;
    w.meta_at = !paged ? up((size_t)B * w.tiles * sizeof(int4)) : 0;
    w.lse_at = w.meta_at + up(w.ctas * sizeof(fa::SpanMeta));
    w.o_at = w.lse_at + up(rows * sizeof(float));
    w.total = w.o_at + up(rows * d * sizeof(float)) + 256;  // (the base is brought to a 256-byte boundary)
    return w;
  }
};

template <int D, int MOD, bool PAIR, bool PAGED>
fa_status launch_span_fwd(const CUtensorMap* maps, const fa::SpanFwdParams<PAGED>& p, unsigned grid, cudaStream_t stream) {
  using C = fa::CrossCfg<D>;
  auto kernel = fa::fa_span_fwd_kernel<D, MOD, PAIR, PAGED>;
  if (set_smem(kernel, C::kSmemBytes) != cudaSuccess) return FA_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  static std::atomic<unsigned long long> known{0};
  if (!has_launch_regs(kernel, C::kLaunchRegs, dev, known)) return FA_ERR_CUDA;
  return launch_early(kernel, dim3(grid), C::kThreads, C::kSmemBytes, stream, maps[0], maps[1], maps[2], p) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

// Clusters of 8, 4 and 2 CTAs of the kernel for few rows that the device holds at once, asked once per device.
template <int D>
fa::CrossClusterFit few_cluster_fit(int dev) {
  using C = fa::FewCfg<D>;
  static std::atomic<unsigned long long> known[64];  // by device: the three numbers and a bit that says so
  return cluster_fit(fa::fa_span_few_kernel<D, true>, C::kThreads, C::kSmemBytes, dev, known);
}

template <int D>
fa_status launch_span_few(const CUtensorMap* maps, fa::SpanFwdParams<true>& p, unsigned grid, int sms, cudaStream_t stream) {
  using C = fa::FewCfg<D>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  // One request of a length that only the device knows counts as half of what its pages hold, as
  // in the cross forward.
  const long long items = (long long)p.B * p.rows.units;
  int blocks = (p.rows.view.C + 127) / 128;
  if (p.B == 1 && blocks > 2) blocks = (blocks + 1) / 2;
  p.cluster = fa::cross_cluster(items, blocks, p.part_rows, p.B == 1, std::min(sms, fa::kCrossMaxCtas),
                                few_cluster_fit<D>(dev));
  if (p.cluster > 1) {
    auto kernel = fa::fa_span_few_kernel<D, true>;
    if (set_smem(kernel, C::kSmemBytes) != cudaSuccess) return FA_ERR_CUDA;
    return launch_early_clusters(kernel, dim3((unsigned)(items * p.cluster)), p.cluster, C::kThreads, C::kSmemBytes, stream,
                                 maps[0], maps[1], maps[2], p) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
  }
  auto kernel = fa::fa_span_few_kernel<D, false>;
  if (set_smem(kernel, C::kSmemBytes) != cudaSuccess) return FA_ERR_CUDA;
  return launch_early(kernel, dim3(grid), C::kThreads, C::kSmemBytes, stream, maps[0], maps[1], maps[2], p) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

template <int D, bool PAIR, bool PAGED>
fa_status launch_span_mod(const CUtensorMap* maps, const fa::SpanFwdParams<PAGED>& p, unsigned grid, cudaStream_t stream) {
  if (p.cap.top > 0.f)
    return p.slopes ? launch_span_fwd<D, 3, PAIR>(maps, p, grid, stream) : launch_span_fwd<D, 2, PAIR>(maps, p, grid, stream);
  return p.slopes ? launch_span_fwd<D, 1, PAIR>(maps, p, grid, stream) : launch_span_fwd<D, 0, PAIR>(maps, p, grid, stream);
}

// The forward's main kernel: two row tiles per item, or (pages) one, or few rows.
template <int D, bool PAGED>
fa_status launch_span_form(const CUtensorMap* maps, fa::SpanFwdParams<PAGED>& p, const SpanFwdPlan& plan, unsigned grid,
                           int sms, cudaStream_t stream) {
  if constexpr (PAGED) {
    if (plan.few) return launch_span_few<D>(maps, p, grid, sms, stream);
    if (!plan.pair) return launch_span_mod<D, false>(maps, p, grid, stream);
  }
  return launch_span_mod<D, true>(maps, p, grid, stream);
}

template <int D, bool PAGED>
fa_status launch_span_combine(const fa::SpanFwdParams<PAGED>& p, const SpanFwdPlan& plan, unsigned grid, cudaStream_t stream) {
  const int per_block = plan.pair ? 32 : 8;  // rows of a block
  const dim3 parts(grid, (unsigned)((plan.part_rows + per_block - 1) / per_block));
  auto combine = fa::fa_span_combine_kernel<D, true, PAGED>;
  if constexpr (PAGED)
    if (!plan.pair) combine = fa::fa_span_combine_kernel<D, false, PAGED>;
  return launch_early(combine, parts, 256, 0, stream, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <bool PAGED>
struct SpanCall {
  fa::SpanRows<PAGED> rows;
  const void* q;
  fa::PageRows k, v;
  int box_rows, tokens, pages;  // of the key and value tensors
  void* o;
  float* lse;
  void* workspace;
  int B, H, Hkv, d;
  float scale, cap;
  const float* slopes;
  cudaStream_t stream;
};

template <bool PAGED>
fa_status run_span_fwd(const SpanCall<PAGED>& a) {
  const fa::SpanView<PAGED>& view = a.rows.view;
  const SpanFwdPlan plan = SpanFwdPlan::of(a.B, a.H, a.rows.unit_heads, view.N, view.C, a.d, PAGED);
  CUtensorMap maps[3];
  if (!encode_units(&maps[0], a.q, a.B * a.rows.units, a.rows.unit_heads, view.N, plan.tokens, a.d) ||
      !encode_pages(&maps[1], a.k, a.tokens, a.Hkv, a.pages, a.box_rows, a.d) ||
      !encode_pages(&maps[2], a.v, a.tokens, a.Hkv, a.pages, a.box_rows, a.d))
    return FA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return FA_ERR_CUDA;
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(a.workspace) + 255) & ~uintptr_t(255));
  fa::SpanFwdParams<PAGED> p{};
  p.rows = a.rows;
  p.rows.tile_tokens = plan.tokens;
  p.rows.tiles = plan.tiles;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.meta = reinterpret_cast<fa::SpanMeta*>(ws + plan.meta_at);
  p.part_lse = reinterpret_cast<float*>(ws + plan.lse_at);
  p.part_o = reinterpret_cast<float*>(ws + plan.o_at);
  p.part_rows = plan.part_rows;
  p.q_bytes = a.rows.unit_heads * plan.tokens * a.d * 2;
  p.B = a.B;
  p.row_tiles = plan.row_tiles;
  p.pages = a.pages;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.cap = span_cap(a.scale, a.cap);
  p.slopes = a.slopes;
  p.wait_limit_ns = wait_limit_ns();
  p.debug_stall = g_debug_stall.load();
  p.o_align32 = aligned32(a.o);
  p.cluster = 1;
  if constexpr (!PAGED) {
    if (view.begin || view.end) {
      int4* bounds = reinterpret_cast<int4*>(ws);
      p.rows.bounds = bounds;
      if (launch_early(fa::fa_span_bounds_kernel, dim3((unsigned)plan.tiles * (unsigned)a.B), 128, 0, a.stream, view,
                       plan.tiles, bounds) != cudaSuccess)
        return FA_ERR_CUDA;
    }
  }
  const unsigned grid = (unsigned)std::min(plan.ctas, sms);
  const fa_status st = a.d == 128 ? launch_span_form<128>(maps, p, plan, grid, sms, a.stream)
                                  : launch_span_form<64>(maps, p, plan, grid, sms, a.stream);
  if (st != FA_OK || !plan.cuts || p.cluster > 1) return st;
  // Nothing is cut where whole items cannot take longer than what cutting costs (span_schedule's rule).
  const long long items = (long long)a.B * a.rows.units * plan.row_tiles;
  if ((items + grid - 1) / grid * ((view.C + 127LL) / 128 + fa::kCrossStart) <= fa::kCrossCut) return FA_OK;
  return a.d == 128 ? launch_span_combine<128>(p, plan, grid, a.stream) : launch_span_combine<64>(p, plan, grid, a.stream);
}

// workspace of the backward: the plan, the spans and their tiles' bounds, the dQ accumulator (more than
// one key block), delta and LSE log2(e) padded to whole blocks, runs of cut items
struct SpanBwdWorkspace {
  size_t first_at, runs_at, cuts_at, hulls_at, order_at, lo_at, hi_at, bounds_at, dq_at, delta_at, lse_at, sums_at, total;
  static SpanBwdWorkspace of(int B, int H, int Hkv, int N, int d) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t nb = ((size_t)N + 127) / 128, npad = nb * 128, entries = (size_t)B * nb;
    SpanBwdWorkspace w;
    w.first_at = up(sizeof(fa::SpanBwdPlan));
    w.runs_at = w.first_at + up(((size_t)B + 1) * sizeof(int));
    w.cuts_at = w.runs_at + up((entries + fa::kSpanBwdSlots) * sizeof(fa::SpanRun));
    w.hulls_at = w.cuts_at + up(fa::kSpanBwdSlots / 2 * sizeof(int4));
    w.order_at = w.hulls_at + up(entries * sizeof(int2));
    w.lo_at = w.order_at + up(entries * sizeof(int));
    w.hi_at = w.lo_at + up(B * npad * sizeof(int));
    w.bounds_at = w.hi_at + up(B * npad * sizeof(int));
    w.dq_at = w.bounds_at + up(entries * sizeof(int4));
    w.delta_at = w.dq_at + (nb > 1 ? up((size_t)B * H * N * d * sizeof(float)) : 0);
    w.lse_at = w.delta_at + up((size_t)B * H * npad * sizeof(float));
    w.sums_at = w.lse_at + up((size_t)B * H * npad * sizeof(float));
    // (no run is shorter than a block, and an item of one is never cut)
    const size_t blocks = (size_t)B * H * nb * nb, runs = H / Hkv * nb > 1 ? std::min<size_t>(fa::kSpanBwdSlots, blocks) : 0;
    w.total = w.sums_at + runs * 2 * 128 * d * sizeof(float) + 256;
    return w;
  }
};

template <int D, int MOD>
fa_status launch_span_bwd(const CUtensorMap* maps, const fa::SpanBwdParams& p, unsigned grid, cudaStream_t stream) {
  using C = fa::BwdCfg<D, true>;
  auto kernel = fa::fa_span_bwd_kernel<D, MOD>;
  if (set_smem(kernel, fa::kSpanBwdSmemBytes<D>) != cudaSuccess) return FA_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  static std::atomic<unsigned long long> known{0};
  if (!has_launch_regs(kernel, C::kLaunchRegs, dev, known)) return FA_ERR_CUDA;
  return launch_early(kernel, dim3(grid), C::kThreads, fa::kSpanBwdSmemBytes<D>, stream, maps[0], maps[1], maps[2],
                      maps[3], maps[4], maps[5], maps[6], p) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

template <int D>
fa_status run_span_bwd(const fa::SpanView<false>& view, const float* slopes, const void* q, const void* k, const void* v,
                       const void* o, const void* dout, const float* lse, void* dq, void* dk, void* dv, void* workspace,
                       int B, int H, int Hkv, float scale, float cap, cudaStream_t stream) {
  const int N = view.N, nb = (N + 127) / 128, npad = nb * 128;
  const SpanBwdWorkspace w = SpanBwdWorkspace::of(B, H, Hkv, N, D);
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
  float* dq_acc = reinterpret_cast<float*>(ws + w.dq_at);
  float* delta = reinterpret_cast<float*>(ws + w.delta_at);
  float* lse2 = reinterpret_cast<float*>(ws + w.lse_at);
  CUtensorMap maps[7];
  if (!encode_bhnd(&maps[0], q, B * H, N, D) || !encode_bhnd(&maps[1], k, B * Hkv, N, D) ||
      !encode_bhnd(&maps[2], v, B * Hkv, N, D) || !encode_bhnd(&maps[3], dout, B * H, N, D) ||
      !encode_f32_rows(&maps[4], lse2, B * H, npad, 128) || !encode_f32_rows(&maps[5], delta, B * H, npad, 128) ||
      !encode_dq_acc(&maps[6], dq_acc, B * H, N, D))
    return FA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return FA_ERR_CUDA;
  // with one key block each query block meets one item: its dQ is written where it is formed
  const bool direct = nb == 1;
  fa::SpanBwdParams p{};
  p.rows.view = view;
  p.rows.bounds = reinterpret_cast<int4*>(ws + w.bounds_at);
  p.rows.unit_heads = 1, p.rows.tile_tokens = 128, p.rows.tiles = nb, p.rows.units = H, p.rows.kv_div = H / Hkv;
  p.lo = reinterpret_cast<int*>(ws + w.lo_at);
  p.hi = reinterpret_cast<int*>(ws + w.hi_at);
  p.plan = reinterpret_cast<fa::SpanBwdPlan*>(ws);
  p.runs = reinterpret_cast<fa::SpanRun*>(ws + w.runs_at);
  p.first = reinterpret_cast<int*>(ws + w.first_at);
  p.cuts = reinterpret_cast<int4*>(ws + w.cuts_at);
  p.hulls = reinterpret_cast<int2*>(ws + w.hulls_at);
  p.order = reinterpret_cast<int*>(ws + w.order_at);
  p.sums = reinterpret_cast<float*>(ws + w.sums_at);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.dq = direct ? static_cast<__nv_bfloat16*>(dq) : nullptr;
  p.B = B, p.H = H, p.Hkv = Hkv, p.N = N, p.nb = nb;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.scale = scale;
  p.cap = span_cap(scale, cap);
  p.slopes = slopes;
  p.wait_limit_ns = wait_limit_ns();
  p.debug_stall = g_debug_stall.load();
  p.out_align32 = aligned32(dk) && aligned32(dv) && aligned32(dq);
  const long long blocks = (long long)B * H * nb * nb;  // (at most: what a mask leaves out is not known here)
  const unsigned grid = (unsigned)std::min<long long>(blocks, std::min(sms, fa::kCrossBwdMaxCtas));
  const long long rows = (long long)B * H * npad, per_block = 256 / (D / 8);
  const long long prep = std::min((rows + per_block - 1) / per_block, 152LL * 16) + ((long long)B * nb + 1) / 2;
  if (launch_early(fa::fa_span_bwd_prep_kernel<D>, dim3((unsigned)prep), 256, 0, stream,
                   static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dout), lse, delta, lse2,
                   direct ? static_cast<float*>(nullptr) : dq_acc, view, const_cast<int*>(p.lo), const_cast<int*>(p.hi),
                   const_cast<int4*>(p.rows.bounds), B, npad, rows) != cudaSuccess)
    return FA_ERR_CUDA;
  if (launch_early(fa::fa_span_plan_kernel, dim3(1), 1024, 0, stream, p) != cudaSuccess) return FA_ERR_CUDA;
  const fa_status st = cap > 0.f ? (slopes ? launch_span_bwd<D, 3>(maps, p, grid, stream) : launch_span_bwd<D, 2>(maps, p, grid, stream))
                                 : (slopes ? launch_span_bwd<D, 1>(maps, p, grid, stream) : launch_span_bwd<D, 0>(maps, p, grid, stream));
  if (st != FA_OK) return st;
  const long long n8 = direct ? 0 : (long long)B * H * N * D / 8;
  const long long post = 4LL * fa::kSpanBwdSlots + std::min((n8 + 255) / 256, 152LL * 16);
  return launch_early(fa::fa_span_bwd_post_kernel<D>, dim3((unsigned)post), 256, 0, stream, p, dq_acc,
                      static_cast<__nv_bfloat16*>(dq), n8) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t fa_span_fwd_workspace_bytes(int B, int H, int Hkv, int N, int d) {
  return check_span_shape(B, H, Hkv, N, d) == FA_OK ? SpanFwdPlan::of(B, H, 1, N, N, d, false).total : 0;
}

fa_status fa_span_fwd(const void* q, const void* k, const void* v, const int* key_begin, const int* key_end,
                      const float* slopes, void* o, float* lse, void* workspace, size_t ws_bytes, int B, int H, int Hkv,
                      int N, int d, float scale, float cap, int window, int causal, cudaStream_t stream) {
  if (!q || !k || !v || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  fa_status st = check_span_shape(B, H, Hkv, N, d);
  if (st != FA_OK) return st;
  if ((st = check_span_args(scale, cap, window, causal)) != FA_OK) return st;
  if (ws_bytes < fa_span_fwd_workspace_bytes(B, H, Hkv, N, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, o, lse, workspace}) || !all_aligned({key_begin, key_end, slopes}, 4))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k, v, o, lse, workspace})) != FA_OK) return st;
  if ((st = check_device_ptrs_given({key_begin, key_end, slopes})) != FA_OK) return st;
  SpanCall<false> a{};
  a.rows.view = {key_begin, key_end, nullptr, nullptr, nullptr, 0, 0, N, N, causal, window};
  a.rows.unit_heads = 1;
  a.rows.units = H;
  a.rows.kv_div = H / Hkv;
  a.q = q;
  a.k = {static_cast<__nv_bfloat16*>(const_cast<void*>(k)), (long long)Hkv * N * d, (long long)N * d, d};
  a.v = {static_cast<__nv_bfloat16*>(const_cast<void*>(v)), (long long)Hkv * N * d, (long long)N * d, d};
  a.box_rows = 128, a.tokens = N, a.pages = B;
  a.o = o, a.lse = lse, a.workspace = workspace;
  a.B = B, a.H = H, a.Hkv = Hkv, a.d = d, a.scale = scale, a.cap = cap, a.slopes = slopes, a.stream = stream;
  return run_span_fwd(a);
}

size_t fa_span_bwd_workspace_bytes(int B, int H, int Hkv, int N, int d) {
  return check_span_shape(B, H, Hkv, N, d) == FA_OK ? SpanBwdWorkspace::of(B, H, Hkv, N, d).total : 0;
}

fa_status fa_span_bwd(const void* q, const void* k, const void* v, const int* key_begin, const int* key_end,
                      const float* slopes, const void* o, const void* dout, const float* lse, void* dq, void* dk,
                      void* dv, void* workspace, size_t ws_bytes, int B, int H, int Hkv, int N, int d, float scale,
                      float cap, int window, int causal, cudaStream_t stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return FA_ERR_INVALID_ARG;
  fa_status st = check_span_shape(B, H, Hkv, N, d);
  if (st != FA_OK) return st;
  if ((st = check_span_args(scale, cap, window, causal)) != FA_OK) return st;
  if (ws_bytes < fa_span_bwd_workspace_bytes(B, H, Hkv, N, d)) return FA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, o, dout, lse, dq, dk, dv, workspace}) || !all_aligned({key_begin, key_end, slopes}, 4))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k, v, o, dout, lse, dq, dk, dv, workspace})) != FA_OK) return st;
  if ((st = check_device_ptrs_given({key_begin, key_end, slopes})) != FA_OK) return st;
  const fa::SpanView<false> view{key_begin, key_end, nullptr, nullptr, nullptr, 0, 0, N, N, causal, window};
  return (d == 128 ? run_span_bwd<128> : run_span_bwd<64>)(view, slopes, q, k, v, o, dout, lse, dq, dk, dv, workspace, B, H,
                                                           Hkv, scale, cap, stream);
}

size_t fa_paged_fwd_workspace_bytes(int B, int H, int Hkv, int T, int C, int d) {
  int R;
  return check_cross_shape(B, H, Hkv, T, C, d, &R) == FA_OK
             ? SpanFwdPlan::of(B, H, span_unit_heads(H / Hkv, T), T, C, d, true).total
             : 0;
}

fa_status fa_paged_fwd(const void* q, const fa_pages* k_pages, const fa_pages* v_pages, const int* page_table,
                       const int* cache_lens, const int* chunk_lens, const float* slopes, void* o, float* lse,
                       void* workspace, size_t ws_bytes, int B, int H, int Hkv, int T, int d, int num_pages,
                       int page_size, int table_width, float scale, float cap, int window, cudaStream_t stream) {
  if (!q || !page_table || !cache_lens || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  const PageShape pages{num_pages, page_size, table_width};
  fa_status st = pages.check();
  if (st != FA_OK) return st;
  int R;
  if ((st = check_cross_shape(B, H, Hkv, T, (int)pages.capacity(), d, &R)) != FA_OK) return st;
  if ((st = check_span_args(scale, cap, window, 1)) != FA_OK) return st;
  if (ws_bytes < fa_paged_fwd_workspace_bytes(B, H, Hkv, T, (int)pages.capacity(), d)) return FA_ERR_INVALID_ARG;
  for (const fa_pages* r : {k_pages, v_pages})
    if ((st = check_pages(r, pages, Hkv)) != FA_OK) return st;
  if (!all_aligned16({q, o, lse, workspace}) || !all_aligned({page_table, cache_lens, chunk_lens, slopes}, 4))
    return FA_ERR_MISALIGNED;
  if ((st = check_device_ptrs({q, k_pages->ptr, v_pages->ptr, page_table, cache_lens, o, lse, workspace})) != FA_OK)
    return st;
  if ((st = check_device_ptrs_given({chunk_lens, slopes})) != FA_OK) return st;
  SpanCall<true> a{};
  a.rows.view = {nullptr, nullptr, cache_lens, chunk_lens, page_table, table_width, pages.shift(), T,
                 (int)pages.capacity(), 1, window};
  a.rows.unit_heads = span_unit_heads(H / Hkv, T);
  a.rows.units = H / a.rows.unit_heads;
  a.rows.kv_div = a.rows.units / Hkv;
  a.q = q;
  a.k = page_rows(k_pages), a.v = page_rows(v_pages);
  a.box_rows = std::min(page_size, 128), a.tokens = page_size, a.pages = num_pages;
  a.o = o, a.lse = lse, a.workspace = workspace;
  a.B = B, a.H = H, a.Hkv = Hkv, a.d = d, a.scale = scale, a.cap = cap, a.slopes = slopes, a.stream = stream;
  return run_span_fwd(a);
}

fa_status fa_span_fwd_packed(const fa_span_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_span_fwd(a->q, a->k, a->v, a->key_begin, a->key_end, a->slopes, a->o, a->lse, a->workspace, a->ws_bytes,
                     a->B, a->H, a->Hkv, a->N, a->d, a->scale, a->cap, a->window, a->causal, a->stream);
}

fa_status fa_span_bwd_packed(const fa_span_bwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_span_bwd(a->q, a->k, a->v, a->key_begin, a->key_end, a->slopes, a->o, a->dout, a->lse, a->dq, a->dk, a->dv,
                     a->workspace, a->ws_bytes, a->B, a->H, a->Hkv, a->N, a->d, a->scale, a->cap, a->window, a->causal,
                     a->stream);
}

fa_status fa_paged_fwd_packed(const fa_paged_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_paged_fwd(a->q, &a->k_pages, &a->v_pages, a->page_table, a->cache_lens, a->chunk_lens, a->slopes, a->o,
                      a->lse, a->workspace, a->ws_bytes, a->B, a->H, a->Hkv, a->T, a->d, a->num_pages, a->page_size,
                      a->table_width, a->scale, a->cap, a->window, a->stream);
}

}  // extern "C"
