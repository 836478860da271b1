// C entry points of the operators around an FP8 projection (layer norm, the
// few-token MoE layer, low-rank adapters): argument checks and launches.
// Included by fp8q_lib.cu after its host helpers.
#pragma once

namespace {

inline bool bad_dtype(int dt) { return dt != FP8Q_OUT_BF16 && dt != FP8Q_OUT_F32; }
inline int64_t elem_size(int dt) { return dt == FP8Q_OUT_F32 ? 4 : 2; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Dynamic shared memory of a kernel instance, set once per device.
template <class Kern>
fp8q_status allow_smem(Kern kern, int bytes, bool* done) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!*done) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return FP8Q_ERR_CUDA;
    *done = true;
  }
  return FP8Q_OK;
}

// Launch that may start while the kernel before it in the stream runs out; the
// kernel itself waits for that one's end (griddepcontrol.wait) before any access.
template <class Kern, class... Args>
fp8q_status launch_after(Kern kern, dim3 grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    cudaGetLastError();
    return FP8Q_ERR_CUDA;
  }
  return FP8Q_OK;
}

// How a layer norm row of N elements is laid over threads: one warp up to 512
// elements, else a block with one vector of eight elements a thread (two above
// `one_vec` elements).
struct NormShape {
  bool warp_row;
  int vpt;
  int threads;
};
NormShape norm_shape(int64_t N, int64_t one_vec) {
  NormShape s;
  const int64_t vecs = ceil_div(N, 8);
  s.warp_row = N <= fp8q::kNormWarpRowMaxN;
  s.vpt = s.warp_row ? (N <= 256 ? 1 : 2) : (N <= one_vec ? 1 : 2);
  s.threads = s.warp_row ? fp8q::kNormWarpRowThreads : static_cast<int>(ceil_div(ceil_div(vecs, s.vpt), 32) * 32);
  return s;
}
constexpr int64_t kNormFwdOneVec = 4096;    // 512 threads
constexpr int64_t kNormBwdOneVec = 8192;    // 1024 threads

// Many rows of whole vectors go through the stream kernels: from four steps an
// SM on, where the ring's start no longer shows, and while a stage of `rows`
// rows of `bytes` a column fits a third of an SM's shared memory.
bool norm_streams(int64_t M, int64_t N, int rows, int64_t bytes) {
  return N % 8 == 0 && N > fp8q::kNormWarpRowMaxN && N <= fp8q::kNormStreamMaxN && M >= 4 * 148 * rows &&
         fp8q::kNormStages * rows * N * bytes <= 192 * 1024;
}
int norm_stream_threads(int64_t N) { return static_cast<int>(ceil_div(N / 8, 64) * 32); }
// Blocks an SM of steps of `rows` rows of `bytes` a column: as many as their registers and their shared memory (the ring,
// and 3 KB a block: the joins' parts and what the system keeps) allow.
int norm_stream_blocks(int64_t N, int rows, int64_t bytes) {
  const int64_t regs = fp8q::kNormStreamThreads / norm_stream_threads(N);
  const int64_t smem = 228 * 1024 / (fp8q::kNormStages * rows * N * bytes + 3 * 1024);
  return static_cast<int>(regs < smem ? regs : smem);
}

// Blocks of the backward pass, and so partial rows: a function of the sizes
// alone, so that the same call always adds in the same order.  A block of the
// streams takes as many steps as its ring has stages at least (that is 198 blocks or more):
// 1184 x 520 BF16 8.0 us with 198 blocks, 10.8 with the 1036 that fit at once; FP32 8192 x 2048
// 39.6 us with the two blocks an SM that fit, 49.3 with three.
int64_t norm_bwd_blocks(int64_t M, int64_t N, int64_t elem) {
  if (norm_streams(M, N, fp8q::kNormBwdRows, 2 * elem)) {
    const int64_t few = ceil_div(ceil_div(M, fp8q::kNormBwdRows), fp8q::kNormStages);
    const int64_t most = 148 * norm_stream_blocks(N, fp8q::kNormBwdRows, 2 * elem);
    return few < most ? few : most;
  }
  const NormShape s = norm_shape(N, kNormBwdOneVec);
  const int64_t rows = s.warp_row ? 2 * (fp8q::kNormWarpRowThreads / 32) : 2;
  const int64_t cap = 148 * (s.threads > 512 ? 1 : (s.threads > 256 ? 2 : 4));
  const int64_t b = ceil_div(M, rows);
  return b < cap ? b : cap;
}

template <typename T, typename W, int VPT, bool kWarpRow>
void launch_norm(const fp8q::LayerNormArgs& a, int64_t grid, int threads, cudaStream_t s) {
  if (a.q != nullptr)
    fp8q::layer_norm_kernel<T, W, VPT, kWarpRow, true><<<static_cast<unsigned>(grid), threads, 0, s>>>(a);
  else
    fp8q::layer_norm_kernel<T, W, VPT, kWarpRow, false><<<static_cast<unsigned>(grid), threads, 0, s>>>(a);
}
template <typename T, typename W>
void launch_norm_shape(const fp8q::LayerNormArgs& a, const NormShape& sh, int64_t grid, cudaStream_t s) {
  if (sh.warp_row) {
    if (sh.vpt == 1) launch_norm<T, W, 1, true>(a, grid, sh.threads, s);
    else launch_norm<T, W, 2, true>(a, grid, sh.threads, s);
  } else {
    if (sh.vpt == 1) launch_norm<T, W, 1, false>(a, grid, sh.threads, s);
    else launch_norm<T, W, 2, false>(a, grid, sh.threads, s);
  }
}
template <typename T, typename W, bool kTiles>
fp8q_status launch_norm_stream(const fp8q::LayerNormArgs& a, DeviceInfo* dev, cudaStream_t s) {
  static bool done[kMaxDevices] = {};
  constexpr int R = sizeof(T) == 4 ? fp8q::kNormFwdRows32 : fp8q::kNormFwdRows16;
  constexpr int kMost = 192 * 1024;
  auto kern = fp8q::layer_norm_stream_kernel<T, W, R, kTiles>;
  fp8q_status st = allow_smem(kern, kMost, &done[dev - g_dev]);
  if (st != FP8Q_OK) return st;
  const int64_t grid = grid_for(ceil_div(a.M, R), dev->sm_count, norm_stream_blocks(a.N, R, sizeof(T)));
  kern<<<static_cast<unsigned>(grid), norm_stream_threads(a.N),
         static_cast<size_t>(fp8q::kNormStages) * R * a.N * sizeof(T), s>>>(a);
  return launch_status();
}
template <typename T, typename W>
fp8q_status launch_norm_any(const fp8q::LayerNormArgs& a, const NormShape& sh, int64_t grid, DeviceInfo* dev,
                            cudaStream_t s) {
  if (norm_streams(a.M, a.N, sizeof(T) == 4 ? fp8q::kNormFwdRows32 : fp8q::kNormFwdRows16, sizeof(T)))
    return a.q != nullptr ? launch_norm_stream<T, W, true>(a, dev, s) : launch_norm_stream<T, W, false>(a, dev, s);
  launch_norm_shape<T, W>(a, sh, grid, s);
  return launch_status();
}
template <typename T, typename W>
fp8q_status launch_norm_bwd_stream(const fp8q::LayerNormBwdArgs& a, int64_t grid, DeviceInfo* dev, cudaStream_t s) {
  static bool done[kMaxDevices] = {};
  constexpr int kRowBytes = fp8q::kNormStages * fp8q::kNormBwdRows * 2 * static_cast<int>(sizeof(T));
  auto kern = fp8q::layer_norm_bwd_stream_kernel<T, W>;
  fp8q_status st = allow_smem(kern, 192 * 1024, &done[dev - g_dev]);
  if (st != FP8Q_OK) return st;
  kern<<<static_cast<unsigned>(grid), norm_stream_threads(a.N), static_cast<size_t>(kRowBytes) * a.N, s>>>(a);
  return launch_status();
}
template <typename T, typename W>
fp8q_status launch_norm_bwd(const fp8q::LayerNormBwdArgs& a, const NormShape& sh, int64_t grid, DeviceInfo* dev,
                            cudaStream_t s) {
  if (norm_streams(a.M, a.N, fp8q::kNormBwdRows, 2 * sizeof(T))) return launch_norm_bwd_stream<T, W>(a, grid, dev, s);
  const unsigned g = static_cast<unsigned>(grid);
  if (sh.warp_row) {
    if (sh.vpt == 1) fp8q::layer_norm_bwd_kernel<T, W, 1, true><<<g, sh.threads, 0, s>>>(a);
    else fp8q::layer_norm_bwd_kernel<T, W, 2, true><<<g, sh.threads, 0, s>>>(a);
  } else {
    if (sh.vpt == 1) fp8q::layer_norm_bwd_kernel<T, W, 1, false><<<g, sh.threads, 0, s>>>(a);
    else fp8q::layer_norm_bwd_kernel<T, W, 2, false><<<g, sh.threads, 0, s>>>(a);
  }
  return launch_status();
}

template <int MODE, int RT, int S>
fp8q_status launch_few_weights(const fp8q::FewArgs& a, DeviceInfo* dev, cudaStream_t s) {
  static bool done[kMaxDevices] = {};
  using Sm = fp8q::FewSmem<MODE, RT, S>;
  auto kern = fp8q::few_weights_kernel<MODE, RT, S>;
  fp8q_status st = allow_smem(kern, Sm::kBytes, &done[dev - g_dev]);
  if (st != FP8Q_OK) return st;
  const int64_t K = MODE == fp8q::kFewDown ? a.I : a.H, rows = static_cast<int64_t>(a.E) * (MODE == fp8q::kFewDown ? a.H : a.I);
  const uint8_t* lo = MODE == fp8q::kFewDown ? a.wd : (MODE == fp8q::kFewGated ? a.wg : a.wu);
  CUtensorMap map_lo, map_hi;
  if ((st = make_tmap(&map_lo, lo, K, rows, K, MODE == fp8q::kFewGated ? 8 * RT : 16 * RT)) != FP8Q_OK) return st;
  map_hi = map_lo;
  if (MODE == fp8q::kFewGated && (st = make_tmap(&map_hi, a.wu, K, rows, K, 8 * RT)) != FP8Q_OK) return st;
  return launch_after(kern, dim3(dev->sm_count), fp8q::kFewWeightThreads, Sm::kBytes, s, map_lo, map_hi, a);
}

// Row tiles an item and stages of the up pass (RT, S) and of the down pass (RTD, SD).
template <int RT, int S, int RTD, int SD>
fp8q_status moe_few(const fp8q::FewArgs& a, int y_dtype, DeviceInfo* dev, cudaStream_t s) {
  fp8q_status st;
  fp8q::few_plan_kernel<<<static_cast<unsigned>(1 + ceil_div(static_cast<int64_t>(a.T) * (a.H / 128), 32)), 1024, 0,
                             s>>>(a);
  if ((st = launch_status()) != FP8Q_OK) return st;
  st = a.wg != nullptr ? launch_few_weights<fp8q::kFewGated, RT, S>(a, dev, s)
                       : launch_few_weights<fp8q::kFewPlain, RT, S>(a, dev, s);
  if (st != FP8Q_OK) return st;
  const int64_t chunks = a.l.max_positions * (a.I / 128);
  const int64_t grid = grid_for(ceil_div(chunks, fp8q::kFewThreads / 32), dev->sm_count, 8);
  st = launch_after(fp8q::few_hidden_kernel, dim3(static_cast<unsigned>(grid)), fp8q::kFewThreads, 0, s, a);
  if (st != FP8Q_OK) return st;
  if ((st = launch_few_weights<fp8q::kFewDown, RTD, SD>(a, dev, s)) != FP8Q_OK) return st;
  const dim3 cg(static_cast<unsigned>(ceil_div(a.H, 512)), static_cast<unsigned>(a.T));
  return y_dtype == FP8Q_OUT_F32 ? launch_after(fp8q::few_combine_kernel<float>, cg, 64, 0, s, a)
                                 : launch_after(fp8q::few_combine_kernel<__nv_bfloat16>, cg, 64, 0, s, a);
}

inline bool few_sizes_ok(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  return T <= fp8q::kFewMaxTokens && T * k <= fp8q::kFewMaxEntries && E <= fp8q::kFewMaxExperts && H <= 65536 &&
         I <= 65536;
}

// How the adapters' shrink is split: whether the groups hold more than eight
// tokens on average (blocks of 32 tokens, else of 8), and the K slices that
// give every SM work when blocks are few.  A function of the sizes alone (the
// group bounds are on the device).  Skewed groups do not turn the choice around: 256 tokens of 32
// adapters of rank 64 (blocks of 8), even, half of them on one adapter and all on one, take 33, 47 and 39 us
// beside 7168 -> 18432 BF16, 257 tokens (blocks of 32) 35, 45 and 45.
struct LoraShape {
  bool many;
  int ranks;        // an item's ranks: 16, 32 or 64
  int64_t blocks;   // at most
  int slices;
};
LoraShape lora_shape(int64_t T, int64_t K, int64_t r, int64_t groups) {
  LoraShape s;
  s.many = T > 8 * groups;
  s.ranks = r <= 16 ? 16 : (r <= 32 ? 32 : 64);
  const int64_t tile = s.many ? 32 : 8;
  s.blocks = T / tile + (groups < T ? groups : T);
  if (s.blocks > T) s.blocks = T;
  const int64_t items = s.blocks * ceil_div(r, s.ranks);
  int64_t n = (s.many ? 148 : 2 * 148) / (items < 1 ? 1 : items);
  const int64_t most = ceil_div(K, 64) / fp8q::kLoraWarps;      // a chunk a warp at least
  if (n > most) n = most;
  s.slices = static_cast<int>(n < 1 ? 1 : n);
  return s;
}

template <int RT, int G, int P, int S>
fp8q_status launch_lora_shrink(const fp8q::LoraArgs& a, const LoraShape& sh, DeviceInfo* dev, cudaStream_t s) {
  static bool done[kMaxDevices] = {};
  using Sm = fp8q::LoraSmem<RT, G, P, S>;
  auto kern = fp8q::lora_shrink_kernel<RT, G, P, S>;
  fp8q_status st = allow_smem(kern, Sm::kBytes, &done[dev - g_dev]);
  if (st != FP8Q_OK) return st;
  const int64_t grid =
      grid_for(sh.blocks * ceil_div(a.r, sh.ranks) * a.slices, dev->sm_count, Sm::kBytes <= 100 * 1024 ? 2 : 1);
  kern<<<static_cast<unsigned>(grid), fp8q::kLoraThreads, Sm::kBytes, s>>>(a);
  return launch_status();
}

// Units of columns an item of the expansion takes: the split of a block's `units`
// with the least rounds x (units + overhead) over the resident blocks; an item
// costs some 3 us before its first column (its group, tokens and v), which is
// `overhead` units.
int lora_col_units(int64_t blocks, int64_t units, int64_t resident, int64_t overhead) {
  int64_t best = units, cost = -1;
  for (int64_t parts = 1; parts <= units && parts <= 64; ++parts) {
    const int64_t u = ceil_div(units, parts);
    const int64_t c = ceil_div(blocks * ceil_div(units, u), resident) * (u + overhead);
    if (cost < 0 || c < cost) {
      cost = c;
      best = u;
    }
  }
  return static_cast<int>(best);
}

template <typename T, int KQ, int MB, int S, int WARPS>
fp8q_status launch_lora_expand(fp8q::LoraArgs a, bool after_shrink, DeviceInfo* dev, cudaStream_t s) {
  static bool done[kMaxDevices] = {};
  using Sm = fp8q::LoraExpandSmem<T, KQ, MB, S, WARPS>;
  auto kern = fp8q::lora_expand_kernel<T, KQ, MB, S, WARPS>;
  constexpr int kThreads = 32 * WARPS;
  fp8q_status st = allow_smem(kern, Sm::kBytes, &done[dev - g_dev]);
  if (st != FP8Q_OK) return st;
  const int per_sm = Sm::kBytes + static_cast<int>(sizeof(fp8q::LoraGroups)) + 1024 <= 113 * 1024 ? 2 : 1;
  int64_t blocks = a.T / (16 * MB) + (a.groups < a.T ? a.groups : a.T);
  if (blocks > a.T) blocks = a.T;
  a.col_units = lora_col_units(blocks, ceil_div(a.N, kThreads), static_cast<int64_t>(per_sm) * dev->sm_count, 1);
  const int64_t grid = grid_for(blocks * ceil_div(ceil_div(a.N, kThreads), a.col_units), dev->sm_count, per_sm);
  if (after_shrink) return launch_after(kern, dim3(static_cast<unsigned>(grid)), kThreads, Sm::kBytes, s, a);
  kern<<<static_cast<unsigned>(grid), kThreads, Sm::kBytes, s>>>(a);
  return launch_status();
}
template <typename T>
fp8q_status lora_expand_few(fp8q::LoraArgs a, bool after_shrink, DeviceInfo* dev, cudaStream_t s) {
  constexpr int kPerSm = 4;
  auto kern = fp8q::lora_expand_few_kernel<T>;
  int64_t blocks = a.T / fp8q::kLoraFewTokens + (a.groups < a.T ? a.groups : a.T);
  if (blocks > a.T) blocks = a.T;
  const int64_t units = ceil_div(a.N, fp8q::kLoraFewColumns);
  a.col_units = lora_col_units(blocks, units, static_cast<int64_t>(kPerSm) * dev->sm_count, 2);
  const int64_t grid = grid_for(blocks * ceil_div(units, a.col_units), dev->sm_count, kPerSm);
  if (after_shrink)
    return launch_after(kern, dim3(static_cast<unsigned>(grid)), fp8q::kLoraThreads, 0, s, a);
  kern<<<static_cast<unsigned>(grid), fp8q::kLoraThreads, 0, s>>>(a);
  return launch_status();
}
template <typename T>
fp8q_status lora_expand(const fp8q::LoraArgs& a, DeviceInfo* dev, cudaStream_t s) {
  constexpr bool kF32 = sizeof(T) == 4;
  const bool after = a.adapters > 0;
  // Few short rows of B a token: FP32 FMAs.  The whole call beside 7168 -> 18432 BF16 with 64 adapters, FMAs and matrix
  // instructions (us): 64 tokens of rank 8 19.1, 25.1, rank 16 22.4, 26.3, rank 32 33.0, 31.5; 128 tokens of rank 16 33.4,
  // 27.9; 300 tokens of 128 adapters of rank 16 67, 47.  The groups' average decides; on skewed groups the FMAs, which read
  // a popular adapter's B once for every two tokens (from L2), stay ahead: 64 tokens of 64 adapters of rank 16, half of
  // them on one adapter and all on one, 18.4 and 17.0, on matrix instructions (65 tokens) 35.3 and 33.8.
  if (a.r <= fp8q::kLoraFewRank && a.T <= a.groups) return lora_expand_few<T>(a, after, dev, s);
  if (a.r <= 32) return launch_lora_expand<T, 1, 2, 2, 16>(a, after, dev, s);
  if (a.r <= 64) return launch_lora_expand<T, 2, kF32 ? 1 : 2, 2, 16>(a, after, dev, s);
  return launch_lora_expand<T, 4, kF32 ? 1 : 2, 2, 8>(a, after, dev, s);
}

}  // namespace

extern "C" {

fp8q_status fp8q_layer_norm(const void* x, int x_dtype, int64_t M, int64_t N, int64_t ldx, const void* gamma,
                            const void* beta, int param_dtype, float eps, void* y, int64_t ldy, float* mean,
                            float* rstd, void* q, int64_t ldq, float* sf, int64_t ld_sf, void* stream) {
  if (bad_dtype(x_dtype) || bad_dtype(param_dtype) || M < 0 || N < 1 || ldx < N || !(eps > 0.0f) || eps > 3.0e38f)
    return FP8Q_ERR_INVALID_ARG;
  if ((q == nullptr) != (sf == nullptr) || (y == nullptr && q == nullptr && M > 0)) return FP8Q_ERR_INVALID_ARG;
  if (y != nullptr && ldy < N) return FP8Q_ERR_INVALID_ARG;
  if (q != nullptr && (N % 128 != 0 || ldq < N || ld_sf < M)) return FP8Q_ERR_INVALID_ARG;
  if (N > fp8q::kNormMaxN) return FP8Q_ERR_UNSUPPORTED;
  if (M == 0) return FP8Q_OK;
  if (x == nullptr) return FP8Q_ERR_INVALID_ARG;
  const int64_t per16 = 16 / elem_size(x_dtype);
  if (!aligned(x, 16) || ldx % per16 != 0 || !aligned(gamma, 16) || !aligned(beta, 16) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || (y != nullptr && (!aligned(y, 16) || ldy % per16 != 0)) ||
      (q != nullptr && (!aligned(q, 16) || ldq % 16 != 0 || !aligned(sf, 4))))
    return FP8Q_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  fp8q_status st = device_info(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::LayerNormArgs a{};
  a.x = x; a.M = M; a.ldx = ldx; a.N = static_cast<int>(N);
  a.gamma = gamma; a.beta = beta; a.eps = eps;
  a.y = y; a.ldy = ldy; a.mean = mean; a.rstd = rstd;
  a.q = static_cast<uint8_t*>(q); a.ldq = ldq; a.sf = sf; a.ld_sf = ld_sf;
  const NormShape sh = norm_shape(N, kNormFwdOneVec);
  const int64_t rows = sh.warp_row ? 2 * (fp8q::kNormWarpRowThreads / 32) : 2;
  const int64_t grid = grid_for(ceil_div(M, rows), dev->sm_count, 2048 / sh.threads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x_dtype == FP8Q_OUT_BF16) {
    return param_dtype == FP8Q_OUT_BF16 ? launch_norm_any<__nv_bfloat16, __nv_bfloat16>(a, sh, grid, dev, s)
                                        : launch_norm_any<__nv_bfloat16, float>(a, sh, grid, dev, s);
  }
  return param_dtype == FP8Q_OUT_BF16 ? launch_norm_any<float, __nv_bfloat16>(a, sh, grid, dev, s)
                                      : launch_norm_any<float, float>(a, sh, grid, dev, s);
}

int64_t fp8q_layer_norm_backward_workspace(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || N > fp8q::kNormMaxN) return 0;
  const int64_t b = norm_bwd_blocks(M, N, 2), f = norm_bwd_blocks(M, N, 4);     // of either type
  return (b > f ? b : f) * 2 * N;
}

fp8q_status fp8q_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int x_dtype, int64_t M,
                                     int64_t N, const void* gamma, int param_dtype, const float* mean,
                                     const float* rstd, void* dx, int64_t lddx, float* dgamma, float* dbeta,
                                     float* workspace, int64_t workspace_len, void* stream) {
  if (bad_dtype(x_dtype) || bad_dtype(param_dtype) || M < 0 || N < 1 || lddy < N || ldx < N ||
      (dx != nullptr && lddx < N))
    return FP8Q_ERR_INVALID_ARG;
  const bool grads = dgamma != nullptr || dbeta != nullptr;
  if (dx == nullptr && !grads && M > 0) return FP8Q_ERR_INVALID_ARG;
  if (N > fp8q::kNormMaxN) return FP8Q_ERR_UNSUPPORTED;
  if (M > 0) {
    if (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr) return FP8Q_ERR_INVALID_ARG;
    if (grads && (workspace == nullptr || workspace_len < fp8q_layer_norm_backward_workspace(M, N)))
      return FP8Q_ERR_INVALID_ARG;
  }
  const int64_t per16 = 16 / elem_size(x_dtype);
  if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return FP8Q_ERR_ALIGNMENT;
  if (M > 0 && (!aligned(dy, 16) || !aligned(x, 16) || lddy % per16 != 0 || ldx % per16 != 0 || !aligned(gamma, 16) ||
                !aligned(mean, 4) || !aligned(rstd, 4) || (grads && !aligned(workspace, 16)) ||
                (dx != nullptr && (!aligned(dx, 16) || lddx % per16 != 0))))
    return FP8Q_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  fp8q_status st = device_info(&dev);
  if (st != FP8Q_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {      // an empty batch's weight gradients are zero
    if (dgamma != nullptr && cudaMemsetAsync(dgamma, 0, sizeof(float) * N, s) != cudaSuccess) return FP8Q_ERR_CUDA;
    if (dbeta != nullptr && cudaMemsetAsync(dbeta, 0, sizeof(float) * N, s) != cudaSuccess) return FP8Q_ERR_CUDA;
    return FP8Q_OK;
  }
  fp8q::LayerNormBwdArgs a{};
  a.dy = dy; a.x = x; a.M = M; a.lddy = lddy; a.ldx = ldx; a.N = static_cast<int>(N);
  a.gamma = gamma; a.mean = mean; a.rstd = rstd; a.dx = dx; a.lddx = lddx;
  a.partial = grads ? workspace : nullptr; a.partial_len = workspace_len;
  const NormShape sh = norm_shape(N, kNormBwdOneVec);
  const int64_t grid = norm_bwd_blocks(M, N, elem_size(x_dtype));
  if (x_dtype == FP8Q_OUT_BF16) {
    st = param_dtype == FP8Q_OUT_BF16 ? launch_norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, sh, grid, dev, s)
                                      : launch_norm_bwd<__nv_bfloat16, float>(a, sh, grid, dev, s);
  } else {
    st = param_dtype == FP8Q_OUT_BF16 ? launch_norm_bwd<float, __nv_bfloat16>(a, sh, grid, dev, s)
                                      : launch_norm_bwd<float, float>(a, sh, grid, dev, s);
  }
  if (st != FP8Q_OK || !grads) return st;
  return launch_after(fp8q::layer_norm_bwd_join_kernel, dim3(static_cast<unsigned>(ceil_div(2 * N, 32))),
                      fp8q::kNormJoinThreads, 0, s, static_cast<const float*>(workspace), static_cast<int>(grid), a.N,
                      dgamma, dbeta);
}

int64_t fp8q_moe_few_tokens_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  if (T <= 0 || k < 1 || k > fp8q::kFewMaxEntries || E < 1 || H < 128 || I < 128 || H % 128 != 0 || I % 128 != 0 ||
      !few_sizes_ok(T, k, E, H, I))
    return 0;
  return fp8q::few_layout(T, k, E, H, I).bytes;
}

fp8q_status fp8q_moe_few_tokens(const void* x, int64_t T, int64_t H, int64_t ldx, const int32_t* expert_ids,
                                const float* expert_weights, int64_t k, int64_t E, const void* w_gate,
                                const float* sf_gate, const void* w_up, const float* sf_up, const void* w_down,
                                const float* sf_down, int64_t I, void* y, int64_t ldy, int y_dtype, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  if (T < 0 || k < 1 || k > fp8q::kFewMaxEntries || E < 1 || H < 128 || H % 128 != 0 || I < 128 || I % 128 != 0 ||
      ldx < H || ldy < H || bad_dtype(y_dtype) || (w_gate == nullptr) != (sf_gate == nullptr))
    return FP8Q_ERR_INVALID_ARG;
  if (!few_sizes_ok(T, k, E, H, I)) return FP8Q_ERR_UNSUPPORTED;
  if (T == 0) return FP8Q_OK;
  if (x == nullptr || expert_ids == nullptr || expert_weights == nullptr || w_up == nullptr || sf_up == nullptr ||
      w_down == nullptr || sf_down == nullptr || y == nullptr || workspace == nullptr)
    return FP8Q_ERR_INVALID_ARG;
  if (workspace_bytes < fp8q_moe_few_tokens_workspace(T, k, E, H, I)) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(y, 16) || ldy % (16 / elem_size(y_dtype)) != 0 ||
      !aligned(expert_ids, 4) || !aligned(expert_weights, 4) || !aligned(w_gate, 16) || !aligned(w_up, 16) ||
      !aligned(w_down, 16) || !aligned(sf_gate, 4) || !aligned(sf_up, 4) || !aligned(sf_down, 4) ||
      !aligned(workspace, 256))
    return FP8Q_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  fp8q_status st = device_info(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::FewArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x); a.ldx = ldx;
  a.T = static_cast<int>(T); a.k = static_cast<int>(k); a.E = static_cast<int>(E);
  a.H = static_cast<int>(H); a.I = static_cast<int>(I);
  a.ids = expert_ids; a.share = expert_weights;
  a.wg = static_cast<const uint8_t*>(w_gate); a.wu = static_cast<const uint8_t*>(w_up);
  a.wd = static_cast<const uint8_t*>(w_down);
  a.sg = sf_gate; a.su = sf_up; a.sd = sf_down;
  a.y = y; a.ldy = ldy;
  a.ws = static_cast<uint8_t*>(workspace);
  a.l = fp8q::few_layout(T, k, E, H, I);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Row tiles an item: few entries need small items to fill the SMs evenly, many are better off with fewer, larger
  // boxes; the down pass, with two parts a column, has room for four stages only from 4 tiles on.  7168 -> 2048 -> 7168,
  // top-8, the call's device time with 2, 4 and 8 tiles (us, a few calls at 1965 MHz): 1 token 72.6, 76.1, 76.8; 4 tokens
  // 201, 204, 212; 16 tokens (64 experts, no gate) 219, 220, 226; 128 tokens 1506, 1429, 1429.  2 tiles and three stages
  // in the down pass too: 1 token 74.6, 16 tokens 234.
  if (T * k <= 64) return moe_few<2, 4, 4, 4>(a, y_dtype, dev, s);
  return T * k <= 512 ? moe_few<4, 5, 4, 4>(a, y_dtype, dev, s) : moe_few<8, 5, 8, 5>(a, y_dtype, dev, s);
}

int64_t fp8q_lora_apply_workspace(int64_t T, int64_t K, int64_t r, int64_t groups) {
  if (T <= 0 || K < 8 || K % 8 != 0 || r < 8 || r % 8 != 0 || r > fp8q::kLoraMaxRank || groups < 1 ||
      groups > fp8q::kLoraMaxGroups)
    return 0;
  return lora_shape(T, K, r, groups).slices * T * r;
}

fp8q_status fp8q_lora_apply(const void* x, int64_t T, int64_t K, int64_t ldx, const int32_t* rows,
                            const int32_t* group_offsets, int64_t groups, const void* a, const void* b, int64_t r,
                            const float* scaling, int64_t adapters, const void* base, int64_t ldb, void* out,
                            int64_t ldo, int dtype, int64_t N, float* workspace, int64_t workspace_len, void* stream) {
  if (T < 0 || K < 8 || K % 8 != 0 || N < 8 || N % 8 != 0 || r < 8 || r % 8 != 0 || ldx < K || ldb < N || ldo < N ||
      groups < 1 || adapters < 0 || bad_dtype(dtype))
    return FP8Q_ERR_INVALID_ARG;
  if (r > fp8q::kLoraMaxRank || groups > fp8q::kLoraMaxGroups || adapters > 0x7FFFFFFF || T > (1 << 24) ||
      K > (1 << 24) || N > (1 << 24))
    return FP8Q_ERR_UNSUPPORTED;
  if (T == 0) return FP8Q_OK;
  if (x == nullptr || rows == nullptr || group_offsets == nullptr || base == nullptr || out == nullptr ||
      workspace == nullptr || (adapters > 0 && (a == nullptr || b == nullptr)))
    return FP8Q_ERR_INVALID_ARG;
  if (base == out && ldb != ldo) return FP8Q_ERR_INVALID_ARG;
  if (workspace_len < fp8q_lora_apply_workspace(T, K, r, groups)) return FP8Q_ERR_INVALID_ARG;
  const int64_t per16 = 16 / elem_size(dtype);
  if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(a, 16) || !aligned(b, 16) || !aligned(base, 16) || ldb % per16 != 0 ||
      !aligned(out, 16) || ldo % per16 != 0 || !aligned(rows, 4) || !aligned(group_offsets, 4) || !aligned(scaling, 4) ||
      !aligned(workspace, 16))
    return FP8Q_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  fp8q_status st = device_info(&dev);
  if (st != FP8Q_OK) return st;
  const LoraShape sh = lora_shape(T, K, r, groups);
  fp8q::LoraArgs g{};
  g.x = static_cast<const __nv_bfloat16*>(x); g.T = T; g.ldx = ldx;
  g.K = static_cast<int>(K); g.N = static_cast<int>(N); g.r = static_cast<int>(r);
  g.groups = static_cast<int>(groups); g.adapters = static_cast<int>(adapters);
  g.rows = rows; g.offsets = group_offsets;
  g.a = static_cast<const __nv_bfloat16*>(a); g.b = static_cast<const __nv_bfloat16*>(b); g.scaling = scaling;
  g.base = base; g.ldb = ldb; g.out = out; g.ldo = ldo;
  g.v = workspace; g.v_len = workspace_len; g.slices = sh.slices;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (adapters > 0) {
    if (sh.many)
      st = sh.ranks == 16   ? launch_lora_shrink<1, 4, 1, 4>(g, sh, dev, s)
           : sh.ranks == 32 ? launch_lora_shrink<2, 4, 1, 4>(g, sh, dev, s)
                            : launch_lora_shrink<4, 4, 1, 3>(g, sh, dev, s);
    else
      st = sh.ranks == 16   ? launch_lora_shrink<1, 1, 2, 4>(g, sh, dev, s)
           : sh.ranks == 32 ? launch_lora_shrink<2, 1, 2, 4>(g, sh, dev, s)
                            : launch_lora_shrink<4, 1, 2, 2>(g, sh, dev, s);
    if (st != FP8Q_OK) return st;
  }
  return dtype == FP8Q_OUT_F32 ? lora_expand<float>(g, dev, s) : lora_expand<__nv_bfloat16>(g, dev, s);
}

}  // extern "C"
