// C entry points of the operators around an FP8 projection (layer norm, the
// few-token MoE layer, low-rank adapters): argument checks and launches.
// Included by fp8q_lib.cu after its host helpers.
#pragma once

namespace {

inline bool bad_dtype(int dt) { return dt != FP8Q_OUT_BF16 && dt != FP8Q_OUT_F32; }
inline int64_t elem_size(int dt) { return dt == FP8Q_OUT_F32 ? 4 : 2; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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

// Blocks of the backward pass, and so partial rows: a function of the sizes
// alone, so that the same call always adds in the same order.
int64_t norm_bwd_blocks(int64_t M, int64_t N) {
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
template <typename T, typename W>
void launch_norm_bwd(const fp8q::LayerNormBwdArgs& a, const NormShape& sh, int64_t grid, cudaStream_t s) {
  const unsigned g = static_cast<unsigned>(grid);
  if (sh.warp_row) {
    if (sh.vpt == 1) fp8q::layer_norm_bwd_kernel<T, W, 1, true><<<g, sh.threads, 0, s>>>(a);
    else fp8q::layer_norm_bwd_kernel<T, W, 2, true><<<g, sh.threads, 0, s>>>(a);
  } else {
    if (sh.vpt == 1) fp8q::layer_norm_bwd_kernel<T, W, 1, false><<<g, sh.threads, 0, s>>>(a);
    else fp8q::layer_norm_bwd_kernel<T, W, 2, false><<<g, sh.threads, 0, s>>>(a);
  }
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
    if (param_dtype == FP8Q_OUT_BF16) launch_norm_shape<__nv_bfloat16, __nv_bfloat16>(a, sh, grid, s);
    else launch_norm_shape<__nv_bfloat16, float>(a, sh, grid, s);
  } else {
    if (param_dtype == FP8Q_OUT_BF16) launch_norm_shape<float, __nv_bfloat16>(a, sh, grid, s);
    else launch_norm_shape<float, float>(a, sh, grid, s);
  }
  return launch_status();
}

int64_t fp8q_layer_norm_backward_workspace(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || N > fp8q::kNormMaxN) return 0;
  return norm_bwd_blocks(M, N) * 2 * N;
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
                !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 4) ||
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
  a.partial = grads ? workspace : nullptr;
  const NormShape sh = norm_shape(N, kNormBwdOneVec);
  const int64_t grid = norm_bwd_blocks(M, N);
  if (x_dtype == FP8Q_OUT_BF16) {
    if (param_dtype == FP8Q_OUT_BF16) launch_norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, sh, grid, s);
    else launch_norm_bwd<__nv_bfloat16, float>(a, sh, grid, s);
  } else {
    if (param_dtype == FP8Q_OUT_BF16) launch_norm_bwd<float, __nv_bfloat16>(a, sh, grid, s);
    else launch_norm_bwd<float, float>(a, sh, grid, s);
  }
  if ((st = launch_status()) != FP8Q_OK || !grads) return st;
  fp8q::layer_norm_bwd_join_kernel<<<static_cast<unsigned>(ceil_div(2 * N, 32)), fp8q::kNormJoinThreads, 0, s>>>(
      workspace, static_cast<int>(grid), a.N, dgamma, dbeta);
  return launch_status();
}

}  // extern "C"
