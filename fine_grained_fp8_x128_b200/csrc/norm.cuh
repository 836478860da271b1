// Layer norm in front of an FP8 projection: forward (into x's type and/or into
// the projection's 1x128 E4M3 tiles) and backward (input, weight and bias
// gradients).  Each element of the inputs is read from HBM once, and the outputs
// leave in the same pass.  The row kernels, for short calls, hold a pair of rows
// in registers; the streams, for many rows, hold them in a ring in shared memory
// and read it twice, for the sums and for the outputs.  By its bytes either is
// HBM's work; what bounds the streams stands there.
//
//   mu = sum x / N,  v = sum (x - mu)^2 / N,  r = 1 / sqrt(v + eps)
//   xh = (x - mu) r,  y = xh gamma + beta
//   backward, g = dy gamma:  dx = r (g - mean(g) - xh mean(g xh))
//   dgamma = sum_m dy xh,  dbeta = sum_m dy
//
// All sums and statistics are FP32.  The variance is the mean square of the
// deviations (never E[x^2] - mu^2, which cancels when |mu| >> sigma): a warp
// takes the deviations from its own mean, and the warps' (sum, M2) are joined
// by the pairwise update of Chan, Golub and LeVeque ("Updating formulae and a
// pairwise algorithm for computing sample variances", 1979), so that a row
// needs one block barrier instead of two.
#pragma once

#include "quant.cuh"

namespace fp8q {

constexpr int kNormMaxN = 16384;       // 1024 threads x 2 vectors of 8 elements
constexpr int kNormWarpRowMaxN = 512;  // up to here one warp owns a row
constexpr int kNormWarpRowThreads = 128;

struct LayerNormArgs {
  const void* x;
  int64_t M, ldx;
  int N;
  const void* gamma;   // may be null: ones
  const void* beta;    // may be null: zeros
  float eps;
  void* y;             // may be null
  int64_t ldy;
  float* mean;         // may be null
  float* rstd;         // may be null
  uint8_t* q;
  int64_t ldq;
  float* sf;
  int64_t ld_sf;
};

// Programmatic dependent launch: let the next launch of the stream begin; wait
// for the end of the launch before (and so, as every launch waits, of all before).
// What the launch before wrote is read through plain pointers: a load the compiler
// may take for one of constant memory (__ldg, const __restrict__) could be moved
// ahead of the wait.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A warp's wait on a barrier.  It has to leave the warp converged: called under a
// condition the compiler cannot see to be uniform (`if (ok) ok = wait`), the warp
// went on in two halves and issued the whole loop body twice (forward stream
// 110 us instead of 66).  So it is called without one, and ends in a __syncwarp;
// after a wait that gave up, the later ones return at once.
__device__ __forceinline__ bool warp_wait_converged(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t where) {
  const bool ok = warp_wait(bar, parity, abort, where);
  __syncwarp();
  return ok;
}

// Eight consecutive elements as they lie in memory (BF16: one 16-byte word,
// FP32: two).
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};

// The first `valid` (0..8) elements from p (16-byte aligned), the rest zero.
template <typename T, bool kStream>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* __restrict__ p, int valid) {
  constexpr int kW = sizeof(T) / 2;
  if (valid == 8) {
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(p) + i;
      r.w[i] = kStream ? __ldcs(src) : __ldg(src);
    }
    return;
  }
  uint32_t u[4 * kW];
#pragma unroll
  for (int i = 0; i < 4 * kW; ++i) u[i] = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j < valid) {
      if (sizeof(T) == 4) {
        u[j] = __ldg(reinterpret_cast<const uint32_t*>(p) + j);
      } else {
        const uint32_t h = __ldg(reinterpret_cast<const unsigned short*>(p) + j);
        u[j / 2] |= h << (16 * (j & 1));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kW; ++i) r.w[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
}

__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&f)[8]) {
  const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(u[i]);
    f[2 * i + 1] = bf16hi(u[i]);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&f)[8]) {
  const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void pack8(Raw8<__nv_bfloat16>& r, const float (&f)[8]) {
  r.w[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void pack8(Raw8<float>& r, const float (&f)[8]) {
  r.w[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  r.w[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
}

// The first `valid` elements of r to p; what lies behind them is not touched.
template <typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, const Raw8<T>& r, int valid) {
  constexpr int kW = sizeof(T) / 2;
  if (valid == 8) {
#pragma unroll
    for (int i = 0; i < kW; ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (sizeof(T) == 4) {
        if (4 * i + k < valid) reinterpret_cast<uint32_t*>(p)[4 * i + k] = u[k];
      } else {
        if (2 * k < valid) reinterpret_cast<unsigned short*>(p)[2 * k] = static_cast<unsigned short>(u[k]);
        if (2 * k + 1 < valid) reinterpret_cast<unsigned short*>(p)[2 * k + 1] = static_cast<unsigned short>(u[k] >> 16);
      }
    }
  }
}

// gamma or beta (may be null: `none` in every place) of vector v.
template <typename W>
__device__ __forceinline__ void load_param8(float (&f)[8], const void* p, int64_t v, int valid, float none) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = none;
    return;
  }
  Raw8<W> r;
  load8<W, false>(r, static_cast<const W*>(p) + v * 8, valid);
  unpack8(r, f);
}

// Sums of two values over the warp: the lower half-warp ends with the total
// of a, the upper with that of b (one exchange, then four steps within the halves).
__device__ __forceinline__ float warp_sum2(float a, float b, int lane) {
  const bool up = (lane & 16) != 0;
  const float give = up ? a : b;
  float keep = up ? b : a;
  keep += __shfl_xor_sync(0xFFFFFFFFu, give, 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) keep += __shfl_xor_sync(0xFFFFFFFFu, keep, o);
  return keep;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// Four values: lanes 8i .. 8i+7 end with the total of value i.
__device__ __forceinline__ float warp_sum4(float a, float b, float c, float d, int lane) {
  const bool up = (lane & 16) != 0;
  float k0 = up ? c : a, k1 = up ? d : b;
  k0 += __shfl_xor_sync(0xFFFFFFFFu, up ? a : c, 16);
  k1 += __shfl_xor_sync(0xFFFFFFFFu, up ? b : d, 16);
  const bool up2 = (lane & 8) != 0;
  float k = up2 ? k1 : k0;
  k += __shfl_xor_sync(0xFFFFFFFFu, up2 ? k0 : k1, 8);
#pragma unroll
  for (int o = 4; o; o >>= 1) k += __shfl_xor_sync(0xFFFFFFFFu, k, o);
  return k;
}

// Elements of a row that warp `w` of a row group with `warps` warps holds.
template <int VPT>
__device__ __forceinline__ int norm_warp_count(int N, int w, int warps) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) n += min(max(N - 256 * (i * warps + w), 0), 256);
  return n;
}

// ---------------------------------------------------------------------------
// Forward.  A row group (one warp for N <= 512, else the block) takes two rows
// at a time: one barrier and one read of gamma and beta serve both, and twice
// the bytes are in flight.  Thread t holds vectors t, t + nt, ... of eight
// elements, so 16 consecutive lanes hold one 128-element tile and a tile's
// maximum is four shuffles.  The tiles quantize y before any rounding to BF16.
// ---------------------------------------------------------------------------
template <typename T, typename W, int VPT, bool kWarpRow, bool kTiles>
__global__ void __launch_bounds__(kWarpRow ? kNormWarpRowThreads : (VPT == 1 ? 512 : 1024))
layer_norm_kernel(const LayerNormArgs a) {
  __shared__ float2 part[2][32][2];     // [row-pair parity][warp][row] = (sum, M2)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nt = kWarpRow ? 32 : blockDim.x;
  const int t = kWarpRow ? lane : threadIdx.x;
  const int warps = nt >> 5;
  const int64_t group = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (kNormWarpRowThreads / 32) + warp : blockIdx.x;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kWarpRow ? kNormWarpRowThreads / 32 : 1);
  const int N = a.N;
  // true divisions by the counts: a row of one value has exactly that mean and no deviations where its sums are exact
  const float n_f = static_cast<float>(N);
  const float nw_f = static_cast<float>(max(norm_warp_count<VPT>(N, kWarpRow ? 0 : warp, warps), 1));
  int parity = 0;
  for (int64_t row0 = group * 2; row0 < a.M; row0 += groups * 2, parity ^= 1) {
    Raw8<T> raw[2][VPT];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nt + t;
        const int valid = row0 + r < a.M ? min(max(N - 8 * v, 0), 8) : 0;
        load8<T, true>(raw[r][i], static_cast<const T*>(a.x) + (row0 + r) * a.ldx + 8 * static_cast<int64_t>(v), valid);
      }
    }
    // the warp's sums, then its deviations from its own means
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float f[8];
        unpack8(raw[r][i], f);
        sum[r] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
      }
    }
    const float wsum = warp_sum2(sum[0], sum[1], lane);       // this half's row
    const float wmean = __fdiv_rn(wsum, nw_f);
    const float mw[2] = {__shfl_sync(0xFFFFFFFFu, wmean, 0), __shfl_sync(0xFFFFFFFFu, wmean, 16)};
    float m2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float f[8];
        unpack8(raw[r][i], f);
        const int valid = min(max(N - 8 * (i * nt + t), 0), 8);
        if (valid == 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = f[j] - mw[r];
            m2[r] = fmaf(d, d, m2[r]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = j < valid ? f[j] - mw[r] : 0.0f;
            m2[r] = fmaf(d, d, m2[r]);
          }
        }
      }
    }
    const float wm2 = warp_sum2(m2[0], m2[1], lane);
    float mean_h, m2_h;                                       // of this half-warp's row
    if (kWarpRow) {
      mean_h = wmean;
      m2_h = wm2;
    } else {
      if ((lane & 15) == 0) part[parity][warp][lane >> 4] = make_float2(wsum, wm2);
      __syncthreads();
      // half-warp h joins row h's warps: lane l takes warps l and l + 16.  The
      // next pair writes the other buffer, so one barrier a pair is enough.
      const int h = lane >> 4, w0 = lane & 15, w1 = w0 + 16;
      const float2 p0 = w0 < warps ? part[parity][w0][h] : make_float2(0.0f, 0.0f);
      const float2 p1 = w1 < warps ? part[parity][w1][h] : make_float2(0.0f, 0.0f);
      mean_h = __fdiv_rn(half_warp_sum(p0.x + p1.x), n_f);
      float s = 0.0f;
      if (w0 < warps) {
        const int n0 = norm_warp_count<VPT>(N, w0, warps);
        const float d = n0 > 0 ? __fdiv_rn(p0.x, static_cast<float>(n0)) - mean_h : 0.0f;
        s = fmaf(static_cast<float>(n0) * d, d, p0.y);
      }
      if (w1 < warps) {
        const int n1 = norm_warp_count<VPT>(N, w1, warps);
        const float d = n1 > 0 ? __fdiv_rn(p1.x, static_cast<float>(n1)) - mean_h : 0.0f;
        s += fmaf(static_cast<float>(n1) * d, d, p1.y);
      }
      m2_h = half_warp_sum(s);
    }
    const float rstd_h = __frcp_rn(__fsqrt_rn(__fdiv_rn(m2_h, n_f) + a.eps));
    const float mean[2] = {__shfl_sync(0xFFFFFFFFu, mean_h, 0), __shfl_sync(0xFFFFFFFFu, mean_h, 16)};
    const float rstd[2] = {__shfl_sync(0xFFFFFFFFu, rstd_h, 0), __shfl_sync(0xFFFFFFFFu, rstd_h, 16)};
    if (t < 2 && row0 + t < a.M) {
      if (a.mean != nullptr) a.mean[row0 + t] = t ? mean[1] : mean[0];
      if (a.rstd != nullptr) a.rstd[row0 + t] = t ? rstd[1] : rstd[0];
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nt + t;
      const int valid = min(max(N - 8 * v, 0), 8);
      float ga[8], be[8];
      load_param8<W>(ga, a.gamma, v, valid, 1.0f);
      load_param8<W>(be, a.beta, v, valid, 0.0f);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float f[8];
        unpack8(raw[r][i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = fmaf((f[j] - mean[r]) * rstd[r], ga[j], be[j]);
        const bool live = row0 + r < a.M;
        if (a.y != nullptr && live && valid > 0 &&
            chk((row0 + r) * a.ldy + 8 * v + valid - 1, rows_extent(a.M, N, a.ldy), CHK_NORM)) {
          Raw8<T> o;
          pack8(o, f);
          store8(static_cast<T*>(a.y) + (row0 + r) * a.ldy + 8 * static_cast<int64_t>(v), o, valid);
        }
        if (kTiles) {
          float m = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
#pragma unroll
          for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const float s = tile_scale(m);
          const float nr = -__frcp_rn(s);
          // y is an FP32 value here, outside the domain on which the corrected
          // quotient was shown equal to the IEEE one: it may be one FP32 step
          // off, which y's own FP32 rounding already is.
          if (live && valid == 8) {
            uint32_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = e4m3x2_neg_quot(f[2 * j], f[2 * j + 1], nr, nr, s, s);
            uint2 o;
            o.x = (c[0] | (c[1] << 16)) ^ kFlipSigns;
            o.y = (c[2] | (c[3] << 16)) ^ kFlipSigns;
            if (chk((row0 + r) * a.ldq + 8 * v + 7, rows_extent(a.M, N, a.ldq), CHK_Q1))
              *reinterpret_cast<uint2*>(a.q + (row0 + r) * a.ldq + 8 * static_cast<int64_t>(v)) = o;
            if ((lane & 15) == 0 && chk((v >> 4) * a.ld_sf + row0 + r, rows_extent(N / 128, a.M, a.ld_sf), CHK_Q1_SF))
              a.sf[(v >> 4) * a.ld_sf + row0 + r] = s;
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Streams, for many rows of 512 < N <= 7168 whole vectors: a block per SM (more
// where rows are short), two vectors of eight columns a thread, and a ring of
// kNormStages stages of rows in shared memory that bulk copies fill ahead, so
// that HBM stays busy while a step's rows are reduced.  gamma, beta and the
// columns' gradients stay in registers for all rows of the block; the rows are
// read from the ring twice, for the sums and for the outputs, rather than kept in
// registers, which spilled.  A step's block barrier also tells that the step
// before is done with its stage.  8192 x 7168 BF16, tiles and backward: 54.5 and
// 70 us (and 4.5 for the join), at 32 and 55 % of DRAM.  Neither HBM nor the issue
// of instructions (57 and 53 % of the slots) is full: what bounds these kernels is
// the latency of a step's two halves and the barrier between them, with 14 warps an SM.
// Rows kept in registers took 57 and 94 us, one vector a thread (twice the warps
// for the joins) 59 and 93, two rows a step forward 62; the row kernels, which
// load a step's rows when it begins, 85 and 126.
// ---------------------------------------------------------------------------
constexpr int kNormStages = 3;
// Two vectors a thread of rows of up to 7168; the kernels take up to 128 registers.  More threads (512 would fit, for 8192
// columns) have not been measured.
constexpr int kNormStreamThreads = 448;
constexpr int kNormStreamMaxN = 16 * kNormStreamThreads;
constexpr int kNormFwdRows16 = 4, kNormFwdRows32 = 2;      // rows a step, BF16 and FP32
constexpr int kNormBwdRows = 2;                            // of x and of dy

__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float2 (&f)[4]) {
  const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(bf16lo(u[i]), bf16hi(u[i]));
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float2 (&f)[4]) {
  f[0] = f2u(r.w[0].x, r.w[0].y);
  f[1] = f2u(r.w[0].z, r.w[0].w);
  f[2] = f2u(r.w[1].x, r.w[1].y);
  f[3] = f2u(r.w[1].z, r.w[1].w);
}
__device__ __forceinline__ void pack8(Raw8<__nv_bfloat16>& r, const float2 (&f)[4]) {
  r.w[0] = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ void pack8(Raw8<float>& r, const float2 (&f)[4]) {
  r.w[0] = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
  r.w[1] = make_uint4(__float_as_uint(f[2].x), __float_as_uint(f[2].y), __float_as_uint(f[3].x), __float_as_uint(f[3].y));
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float sum8(const float2 (&f)[4]) {
  const float2 s = fadd2(fadd2(f[0], f[1]), fadd2(f[2], f[3]));
  return s.x + s.y;
}
// Sum over 32 lanes of R values (2 or 4): lanes (32 / R) i .. end with that of value i.
template <int R>
__device__ __forceinline__ float warp_sum_rows(const float (&v)[R], int lane) {
  if constexpr (R == 2) return warp_sum2(v[0], v[1], lane);
  else return warp_sum4(v[0], v[1], v[2], v[3], lane);
}
// Sum over the 32 / R lanes that share a row.
template <int R>
__device__ __forceinline__ float row_lanes_sum(float v) {
#pragma unroll
  for (int o = 16 / R; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// x / n, correctly rounded, with inv = fl(1 / n): a product and one correction
// step of Markstein's division (see e4m3x2_neg_quot).
__device__ __forceinline__ float div_by(float x, float n, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, n, x), inv, q);
}

// What a thread, a warp and a row of a stream hold: two vectors a thread, t and
// t + T of the row's N / 8.
struct NormStream {
  int N, t, lane, warp, warps;
  bool mine[2];
  float n, inv_n;          // of the row
  float n_w, inv_nw;       // of this warp
  float inv_nt;            // of this thread
  __device__ __forceinline__ explicit NormStream(int N_) : N(N_) {
    t = threadIdx.x;
    lane = t & 31;
    warp = t >> 5;
    warps = blockDim.x >> 5;
    mine[0] = 8 * t < N;
    mine[1] = 8 * (t + static_cast<int>(blockDim.x)) < N;
    n = static_cast<float>(N);
    inv_n = __frcp_rn(n);
    n_w = count(warp);
    inv_nw = __frcp_rn(fmaxf(n_w, 1.0f));
    inv_nt = mine[1] ? 0.0625f : 0.125f;
  }
  __device__ __forceinline__ float count(int w) const {      // of warp w
    return w < warps ? static_cast<float>(norm_warp_count<2>(N, w, warps)) : 0.0f;
  }
  __device__ __forceinline__ int vec(int i) const { return t + i * static_cast<int>(blockDim.x); }
};

template <typename T>
__device__ __forceinline__ void stream_read(Raw8<T>& r, const uint8_t* row, int vec, bool live) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    r.w[i] = live ? reinterpret_cast<const uint4*>(row + vec * 8 * sizeof(T))[i] : make_uint4(0, 0, 0, 0);
}
template <typename W>
__device__ __forceinline__ void stream_param(float2 (&p)[4], const void* src, int vec, bool live, float none) {
  float f[8];
  load_param8<W>(f, src, vec, live ? 8 : 0, none);
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = make_float2(f[2 * j], f[2 * j + 1]);
}

template <typename T, typename W, int R, bool kTiles>
__global__ void __launch_bounds__(kNormStreamThreads, 1) layer_norm_stream_kernel(const LayerNormArgs a) {
  constexpr int kL = 32 / R;                     // lanes that share a row in the warps' joins
  constexpr int kJoin = (kNormStreamThreads / 32 + kL - 1) / kL;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 part[2][32][R];
  __shared__ __align__(8) uint64_t full[kNormStages];
  __shared__ int abort_flag;
  const NormStream c(a.N);
  const int t = c.t, lane = c.lane;
  const uint32_t row_bytes = a.N * sizeof(T);
  const int64_t steps = (a.M + R - 1) / R;
  if (t == 0) {
#pragma unroll
    for (int s = 0; s < kNormStages; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  uint32_t issued = 0;
  auto request = [&](int64_t step, int s) {      // thread 0
    const int64_t row0 = step * R;
    const int rows = static_cast<int>(a.M - row0 < R ? a.M - row0 : R);
    ++issued;
    mbar_arrive_expect_tx(&full[s], rows * row_bytes);
    for (int r = 0; r < rows; ++r)
      bulk_load(smem + (s * R + r) * row_bytes, static_cast<const T*>(a.x) + (row0 + r) * a.ldx, row_bytes, &full[s]);
  };
  if (t == 0) {
    int s = 0;
    for (int64_t step = blockIdx.x; step < steps && s < kNormStages; step += gridDim.x, ++s) request(step, s);
  }
  float2 ga[2][4], be[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    stream_param<W>(ga[i], a.gamma, c.vec(i), c.mine[i], 1.0f);
    stream_param<W>(be[i], a.beta, c.vec(i), c.mine[i], 0.0f);
  }
  // the warps whose parts this lane joins: of row lane / kL
  float count[kJoin];
#pragma unroll
  for (int k = 0; k < kJoin; ++k) count[k] = c.count(lane % kL + kL * k);
  int stage = 0, parity = 0;
  uint32_t phase = 0;
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x, parity ^= 1) {
    warp_wait_converged(&full[stage], phase, &abort_flag, WAIT_STAGE);
    float sum[R], m2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // the thread's sum, and its deviations from its own mean
      float2 f[2][4], q = f2(0.0f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Raw8<T> raw;
        stream_read(raw, smem + (stage * R + r) * row_bytes, c.vec(i), c.mine[i]);
        unpack8(raw, f[i]);
      }
      sum[r] = sum8(f[0]) + sum8(f[1]);
      const float2 m = f2(-c.inv_nt * sum[r]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (c.mine[i]) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 d = fadd2(f[i][j], m);
            q = ffma2(d, d, q);
          }
        }
      }
      m2[r] = q.x + q.y;
    }
    // the warp's: the deviations add up to the threads' own and those of their means
    const float wsum = warp_sum_rows<R>(sum, lane);
    const float wmean = div_by(wsum, fmaxf(c.n_w, 1.0f), c.inv_nw);
    const float n_t = c.mine[1] ? 16.0f : (c.mine[0] ? 8.0f : 0.0f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float d = fmaf(c.inv_nt, sum[r], -__shfl_sync(0xFFFFFFFFu, wmean, r * kL));
      m2[r] = fmaf(n_t * d, d, m2[r]);
    }
    const float wm2 = warp_sum_rows<R>(m2, lane);
    if (lane % kL == 0) part[parity][c.warp][lane / kL] = make_float2(wmean, wm2);
    __syncthreads();
    // all are done with the stage of the step before: request the step that comes into it
    const int64_t coming = step + (kNormStages - 1) * static_cast<int64_t>(gridDim.x);
    if (t == 0 && step > blockIdx.x && coming < steps) {
      fence_proxy_async_shared();
      request(coming, stage > 0 ? stage - 1 : kNormStages - 1);
    }
    const uint8_t* rows_at = smem + stage * R * row_bytes;
    if (++stage == kNormStages) {
      stage = 0;
      phase ^= 1;
    }
    // the row's, in the same way from the warps
    float2 p[kJoin];
    float total = 0.0f, dev = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      const int w = lane % kL + kL * k;
      p[k] = w < c.warps ? part[parity][w][lane / kL] : make_float2(0.0f, 0.0f);
      total = fmaf(count[k], p[k].x, total);
    }
    const float mean_l = div_by(row_lanes_sum<R>(total), c.n, c.inv_n);
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      const float d = p[k].x - mean_l;
      dev += fmaf(count[k] * d, d, p[k].y);
    }
    // as the row kernels round it; the hardware's approximate reciprocal root is off by up to two FP32 steps (and took
    // 53.3 us where this takes 54.5 for 8192 x 7168 BF16 into tiles)
    const float rstd_l = __frcp_rn(__fsqrt_rn(div_by(row_lanes_sum<R>(dev), c.n, c.inv_n) + a.eps));
    const int64_t row0 = step * R;
    if (c.warp == 0 && lane % kL == 0 && row0 + lane / kL < a.M) {
      if (a.mean != nullptr) a.mean[row0 + lane / kL] = mean_l;
      if (a.rstd != nullptr) a.rstd[row0 + lane / kL] = rstd_l;
    }
#pragma unroll
    for (int r0 = 0; r0 < R; r0 += 2) {          // two rows, and so four tiles, at a time
      float2 y[2][2][4];
      float amax[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = r0 + u;
        const float2 m = f2(-__shfl_sync(0xFFFFFFFFu, mean_l, r * kL)), k = f2(__shfl_sync(0xFFFFFFFFu, rstd_l, r * kL));
        const bool live = row0 + r < a.M;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 (&f)[4] = y[u][i];
          Raw8<T> raw;
          stream_read(raw, rows_at + r * row_bytes, c.vec(i), c.mine[i]);
          unpack8(raw, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = ffma2(fmul2(fadd2(f[j], m), k), ga[i][j], be[i][j]);
          if (a.y != nullptr && c.mine[i] && live &&
              chk((row0 + r) * a.ldy + 8 * c.vec(i) + 7, rows_extent(a.M, a.N, a.ldy), CHK_NORM)) {
            Raw8<T> o;
            pack8(o, f);
            store8(static_cast<T*>(a.y) + (row0 + r) * a.ldy + 8 * c.vec(i), o, 8);
          }
          if (kTiles) {
            float m4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) m4[j] = fmaxf(fabsf(f[j].x), fabsf(f[j].y));
            amax[2 * u + i] = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          }
        }
      }
      if constexpr (kTiles) {
        // the four tiles' maxima over 16 lanes: lanes 4 i .. 4 i + 3 of the 16 end
        // with that of tile i = 2 (row) + (vector), and so its scale
        const bool up = (lane & 8) != 0, up2 = (lane & 4) != 0;
        const float k0 = fmaxf(up ? amax[2] : amax[0], __shfl_xor_sync(0xFFFFFFFFu, up ? amax[0] : amax[2], 8));
        const float k1 = fmaxf(up ? amax[3] : amax[1], __shfl_xor_sync(0xFFFFFFFFu, up ? amax[1] : amax[3], 8));
        float m = fmaxf(up2 ? k1 : k0, __shfl_xor_sync(0xFFFFFFFFu, up2 ? k0 : k1, 4));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        const float s_l = tile_scale(m);
        const float nr_l = -__frcp_rn(s_l);
        const int64_t own = row0 + r0 + (up ? 1 : 0);
        if ((lane & 3) == 0 && (up2 ? c.mine[1] : c.mine[0]) && own < a.M &&
            chk((c.vec(up2 ? 1 : 0) >> 4) * a.ld_sf + own, rows_extent(a.N / 128, a.M, a.ld_sf), CHK_Q1_SF))
          a.sf[(c.vec(up2 ? 1 : 0) >> 4) * a.ld_sf + own] = s_l;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int from = (lane & 16) + 4 * (2 * u + i);
            const float s = __shfl_sync(0xFFFFFFFFu, s_l, from), nr = __shfl_sync(0xFFFFFFFFu, nr_l, from);
            const float2 (&f)[4] = y[u][i];
            // y is an FP32 value here: see the row kernel
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = e4m3x2_neg_quot(f[j].x, f[j].y, nr, nr, s, s);
            uint2 o;
            o.x = (q[0] | (q[1] << 16)) ^ kFlipSigns;
            o.y = (q[2] | (q[3] << 16)) ^ kFlipSigns;
            if (c.mine[i] && row0 + r0 + u < a.M &&
                chk((row0 + r0 + u) * a.ldq + 8 * c.vec(i) + 7, rows_extent(a.M, a.N, a.ldq), CHK_Q1))
              *reinterpret_cast<uint2*>(a.q + (row0 + r0 + u) * a.ldq + 8 * c.vec(i)) = o;
          }
      }
    }
  }
  // a wait that gave up leaves copies in flight, which still write this block's memory
  for (uint32_t j = issued > kNormStages ? issued - kNormStages : 0; j < issued; ++j)
    mbar_wait(&full[j % kNormStages], (j / kNormStages) & 1, nullptr, WAIT_DRAIN, 1ll << 22);
}

// ---------------------------------------------------------------------------
// Backward.  Row groups as in the forward pass, two rows at a time; mean and
// rstd come from it.  The two row sums of both rows are one four-value warp
// reduction and one barrier.  Each thread keeps its columns' dgamma and dbeta
// in registers over all rows of its block, so the columns cost no further read;
// a block leaves one partial row of each in the workspace and a second kernel
// adds the blocks' rows in a fixed order (no atomics: the result does not
// depend on which block ends first).
// ---------------------------------------------------------------------------
struct LayerNormBwdArgs {
  const void* dy;
  const void* x;
  int64_t M, lddy, ldx;
  int N;
  const void* gamma;    // may be null: ones
  const float* mean;
  const float* rstd;
  void* dx;             // may be null
  int64_t lddx;
  float* partial;       // [gridDim.x][2][N]; null: no weight gradients
  int64_t partial_len;  // elements there
};

template <typename T, typename W, int VPT, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? kNormWarpRowThreads : 1024)
layer_norm_bwd_kernel(const LayerNormBwdArgs a) {
  constexpr int kColumns = kWarpRow ? kNormWarpRowMaxN : 1;
  __shared__ float part[2][32][4];                // [row-pair parity][warp][row 0: g, g xh; row 1: g, g xh]
  __shared__ float cols[kWarpRow ? kNormWarpRowThreads / 32 : 1][kColumns];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nt = kWarpRow ? 32 : blockDim.x;
  const int t = kWarpRow ? lane : threadIdx.x;
  const int warps = nt >> 5;
  const int64_t group = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (kNormWarpRowThreads / 32) + warp : blockIdx.x;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kWarpRow ? kNormWarpRowThreads / 32 : 1);
  const int N = a.N;
  const float inv_n = 1.0f / static_cast<float>(N);
  pdl_launch();
  float dga[VPT][8], dbe[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dga[i][j] = dbe[i][j] = 0.0f;
  int parity = 0;
  for (int64_t row0 = group * 2; row0 < a.M; row0 += groups * 2, parity ^= 1) {
    Raw8<T> rx[2][VPT], rd[2][VPT];
    float mean[2], rstd[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool live = row0 + r < a.M;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int64_t v = i * nt + t;
        const int valid = live ? min(max(N - 8 * static_cast<int>(v), 0), 8) : 0;
        load8<T, true>(rx[r][i], static_cast<const T*>(a.x) + (row0 + r) * a.ldx + 8 * v, valid);
        load8<T, true>(rd[r][i], static_cast<const T*>(a.dy) + (row0 + r) * a.lddy + 8 * v, valid);
      }
      mean[r] = live ? __ldg(a.mean + row0 + r) : 0.0f;
      rstd[r] = live ? __ldg(a.rstd + row0 + r) : 0.0f;
    }
    float s1[2] = {0.0f, 0.0f}, s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nt + t;
      float ga[8];
      load_param8<W>(ga, a.gamma, v, min(max(N - 8 * v, 0), 8), 1.0f);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float fx[8], fd[8];
        unpack8(rx[r][i], fx);
        unpack8(rd[r][i], fd);
#pragma unroll
        for (int j = 0; j < 8; ++j) {                   // places outside the row have dy = 0
          const float xh = (fx[j] - mean[r]) * rstd[r];
          const float g = fd[j] * ga[j];
          s1[r] += g;
          s2[r] = fmaf(g, xh, s2[r]);
          dga[i][j] = fmaf(fd[j], xh, dga[i][j]);
          dbe[i][j] += fd[j];
        }
      }
    }
    const float ws = warp_sum4(s1[0], s2[0], s1[1], s2[1], lane);
    float tot = ws;
    if (!kWarpRow) {
      if ((lane & 7) == 0) part[parity][warp][lane >> 3] = ws;
      __syncthreads();
      tot = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int w = (lane & 7) + 8 * k;
        if (w < warps) tot += part[parity][w][lane >> 3];
      }
#pragma unroll
      for (int o = 4; o; o >>= 1) tot += __shfl_xor_sync(0xFFFFFFFFu, tot, o);
    }
    tot *= inv_n;
    const float c1[2] = {__shfl_sync(0xFFFFFFFFu, tot, 0), __shfl_sync(0xFFFFFFFFu, tot, 16)};
    const float c2[2] = {__shfl_sync(0xFFFFFFFFu, tot, 8), __shfl_sync(0xFFFFFFFFu, tot, 24)};
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nt + t;
        const int valid = min(max(N - 8 * v, 0), 8);
        float ga[8];
        load_param8<W>(ga, a.gamma, v, valid, 1.0f);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float fx[8], fd[8];
          unpack8(rx[r][i], fx);
          unpack8(rd[r][i], fd);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xh = (fx[j] - mean[r]) * rstd[r];
            fd[j] = rstd[r] * (fmaf(fd[j], ga[j], -c1[r]) - xh * c2[r]);
          }
          if (row0 + r < a.M && valid > 0 &&
              chk((row0 + r) * a.lddx + 8 * v + valid - 1, rows_extent(a.M, N, a.lddx), CHK_NORM)) {
            Raw8<T> o;
            pack8(o, fd);
            store8(static_cast<T*>(a.dx) + (row0 + r) * a.lddx + 8 * static_cast<int64_t>(v), o, valid);
          }
        }
      }
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * N;
  if constexpr (kWarpRow) {
    // the block's warps, one after the other per column
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = 8 * (i * 32 + lane) + j;
          if (c < N) cols[warp][c] = which ? dbe[i][j] : dga[i][j];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < N; c += blockDim.x) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kNormWarpRowThreads / 32; ++w) s += cols[w][c];
        if (chk(out - a.partial + which * N + c, a.partial_len, CHK_NORM)) out[which * N + c] = s;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nt + t;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (8 * v + j < N && chk(out - a.partial + N + 8 * v + j, a.partial_len, CHK_NORM)) {
          out[8 * v + j] = dga[i][j];
          out[N + 8 * v + j] = dbe[i][j];
        }
      }
    }
  }
}

// The backward pass as a stream: a stage holds kNormBwdRows rows of x and of dy.
template <typename T, typename W>
__global__ void __launch_bounds__(kNormStreamThreads, 1) layer_norm_bwd_stream_kernel(const LayerNormBwdArgs a) {
  constexpr int R = kNormBwdRows;
  constexpr int kJoin = (kNormStreamThreads / 32 + 7) / 8;
  static_assert(R == 2, "two sums of two rows: a four-value reduction");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float part[2][32][4];
  __shared__ __align__(8) uint64_t full[kNormStages];
  __shared__ int abort_flag;
  const NormStream c(a.N);
  const int t = c.t, lane = c.lane;
  const uint32_t row_bytes = a.N * sizeof(T);
  const int64_t steps = (a.M + R - 1) / R;
  pdl_launch();
  if (t == 0) {
#pragma unroll
    for (int s = 0; s < kNormStages; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  uint32_t issued = 0;
  auto request = [&](int64_t step, int s) {      // thread 0
    const int64_t row0 = step * R;
    const int rows = static_cast<int>(a.M - row0 < R ? a.M - row0 : R);
    ++issued;
    mbar_arrive_expect_tx(&full[s], 2 * rows * row_bytes);
    for (int r = 0; r < rows; ++r) {
      uint8_t* dst = smem + (s * R + r) * 2 * row_bytes;
      bulk_load(dst, static_cast<const T*>(a.x) + (row0 + r) * a.ldx, row_bytes, &full[s]);
      bulk_load(dst + row_bytes, static_cast<const T*>(a.dy) + (row0 + r) * a.lddy, row_bytes, &full[s]);
    }
  };
  if (t == 0) {
    int s = 0;
    for (int64_t step = blockIdx.x; step < steps && s < kNormStages; step += gridDim.x, ++s) request(step, s);
  }
  float2 ga[2][4], dga[2][4], dbe[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    stream_param<W>(ga[i], a.gamma, c.vec(i), c.mine[i], 1.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) dga[i][j] = dbe[i][j] = f2(0.0f);
  }
  // the statistics of a step's rows, a step ahead (a row past the end takes those of the step's first)
  float mean_next[R], rstd_next[R];
  auto statistics = [&](int64_t step) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = step * R + r < a.M ? step * R + r : step * R;
      mean_next[r] = step < steps ? __ldg(a.mean + row) : 0.0f;
      rstd_next[r] = step < steps ? __ldg(a.rstd + row) : 0.0f;
    }
  };
  statistics(blockIdx.x);
  int stage = 0, parity = 0;
  uint32_t phase = 0;
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x, parity ^= 1) {
    const int64_t row0 = step * R;
    float2 mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = f2(-mean_next[r]);
      rstd[r] = f2(rstd_next[r]);
    }
    statistics(step + gridDim.x);
    warp_wait_converged(&full[stage], phase, &abort_flag, WAIT_STAGE);
    float v[4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint8_t* src = smem + (stage * R + r) * 2 * row_bytes;
      const bool live = row0 + r < a.M;          // what lies past the end counts as zero
      float2 s1 = f2(0.0f), s2 = f2(0.0f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Raw8<T> rx, rd;
        stream_read(rx, src, c.vec(i), c.mine[i] && live);
        stream_read(rd, src + row_bytes, c.vec(i), c.mine[i] && live);
        float2 x[4], d[4];
        unpack8(rx, x);
        unpack8(rd, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 xh = fmul2(fadd2(x[j], mean[r]), rstd[r]), g = fmul2(d[j], ga[i][j]);
          s1 = fadd2(s1, g);
          s2 = ffma2(g, xh, s2);
          dga[i][j] = ffma2(d[j], xh, dga[i][j]);
          dbe[i][j] = fadd2(dbe[i][j], d[j]);
        }
      }
      v[2 * r] = s1.x + s1.y;
      v[2 * r + 1] = s2.x + s2.y;
    }
    const float ws = warp_sum4(v[0], v[1], v[2], v[3], lane);
    if ((lane & 7) == 0) part[parity][c.warp][lane >> 3] = ws;
    __syncthreads();
    const int64_t coming = step + (kNormStages - 1) * static_cast<int64_t>(gridDim.x);
    if (t == 0 && step > blockIdx.x && coming < steps) {
      fence_proxy_async_shared();
      request(coming, stage > 0 ? stage - 1 : kNormStages - 1);
    }
    const uint8_t* rows_at = smem + stage * R * 2 * row_bytes;
    if (++stage == kNormStages) {
      stage = 0;
      phase ^= 1;
    }
    float tot = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      const int w = (lane & 7) + 8 * k;
      if (w < c.warps) tot += part[parity][w][lane >> 3];
    }
    tot = row_lanes_sum<4>(tot) * c.inv_n;
    if (a.dx != nullptr) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 c1 = f2(-__shfl_sync(0xFFFFFFFFu, tot, 16 * r)), c2 = f2(-__shfl_sync(0xFFFFFFFFu, tot, 16 * r + 8));
        const bool live = row0 + r < a.M;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          Raw8<T> rx, rd;
          const uint8_t* src = rows_at + r * 2 * row_bytes;
          stream_read(rx, src, c.vec(i), c.mine[i] && live);
          stream_read(rd, src + row_bytes, c.vec(i), c.mine[i] && live);
          float2 x[4], d[4];
          unpack8(rx, x);
          unpack8(rd, d);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 xh = fmul2(fadd2(x[j], mean[r]), rstd[r]);
            d[j] = fmul2(rstd[r], ffma2(xh, c2, ffma2(d[j], ga[i][j], c1)));
          }
          if (c.mine[i] && live && chk((row0 + r) * a.lddx + 8 * c.vec(i) + 7, rows_extent(a.M, a.N, a.lddx), CHK_NORM)) {
            Raw8<T> o;
            pack8(o, d);
            store8(static_cast<T*>(a.dx) + (row0 + r) * a.lddx + 8 * c.vec(i), o, 8);
          }
        }
      }
    }
  }
  // a wait that gave up leaves copies in flight, which still write this block's memory
  for (uint32_t j = issued > kNormStages ? issued - kNormStages : 0; j < issued; ++j)
    mbar_wait(&full[j % kNormStages], (j / kNormStages) & 1, nullptr, WAIT_DRAIN, 1ll << 22);
  if (a.partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!c.mine[i]) continue;
    float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.N + 8 * c.vec(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!chk(out - a.partial + a.N + 2 * j + 1, a.partial_len, CHK_NORM)) continue;
      *reinterpret_cast<float2*>(out + 2 * j) = dga[i][j];
      *reinterpret_cast<float2*>(out + a.N + 2 * j) = dbe[i][j];
    }
  }
}

// dgamma[c], dbeta[c] <- the sum over `rows` partial rows: 32 columns a block,
// 32 threads a column, then a fixed tree.
constexpr int kNormJoinThreads = 1024;
__global__ void __launch_bounds__(kNormJoinThreads)
layer_norm_bwd_join_kernel(const float* partial, int rows, int N, float* dgamma, float* dbeta) {
  __shared__ float s[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;               // of 2 N columns: dgamma's, then dbeta's
  pdl_wait();
  float v = 0.0f;
  if (c < 2 * N)
    for (int r = ry; r < rows; r += 32) v += partial[static_cast<int64_t>(r) * 2 * N + c];
  s[ry][cx] = v;
  __syncthreads();
  v = s[cx][ry];                                    // warp ry now holds column ry
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int oc = blockIdx.x * 32 + ry;
  if (cx == 0 && oc < 2 * N) {
    if (oc < N) {
      if (dgamma != nullptr) dgamma[oc] = v;
    } else if (dbeta != nullptr) {
      dbeta[oc - N] = v;
    }
  }
}

}  // namespace fp8q
