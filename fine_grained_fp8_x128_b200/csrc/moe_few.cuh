// A whole mixture-of-experts layer for a few tokens (decoding), over the same
// E4M3 expert weights with 128x128 scales as the grouped GEMM:
//
//   y[t] = sum_j w[t,j] Wd[e] h,   h = silu(Wg[e] x[t]) * (Wu[e] x[t]),  e = ids[t,j]
//   (without a gate matrix h = Wu[e] x[t])
//
// With a handful of tokens an expert every weight byte is used once or a few
// times, so the layer is bound by reading the picked experts' codes once.  The
// activations are NOT quantized: they go to the tensor cores as FP16 with an
// exact power-of-two scale per 128-wide chunk, the codes are widened E4M3 ->
// FP16 in registers (exact), products are summed in FP32 over one 128-wide
// chunk and then multiplied by the weight block's and the chunk's scales.
// mma.sync rather than tcgen05: the widened codes would have to go back through
// shared memory to be a tcgen05 operand, twice the bytes that came in, and at
// these token counts the matrix instructions are far from their limit.
//
// Five launches:
//   plan     tokens by expert in blocks of 8 G columns; x to FP16 chunks
//   up       hidden rows, FP32
//   hidden   hidden rows to FP16 chunks
//   down     each (token, slot)'s output row, FP32
//   combine  the weighted sum over a token's slots, in slot order
// No atomic touches a result: equal inputs give equal bits.
#pragma once

#include <cuda_fp16.h>

#include "norm.cuh"

namespace fp8q {

constexpr int kFewMaxTokens = 128;
constexpr int kFewMaxEntries = 1024;
constexpr int kFewMaxExperts = 1024;
constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;

// What the plan leaves for the other launches.  Positions number the entries
// (token, slot) expert by expert, each expert's first position a multiple of 8.
struct FewPlan {
  int blocks;        // column blocks over all experts
  int positions;     // padded positions in use
  int pad[2];
  // followed by (see FewLayout):
  //   int block_expert[max_blocks], block_start[max_blocks], block_count[max_blocks]
  //   int entry[max_positions]  (-1: padding)
};

// Workspace layout, in bytes from its 256-byte aligned start; host and device
// compute it from the same sizes.
struct FewLayout {
  int64_t max_blocks, max_positions;
  int64_t block_expert, block_start, block_count, entry;
  int64_t xh, xs;       // FP16 [T][H], FP32 [H/128][ld_xs]
  int64_t hid;          // FP32 [max_positions][I]
  int64_t hh, hs;       // FP16 [max_positions][I], FP32 [I/128][max_positions]
  int64_t yp;           // FP32 [T k][H]
  int64_t ld_xs;
  int64_t bytes;
};
__host__ __device__ inline int64_t few_align(int64_t v) { return (v + 255) / 256 * 256; }
__host__ __device__ inline FewLayout few_layout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  FewLayout l;
  const int64_t n = T * k;
  const int64_t groups = n < E ? n : E;
  l.max_positions = (n + 7 * groups + 7) / 8 * 8;
  l.max_blocks = l.max_positions / 8;
  l.ld_xs = (T + 3) / 4 * 4;
  int64_t o = few_align(sizeof(FewPlan));
  l.block_expert = o; o = few_align(o + 4 * l.max_blocks);
  l.block_start = o; o = few_align(o + 4 * l.max_blocks);
  l.block_count = o; o = few_align(o + 4 * l.max_blocks);
  l.entry = o; o = few_align(o + 4 * l.max_positions);
  l.xh = o; o = few_align(o + 2 * T * H);
  l.xs = o; o = few_align(o + 4 * (H / 128) * l.ld_xs);
  l.hid = o; o = few_align(o + 4 * l.max_positions * I);
  l.hh = o; o = few_align(o + 2 * l.max_positions * I);
  l.hs = o; o = few_align(o + 4 * (I / 128) * l.max_positions);
  l.yp = o; o = few_align(o + 4 * n * H);
  l.bytes = o;
  return l;
}

struct FewArgs {
  const __nv_bfloat16* x;
  int64_t ldx;
  int T, k, E, H, I;
  const int32_t* ids;
  const float* share;              // [T][k]
  const uint8_t *wg, *wu, *wd;     // wg may be null
  const float *sg, *su, *sd;
  void* y;
  int64_t ldy;
  uint8_t* ws;
  FewLayout l;
};

__device__ __forceinline__ const FewPlan* few_plan(const FewArgs& a) { return reinterpret_cast<const FewPlan*>(a.ws); }
template <typename T>
__device__ __forceinline__ T* few_at(const FewArgs& a, int64_t off) { return reinterpret_cast<T*>(a.ws + off); }

// ---------------------------------------------------------------------------
// FP16 chunks: 128 values times a power of two that takes their largest
// magnitude into [2^14, 2^15).  The scaling is exact, FP16 keeps 11 bits (a
// BF16 value has 8, so x is exact) down to 2^-28 of the chunk's maximum, and
// what lies below is off by at most 2^-40 of that maximum, under the FP32
// accumulation's own rounding.  A hidden value is off by at most 2^-11 of itself.
// The power is at most 2^84, so that its inverse times a block scale (>= 1e-12)
// is a normal FP32 number: a chunk under 2^-98 loses bits, 2^-109 at most.
// A warp owns one chunk, four consecutive values a lane.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void few_chunk(const float (&f)[4], __half* dst, float* scale, int lane) {
  float m = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;   // m >= 0: no sign bit
  e = max(e, -70);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
  const __half2 h0 = __floats2half2_rn(f[0] * up, f[1] * up), h1 = __floats2half2_rn(f[2] * up, f[3] * up);
  uint2 o;
  o.x = *reinterpret_cast<const uint32_t*>(&h0);
  o.y = *reinterpret_cast<const uint32_t*>(&h1);
  *reinterpret_cast<uint2*>(dst + 4 * lane) = o;
  if (lane == 0) *scale = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
}

// Inclusive scan of two counters over 1024 threads.
__device__ __forceinline__ int2 few_scan(int2 v, int2 (&sums)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, v.x, o), b = __shfl_up_sync(0xFFFFFFFFu, v.y, o);
    if (lane >= o) { v.x += a; v.y += b; }
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int2 s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xFFFFFFFFu, s.x, o), b = __shfl_up_sync(0xFFFFFFFFu, s.y, o);
      if (lane >= o) { s.x += a; s.y += b; }
    }
    sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) { v.x += sums[warp - 1].x; v.y += sums[warp - 1].y; }
  return v;
}

// Block 0 orders the entries; the others turn x into FP16 chunks.
template <int G>
__global__ void __launch_bounds__(1024) few_plan_kernel(const FewArgs a) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (blockIdx.x > 0) {
    const int chunks = a.H / 128;
    const int item = (blockIdx.x - 1) * 32 + (tid >> 5);
    if (item >= a.T * chunks) return;
    const int t = item / chunks, kb = item - t * chunks;
    const uint2 r = *reinterpret_cast<const uint2*>(a.x + t * a.ldx + kb * 128 + 4 * lane);
    const float f[4] = {bf16lo(r.x), bf16hi(r.x), bf16lo(r.y), bf16hi(r.y)};
    few_chunk(f, few_at<__half>(a, a.l.xh) + static_cast<int64_t>(t) * a.H + kb * 128,
              few_at<float>(a, a.l.xs) + kb * a.l.ld_xs + t, lane);
    return;
  }
  __shared__ int count[kFewMaxExperts], start[kFewMaxExperts];
  __shared__ int2 sums[32];
  const int n = a.T * a.k;
  int* entry = few_at<int>(a, a.l.entry);
  count[tid] = 0;
  for (int i = tid; i < a.l.max_positions; i += 1024) entry[i] = -1;
  __syncthreads();
  int e = -1;
  if (tid < n) {
    e = a.ids[tid];
    if (e >= a.E) {
      report_status(FP8Q_ERR_INVALID_ARG, BAD_EXPERT_ID);
      e = -1;
    }
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  const int c = count[tid];
  const int2 mine = make_int2((c + 7) / 8 * 8, (c + 8 * G - 1) / (8 * G));   // padded positions, column blocks
  const int2 upto = few_scan(mine, sums);
  start[tid] = upto.x - mine.x;
  for (int b = 0; b < mine.y; ++b) {
    const int at = upto.y - mine.y + b;
    if (chk(at, a.l.max_blocks, CHK_FEW)) {
      few_at<int>(a, a.l.block_expert)[at] = tid;
      few_at<int>(a, a.l.block_start)[at] = upto.x - mine.x + 8 * G * b;
      few_at<int>(a, a.l.block_count)[at] = min(c - 8 * G * b, 8 * G);
    }
  }
  if (tid == 1023) {
    FewPlan* p = reinterpret_cast<FewPlan*>(a.ws);
    p->blocks = upto.y;
    p->positions = upto.x;
  }
  count[tid] = 0;
  __syncthreads();
  // Which of an expert's positions an entry gets does not reach the results:
  // every entry is a column of its own.
  if (e >= 0) {
    const int at = start[e] + atomicAdd(&count[e], 1);
    if (chk(at, a.l.max_positions, CHK_FEW)) entry[at] = tid;
  }
}

// ---------------------------------------------------------------------------
// The two weight passes.  An item is MT tiles of 16 weight rows of one expert
// times one block of up to 8 G of its columns; the block's eight warps split
// the 128-wide K chunks (warp w: chunks w, w + 8, ...), which keeps 1 KB of a row
// together in time, and their FP32 sums are joined in shared memory in warp order.
//
// A tile's operand order is free along K as long as both operands share it, so
// lane (g, t) of a warp takes bytes 16 t .. and 64 + 16 t .. of rows g and g + 8:
// 16-byte loads straight into fragment order.  Every lane reads back only what
// it copied itself (cp.async, 512 contiguous bytes a warp instruction), so the
// ring of S units (one unit: one chunk of one item) needs no barrier, and runs on
// across items: the next item's weights are in flight while this one is joined.
// Only the few scales of a unit are shared by the lanes.
// ---------------------------------------------------------------------------
enum : int { kFewGated = 0, kFewPlain = 1, kFewDown = 2 };

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void* gmem, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_or_zero(uint32_t smem, const void* gmem, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem), "l"(gmem), "r"(live ? 4 : 0) : "memory");
}
// Four E4M3 codes (element order) -> two FP16 pairs; exact.
__device__ __forceinline__ void widen4(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int MT, int G, int S>
struct FewSmem {
  static constexpr int kUnit = (MT * 4 + G * 4) * 512 + 256;   // weights, columns, scales (64 floats)
  static constexpr int kRing = kFewWarps * S * kUnit;
  static constexpr int kJoin = kFewWarps * MT * G * 512;
  static constexpr int kBytes = kRing + kJoin;
  static_assert(8 * G + 2 <= 64, "a unit's scales");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int MODE, int MT, int G, int S>
__global__ void __launch_bounds__(kFewThreads) few_weights_kernel(const FewArgs a) {
  using Sm = FewSmem<MT, G, S>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int K = MODE == kFewDown ? a.I : a.H;
  const int N = MODE == kFewDown ? a.H : a.I;
  constexpr int kRows = MODE == kFewGated ? 8 * MT : 16 * MT;      // output rows an item
  const int KB = K / 128;
  const int row_blocks = N / kRows;
  const int blocks = few_plan(a)->blocks;
  const int64_t items = static_cast<int64_t>(blocks) * row_blocks;
  const int* block_expert = few_at<const int>(a, a.l.block_expert);
  const int* block_start = few_at<const int>(a, a.l.block_start);
  const int* block_count = few_at<const int>(a, a.l.block_count);
  const int* entry = few_at<const int>(a, a.l.entry);
  const uint8_t* w_lo = MODE == kFewDown ? a.wd : (MODE == kFewGated ? a.wg : a.wu);
  const uint8_t* w_hi = MODE == kFewDown ? a.wd : a.wu;
  const float* s_lo = MODE == kFewDown ? a.sd : (MODE == kFewGated ? a.sg : a.su);
  const float* s_hi = MODE == kFewDown ? a.sd : a.su;
  const __half* cols = few_at<const __half>(a, MODE == kFewDown ? a.l.hh : a.l.xh);
  const float* col_scale = few_at<const float>(a, MODE == kFewDown ? a.l.hs : a.l.xs);
  const int64_t ld_cs = MODE == kFewDown ? a.l.max_positions : a.l.ld_xs;

  uint8_t* ring = smem + warp * S * Sm::kUnit;
  const uint32_t ring_u32 = smem_u32(ring);
  float4* join = reinterpret_cast<float4*>(smem + Sm::kRing);

  // ---- the load cursor: (item, chunk) of the next unit to request ----
  int64_t l_item = blockIdx.x;
  int l_chunk = warp;
  int l_slot = 0;
  const uint8_t *p_lo[MT], *p_hi[MT];
  const __half* p_col[G];
  bool live[G];
  const float *p_s0 = nullptr, *p_s1 = nullptr;   // this lane's one or two scales of the unit
  int64_t ld_s0 = 0, ld_s1 = 0;
  auto load_item = [&]() {
    const int b = static_cast<int>(l_item % blocks);
    const int row0 = static_cast<int>(l_item / blocks) * kRows;
    const int64_t e = block_expert[b];
    const int start = block_start[b], count = block_count[b];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r_lo = row0 + (MODE == kFewGated ? 8 * m : 16 * m) + g;
      const int r_hi = MODE == kFewGated ? r_lo : r_lo + 8;
      p_lo[m] = w_lo + (e * N + r_lo) * K + 16 * t;
      p_hi[m] = w_hi + (e * N + r_hi) * K + 16 * t;
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int c = 8 * j + g;
      live[j] = c < count;
      const int64_t row = !live[j] ? 0 : (MODE == kFewDown ? start + c : entry[start + c] / a.k);
      p_col[j] = cols + row * K + 16 * t;
    }
    // scales of a unit: [0, 8 G) the columns', 8 G and 8 G + 1 the weight rows'
    const int64_t blk = (e * (N / 128) + row0 / 128) * KB;
    auto scale_at = [&](int i, const float*& p, int64_t& ld) {
      if (i < 8 * G) {
        p = i < count ? col_scale + (MODE == kFewDown ? start + i : entry[start + i] / a.k) : nullptr;
        ld = ld_cs;
      } else {
        p = i == 8 * G ? s_lo + blk : (i == 8 * G + 1 ? s_hi + blk : nullptr);
        ld = 1;
      }
    };
    scale_at(lane, p_s0, ld_s0);
    scale_at(lane + 32, p_s1, ld_s1);
  };
  auto request = [&]() {
    if (l_item < items && l_chunk < KB) {
      const uint32_t unit = ring_u32 + l_slot * Sm::kUnit + lane * 16;
      const int64_t o = static_cast<int64_t>(l_chunk) * 128;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        cp_async16_or_zero(unit + (4 * m + 0) * 512, p_lo[m] + o, true);
        cp_async16_or_zero(unit + (4 * m + 1) * 512, p_hi[m] + o, true);
        cp_async16_or_zero(unit + (4 * m + 2) * 512, p_lo[m] + o + 64, true);
        cp_async16_or_zero(unit + (4 * m + 3) * 512, p_hi[m] + o + 64, true);
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint32_t c = unit + (4 * MT + 4 * j) * 512;
        cp_async16_or_zero(c, p_col[j] + o, live[j]);
        cp_async16_or_zero(c + 512, p_col[j] + o + 8, live[j]);
        cp_async16_or_zero(c + 1024, p_col[j] + o + 64, live[j]);
        cp_async16_or_zero(c + 1536, p_col[j] + o + 72, live[j]);
      }
      const uint32_t sc = ring_u32 + l_slot * Sm::kUnit + (MT * 4 + G * 4) * 512 + lane * 4;
      const float* any = s_lo;
      cp_async4_or_zero(sc, p_s0 != nullptr ? p_s0 + l_chunk * ld_s0 : any, p_s0 != nullptr);
      if (8 * G + 2 > 32) cp_async4_or_zero(sc + 128, p_s1 != nullptr ? p_s1 + l_chunk * ld_s1 : any, p_s1 != nullptr);
      l_slot = l_slot + 1 == S ? 0 : l_slot + 1;
      l_chunk += kFewWarps;
      if (l_chunk >= KB) {
        l_chunk = warp;
        l_item += gridDim.x;
        if (l_item < items) load_item();
      }
    }
    cp_async_commit();
  };
  if (l_item < items && warp < KB) load_item();
  else l_item = items;                       // a warp without chunks requests nothing
#pragma unroll
  for (int i = 0; i < S - 1; ++i) request();

  int slot = 0;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    float acc[MT][G][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.0f;
    const int b = static_cast<int>(item % blocks);
    const int count = block_count[b], start = block_start[b];
    const int row0 = static_cast<int>(item / blocks) * kRows;
    for (int kb = warp; kb < KB; kb += kFewWarps) {
      cp_async_wait<S - 2>();
      __syncwarp();                          // the unit's scales; and the slot before it is free
      request();
      const uint8_t* unit = ring + slot * Sm::kUnit;
      const uint4* u4 = reinterpret_cast<const uint4*>(unit) + lane;
      const float* sc = reinterpret_cast<const float*>(unit + (MT * 4 + G * 4) * 512);
      slot = slot + 1 == S ? 0 : slot + 1;
      float part[MT][G][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) part[m][j][c] = 0.0f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t lo[MT][4], hi[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 p = u4[(4 * m + 2 * half) * 32], q = u4[(4 * m + 2 * half + 1) * 32];
          lo[m][0] = p.x; lo[m][1] = p.y; lo[m][2] = p.z; lo[m][3] = p.w;
          hi[m][0] = q.x; hi[m][1] = q.y; hi[m][2] = q.z; hi[m][3] = q.w;
        }
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {     // eight of the piece's sixteen elements: two k16 steps
          uint32_t al[MT][4], ah[MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            widen4(lo[m][2 * s2], al[m][0], al[m][1]);
            widen4(lo[m][2 * s2 + 1], al[m][2], al[m][3]);
            widen4(hi[m][2 * s2], ah[m][0], ah[m][1]);
            widen4(hi[m][2 * s2 + 1], ah[m][2], ah[m][3]);
          }
#pragma unroll
          for (int j = 0; j < G; ++j) {
            if (G > 1 && 8 * j >= count) continue;
            const uint4 c = u4[(4 * MT + 4 * j + 2 * half + s2) * 32];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma_f16(part[m][j], al[m][0], ah[m][0], al[m][1], ah[m][1], c.x, c.y);
              mma_f16(part[m][j], al[m][2], ah[m][2], al[m][3], ah[m][3], c.z, c.w);
            }
          }
        }
      }
      const float w0 = sc[8 * G], w1 = sc[8 * G + 1];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const float2 cs = *reinterpret_cast<const float2*>(sc + 8 * j + 2 * t);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[m][j][0] = fmaf(part[m][j][0], w0 * cs.x, acc[m][j][0]);
          acc[m][j][1] = fmaf(part[m][j][1], w0 * cs.y, acc[m][j][1]);
          acc[m][j][2] = fmaf(part[m][j][2], w1 * cs.x, acc[m][j][2]);
          acc[m][j][3] = fmaf(part[m][j][3], w1 * cs.y, acc[m][j][3]);
        }
      }
    }
    // join the warps' sums
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < G; ++j)
        join[(warp * MT * G + m * G + j) * 32 + lane] =
            make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
    __syncthreads();
    for (int i = threadIdx.x; i < MT * G * 32; i += kFewThreads) {
      const int m = i / (G * 32), j = i / 32 % G;
      if (8 * j >= count) continue;
      float4 s = join[i];
#pragma unroll
      for (int w = 1; w < kFewWarps; ++w) {
        const float4 v = join[w * MT * G * 32 + i];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
      // s: rows g and g + 8 (.xy, .zw) of tile m, columns 2 t and 2 t + 1 of group j
      const float lo[2] = {s.x, s.y}, hi[2] = {s.z, s.w};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * j + 2 * t + c;
        if (col >= count) continue;
        const int at = start + col;
        if (MODE == kFewGated) {
          const float h = lo[c] / (1.0f + expf(-lo[c])) * hi[c];
          if (chk(at, a.l.max_positions, CHK_FEW))
            few_at<float>(a, a.l.hid)[static_cast<int64_t>(at) * N + row0 + 8 * m + g] = h;
        } else {
          const int64_t row = MODE == kFewDown ? entry[at] : at;
          float* dst = few_at<float>(a, MODE == kFewDown ? a.l.yp : a.l.hid) + row * N + row0 + 16 * m + g;
          if (chk(row, MODE == kFewDown ? a.T * a.k : a.l.max_positions, CHK_FEW)) {
            dst[0] = lo[c];
            dst[8] = hi[c];
          }
        }
      }
    }
    __syncthreads();                         // join is free for the next item
  }
}

// Hidden rows to FP16 chunks: a warp a chunk.
__global__ void __launch_bounds__(kFewThreads) few_hidden_kernel(const FewArgs a) {
  const int lane = threadIdx.x & 31;
  const int chunks = a.I / 128;
  const int items = few_plan(a)->positions * chunks;
  const int* entry = few_at<const int>(a, a.l.entry);
  for (int item = blockIdx.x * kFewWarps + (threadIdx.x >> 5); item < items; item += gridDim.x * kFewWarps) {
    const int p = item / chunks, kb = item - p * chunks;
    if (entry[p] < 0) continue;
    const int64_t o = static_cast<int64_t>(p) * a.I + kb * 128;
    const float4 v = *reinterpret_cast<const float4*>(few_at<const float>(a, a.l.hid) + o + 4 * lane);
    const float f[4] = {v.x, v.y, v.z, v.w};
    few_chunk(f, few_at<__half>(a, a.l.hh) + o, few_at<float>(a, a.l.hs) + kb * a.l.max_positions + p, lane);
  }
}

// y[t] = sum_j share[t,j] * (slot j's row), in slot order; a token none of
// whose slots names an expert gets zeros.  Eight columns a thread.
template <typename T>
__global__ void __launch_bounds__(128) few_combine_kernel(const FewArgs a) {
  const int t = blockIdx.y;
  const int n = (blockIdx.x * 128 + threadIdx.x) * 8;
  if (n >= a.H) return;
  float s[8] = {};
  for (int j = 0; j < a.k; ++j) {
    const int e = __ldg(a.ids + t * a.k + j);
    if (e < 0 || e >= a.E) continue;
    const float w = __ldg(a.share + t * a.k + j);
    const float4* src = reinterpret_cast<const float4*>(few_at<const float>(a, a.l.yp) +
                                                        (static_cast<int64_t>(t) * a.k + j) * a.H + n);
    const float4 u = src[0], v = src[1];
    s[0] = fmaf(w, u.x, s[0]); s[1] = fmaf(w, u.y, s[1]); s[2] = fmaf(w, u.z, s[2]); s[3] = fmaf(w, u.w, s[3]);
    s[4] = fmaf(w, v.x, s[4]); s[5] = fmaf(w, v.y, s[5]); s[6] = fmaf(w, v.z, s[6]); s[7] = fmaf(w, v.w, s[7]);
  }
  Raw8<T> o;
  pack8(o, s);
  if (chk(n + 7, a.ldy, CHK_FEW)) store8(static_cast<T*>(a.y) + t * a.ldy + n, o, 8);
}

}  // namespace fp8q
