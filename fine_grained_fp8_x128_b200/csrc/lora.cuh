// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + s_a B_a (A_a x[t]),   a = the adapter of token t
//
// base is the projection's output (fp8q_gemm_blockscaled); tokens come grouped
// by adapter (fp8q_moe_dispatch_layout).  Two launches:
//   shrink   v = A_a x, FP32, in K slices where tokens are few
//   expand   out = base + s_a B_a v
// With few tokens an adapter the bound is reading A and B once, with many it is
// x, base and out; the products are 2 r (K + N) a token, far under either.  The
// shrink and the expansion run on mma.sync with operands loaded straight into
// fragment order; for a token an adapter and rows of B of 32 bytes at most the
// expansion runs on FP32 FMAs (a tile would be one row in sixteen full, and its
// loads half empty).
// x, A and B are BF16 as given; as an MMA operand v is split into BF16 parts (two
// for a BF16 output, which keep v to 2^-16 of itself; three for FP32, 2^-24), so
// that its rounding stays under the output's.
#pragma once

#include <type_traits>

#include "moe_few.cuh"

namespace fp8q {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxGroups = 1024;
constexpr int kLoraMaxRank = 128;

struct LoraArgs {
  const __nv_bfloat16* x;
  int64_t T, ldx;
  int K, N, r;
  int groups, adapters;           // groups at or above `adapters` have none: out = base
  const int32_t* rows;
  const int32_t* offsets;
  const __nv_bfloat16* a;         // [adapters][r][K]
  const __nv_bfloat16* b;         // [adapters][N][r]
  const float* scaling;           // [adapters]; may be null: ones
  const void* base;
  int64_t ldb;
  void* out;
  int64_t ldo;
  float* v;                       // [slices][T][r]
  int64_t v_len;                  // elements there
  int slices;
  int col_units;                  // an item of the expansion's units, which are 32 columns a warp, for a token a group 64
};

// The groups' token ranges and the running count of their blocks of `tile`
// tokens, in shared memory; returns the number of blocks.  A group's bounds
// are clamped to [0, T]; bounds that decrease or leave it are reported.
struct LoraGroups {
  int first[kLoraMaxGroups];
  int count[kLoraMaxGroups];
  int upto[kLoraMaxGroups];       // blocks of groups 0 .. i
  int sums[16];                   // of the warps, sixteen at most
};
template <int THREADS>
__device__ __forceinline__ int lora_groups(LoraGroups& s, const LoraArgs& a, int groups, int tile) {
  constexpr int kPer = kLoraMaxGroups / THREADS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int mine[kPer], total = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = threadIdx.x * kPer + i;
    int n = 0;
    if (g < groups) {
      const int lo = __ldg(a.offsets + g), hi = __ldg(a.offsets + g + 1);
      if ((lo < 0 || hi < lo || hi > a.T) && blockIdx.x == 0) report_status(FP8Q_ERR_INVALID_ARG, BAD_GROUP_OFFSETS);
      const int T = static_cast<int>(a.T);
      const int l = min(max(lo, 0), T), h = min(max(hi, 0), T);
      s.first[g] = l;
      s.count[g] = max(h - l, 0);
      n = (max(h - l, 0) + tile - 1) / tile;
    }
    total += n;
    mine[i] = total;
  }
  int scan = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) s.sums[warp] = scan;
  __syncthreads();
  int before = scan - total;
  for (int w = 0; w < warp; ++w) before += s.sums[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = threadIdx.x * kPer + i;
    if (g < groups) s.upto[g] = before + mine[i];
  }
  __syncthreads();
  return groups > 0 ? s.upto[groups - 1] : 0;
}
// The group of block b and the block's number within it.
__device__ __forceinline__ int2 lora_find(const LoraGroups& s, int groups, int b) {
  int lo = 0, hi = groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s.upto[mid] > b) hi = mid;
    else lo = mid + 1;
  }
  return make_int2(lo, b - (lo > 0 ? s.upto[lo - 1] : 0));
}
// The token of a grouped position; one outside [0, T) is reported and skipped (-1).
__device__ __forceinline__ int64_t lora_token(const LoraArgs& a, int pos) {
  const int t = __ldg(a.rows + pos);
  if (t < 0 || t >= a.T) {
    report_status(FP8Q_ERR_INVALID_ARG, BAD_ROW_INDEX);
    return -1;
  }
  return t;
}

// The first `bytes` (at most 128 KB, so that all resident blocks' stay in L2) from p into L2; both multiples of 16.
__device__ __forceinline__ void bulk_prefetch(const void* p, int64_t bytes) {
  const uint32_t n = static_cast<uint32_t>(min(bytes, static_cast<int64_t>(128 * 1024)));
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void* gmem, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// ---------------------------------------------------------------------------
// Shrink.  An item is a block of up to 8 G tokens of one adapter times up to
// 16 RT of its ranks times one K slice; the block's warps split the slice's
// chunks of 32 P elements and join their FP32 sums in shared memory.  The
// operands' order along K is free as long as both share it: lane (g, t) takes
// the 16-byte piece t of a chunk of rows g and g + 8, in fragment order.  Every lane
// reads back only what it copied itself (cp.async), so the ring of S units (one
// unit: one chunk of one item) needs no barrier, and runs on across items.
// ---------------------------------------------------------------------------
struct LoraTrue { static constexpr bool value = true; };
struct LoraFalse { static constexpr bool value = false; };

template <int RT, int G, int P, int S>
struct LoraSmem {
  static constexpr int kUnit = P * (2 * RT + G) * 512;
  static constexpr int kRing = kLoraWarps * S * kUnit;
  static constexpr int kJoin = kLoraWarps * RT * G * 512;
  static constexpr int kBytes = kRing + kJoin;
  static_assert(kBytes + static_cast<int>(sizeof(LoraGroups)) <= 227 * 1024, "shared memory");
};

template <int RT, int G, int P, int S>
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(const LoraArgs a) {
  using Sm = LoraSmem<RT, G, P, S>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ LoraGroups gr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_launch();
  const int groups = min(a.groups, a.adapters);          // the others shrink to nothing
  const int blocks = lora_groups<kLoraThreads>(gr, a, groups, 8 * G);
  const int rank_blocks = (a.r + 16 * RT - 1) / (16 * RT);
  const int chunks = (a.K + 32 * P - 1) / (32 * P);
  const int per_slice = (chunks + a.slices - 1) / a.slices;
  const int64_t items = static_cast<int64_t>(blocks) * rank_blocks * a.slices;

  uint8_t* ring = smem + warp * S * Sm::kUnit;
  const uint32_t ring_u32 = smem_u32(ring);
  float4* join = reinterpret_cast<float4*>(smem + Sm::kRing);

  struct Where {
    int adapter, first, count, rank0, slice, chunk0, chunk1;
  };
  auto where = [&](int64_t item) {
    Where w;
    const int b = static_cast<int>(item % blocks);
    const int rest = static_cast<int>(item / blocks);
    const int2 f = lora_find(gr, groups, b);
    w.adapter = f.x;
    w.first = gr.first[f.x] + f.y * 8 * G;
    w.count = min(gr.count[f.x] - f.y * 8 * G, 8 * G);
    w.rank0 = rest % rank_blocks * 16 * RT;
    w.slice = rest / rank_blocks;
    w.chunk0 = min(w.slice * per_slice, chunks);
    w.chunk1 = min(w.chunk0 + per_slice, chunks);
    return w;
  };

  // ---- the load cursor ----
  int64_t l_item = blockIdx.x;
  int l_chunk = 0, l_end = 0, l_slot = 0;
  const __nv_bfloat16 *p_lo[RT], *p_hi[RT], *p_x[G];
  bool lo_live[RT], hi_live[RT], x_live[G];
  auto load_item = [&]() {                               // the next item with a chunk for this warp
    for (; l_item < items; l_item += gridDim.x) {
      const Where w = where(l_item);
      l_chunk = w.chunk0 + warp;
      l_end = w.chunk1;
      if (l_chunk >= l_end) continue;
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const int r_lo = w.rank0 + 16 * m + g, r_hi = r_lo + 8;
        lo_live[m] = r_lo < a.r;
        hi_live[m] = r_hi < a.r;
        const __nv_bfloat16* base = a.a + static_cast<int64_t>(w.adapter) * a.r * a.K + 8 * t;
        p_lo[m] = base + (lo_live[m] ? static_cast<int64_t>(r_lo) * a.K : 0);
        p_hi[m] = base + (hi_live[m] ? static_cast<int64_t>(r_hi) * a.K : 0);
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int c = 8 * j + g;
        const int64_t tok = c < w.count ? lora_token(a, w.first + c) : -1;
        x_live[j] = tok >= 0;
        p_x[j] = a.x + (tok >= 0 ? tok * a.ldx : 0) + 8 * t;
      }
      return;
    }
  };
  auto request = [&]() {
    if (l_item < items) {
      const uint32_t unit = ring_u32 + l_slot * Sm::kUnit + lane * 16;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int k = l_chunk * 32 * P + 32 * p;         // this lane's piece: elements k + 8 t ..
        const bool in = k + 8 * t < a.K;
        const int o = in ? k : -8 * t;                   // outside: any address of the row
        const uint32_t at = unit + p * (2 * RT + G) * 512;
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          cp_async16_or_zero(at + (2 * m) * 512, p_lo[m] + o, in && lo_live[m]);
          cp_async16_or_zero(at + (2 * m + 1) * 512, p_hi[m] + o, in && hi_live[m]);
        }
#pragma unroll
        for (int j = 0; j < G; ++j) cp_async16_or_zero(at + (2 * RT + j) * 512, p_x[j] + o, in && x_live[j]);
      }
      l_slot = l_slot + 1 == S ? 0 : l_slot + 1;
      l_chunk += kLoraWarps;
      if (l_chunk >= l_end) {
        l_item += gridDim.x;
        load_item();
      }
    }
    cp_async_commit();
  };
  load_item();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) request();

  int slot = 0;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const Where w = where(item);
    // Sums of 64 products come from the tensor cores (2 / P chunks of 32 P), then an FP32 addition.
    float2 acc[RT][G][2];
    float part[RT][G][4];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int j = 0; j < G; ++j) acc[m][j][0] = acc[m][j][1] = f2(0.0f);
    auto promote = [&]() {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if (G > 1 && 8 * j >= w.count) continue;
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          acc[m][j][0] = fadd2(acc[m][j][0], make_float2(part[m][j][0], part[m][j][1]));
          acc[m][j][1] = fadd2(acc[m][j][1], make_float2(part[m][j][2], part[m][j][3]));
        }
      }
    };
    auto multiply = [&](auto onto_zero) {
      cp_async_wait<S - 2>();
      // every lane reads only what it copied itself: no other wait.  The slot that is
      // requested now was read by this lane in the step before.
      request();
      const uint4* u4 = reinterpret_cast<const uint4*>(ring + slot * Sm::kUnit) + lane;
      slot = slot + 1 == S ? 0 : slot + 1;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        uint4 xb[G];
#pragma unroll
        for (int j = 0; j < G; ++j) xb[j] = u4[(p * (2 * RT + G) + 2 * RT + j) * 32];
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const uint4 lo = u4[(p * (2 * RT + G) + 2 * m) * 32], hi = u4[(p * (2 * RT + G) + 2 * m + 1) * 32];
#pragma unroll
          for (int j = 0; j < G; ++j) {
            if (G > 1 && 8 * j >= w.count) continue;
            if (decltype(onto_zero)::value && p == 0) mma_bf16_first(part[m][j], lo.x, hi.x, lo.y, hi.y, xb[j].x, xb[j].y);
            else mma_bf16(part[m][j], lo.x, hi.x, lo.y, hi.y, xb[j].x, xb[j].y);
            mma_bf16(part[m][j], lo.z, hi.z, lo.w, hi.w, xb[j].z, xb[j].w);
          }
        }
      }
    };
    for (int chunk = w.chunk0 + warp; chunk < w.chunk1; chunk += kLoraWarps) {
      multiply(LoraTrue{});
      if (P == 1 && chunk + kLoraWarps < w.chunk1) {
        chunk += kLoraWarps;
        multiply(LoraFalse{});
      }
      promote();
    }
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int j = 0; j < G; ++j)
        join[(warp * RT * G + m * G + j) * 32 + lane] =
            make_float4(acc[m][j][0].x, acc[m][j][0].y, acc[m][j][1].x, acc[m][j][1].y);
    __syncthreads();
    for (int i = threadIdx.x; i < RT * G * 32; i += kLoraThreads) {
      const int m = i / (G * 32), j = i / 32 % G;
      float4 s = join[i];
#pragma unroll
      for (int u = 1; u < kLoraWarps; ++u) {
        const float4 q = join[u * RT * G * 32 + i];
        s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
      }
      const float lo[2] = {s.x, s.y}, hi[2] = {s.z, s.w};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * j + 2 * t + c;
        const int rank = w.rank0 + 16 * m + g;
        const int64_t pos = w.first + col;
        if (col < w.count) {
          const int64_t at = (w.slice * a.T + pos) * a.r + rank;
          if (rank < a.r && chk(at, a.v_len, CHK_LORA)) a.v[at] = lo[c];
          if (rank + 8 < a.r && chk(at + 8, a.v_len, CHK_LORA)) a.v[at + 8] = hi[c];
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Expand on matrix instructions.  An item is a block of up to 16 MB tokens of one group times
// a.col_units units of 32 columns a warp.  Tokens are the rows of the
// product, v's parts its first operand (in shared memory, fragment order), B's
// rows the second.  The 8 columns of an instruction stand for columns
// 8 (c / 2) + 2 j + c % 2 of the warp's 32 (j: the instruction's number of four),
// so that a lane ends with 8 consecutive columns: base and out move in 16-byte
// words, 64 contiguous bytes a row.  base and B of the coming units are on their
// way (cp.async into a ring of S units a warp; a lane reads only what it copied)
// while a unit is multiplied: read when they are needed, 4096 tokens of 8
// adapters of rank 64 beside 7168 -> 18432 took 108 us, now 80: 49 % of the tensor
// pipe, half of it for v's second part, and 44 % of the issue slots; so the addresses
// are kept and advanced.  Places that no copy fills: a column
// past N or a token that is none holds anything, which stays in that column or
// row and is not stored; ranks past r multiply zeros of v, so they are zeros
// from the start.
// ---------------------------------------------------------------------------
template <typename T, int KQ, int MB, int S, int WARPS>
struct LoraExpandSmem {
  static constexpr int kParts = sizeof(T) == 4 ? 3 : 2;
  static constexpr int kWords = sizeof(T) / 2;                         // 16-byte words of 8 elements
  static constexpr int kUnit = (KQ * 4 + MB * 2 * kWords) * 512;
  static constexpr int kV = MB * KQ * kParts * 1024;
  static constexpr int kBytes = kV + WARPS * S * kUnit;
  static_assert(kBytes + static_cast<int>(sizeof(LoraGroups)) <= 227 * 1024, "shared memory");
};

template <typename T, int KQ, int MB, int S, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) lora_expand_kernel(const LoraArgs a) {
  using Sm = LoraExpandSmem<T, KQ, MB, S, WARPS>;
  constexpr int kCols = 32 * WARPS;              // of a unit
  constexpr int kParts = Sm::kParts, kWords = Sm::kWords;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ LoraGroups gr;
  uint4* vs = reinterpret_cast<uint4*>(smem);    // [tile][32 ranks][part][rows g | g + 8][lane]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + Sm::kV + warp * S * Sm::kUnit;
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int q = 0; q < KQ; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (32 * q + 8 * t >= a.r)
          reinterpret_cast<uint4*>(ring + i * Sm::kUnit)[(4 * q + j) * 32 + lane] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  const int blocks = lora_groups<kCols>(gr, a, a.groups, 16 * MB);
  const int units = (a.N + kCols - 1) / kCols;
  const int col_blocks = (units + a.col_units - 1) / a.col_units;
  const int64_t items = static_cast<int64_t>(blocks) * col_blocks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int bl = static_cast<int>(item / col_blocks);
    const int unit0 = static_cast<int>(item % col_blocks) * a.col_units, unit1 = min(unit0 + a.col_units, units);
    const int2 f = lora_find(gr, a.groups, bl);
    const int first = gr.first[f.x] + f.y * 16 * MB;
    const int count = min(gr.count[f.x] - f.y * 16 * MB, 16 * MB);
    const bool adapted = f.x < a.adapters;
    if (!adapted && a.base == a.out) continue;                   // nothing to add, nowhere to copy
    // this lane's rows of base and out and its rows of B, at the unit to request and at the unit to store
    const int col0 = unit0 * kCols + warp * 32;
    const T* p_base[MB][2];
    T* p_out[MB][2];
    bool live[MB][2];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 16 * m + 8 * h + g;
        const int64_t tok = c < count ? lora_token(a, first + c) : -1;
        live[m][h] = tok >= 0;
        p_base[m][h] = static_cast<const T*>(a.base) + max(tok, static_cast<int64_t>(0)) * a.ldb + col0 + 8 * t;
        p_out[m][h] = static_cast<T*>(a.out) + max(tok, static_cast<int64_t>(0)) * a.ldo + col0 + 8 * t;
      }
    const __nv_bfloat16* p_b = a.b + (static_cast<int64_t>(f.x) * a.N + col0 + 8 * (g >> 1) + (g & 1)) * a.r + 8 * t;
    int r_col = col0;                            // the column of the warp's next request
    auto request = [&](int u, int slot) {
      if (u < unit1) {
        uint4* at = reinterpret_cast<uint4*>(ring + slot * Sm::kUnit) + lane;
        if (adapted) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat16* row = p_b + 2 * j * a.r;
            const bool in = r_col + 8 * (g >> 1) < a.N;          // N is a multiple of eight
#pragma unroll
            for (int q = 0; q < KQ; ++q)
              if (in && 32 * q + 8 * t < a.r) cp_async16(at + (4 * q + j) * 32, row + 32 * q);
          }
          p_b += kCols * static_cast<int64_t>(a.r);
        }
        const bool in = r_col + 8 * t < a.N;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (in && live[m][h]) {
#pragma unroll
              for (int w = 0; w < kWords; ++w)
                cp_async16(at + (KQ * 4 + (2 * m + h) * kWords + w) * 32, reinterpret_cast<const uint4*>(p_base[m][h]) + w);
            }
            p_base[m][h] += kCols;
          }
        r_col += kCols;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) request(unit0 + i, i);
    if (adapted) {
      __syncthreads();                                           // the item before is done with vs
      const float scale = a.scaling != nullptr ? __ldg(a.scaling + f.x) : 1.0f;
      for (int i = threadIdx.x; i < MB * KQ * 2 * 32; i += 32 * WARPS) {
        const int q = i / 64 % KQ, m = i / (64 * KQ), h = i / 32 & 1;
        const int c = 16 * m + 8 * h + g, rank = 32 * q + 8 * t;
        float s[8] = {};
        if (c < count && rank < a.r) {
          const float* src = a.v + static_cast<int64_t>(first + c) * a.r + rank;
          for (int u = 0; u < a.slices; ++u, src += a.T * a.r) {
            const float4 p = *reinterpret_cast<const float4*>(src), w = *reinterpret_cast<const float4*>(src + 4);
            s[0] += p.x; s[1] += p.y; s[2] += p.z; s[3] += p.w;
            s[4] += w.x; s[5] += w.y; s[6] += w.z; s[7] += w.w;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] *= scale;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {              // the leading 8 bits, the next, the rest
          Raw8<__nv_bfloat16> o;
          pack8(o, s);
          vs[(((m * KQ + q) * kParts + part) * 2 + h) * 32 + lane] = o.w[0];
          float d[8];
          unpack8(o, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] -= d[e];
        }
      }
      __syncthreads();
    }
    int slot = 0;
#pragma unroll 1
    for (int u = unit0; u < unit1; ++u) {
      cp_async_wait<S - 2>();
      // every lane reads only what it copied itself; the slot that is requested now
      // was read by this lane in the unit before
      request(u + S - 1, slot + S - 1 >= S ? slot - 1 : slot + S - 1);
      const uint4* u4 = reinterpret_cast<const uint4*>(ring + slot * Sm::kUnit) + lane;
      slot = slot + 1 == S ? 0 : slot + 1;
      const int mine = u * kCols + warp * 32 + 8 * t;              // this lane's 8 output columns
      uint4 bw[KQ][4];
      if (adapted) {
#pragma unroll
        for (int q = 0; q < KQ; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) bw[q][j] = u4[(4 * q + j) * 32];
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if (16 * m >= count) break;
        float acc[4][4];
        if (adapted) {
#pragma unroll
          for (int q = 0; q < KQ; ++q)
#pragma unroll
            for (int part = kParts - 1; part >= 0; --part) {     // the small parts first
              const uint4* v = vs + ((m * KQ + q) * kParts + part) * 64 + lane;
              const uint4 lo = v[0], hi = v[32];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (q == 0 && part == kParts - 1) mma_bf16_first(acc[j], lo.x, hi.x, lo.y, hi.y, bw[q][j].x, bw[q][j].y);
                else mma_bf16(acc[j], lo.x, hi.x, lo.y, hi.y, bw[q][j].x, bw[q][j].y);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) mma_bf16(acc[j], lo.z, hi.z, lo.w, hi.w, bw[q][j].z, bw[q][j].w);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (mine < a.N && live[m][h] &&
              chk(p_out[m][h] - static_cast<const T*>(a.out) + 7, rows_extent(a.T, a.N, a.ldo), CHK_LORA)) {
            Raw8<T> base;
#pragma unroll
            for (int w = 0; w < kWords; ++w) base.w[w] = u4[(KQ * 4 + (2 * m + h) * kWords + w) * 32];
            if (adapted) {
              float2 o[4];
              unpack8(base, o);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[j] = fadd2(o[j], make_float2(acc[j][2 * h], acc[j][2 * h + 1]));
              pack8(base, o);
            }
            store8(p_out[m][h], base, 8);
          }
          p_out[m][h] += kCols;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Expand, r <= 16 and a token a group on average.  An item is a block of one or two tokens of one
// group times a.col_units units of 512 columns, 64 a warp.  B's rows are 16 or 32 bytes and lie together,
// so a warp reads them as they lie, 16 bytes (8 ranks) a lane: a column's one or two
// lanes share its sum, and 32 or 16 columns make a step.  A lane's ranks are the same in
// every step, and its part of v stays in registers.  The sums go through shared memory
// to the lanes that own two neighbouring columns of base and out.  Sums and products are
// FP32.  An item's part of B and base is on its way to L2 while v is awaited.
// 64 tokens with an adapter each of rank 16 beside 7168 -> 18432: 14.5 us (a lane with whole
// rows of B: 16, on matrix instructions 18.5), 2.9 TB/s; what bounds it is the latency of an
// item's steps (group, token, v, B), which one round of items does not overlap.
// ---------------------------------------------------------------------------
constexpr int kLoraFewColumns = 2 * kLoraThreads;
constexpr int kLoraFewRank = 16, kLoraFewTokens = 2;
constexpr int kLoraFewSteps = 4;       // loads a lane keeps on their way

// The item's units for TC tokens; sums: this warp's.
template <typename T, int TC>
__device__ __forceinline__ void lora_few_units(const LoraArgs& a, int group, bool adapted, int unit0, int unit1,
                                               const float (*vs)[kLoraFewRank], const int64_t* tokens,
                                               float (*sums)[64]) {
  using Pair = typename std::conditional<sizeof(T) == 4, float2, uint32_t>::type;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool two = a.r > 8;                                       // lanes a column
  const int columns = two ? 16 : 32, q = two ? lane & 1 : 0, lc = two ? lane >> 1 : lane;
  float2 v[TC][4];
#pragma unroll
  for (int c = 0; c < TC; ++c) {
    const float4 lo = *reinterpret_cast<const float4*>(&vs[c][8 * q]), hi = *reinterpret_cast<const float4*>(&vs[c][8 * q + 4]);
    v[c][0] = make_float2(lo.x, lo.y); v[c][1] = make_float2(lo.z, lo.w);
    v[c][2] = make_float2(hi.x, hi.y); v[c][3] = make_float2(hi.z, hi.w);
  }
  for (int u = unit0; u < unit1; ++u) {
    const int col0 = u * kLoraFewColumns + 64 * warp, col = col0 + 2 * lane;
    if (col0 >= a.N) break;
    const bool mine = col < a.N;                                  // N is a multiple of eight
    Pair base[TC];                                                // on their way while B is multiplied
#pragma unroll
    for (int c = 0; c < TC; ++c)
      if (mine)
        base[c] = __ldcs(reinterpret_cast<const Pair*>(static_cast<const T*>(a.base) +
                                                       max(tokens[c], static_cast<int64_t>(0)) * a.ldb + col));
    if (adapted) {
      const __nv_bfloat16* rows = a.b + (static_cast<int64_t>(group) * a.N + col0) * a.r + 8 * lane;
      const int end = min(64, a.N - col0);                        // of the warp's columns
      for (int c0 = 0; c0 < end; c0 += kLoraFewSteps * columns) {
        Raw8<__nv_bfloat16> raw[kLoraFewSteps];
#pragma unroll
        for (int i = 0; i < kLoraFewSteps; ++i) {
          const int at = c0 + i * columns;
          raw[i].w[0] = make_uint4(0, 0, 0, 0);
          if (at + lc < end) raw[i].w[0] = __ldg(reinterpret_cast<const uint4*>(rows + static_cast<int64_t>(at) * a.r));
        }
#pragma unroll
        for (int i = 0; i < kLoraFewSteps; ++i) {
          float2 b[4];
          unpack8(raw[i], b);
          const int at = c0 + i * columns + lc;
#pragma unroll
          for (int c = 0; c < TC; ++c) {
            float2 p = fmul2(v[c][0], b[0]);
#pragma unroll
            for (int j = 1; j < 4; ++j) p = ffma2(v[c][j], b[j], p);
            float sum = p.x + p.y;
            if (two) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            if (q == 0 && at < end) sums[c][at] = sum;
          }
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < TC; ++c) {
      const int64_t tok = tokens[c];
      if (!mine || tok < 0 || !chk(tok * a.ldo + col + 1, rows_extent(a.T, a.N, a.ldo), CHK_LORA)) continue;
      const float2 d = adapted ? *reinterpret_cast<const float2*>(&sums[c][2 * lane]) : f2(0.0f);
      Pair* out = reinterpret_cast<Pair*>(static_cast<T*>(a.out) + tok * a.ldo + col);
      if constexpr (sizeof(T) == 4) {
        *out = adapted ? fadd2(base[c], d) : base[c];
      } else {
        const float2 o = fadd2(make_float2(bf16lo(base[c]), bf16hi(base[c])), d);
        *out = adapted ? pack_bf16x2(o.x, o.y) : base[c];
      }
    }
    __syncwarp();                                                 // sums is free again
  }
}

template <typename T>
__global__ void __launch_bounds__(kLoraThreads, 4) lora_expand_few_kernel(const LoraArgs a) {
  __shared__ LoraGroups gr;
  __shared__ __align__(16) float vs[kLoraFewTokens][kLoraFewRank];
  __shared__ __align__(16) float sums[kLoraWarps][kLoraFewTokens][64];
  __shared__ int64_t tokens[kLoraFewTokens];
  const int blocks = lora_groups<kLoraThreads>(gr, a, a.groups, kLoraFewTokens);
  const int units = (a.N + kLoraFewColumns - 1) / kLoraFewColumns;
  const int col_blocks = (units + a.col_units - 1) / a.col_units;
  const int64_t items = static_cast<int64_t>(blocks) * col_blocks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int bl = static_cast<int>(item / col_blocks);
    const int unit0 = static_cast<int>(item % col_blocks) * a.col_units, unit1 = min(unit0 + a.col_units, units);
    const int2 f = lora_find(gr, a.groups, bl);
    const int first = gr.first[f.x] + f.y * kLoraFewTokens;
    const int count = min(gr.count[f.x] - f.y * kLoraFewTokens, kLoraFewTokens);
    const bool adapted = f.x < a.adapters;
    if (!adapted && a.base == a.out) continue;                   // nothing to add, nowhere to copy
    const int64_t col0 = static_cast<int64_t>(unit0) * kLoraFewColumns;
    const int cols = static_cast<int>(min(static_cast<int64_t>(unit1) * kLoraFewColumns, static_cast<int64_t>(a.N)) - col0);
    if (threadIdx.x == 32 && adapted)
      bulk_prefetch(a.b + (static_cast<int64_t>(f.x) * a.N + col0) * a.r, static_cast<int64_t>(cols) * a.r * 2);
    __syncthreads();                                             // the item before is done with vs
    if (static_cast<int>(threadIdx.x) < count) {
      const int64_t tok = lora_token(a, first + threadIdx.x);
      tokens[threadIdx.x] = tok;
      if (tok >= 0) bulk_prefetch(static_cast<const T*>(a.base) + tok * a.ldb + col0, static_cast<int64_t>(cols) * sizeof(T));
    }
    pdl_wait();
    const float scale = adapted && a.scaling != nullptr ? __ldg(a.scaling + f.x) : 1.0f;
    if (adapted && static_cast<int>(threadIdx.x) < count * a.r) {
      const int c = threadIdx.x / a.r, rank = threadIdx.x - c * a.r;
      const float* src = a.v + static_cast<int64_t>(first + c) * a.r + rank;
      float s = 0.0f;
#pragma unroll 4
      for (int u = 0; u < a.slices; ++u) s += src[u * a.T * a.r];
      vs[c][rank] = s * scale;
    }
    __syncthreads();
    if (count == 1) lora_few_units<T, 1>(a, f.x, adapted, unit0, unit1, vs, tokens, sums[threadIdx.x >> 5]);
    else lora_few_units<T, 2>(a, f.x, adapted, unit0, unit1, vs, tokens, sums[threadIdx.x >> 5]);
  }
  pdl_wait();                                                    // of a block without an item, too
}

}  // namespace fp8q
