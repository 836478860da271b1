// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + s_a B_a (A_a x[t]),   a = the adapter of token t
//
// base is the projection's output (fp8q_gemm_blockscaled); tokens come grouped
// by adapter (fp8q_moe_dispatch_layout).  Two launches:
//   shrink   v = A_a x, FP32, in K slices where tokens are few
//   expand   out = base + s_a B_a v
// With few tokens an adapter the bound is reading A and B once, with many it is
// x, base and out; the products are 2 r (K + N) a token, far under either, so
// both run on mma.sync with operands loaded straight into fragment order.
// x, A and B are BF16 as given; v is split into BF16 parts (two for a BF16
// output, which keep v to 2^-16 of itself; three for FP32, 2^-24), so that its
// rounding stays under the output's.
#pragma once

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
  int slices;
};

// The groups' token ranges and the running count of their blocks of `tile`
// tokens, in shared memory; returns the number of blocks.  A group's bounds
// are clamped to [0, T]; bounds that decrease or leave it are reported.
struct LoraGroups {
  int first[kLoraMaxGroups];
  int count[kLoraMaxGroups];
  int upto[kLoraMaxGroups];       // blocks of groups 0 .. i
  int sums[kLoraWarps];
};
__device__ __forceinline__ int lora_groups(LoraGroups& s, const LoraArgs& a, int groups, int tile) {
  constexpr int kPer = kLoraMaxGroups / kLoraThreads;
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

// ---------------------------------------------------------------------------
// Shrink.  An item is a block of up to 8 G tokens of one adapter times up to
// 16 RT of its ranks times one K slice; the block's warps split the slice's
// chunks of 32 P elements and join their FP32 sums in shared memory.  The
// operands' order along K is free as long as both share it: lane (g, t) takes
// the 16-byte piece t of a chunk of rows g and g + 8, in fragment order.  Every lane
// reads back only what it copied itself (cp.async), so the ring of S units (one
// unit: one chunk of one item) needs no barrier, and runs on across items.
// ---------------------------------------------------------------------------
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
  const int groups = min(a.groups, a.adapters);          // the others shrink to nothing
  const int blocks = lora_groups(gr, a, groups, 8 * G);
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
    float acc[RT][G][4];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.0f;
    for (int chunk = w.chunk0 + warp; chunk < w.chunk1; chunk += kLoraWarps) {
      cp_async_wait<S - 2>();
      // every lane reads only what it copied itself: no other wait.  The slot that is
      // requested now was read by this lane in the step before.
      request();
      const uint4* u4 = reinterpret_cast<const uint4*>(ring + slot * Sm::kUnit) + lane;
      slot = slot + 1 == S ? 0 : slot + 1;
      // the tensor cores add at most 4 P instructions' products before an FP32 addition
      float part[RT][G][4];
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) part[m][j][c] = 0.0f;
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
            mma_bf16(part[m][j], lo.x, hi.x, lo.y, hi.y, xb[j].x, xb[j].y);
            mma_bf16(part[m][j], lo.z, hi.z, lo.w, hi.w, xb[j].z, xb[j].w);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[m][j][c] += part[m][j][c];
    }
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int j = 0; j < G; ++j)
        join[(warp * RT * G + m * G + j) * 32 + lane] =
            make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
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
        if (col < w.count && chk(pos, a.T, CHK_LORA)) {
          float* dst = a.v + (w.slice * a.T + pos) * a.r + rank;
          if (rank < a.r) dst[0] = lo[c];
          if (rank + 8 < a.r) dst[8] = hi[c];
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Expand.  An item is a block of up to 16 MB tokens of one group times 256 CB
// columns; a warp takes 32 columns at a time.  Tokens are the rows of the
// product, v's parts its first operand (in shared memory, fragment order), B's
// rows the second, loaded once an item into registers.  The 8 columns of an
// instruction stand for columns 8 (c / 2) + 2 j + c % 2 of the warp's 32 (j: the
// instruction's number of four), so that a lane ends with 8 consecutive columns:
// base and out move in 16-byte words, 64 contiguous bytes a row.
// ---------------------------------------------------------------------------
template <typename T, int KQ, int MB, int CB>
__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(const LoraArgs a) {
  constexpr int kParts = sizeof(T) == 4 ? 3 : 2;
  __shared__ LoraGroups gr;
  __shared__ __align__(16) uint4 vs[MB][KQ][kParts][2][32];      // [tile][32 ranks][part][rows g | g + 8][lane]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int blocks = lora_groups(gr, a, a.groups, 16 * MB);
  const int col_blocks = (a.N + 256 * CB - 1) / (256 * CB);
  const int64_t items = static_cast<int64_t>(blocks) * col_blocks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int bl = static_cast<int>(item / col_blocks);
    const int col0 = static_cast<int>(item % col_blocks) * 256 * CB;
    const int2 f = lora_find(gr, a.groups, bl);
    const int first = gr.first[f.x] + f.y * 16 * MB;
    const int count = min(gr.count[f.x] - f.y * 16 * MB, 16 * MB);
    const bool adapted = f.x < a.adapters;
    if (!adapted && a.base == a.out) continue;                   // nothing to add, nowhere to copy
    int64_t tok[MB][2];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 16 * m + 8 * h + g;
        tok[m][h] = c < count ? lora_token(a, first + c) : -1;
      }
    if (adapted) {
      __syncthreads();                                           // the item before is done with vs
      const float scale = a.scaling != nullptr ? __ldg(a.scaling + f.x) : 1.0f;
      for (int i = threadIdx.x; i < MB * KQ * 2 * 32; i += kLoraThreads) {
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
          vs[m][q][part][h][lane] = o.w[0];
          float d[8];
          unpack8(o, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] -= d[e];
        }
      }
      __syncthreads();
    }
#pragma unroll 1
    for (int cb = 0; cb < CB; ++cb) {
      const int c0 = col0 + cb * 256 + warp * 32;
      if (c0 >= a.N) break;
      const int mine = c0 + 8 * t;                               // this lane's 8 output columns
      const bool in = mine < a.N;
      uint4 bw[KQ][4];
      if (adapted) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
          const __nv_bfloat16* src = a.b + (static_cast<int64_t>(f.x) * a.N + col) * a.r + 8 * t;
#pragma unroll
          for (int q = 0; q < KQ; ++q)
            bw[q][j] = col < a.N && 32 * q + 8 * t < a.r ? __ldg(reinterpret_cast<const uint4*>(src + 32 * q))
                                                         : make_uint4(0, 0, 0, 0);
        }
      }
      Raw8<T> bs[MB][2];
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (in && tok[m][h] >= 0) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
              bs[m][h].w[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(a.base) +
                                                                   tok[m][h] * a.ldb + mine) + i);
          }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if (16 * m >= count) break;
        float acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[j][c] = 0.0f;
        if (adapted) {
#pragma unroll
          for (int q = 0; q < KQ; ++q)
#pragma unroll
            for (int part = kParts - 1; part >= 0; --part) {     // the small parts first
              const uint4 lo = vs[m][q][part][0][lane], hi = vs[m][q][part][1][lane];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                mma_bf16(acc[j], lo.x, hi.x, lo.y, hi.y, bw[q][j].x, bw[q][j].y);
                mma_bf16(acc[j], lo.z, hi.z, lo.w, hi.w, bw[q][j].z, bw[q][j].w);
              }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (in && tok[m][h] >= 0 && chk(mine + 7, a.ldo, CHK_LORA)) {
            float o[8];
            unpack8(bs[m][h], o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              o[2 * j] += acc[j][2 * h];
              o[2 * j + 1] += acc[j][2 * h + 1];
            }
            Raw8<T> w;
            if (adapted) pack8(w, o);
            else w = bs[m][h];
            store8(static_cast<T*>(a.out) + tok[m][h] * a.ldo + mine, w, 8);
          }
      }
    }
  }
}

}  // namespace fp8q
