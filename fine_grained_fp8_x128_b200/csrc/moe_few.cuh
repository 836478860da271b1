// A whole mixture-of-experts layer for a few tokens (decoding), over the same
// E4M3 expert weights with 128x128 scales as the grouped GEMM:
//
//   y[t] = sum_j w[t,j] Wd[e] h,   h = silu(Wg[e] x[t]) * (Wu[e] x[t]),  e = ids[t,j]
//   (without a gate matrix h = Wu[e] x[t])
//
// With a handful of tokens an expert every weight byte is used once or a few
// times, so the layer is bound by reading the picked experts' codes once.  The
// activations are NOT quantized: they go to the tensor cores as FP16 with an
// exact power-of-two scale per 128-wide chunk (a hidden row as two FP16 parts,
// which keep it to 2^-22), the codes are widened E4M3 -> FP16 in registers
// (exact), products are summed in FP32 over one 128-wide chunk and then
// multiplied by the weight block's and the chunk's scales.
// mma.sync rather than tcgen05: the widened codes would have to go back through
// shared memory to be a tcgen05 operand, twice the bytes that came in, and at
// these token counts the matrix instructions are far from their limit.
//
// Five launches, each started while the one before runs out (programmatic
// dependent launch) and waiting for its end before any access:
//   plan     tokens by expert in blocks of 8 columns; x to FP16 records
//   up       hidden rows, FP32
//   hidden   hidden rows to FP16 records
//   down     each (token, slot)'s output row, FP32
//   combine  the weighted sum over a token's slots, in slot order
// No atomic touches a result: equal inputs give equal bits.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "norm.cuh"

namespace fp8q {

constexpr int kFewMaxTokens = 128;
constexpr int kFewMaxEntries = 1024;
constexpr int kFewMaxExperts = 1024;
constexpr int kFewThreads = 256;              // hidden
constexpr int kFewWarps = 8;                  // of a weight pass, which multiply
constexpr int kFewLoaders = 4;                // and of those that load
constexpr int kFewWeightThreads = 32 * (kFewWarps + kFewLoaders);
constexpr int kFewTiles = 2;                  // row tiles a multiplying warp takes
// a chunk's record: 128 FP16 values, as many lower parts in a hidden row's, and the scale, in 16-byte units
constexpr int kFewRecord = 272, kFewHiddenRecord = 528;

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
  int64_t xr;           // records [T][H/128]
  int64_t hid;          // FP32 [max_positions][I]
  int64_t hr;           // records [max_positions][I/128]
  int64_t yp;           // FP32 [T k][H]
  int64_t bytes;
};
__host__ __device__ inline int64_t few_align(int64_t v) { return (v + 255) / 256 * 256; }
__host__ __device__ inline FewLayout few_layout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  FewLayout l;
  const int64_t n = T * k;
  const int64_t groups = n < E ? n : E;
  l.max_positions = (n + 7 * groups + 7) / 8 * 8;
  l.max_blocks = l.max_positions / 8;
  int64_t o = few_align(sizeof(FewPlan));
  l.block_expert = o; o = few_align(o + 4 * l.max_blocks);
  l.block_start = o; o = few_align(o + 4 * l.max_blocks);
  l.block_count = o; o = few_align(o + 4 * l.max_blocks);
  l.entry = o; o = few_align(o + 4 * l.max_positions);
  l.xr = o; o = few_align(o + kFewRecord * T * (H / 128));
  l.hid = o; o = few_align(o + 4 * l.max_positions * I);
  l.hr = o; o = few_align(o + kFewHiddenRecord * l.max_positions * (I / 128));
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
// FP16 records: 128 values times a power of two that takes their largest
// magnitude into [2^14, 2^15), and the inverse power.  The scaling is exact, FP16
// keeps 11 bits (a BF16 value has 8, so x is exact) down to 2^-28 of the
// chunk's maximum, and what lies below is off by at most 2^-40 of that maximum,
// under the FP32 accumulation's own rounding.  A hidden value is two of them,
// the nearest and what is left (kTwo), and off by at most 2^-22 of itself or
// 2^-40 of the maximum.  The power is at most 2^84, so that its inverse times a block
// scale (>= 1e-12) is a normal FP32 number: a chunk under 2^-98 loses bits,
// 2^-109 at most.
// Value k = 32 t + 8 q + i lies at 16-byte unit 4 q + t, place i: the order in
// which lanes t of a warp read their multiplier operand, without bank conflicts.
// A warp owns one chunk, four consecutive values a lane.
// ---------------------------------------------------------------------------
template <bool kTwo>
__device__ __forceinline__ void few_record(const float (&f)[4], uint8_t* dst, int lane) {
  float m = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;   // m >= 0: no sign bit
  e = max(e, -70);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
  float v[4] = {f[0] * up, f[1] * up, f[2] * up, f[3] * up};
  const int t = lane >> 3, q = (lane & 7) >> 1;
  uint8_t* at = dst + (4 * q + t) * 16 + 8 * (lane & 1);
#pragma unroll
  for (int part = 0; part < (kTwo ? 2 : 1); ++part) {
    const __half2 h0 = __floats2half2_rn(v[0], v[1]), h1 = __floats2half2_rn(v[2], v[3]);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t*>(&h0);
    o.y = *reinterpret_cast<const uint32_t*>(&h1);
    *reinterpret_cast<uint2*>(at + 256 * part) = o;
    const float d[4] = {__low2float(h0), __high2float(h0), __low2float(h1), __high2float(h1)};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = isinf(d[i]) ? 0.0f : v[i] - d[i];
  }
  if (lane == 0) *reinterpret_cast<float*>(dst + (kTwo ? 512 : 256)) = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
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
__global__ void __launch_bounds__(1024) few_plan_kernel(const FewArgs a) {
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_launch();
  if (blockIdx.x > 0) {
    const int chunks = a.H / 128;
    const int item = (blockIdx.x - 1) * 32 + (tid >> 5);
    if (item >= a.T * chunks) return;
    const int t = item / chunks, kb = item - t * chunks;
    const uint2 r = *reinterpret_cast<const uint2*>(a.x + t * a.ldx + kb * 128 + 4 * lane);
    const float f[4] = {bf16lo(r.x), bf16hi(r.x), bf16lo(r.y), bf16hi(r.y)};
    const int64_t at = a.l.xr + static_cast<int64_t>(item) * kFewRecord;
    if (chk(at + kFewRecord - 1, a.l.hid, CHK_FEW)) few_record<false>(f, few_at<uint8_t>(a, at), lane);
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
  const int2 mine = make_int2((c + 7) / 8 * 8, (c + 7) / 8);   // padded positions, column blocks
  const int2 upto = few_scan(mine, sums);
  start[tid] = upto.x - mine.x;
  for (int b = 0; b < mine.y; ++b) {
    const int at = upto.y - mine.y + b;
    if (chk(at, a.l.max_blocks, CHK_FEW)) {
      few_at<int>(a, a.l.block_expert)[at] = tid;
      few_at<int>(a, a.l.block_start)[at] = upto.x - mine.x + 8 * b;
      few_at<int>(a, a.l.block_count)[at] = min(c - 8 * b, 8);
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
// The two weight passes.  An item is RT tiles of 16 weight rows of one expert
// times one block of up to 8 of its columns.  A block's 8 multiplying warps
// take an item in stages of KC 128-wide K chunks, RT KC = 16: a warp multiplies two
// tiles by one chunk of the stage, so that the columns' operands and a stage's
// bookkeeping serve 4 KB of codes, and the warps' FP32 sums are joined once an
// item, in chunk order.  (Sixteen warps of one tile each were bound by their
// instructions: 59 us for one token's up pass, 8 experts of 7168 -> 2048, which
// now takes 38.6, 6.1 TB/s of codes; the down pass 23.7, 4.9 TB/s.  With 128 tokens
// over 256 experts the passes take 876 and 536 us at 1965 MHz, bound by the latency
// of a stage's multiplications; in a row of calls the power limit lowers the clock
// and they take a quarter longer.)
// The down pass multiplies both parts of a hidden row: with one FP16 number a row it
// took 21.5 and 443 us, and every result, the FP32 ones too, was off by some 2^-12.
// Lower parts in the columns that a block of four or fewer leaves spare gained
// nothing: a loop for each form 71.7 us against 72.5 for the one-token call, a
// branch within the loop 76.7.
// Four more warps keep the ring of S stages full, across items.  One lane issues
// a copy in some 100 clocks, so the work is spread: three warps issue the TMA
// boxes of rows x 128 bytes, the fourth one bulk copy a column for its KC records
// and the stage's block scales, which start on no 16-byte boundary and so are
// per-thread copies that arrive on the stage's barrier.  They look up an item's
// block and columns while they load the item before, and hand it on with the stage.
//
// Along K an instruction's operands may be taken in any order that both share:
// lane (g, t) takes bytes 32 t .. 32 t + 31 of rows g and g + 8, which under the
// TMA's 128-byte swizzle are two conflict-free 16-byte reads a row.
// Columns past the block's count hold what the ring held before: a column's
// garbage stays in that column, and is not stored.
// ---------------------------------------------------------------------------
enum : int { kFewGated = 0, kFewPlain = 1, kFewDown = 2 };

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
// A four-byte asynchronous copy, and this lane's arrival once its copies so far are done.
__device__ __forceinline__ void cp_async4(void* smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// The multiplying warps' own barrier.
__device__ __forceinline__ void few_join_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory");
}

template <int MODE, int RT, int S>
struct FewSmem {
  static constexpr int kRecord = MODE == kFewDown ? kFewHiddenRecord : kFewRecord;
  static constexpr int kKC = kFewWarps * kFewTiles / RT;
  static constexpr int kChunkBytes = RT * 16 * 128;                      // a chunk's codes
  // a column's records, an odd number of 64-byte halves apart: neighbouring columns use the other half of the banks
  static constexpr int kColumn = (kKC * kRecord + 63) / 128 * 128 + 64;
  static constexpr int kScales = kKC * kChunkBytes + 8 * kColumn;    // 2 KC block scales
  static constexpr int kStage = (kScales + 8 * kKC + 1023) / 1024 * 1024;
  static constexpr int kRing = S * kStage;
  static constexpr int kJoin = kFewWarps * kFewTiles * 512;
  static constexpr int kBytes = 1024 + kRing + kJoin + 32 * S + 16;      // 1024: the ring's alignment
  static_assert(kColumn >= kKC * kRecord && kColumn % 128 == 64, "column stride");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int MODE, int RT, int S>
__global__ void __launch_bounds__(kFewWeightThreads)
few_weights_kernel(const __grid_constant__ CUtensorMap map_lo, const __grid_constant__ CUtensorMap map_hi,
                   const FewArgs a) {
  using Sm = FewSmem<MODE, RT, S>;
  constexpr int KC = Sm::kKC;
  constexpr int kRecord = Sm::kRecord, kParts = MODE == kFewDown ? 2 : 1;
  constexpr int kRows = MODE == kFewGated ? 8 * RT : 16 * RT;            // output rows an item, and a box's
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* join = reinterpret_cast<float4*>(ring + Sm::kRing);
  int4* stage_item = reinterpret_cast<int4*>(ring + Sm::kRing + Sm::kJoin);   // a stage's item: columns, first position, row
  uint64_t* full = reinterpret_cast<uint64_t*>(stage_item + S);
  uint64_t* empty = full + S;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + S);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 33);       // the bytes' announcement and the lanes that copy scales
      mbar_init(&empty[s], kFewWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_launch();
  pdl_wait();
  const int K = MODE == kFewDown ? a.I : a.H;
  const int N = MODE == kFewDown ? a.H : a.I;
  const int KB = K / 128;
  const int steps = (KB + KC - 1) / KC;
  const uint32_t blocks = few_plan(a)->blocks;
  const uint32_t items = blocks * static_cast<uint32_t>(N / kRows);      // at most 1024 x 4096
  const int* entry = few_at<const int>(a, a.l.entry);

  if (warp >= kFewWarps) {
    // ---- the loading warps: the last one the columns and the scales, the others the boxes in turn ----
    const int loader = warp - kFewWarps;
    constexpr int kBoxLoaders = kFewLoaders - 1, kBoxes = MODE == kFewGated ? 2 * KC : KC;
    const bool columns = loader == kBoxLoaders;
    const int* block_expert = few_at<const int>(a, a.l.block_expert);
    const int* block_start = few_at<const int>(a, a.l.block_start);
    const int* block_count = few_at<const int>(a, a.l.block_count);
    const uint8_t* records = few_at<const uint8_t>(a, MODE == kFewDown ? a.l.hr : a.l.xr);
    // lanes 0 .. KC - 1 fetch the lower rows' scales, with a gate the next KC the upper rows'
    const float* scales = MODE == kFewDown ? a.sd : (MODE == kFewGated ? (lane < KC ? a.sg : a.su) : a.su);
    const int sc = lane % KC;
    struct Item {
      int expert, start, count, row, record;      // record: this lane's column (or -1)
    };
    auto look_up = [&](uint32_t item) {
      Item i{0, 0, 0, 0, -1};
      if (item < items) {
        const uint32_t rb = item / blocks, b = item - rb * blocks;
        i.expert = block_expert[b];
        i.start = block_start[b];
        i.count = block_count[b];
        i.row = static_cast<int>(rb) * kRows;
      }
      return i;
    };
    auto look_up_column = [&](Item& i) {
      if (columns && lane < i.count) i.record = MODE == kFewDown ? i.start + lane : entry[i.start + lane] / a.k;
    };
    Item now = look_up(blockIdx.x);
    look_up_column(now);
    Item next = look_up(blockIdx.x + gridDim.x);
    uint32_t it = 0, slot = 0, phase = 1;
    bool ok = true;
    for (uint32_t item = blockIdx.x; item < items && ok; item += gridDim.x) {
      look_up_column(next);
      const Item after = look_up(item + 2 * gridDim.x);
      const int row0 = now.expert * N + now.row;
      const float* scale = scales + static_cast<int64_t>(row0 / 128) * KB + sc;
      const uint8_t* col = records + static_cast<int64_t>(max(now.record, 0)) * KB * kRecord;
      for (int c0 = 0; c0 < KB; c0 += KC) {
        if (!warp_wait_converged(&empty[slot], phase, abort_flag, WAIT_PRODUCER_EMPTY)) { ok = false; break; }
        const int n = min(KC, KB - c0);
        uint8_t* stage = ring + slot * Sm::kStage;
        if (columns) {
          if (now.record >= 0)
            bulk_load(stage + KC * Sm::kChunkBytes + lane * Sm::kColumn, col + c0 * kRecord, n * kRecord,
                      &full[slot]);
          if (lane < kBoxes && sc < n) cp_async4(stage + Sm::kScales + 4 * lane, scale + c0);
          cp_async_arrive(&full[slot]);
        } else if (lane == 0) {
          if (loader == 0) {
            stage_item[slot] = make_int4(now.count, now.start, now.row, 0);
            mbar_arrive_expect_tx(&full[slot], n * (Sm::kChunkBytes + now.count * kRecord));
          }
#pragma unroll
          for (int i = 0; i < (kBoxes + kBoxLoaders - 1) / kBoxLoaders; ++i) {
            const int box = i * kBoxLoaders + loader, c = box % KC;      // with a gate: KC boxes of it, then of the other
            if (box < kBoxes && c < n)
              tma_load_2d_nohint(stage + c * Sm::kChunkBytes + (box >= KC ? RT * 1024 : 0), box >= KC ? &map_hi : &map_lo,
                                 &full[slot], (c0 + c) * 128, row0);
          }
        }
        __syncwarp();
        ++it;
        slot = slot + 1 == S ? 0 : slot + 1;
        phase ^= slot == 0 ? 1 : 0;
      }
      now = next;
      next = after;
    }
    // a wait that gave up leaves copies in flight, which still write this block's memory
    for (uint32_t j = it > S ? it - S : 0; j < it; ++j)
      mbar_wait(&full[j % S], (j / S) & 1, nullptr, WAIT_DRAIN, 1ll << 22);
    return;
  }

  // ---- the multiplying warps ----
  constexpr int TW = kFewTiles;
  const int g = lane >> 2, t = lane & 3;
  const int kc = warp % KC, rt0 = warp / KC * TW;
  // codes: rows g of the two halves of the first tile; the next tile lies kTileStep further on
  constexpr int kTileStep = (MODE == kFewGated ? 8 : 16) * 128;
  const int code_lo = kc * Sm::kChunkBytes + (MODE == kFewGated ? 8 * rt0 + g : 16 * rt0 + g) * 128;
  const int code_hi = code_lo + (MODE == kFewGated ? 8 * RT : 8) * 128;
  const int sw0 = ((2 * t) ^ g) * 16, sw1 = ((2 * t + 1) ^ g) * 16;
  const int col_at = KC * Sm::kChunkBytes + kc * kRecord;
  uint32_t slot = 0, phase = 0;
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    float acc[TW][4];
#pragma unroll
    for (int m = 0; m < TW; ++m)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][c] = 0.0f;
    int count = 0, start = 0, row0 = 0;
    for (int st = 0; st < steps; ++st) {
      const int kb = st * KC + kc;
      const bool ok = warp_wait_converged(&full[slot], phase, abort_flag, WAIT_STAGE);
      if (ok && st == 0) {
        const int4 i = stage_item[slot];
        count = i.x;
        start = i.y;
        row0 = i.z;
      }
      if (ok && kb < KB) {
        const uint8_t* stage = ring + slot * Sm::kStage;
        const float* block_scale = reinterpret_cast<const float*>(stage + Sm::kScales) + kc;
        const float w0 = block_scale[0], w1 = MODE == kFewGated ? block_scale[KC] : w0;
        float part[kParts][TW][4];            // a hidden row's parts have sums of their own: neither waits for the other
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
          for (int m = 0; m < TW; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) part[p][m][c] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t l4[TW][4], h4[TW][4];
#pragma unroll
          for (int m = 0; m < TW; ++m) {
            const uint4 lo = *reinterpret_cast<const uint4*>(stage + code_lo + m * kTileStep + (h ? sw1 : sw0));
            const uint4 hi = *reinterpret_cast<const uint4*>(stage + code_hi + m * kTileStep + (h ? sw1 : sw0));
            l4[m][0] = lo.x; l4[m][1] = lo.y; l4[m][2] = lo.z; l4[m][3] = lo.w;
            h4[m][0] = hi.x; h4[m][1] = hi.y; h4[m][2] = hi.z; h4[m][3] = hi.w;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t al[TW][4], ah[TW][4];
#pragma unroll
            for (int m = 0; m < TW; ++m) {
              widen4(l4[m][2 * q], al[m][0], al[m][1]);
              widen4(l4[m][2 * q + 1], al[m][2], al[m][3]);
              widen4(h4[m][2 * q], ah[m][0], ah[m][1]);
              widen4(h4[m][2 * q + 1], ah[m][2], ah[m][3]);
            }
            uint4 c[kParts];
#pragma unroll
            for (int p = 0; p < kParts; ++p)
              c[p] = *reinterpret_cast<const uint4*>(stage + col_at + g * Sm::kColumn + 256 * p + (4 * (2 * h + q) + t) * 16);
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
              for (int m = 0; m < TW; ++m) mma_f16(part[p][m], al[m][0], ah[m][0], al[m][1], ah[m][1], c[p].x, c[p].y);
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
              for (int m = 0; m < TW; ++m) mma_f16(part[p][m], al[m][2], ah[m][2], al[m][3], ah[m][3], c[p].z, c[p].w);
          }
        }
        const uint8_t* sc = stage + col_at + 2 * t * Sm::kColumn + 256 * kParts;
        const float c0 = *reinterpret_cast<const float*>(sc), c1 = *reinterpret_cast<const float*>(sc + Sm::kColumn);
#pragma unroll
        for (int m = 0; m < TW; ++m) {
          if constexpr (kParts == 2) {
#pragma unroll
            for (int c = 0; c < 4; ++c) part[0][m][c] += part[1][m][c];
          }
          acc[m][0] = fmaf(part[0][m][0], w0 * c0, acc[m][0]);
          acc[m][1] = fmaf(part[0][m][1], w0 * c1, acc[m][1]);
          acc[m][2] = fmaf(part[0][m][2], w1 * c0, acc[m][2]);
          acc[m][3] = fmaf(part[0][m][3], w1 * c1, acc[m][3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      slot = slot + 1 == S ? 0 : slot + 1;
      phase ^= slot == 0 ? 1 : 0;
    }
    few_join_barrier();                       // the item before has been read out of join
#pragma unroll
    for (int m = 0; m < TW; ++m)
      join[(kc * RT + rt0 + m) * 32 + lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
    few_join_barrier();
    static_assert(RT <= kFewWarps, "a tile's sums a warp");
    if (warp < RT) {
      const int m = warp;
      float4 s = join[m * 32 + lane];
#pragma unroll
      for (int u = 1; u < KC; ++u) {
        const float4 v = join[(u * RT + m) * 32 + lane];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
      // rows g and g + 8 (.xy, .zw) of the tile, columns 2 t and 2 t + 1
      const float lo[2] = {s.x, s.y}, hi[2] = {s.z, s.w};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 2 * t + c;
        if (col >= count) continue;
        const int at = start + col;
        if (MODE == kFewGated) {
          const float h = lo[c] / (1.0f + expf(-lo[c])) * hi[c];
          const int64_t to = static_cast<int64_t>(at) * N + row0 + 8 * m + g;
          if (chk(to, a.l.max_positions * a.I, CHK_FEW)) few_at<float>(a, a.l.hid)[to] = h;
        } else {
          const int64_t row = MODE == kFewDown ? entry[at] : at;
          const int64_t to = row * N + row0 + 16 * m + g;
          float* dst = few_at<float>(a, MODE == kFewDown ? a.l.yp : a.l.hid) + to;
          const int64_t extent = (MODE == kFewDown ? static_cast<int64_t>(a.T) * a.k : a.l.max_positions) * N;
          if (chk(to, extent, CHK_FEW) && chk(to + 8, extent, CHK_FEW)) {
            dst[0] = lo[c];
            dst[8] = hi[c];
          }
        }
      }
    }
  }
}

// Hidden rows to FP16 records: a warp a chunk.
__global__ void __launch_bounds__(kFewThreads) few_hidden_kernel(const FewArgs a) {
  pdl_launch();
  pdl_wait();
  constexpr int kWarps = kFewThreads / 32;
  const int lane = threadIdx.x & 31;
  const int chunks = a.I / 128;
  const int items = few_plan(a)->positions * chunks;
  const int* entry = few_at<const int>(a, a.l.entry);
  for (int item = blockIdx.x * kWarps + (threadIdx.x >> 5); item < items; item += gridDim.x * kWarps) {
    const int p = item / chunks;
    if (entry[p] < 0) continue;
    const float4 v = *reinterpret_cast<const float4*>(few_at<const float>(a, a.l.hid) + static_cast<int64_t>(item) * 128 +
                                                      4 * lane);
    const float f[4] = {v.x, v.y, v.z, v.w};
    const int64_t at = a.l.hr + static_cast<int64_t>(item) * kFewHiddenRecord;
    if (chk(at + kFewHiddenRecord - 1, a.l.yp, CHK_FEW)) few_record<true>(f, few_at<uint8_t>(a, at), lane);
  }
}

// y[t] = sum_j share[t,j] * (slot j's row), in slot order; a token none of
// whose slots names an expert gets zeros.  Eight columns a thread; a skipped
// slot's row is read with the others (its place holds anything) and not used.
template <typename T>
__global__ void __launch_bounds__(64) few_combine_kernel(const FewArgs a) {
  const int t = blockIdx.y;
  const int n = (blockIdx.x * 64 + threadIdx.x) * 8;
  pdl_wait();
  if (n >= a.H) return;
  float s[8] = {};
  const float* rows = few_at<const float>(a, a.l.yp) + static_cast<int64_t>(t) * a.k * a.H + n;
#pragma unroll 8
  for (int j = 0; j < a.k; ++j) {
    const int e = __ldg(a.ids + t * a.k + j);
    const float w = __ldg(a.share + t * a.k + j);
    const float4* src = reinterpret_cast<const float4*>(rows + static_cast<int64_t>(j) * a.H);
    const float4 u = src[0], v = src[1];
    if (e >= 0 && e < a.E) {
      s[0] = fmaf(w, u.x, s[0]); s[1] = fmaf(w, u.y, s[1]); s[2] = fmaf(w, u.z, s[2]); s[3] = fmaf(w, u.w, s[3]);
      s[4] = fmaf(w, v.x, s[4]); s[5] = fmaf(w, v.y, s[5]); s[6] = fmaf(w, v.z, s[6]); s[7] = fmaf(w, v.w, s[7]);
    }
  }
  Raw8<T> o;
  pack8(o, s);
  if (chk(t * a.ldy + n + 7, rows_extent(a.T, a.H, a.ldy), CHK_FEW)) store8(static_cast<T*>(a.y) + t * a.ldy + n, o, 8);
}

}  // namespace fp8q
