// matmul.cu -- the experts' matrix products on the tensor cores, forward and
// backward, over the rows of the dispatch layouts (or one dense matrix).
//
//   kForward  P[r, f] = sum_k x[r, k] * W_e[f, k] (+ bias), then the activation,
//             the gate and the residual;            reduction over k
//   kGradX    dx[r, k] = sum_n g[r, n] * W_e[n, k];  reduction over n
//   kGradW    dW_e[n, k] = sum_{r in e} g[r, n] * x[r, k];  over the rows of e
//
// One orientation serves all three: the 128 "feature" lanes of an accumulator
// (the M side of tcgen05.mma) are the contiguous dimension of the output (f, k,
// k) and its columns (the N side) are output rows (r, r, n). So
//  - an expert's rows sit on the N side, whose size is set per instruction in
//    steps of 16: a tile of 40 rows costs 48 columns, not 128 (experts of a
//    prefill hold a few hundred rows, of a decode batch a few), and the rows of
//    an expert are cut into equal tiles of at most 256 (e4m3: 240, e2m1: 208);
//  - the epilogue reads tensor memory as 8x8 fragments, transposes them through
//    a small staging area (stmatrix) and stores 16-byte pieces of output rows.
// With a gated activation a tile of 128 weight rows is 64 gate and 64 up rows
// interleaved by 16 (one 5-D tensor map does it), so gate and up of a feature
// are 16 lanes apart and arrive in the same register position of one thread.
//
// Two CTAs with neighbouring feature blocks form a pair (cta_group::2): each
// holds its own 128 weight rows and half of the tile's rows, and the pair's
// products read both halves. With one CTA per product the shared-memory port
// was the bound: filling and reading 48 KB each per 128 bytes of reduction of a
// 128 x 256 tile takes 768 cycles at 128 bytes a cycle where the products take
// 512 (measured 727); a pair moves 32 KB.
// Warp roles: 0 and 8 load (TMA), 1 (of the pair's first CTA) issues the products, 2
// and 3 lay out the e4m3 scales, or 2 copies the e2m1 scales and 3, 9 and 10 lay them
// out, or 2 zeroes the last lines of kGradW, 4-7 the epilogue, one warp per 32 lanes of
// tensor memory; two accumulators (columns 0.. and kRows..) let the epilogue of a tile
// overlap the products of the next.
// The grid is persistent; the tile list is formed on the device from the
// segment ends, so a captured graph can be replayed with other counts.
//
// Few tiles (one dense matrix with few rows): the reduction is cut into up to
// four runs, one pair of a larger cluster each. When its own products are done
// the first pair lets the others write their accumulators into its ring (st.async
// over distributed shared memory) and adds them in a fixed order; every cluster
// then has one tile at most, so nothing has to be handed back.
//
// Measured on GB300 (2 x features counted for gated weights), single passes: bf16, 16
// experts, 16382 rows, 2048 x 2816, P kept: 124 us, 1520 TFLOP/s, tensor cores 78% busy;
// its dx 110 us (1710, 87%), dW 115 us (1640, 84%); e4m3, 64 experts, 32768 rows, 7168 x
// 4096: 664 us (2900 TFLOP/s, 68%). Pass after pass the 1400 W power cap lowers the clock:
// 140 to 145 us at 1600 to 1650 MHz, e4m3 721 to 737 us at 1250 to 1350 MHz. e4m3 decode,
// 32 experts with 4 rows each, 7168 x 4096: 136 to 140 us, 6.7 TB/s of weights. Large
// products are bound by the tensor cores and the shared-memory port (a tile of 176 rows
// moves 55 KB per 352 cycles of products), decode by HBM, a weight gradient over few
// rows by its epilogue.
//
// The gradient of the pre-activations enters both backward products in 16 bits. While
// the experts hold few rows it comes as two terms, its rounding and what that left
// over: both are multiplied against the same staged weights (or rows), at next to no
// cost while the tensor cores are not the bound.
//
// Rows outside every segment are read at most as columns that are not stored.
// In kGradW rows are the reduction: lines of the last block past the segment's
// end are zeroed in shared memory before the product, so padding rows may hold
// anything (NaN included).
#include <cuda.h>
#include <stddef.h>

#include <mutex>

#include "activation.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "segments.cuh"
#include "tcgen05.cuh"

namespace moeperm {

namespace {

constexpr int kForward = 0, kGradX = 1, kGradW = 2;
// Operands: 16 bits, e4m3 with a scale per 128, or e2m1 with a scale per 32 or per 16.
constexpr int kHalf = 0, kFp8 = 1, kFp4Mx = 2, kFp4Nv = 3;
constexpr bool is_fp4(int kind) { return kind >= kFp4Mx; }
// Warps: nine, and two more that lay out the scales of e2m1 operands.
constexpr int kTransposers = 3;
template <int KIND>
constexpr int kThreadsOf = 288 + (is_fp4(KIND) ? 32 * (kTransposers - 1) : 0);
constexpr int kMaxSplits = 4;
constexpr int kMaxStages = 10;
constexpr int kABytes = 16384;            // 128 rows x 128 bytes

constexpr int kTmemCols = 512;
// Scales go through buffers in shared memory and two in tensor memory. e4m3: a word of the
// 128 weight rows and of up to 256 rows, 12 columns; e2m1: a piece of four words each.
constexpr int kMaxScaleBufs = 8;
template <int KIND>
constexpr int kScaleBufs = is_fp4(KIND) ? 6 : kMaxScaleBufs;
template <int KIND>
constexpr int kScaleBytes = (is_fp4(KIND) ? 4 : 1) * (512 + 1024);
template <int KIND>
constexpr int kScaleWidth = is_fp4(KIND) ? 48 : 12;  // columns of a buffer
template <int KIND>
constexpr int kScaleCols = is_fp4(KIND) ? 416 : 480;
// Reduction blocks (128 bytes of a row) that share a buffer of scales.
template <int KIND>
constexpr int kScaleBlocks = KIND == kFp4Nv ? 1 : KIND == kFp4Mx ? 2 : 4;
constexpr int kBoxes = 7;                 // heights of the row boxes a CTA may load
__host__ __device__ constexpr int box_rows(int i) {
  return i < 3 ? 8 << i : i < 5 ? 32 * (i - 1) : 16 * (i + 2);  // 8 16 32 64 96 112 128
}

// Rows of one tile (the N side): two accumulators fill tensor memory, but for
// the room that scale words take.
template <int KIND>
constexpr int kRows = KIND == kHalf ? 256 : KIND == kFp8 ? 240 : 208;

struct Maps {
  CUtensorMap a;
  CUtensorMap b[kBoxes];
};

struct Args {
  const int32_t* seg_begin;  // [L] (nullptr: dense, or slabs when cap > 0)
  const int32_t* seg_end;    // [L] segment ends; slabs: rows per expert
  int32_t cap;               // rows per slab (0: not slabs)
  int32_t R, L;
  int32_t red;               // reduction length (not kGradW)
  int32_t feats;             // features of an output row
  int32_t wrows;             // weight rows per expert (kGradW: output rows)
  int32_t gated, act, f16, out_f32;
  int32_t splits;            // pairs per cluster, each with a run of the reduction
  int32_t terms;             // 2: the row operand is a sum of two tensors; or kTermsByRows
  int32_t ring_bytes;
  const float* bias;         // [L, wrows]
  const void* residual;
  int64_t ld_res;
  void* out;
  int64_t ldo;
  void* pre;
  int64_t ld_pre;
  const uint32_t* xs;        // packed scale words of the rows
  int64_t ld_xs;
  const uint32_t* ws;        // and of the weights
  int64_t ld_ws;
  int32_t G4;
  const float* x_tscale;     // e2m1: tensor scales, or nullptr
  const float* w_tscale;
  int32_t* status;
};

struct Bars {  // one barrier of each kind per stage
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t raw[kMaxStages];  // kGradW: the last block of a segment has landed in this CTA
};

struct Tile {
  int e, fb;        // expert, feature block of this CTA
  int row0, rows;   // first output row (kGradW: within the expert), rows of the tile
  int n;            // N of the products (rows rounded up to 16)
  int kb0, nkb;     // this CTA's reduction blocks: first, count
  int red_row0;     // kGradW: first row of the segment
  int tail;         // kGradW: valid lines of the last block
};

__host__ __device__ constexpr int box_index(int half) {  // smallest box of at least `half` rows
  int i = 0;
  while (i < kBoxes - 1 && box_rows(i) < half) ++i;
  return i;
}

// A bounded wait that other roles can cut short.
__device__ __forceinline__ bool wait_or_stop(uint32_t bar, uint32_t parity, volatile int* stop,
                                             long long limit = kWaitCycles) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if (clock64() - t0 > limit) {
      *stop = 1;
      return false;
    }
  }
  return true;
}

// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait_or_stop(uint32_t bar, uint32_t parity, volatile int* stop,
                                                  long long limit = kWaitCycles) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, stop, limit));
}

// The wait of a converged warp whose next steps are uniform: one vote where the phase is
// over already.
__device__ __forceinline__ bool warp_ready(uint32_t bar, uint32_t parity, volatile int* stop) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_or_stop(bar, parity, stop);
}

// The limit of a wait that lasts while `blocks` reduction blocks go through the
// products: a block takes about 500 cycles, 2100 where all SMs wait for HBM.
__device__ __forceinline__ long long limit_for(long long blocks) { return kWaitCycles + blocks * 8192; }

__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool f16) {
  return f16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
__device__ __forceinline__ float2 unpack2(uint32_t w, bool f16) {
  return f16 ? f16x2_to_float2(w) : make_float2(bf16_lo(w), bf16_hi(w));
}

// The epilogue's staging area: per warp 32 output rows of up to 32 features
// (64 bytes), so that fragments of tensor memory (feature-major) leave as whole
// 16-byte pieces of output rows. A pitch of 80 bytes puts the 8 rows of a block
// into different banks.
constexpr int kPitch = 80;
constexpr int kStageBytes = 4 * 32 * kPitch;

// Rows of 16-bit elements in global memory; `vec`: 16-byte pieces are aligned.
struct Rows16 {
  uint16_t* p;
  int64_t ld;
  bool vec;
};
__device__ __forceinline__ Rows16 rows16(const void* p, int64_t ld) {
  return {static_cast<uint16_t*>(const_cast<void*>(p)), ld, ((reinterpret_cast<uintptr_t>(p) | (uint64_t)(ld * 2)) & 15) == 0};
}
__device__ __forceinline__ void put8(const Rows16& r, int64_t row, int col, const uint4& v) {
  uint16_t* dst = r.p + row * r.ld + col;
  if (r.vec) {
    st_v4(dst, v);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dst[2 * i] = (uint16_t)w[i];
      dst[2 * i + 1] = (uint16_t)(w[i] >> 16);
    }
  }
}
// Staged pieces of rows r0, r0 + STEP, ... to rows row + r of the output, where r < nr. All
// are read before the first is stored and the alignment is asked for once: short reductions
// are bound by the epilogue (e2m1, 32768 rows x 4096 features over K = 1792: with this 760 ->
// 480 cycles per 32 rows, and with the tile's scales and biases loaded before the wait 198 ->
// 141 us. Eight epilogue warps instead of four: 141, and 421 against 408 at K = 7168).
template <int N, int STEP>
__device__ __forceinline__ void put_rows(const Rows16& out, int64_t row, int col, int nr, int r0, const uint8_t* st) {
  uint4 v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = *reinterpret_cast<const uint4*>(st + k * STEP * kPitch);
  if (out.vec) {
    uint16_t* dst = out.p + (row + r0) * out.ld + col;
#pragma unroll
    for (int k = 0; k < N; ++k, dst += STEP * out.ld)
      if (r0 + k * STEP < nr) st_v4(dst, v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (r0 + k * STEP < nr) put8(out, row + r0 + k * STEP, col, v[k]);
  }
}
__device__ __forceinline__ uint4 get8(const Rows16& r, int64_t row, int col) {
  const uint16_t* src = r.p + row * r.ld + col;
  if (r.vec) return ld_nc_v4(src);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(src + 2 * i) | ((uint32_t)__ldg(src + 2 * i + 1) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One warp: the 32 x 32 fragments a (features 0-15) and b (16-31) to the
// staging area and from there to `nr` rows; a lane's 16-byte piece c = lane & 3
// goes to column col[c >> 1] + 8 * (c & 1), if that is below lim[c >> 1].
__device__ __forceinline__ void store_32x32(uint8_t* st, const float (&a)[16], const float (&b)[16], bool f16,
                                            const Rows16& out, int64_t row, int nr, int col0, int col1, int lim0,
                                            int lim1) {
  const int lane = threadIdx.x & 31;
  const uint32_t sa = smem_addr(st) + (lane & 7) * kPitch + (lane >> 3) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    stmatrix_trans(sa + i * 8 * kPitch, pack2(a[4 * i], a[4 * i + 1], f16), pack2(a[4 * i + 2], a[4 * i + 3], f16),
                   pack2(b[4 * i], b[4 * i + 1], f16), pack2(b[4 * i + 2], b[4 * i + 3], f16));
  __syncwarp();
  const int c = lane & 3;
  const int col = (c >> 1 ? col1 : col0) + 8 * (c & 1);
  const bool ok = col < (c >> 1 ? lim1 : lim0);
  put_rows<4, 8>(out, row, col, ok ? nr : 0, lane >> 2, st + (lane >> 2) * kPitch + c * 16);
  __syncwarp();
}
// The same for 16 features (fragments a).
__device__ __forceinline__ void store_16x32(uint8_t* st, const float (&a)[16], bool f16, const Rows16& out,
                                            int64_t row, int nr, int col0, int lim) {
  const int lane = threadIdx.x & 31;
  const uint32_t sa = smem_addr(st) + ((lane & 7) + 8 * (lane >> 4)) * kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
  for (int i = 0; i < 4; i += 2)
    stmatrix_trans(sa + i * 8 * kPitch, pack2(a[4 * i], a[4 * i + 1], f16), pack2(a[4 * i + 2], a[4 * i + 3], f16),
                   pack2(a[4 * i + 4], a[4 * i + 5], f16), pack2(a[4 * i + 6], a[4 * i + 7], f16));
  __syncwarp();
  const int col = col0 + 8 * (lane & 1);
  put_rows<2, 16>(out, row, col, col < lim ? nr : 0, lane >> 1, st + (lane >> 1) * kPitch + (lane & 1) * 16);
  __syncwarp();
}
// Residual rows into fragments, added to a (features 0-15) and, with kWide, b.
template <bool kWide>
__device__ __forceinline__ void add_rows(uint8_t* st, float (&a)[16], float (&b)[16], bool f16, const Rows16& res,
                                         int64_t row, int nr, int col0, int lim) {
  const int lane = threadIdx.x & 31;
  constexpr int kPieces = kWide ? 4 : 2, kPer = 32 / kPieces;  // 16-byte pieces a row, rows at once
  const int c = lane % kPieces, col = col0 + 8 * c;
#pragma unroll
  for (int k = 0; k < 32 / kPer; ++k) {
    const int r = lane / kPieces + kPer * k;
    const uint4 v = col < lim && r < nr ? get8(res, row + r, col) : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(st + r * kPitch + c * 16) = v;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; i += kWide ? 1 : 2) {
    uint32_t w[4];
    if constexpr (kWide) {
      ldmatrix_trans(smem_addr(st) + ((lane & 7) + 8 * i) * kPitch + (lane >> 3) * 16, w);
    } else {
      ldmatrix_trans(smem_addr(st) + ((lane & 7) + 8 * (i + (lane >> 4))) * kPitch + ((lane >> 3) & 1) * 16, w);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float2 f = unpack2(w[m], f16);
      float (&dst)[16] = (kWide && m >= 2) ? b : a;
      const int at = kWide ? 4 * i + 2 * (m & 1) : 4 * (i + (m >> 1)) + 2 * (m & 1);
      dst[at] += f.x;
      dst[at + 1] += f.y;
    }
  }
  __syncwarp();
}

template <int MODE, int KIND>
__global__ void __launch_bounds__(kThreadsOf<KIND>, 1)
    matmul_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  extern __shared__ uint8_t dyn[];
  __shared__ Bars s_bars;
  uint64_t *s_full = s_bars.full, *s_empty = s_bars.empty, *s_raw = s_bars.raw;
  __shared__ uint64_t s_tfull[2], s_tempty[2], s_sraw[kMaxScaleBufs], s_sfull[kMaxScaleBufs], s_sempty[kMaxScaleBufs],
      s_drain;
  __shared__ uint64_t s_go, s_recv;  // splits: the ring may be written; the accumulators have arrived
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_stop;
  __shared__ int s_max, s_held;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int crank = (int)cluster_rank(), rank = crank & 1;  // rank 0 issues the pair's products
  const int split = crank >> 1, leader = crank & ~1;        // cluster rank of the pair's first CTA
  const uint16_t both = (uint16_t)(3 << leader);
  const int pair = blockIdx.x / (2 * p.splits), npairs = gridDim.x / (2 * p.splits);  // (clusters)
  constexpr int kTileRows = kRows<KIND>, kThreads = kThreadsOf<KIND>;
  constexpr bool kScaled = KIND != kHalf, FP8 = KIND == kFp8, FP4 = is_fp4(KIND);
  constexpr int kBufs = kScaleBufs<KIND>, kBufBytes = kScaleBytes<KIND>, kPerBuf = kScaleBlocks<KIND>;
  constexpr int kRedBlock = kScaled ? 128 : 64;  // reduction elements per stage (e2m1: pairs of them)

  uint8_t* ring = dyn + ((1024 - (smem_addr(dyn) & 1023)) & 1023);
  uint8_t* s_scale = ring + p.ring_bytes;                                 // kBufs buffers
  uint8_t* s_stage = s_scale + (kScaled ? kBufs * kBufBytes : 0);                  // the epilogue's
  int32_t* s_tiles = reinterpret_cast<int32_t*>(s_stage + kStageBytes);   // [L + 1]
  int32_t* s_begin = s_tiles + p.L + 1;
  int32_t* s_count = s_begin + p.L;
  int32_t* s_per = s_count + p.L;  // rows of an expert's tiles

  // ---- set-up
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(smem_addr(s_full + i), MODE == kGradW ? 2 : FP4 ? 3 : 1);
      mbar_init(smem_addr(s_empty + i), 1);
      mbar_init(smem_addr(s_raw + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(s_tfull + i), 1);
      mbar_init(smem_addr(s_tempty + i), 8);  // four epilogue warps of each CTA
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_addr(s_sraw + i), FP4 ? 1 : 32);
      mbar_init(smem_addr(s_sfull + i), 2);  // one of each CTA
      mbar_init(smem_addr(s_sempty + i), 1);
    }
    mbar_init(smem_addr(&s_drain), 1);
    mbar_init(smem_addr(&s_go), 1);
    mbar_init(smem_addr(&s_recv), 1);
    mbar_init_fence();
    s_stop = 0;
    s_max = s_held = 0;
    prefetch_map(&maps.a);
  }
  if (warp == 3) tmem_alloc(smem_addr(&s_tmem), kTmemCols);
  __syncthreads();
  int mx = 0, held = 0;
  bool ascending = true;  // as every layout makes them: then no two share a row
  for (int e = tid; e < p.L; e += kThreads) {
    int64_t b, c;
    const bool ok = segment(p, e, b, c);
    if (!ok && blockIdx.x == 0) set_status(p.status, kStBadLayout);
    if (p.seg_begin != nullptr) ascending &= ok && (e + 1 == p.L || b + c <= __ldg(p.seg_begin + e + 1));
    s_begin[e] = (int)b;
    s_count[e] = (int)c;
    mx = max(mx, (int)c);
    held += rows_held(c);
  }
  atomicMax(&s_max, mx);
  if (MODE != kForward && p.terms == kTermsByRows) {
    held = __reduce_add_sync(0xffffffffu, held);
    if (lane == 0) atomicAdd(&s_held, held);
  }
  if (!__syncthreads_and(ascending)) {
    // Each against all before it. One that shares rows with an earlier one counts as
    // empty: its rows are written once, and there are no more tiles than the host
    // counted (with split reductions a cluster has one tile at most).
    uint32_t hit = 0;  // bit i: this thread's i-th segment
    for (int e = tid, i = 0; e < p.L; e += kThreads, ++i)
      for (int f = 0; f < e; ++f)
        if (share_rows(s_begin[e], s_count[e], s_begin[f], s_count[f])) hit |= 1u << i;
    __syncthreads();
    for (int e = tid, i = 0; e < p.L; e += kThreads, ++i)
      if ((hit >> i) & 1u) {
        s_count[e] = 0;
        if (blockIdx.x == 0) set_status(p.status, kStBadLayout);
      }
    __syncthreads();
  }
  if (warp == 0) {  // row tiles before each expert
    int base = 0;
    for (int e0 = 0; e0 < p.L; e0 += 32) {
      const int e = e0 + lane;
      int v = e < p.L ? (s_count[e] + kTileRows - 1) / kTileRows : 0;
      int incl = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int nb = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += nb;
      }
      if (e < p.L) {
        s_tiles[e] = base + incl - v;
        s_per[e] = v > 0 ? ((s_count[e] + v - 1) / v + 15) / 16 * 16 : 0;  // equal tiles
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_tiles[p.L] = base;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the other CTA's barriers are ready before anything arrives on them
  const uint32_t tmem = s_tmem;

  // ---- tile list (the same for every role and both CTAs)
  const int fblk = p.gated && MODE == kForward ? 64 : 128;  // features per block
  const int nfp = (p.feats + 2 * fblk - 1) / (2 * fblk);    // pairs of blocks
  const int nnb = MODE == kGradW ? (p.wrows + 255) / 256 : 0;       // kGradW: row blocks per expert
  // the run of the reduction this pair takes: whole scale words (four blocks); the
  // host gives every run some
  const int red_blocks = (p.red + kRedBlock - 1) / kRedBlock;
  const int run_kb0 = red_blocks * split / p.splits & ~3;
  const int run_nkb = (split + 1 == p.splits ? red_blocks : red_blocks * (split + 1) / p.splits & ~3) - run_kb0;
  // A role's walk over its pair's tiles: tile w = rb * nfp + fp is followed by
  // w + npairs. Steps add with carries and the expert only moves forward, so a
  // step costs about 100 cycles (divisions and a search took 900, between tiles).
  struct Walk {
    int rb, fp, e;
  };
  const int d_rb = npairs / nfp, d_fp = npairs % nfp;
  auto settle = [&](Walk& k) {  // kGradW: rb counts within expert e
    if constexpr (MODE == kGradW) {
      while (k.rb >= nnb) {
        k.rb -= nnb;
        ++k.e;
      }
    } else {
      while (k.rb >= s_tiles[k.e + 1]) ++k.e;
    }
  };
  auto more = [&](const Walk& k) { return MODE == kGradW ? k.e < p.L : k.rb < s_tiles[p.L]; };
  auto first = [&] {
    Walk k{pair / nfp, pair % nfp, 0};
    if (MODE == kGradW || more(k)) settle(k);
    return k;
  };
  auto step = [&](Walk& k) {
    k.rb += d_rb;
    k.fp += d_fp;
    if (k.fp >= nfp) {
      k.fp -= nfp;
      ++k.rb;
    }
    if (MODE == kGradW || more(k)) settle(k);
  };
  auto tile_at = [&](const Walk& k) {
    Tile t;
    t.e = k.e;
    t.fb = k.fp * 2 + rank;
    if constexpr (MODE == kGradW) {
      t.row0 = k.rb * 256;
      t.rows = min(256, p.wrows - t.row0);
      t.red_row0 = s_begin[t.e];
      t.kb0 = 0;
      t.nkb = (s_count[t.e] + 63) / 64;
      t.tail = s_count[t.e] - (t.nkb - 1) * 64;
    } else {
      const int per = s_per[t.e], j = k.rb - s_tiles[t.e];
      t.row0 = s_begin[t.e] + j * per;
      t.rows = min(per, s_count[t.e] - j * per);
      t.kb0 = run_kb0;
      t.nkb = run_nkb;
      t.red_row0 = t.tail = 0;
    }
    t.n = (t.rows + 15) / 16 * 16;
    return t;
  };

  // ---- ring geometry: as many stages as the largest row tile allows
  const int max_n = MODE == kGradW ? 256 : min(kTileRows, (s_max + 15) / 16 * 16);
  const int b_bytes = MODE == kGradW ? min((p.wrows + 127) / 128, 2) * 8192
                                     : box_rows(box_index(max_n / 2)) * 128;
  const int terms = MODE == kForward ? 1 : p.terms == kTermsByRows ? terms_of(s_held, p.L) : p.terms;
  const int stage_bytes = kABytes + terms * b_bytes;
  const int stages = min(kMaxStages, p.ring_bytes / stage_bytes);
  const uint32_t ring_s = smem_addr(ring);

  if (warp == 0 || warp == 8) {
    // ------------------------------------------------------------------ loads
    // Warp 0 loads this CTA's weight rows (kGradW: its features of x), warp 8 its
    // half of the tile's rows: issuing is serial in a thread (about 400 cycles a
    // stage for both together, close to the products' 512), so two threads share
    // it as a margin (one thread for both measured the same). The bytes of both
    // CTAs count on the first CTA's barrier. In kGradW a block that ends inside
    // counts on this CTA's own barrier and goes on through warp 2 (the first CTA's
    // barrier then takes an arrival of each CTA's warp 2 instead of the loads').
    if (elect_one()) {
      const bool weights = warp == 0;
      const uint32_t empty0 = smem_addr(s_empty), raw0 = smem_addr(s_raw);
      const uint32_t full0 = map_to_rank(smem_addr(s_full), leader);
      const uint32_t dst0 = ring_s + (weights ? 0 : kABytes);
      uint32_t empty = empty0, full = full0, raw = raw0, dst = dst0, ph = 1;
      int left = stages, issued = 0;
      bool ok = true;
      for (Walk k = first(); ok && more(k); step(k)) {
        const Tile t = tile_at(k);
        const int half = t.n / 2;
        const int box = MODE == kGradW ? 0 : box_index(half);
        const int nbox = (half + 63) / 64;  // kGradW: 64-wide boxes of the row side
        const uint32_t b_tile = terms * (MODE == kGradW ? nbox * 8192 : box_rows(box) * 128);
        const CUtensorMap* mb = &maps.b[box];
        const int f = t.fb * 128, brow = t.row0 + rank * half;
        int red = t.kb0 * kRedBlock;
        for (int kb = 0; kb < t.nkb; ++kb, red += kRedBlock) {
          if (!(ok = wait_or_stop(empty, ph, &s_stop))) break;
          const bool tail = MODE == kGradW && kb == t.nkb - 1 && t.tail < 64;
          const uint32_t bar = tail ? raw : full;
          if (weights) {
            // one arrival arms the barrier for all bytes that will count on it
            if (tail) mbar_expect_tx(bar, kABytes + b_tile);
            else if (rank == 0) mbar_expect_tx(smem_addr(s_full) + (full - full0), 2 * (kABytes + b_tile));
            else if (MODE == kGradW) mbar_arrive_mapped(bar);
            if constexpr (MODE == kForward) {
              if (p.gated) tma_load_5d(dst, &maps.a, bar, red, 0, 0, t.fb * 4, t.e);
              else tma_load_3d(dst, &maps.a, bar, red, f, t.e);
            } else if constexpr (MODE == kGradX) {
              tma_load_3d(dst, &maps.a, bar, f, red, t.e);
              tma_load_3d(dst + 8192, &maps.a, bar, f + 64, red, t.e);
            } else {
              tma_load_2d(dst, &maps.a, bar, f, t.red_row0 + red);
              tma_load_2d(dst + 8192, &maps.a, bar, f + 64, t.red_row0 + red);
            }
          } else {
            if constexpr (MODE == kForward) {
              tma_load_2d(dst, mb, bar, red, brow);
            } else {
              for (int term = 0; term < terms; ++term) {
                const uint32_t to = dst + term * b_bytes;
                if constexpr (MODE == kGradW) {
                  for (int i = 0; i < nbox; ++i)
                    tma_load_3d(to + i * 8192, mb, bar, brow + i * 64, t.red_row0 + red, term);
                } else {
                  tma_load_3d(to, mb, bar, red, brow, term);
                }
              }
            }
          }
          ++issued;
          dst += stage_bytes;
          empty += 8;
          full += 8;
          raw += 8;
          if (--left == 0) {
            left = stages;
            empty = empty0;
            full = full0;
            raw = raw0;
            dst = dst0;
            ph ^= 1;
          }
        }
      }
      // a wait ran out: let the copies in flight land, again with a limit (they
      // count on the first CTA's barriers, whose CTA stays until the end)
      if (!ok && rank == 0 && weights)
        for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
          if (!mbar_wait(smem_addr(s_full + i % stages), (i / stages) & 1)) break;  // (all had that time)
    }
  } else if (FP4 && warp == 1) {
    // --------------------------------------------------------- products, e2m1
    // A block of 128 bytes is four products, as with the other types, but they take half
    // the time (332 cycles for 176 rows), and copies of scales come on top. The warp stays
    // converged, so that operands stay in uniform registers (a thread alone moves each there
    // first), and waits once a block: 4096 tokens x top-8 of 64 experts, 7168 x 4096, scales
    // per 16: 478 us with a thread alone and three waits, 430 converged, 371 with one wait and
    // three copies a piece of scales, the tensor cores 58% active. Without loads of rows and
    // weights it would take 345, without copies of scales 365; a warp of its own for the
    // copies took 386 (scales per 32: 332 -> 324).
    if (uniform(rank) == 0) {
      const uint32_t lead = elect_one(), tm = uniform(tmem), lo_step = uniform(stage_bytes >> 4);
      const int nstages = (int)uniform(stages);
      const uint32_t lo0 = desc_lo(ring_s, 0), bar0 = smem_addr(s_bars.full);
      constexpr uint32_t kEmptyOffset = offsetof(Bars, empty) - offsetof(Bars, full);
      const uint32_t sm0 = desc_lo(smem_addr(s_scale), 0), sempty0 = smem_addr(s_sempty);
      const uint16_t mask = (uint16_t)uniform(both);
      uint32_t lo = lo0, bar = bar0, ph = 0;
      int left = nstages;
      uint32_t buf = 0, cols = 0;  // of the next piece of scales
      int acc_it = 0;
      bool ok = true;
      for (Walk k = first(); ok && __any_sync(0xffffffffu, more(k)); step(k)) {
        const Tile t = tile_at(k);
        const int n = (int)uniform(t.n), nkb = (int)uniform(t.nkb), kb0 = (int)uniform(t.kb0);
        const int as = acc_it & 1;
        if (!(ok = warp_ready(smem_addr(s_tempty + as), ((acc_it >> 1) & 1) ^ 1, &s_stop))) break;
        tc_fence_after();
        const uint32_t d = tm + as * kTileRows;
        const uint32_t idesc = idesc_e2m1(n, KIND == kFp4Mx, 0);
        for (int kb = 0; kb < nkb; kb += kPerBuf) {
          // A piece of scales (four words a row) serves one block (a word per product) or two
          // (half a word). A wait costs about 100 cycles even if it passes at once, so there
          // is one a block: the warps that lay out the scales arrive on its barrier too, and
          // not before the columns that the piece takes are free.
          const uint32_t sfa = tm + kScaleCols<KIND> + cols, sfb = sfa + 16, sm = sm0 + buf * (kBufBytes >> 4);
#pragma unroll
          for (int j = 0; j < kPerBuf; ++j) {
            if (kb + j >= nkb) break;
            if (!(ok = warp_ready(bar, ph, &s_stop))) break;
            const int left_red = p.red - (kb0 + kb + j) * 128;  // bytes: 32 a product
            const uint32_t acc = j > 0 ? 1u : (uint32_t)kb, empty = bar + kEmptyOffset;
            if (lead) {
              if (j == 0) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                  tmem_copy_scales(sfa + 4 * w, sm + w * (512 >> 4));
                  tmem_copy_scales(sfb + 8 * w, sm + (2048 >> 4) + w * (512 >> 4));
                }
                if (n > 128) {
#pragma unroll
                  for (int w = 0; w < 4; ++w) tmem_copy_scales(sfb + 8 * w + 4, sm + (4096 >> 4) + w * (512 >> 4));
                }
              }
              auto product = [&](int k) {
                const int w = KIND == kFp4Nv ? k : 2 * j + k / 2;
                const uint32_t sf = KIND == kFp4Nv ? 0 : 2 * (k & 1);
                mma_e2m1<KIND == kFp4Mx>(d, lo + 2 * k, lo + (kABytes >> 4) + 2 * k, idesc | (sf << 4) | (sf << 29),
                                         sfa + 4 * w, sfb + 8 * w, k > 0 ? 1u : acc);
              };
              product(0);
              if (left_red > 96) {
                product(1);
                product(2);
                product(3);
              } else {
                if (left_red > 32) product(1);
                if (left_red > 64) product(2);
              }
              mma_commit_pair(empty, mask);
              if (j == kPerBuf - 1 || kb + j + 1 >= nkb) mma_commit_pair(sempty0 + 8 * buf, mask);
            }
            __syncwarp();
            lo += lo_step;
            bar += 8;
            if (--left == 0) {
              left = nstages;
              lo = lo0;
              bar = bar0;
              ph ^= 1;
            }
          }
          if (!ok) break;
          if (++buf == kBufs) buf = 0;
          cols = kScaleWidth<KIND> - cols;
        }
        if (lead) mma_commit_pair(smem_addr(s_tfull + as), mask);
        __syncwarp();
        ++acc_it;
      }
      if (!ok) {  // products in flight end before tensor memory is freed
        if (lead) mma_commit_pair(smem_addr(&s_drain), mask);
        __syncwarp();
        mbar_wait(smem_addr(&s_drain), 0);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- products
    if (rank == 0 && elect_one()) {
      int acc_it = 0, sf_it = 0;
      // the stage's descriptor word and barrier, stepped rather than indexed: one
      // thread issues alone, so every instruction of this loop counts
      const uint32_t lo0 = desc_lo(ring_s, 0), bar0 = smem_addr(s_bars.full);
      constexpr uint32_t kEmptyOffset = offsetof(Bars, empty) - offsetof(Bars, full);
      uint32_t lo = lo0, bar = bar0, ph = 0;
      int left = stages;
      bool ok = true;
      for (Walk k = first(); ok && more(k); step(k)) {
        const Tile t = tile_at(k);
        if (t.nkb == 0) continue;  // kGradW: an expert without rows; the epilogue writes zeros
        const int as = acc_it & 1;
        if (!(ok = wait_or_stop(smem_addr(s_tempty + as), ((acc_it >> 1) & 1) ^ 1, &s_stop))) break;
        tc_fence_after();
        const uint32_t d = tmem + as * kTileRows;
        const uint32_t idesc = FP8 ? idesc_e4m3(t.n, 0) : idesc_16bit(!p.f16, MODE != kForward, MODE == kGradW, t.n);
        auto advance = [&] {  // hand the stage back and move on to the next
          mma_commit_pair(bar + kEmptyOffset, both);
          lo += stage_bytes >> 4;
          bar += 8;
          if (--left == 0) {
            left = stages;
            lo = lo0;
            bar = bar0;
            ph ^= 1;
          }
        };
        if constexpr (FP8) {
          // four blocks share a scale word, each its own byte of it
          for (int kb = 0; kb < t.nkb && ok; kb += 4, ++sf_it) {
            const int sb = sf_it % kBufs;
            if (!(ok = wait_or_stop(smem_addr(s_sfull + sb), (sf_it / kBufs) & 1, &s_stop))) break;
            const uint32_t sfa = tmem + kScaleCols<KIND> + kScaleWidth<KIND> * (sf_it & 1), sfb = sfa + 4;
            const uint32_t sm = desc_lo(smem_addr(s_scale + sb * kBufBytes), 0);
            tmem_copy_scales(sfa, sm);
            tmem_copy_scales(sfb, sm + (512 >> 4));
            if (t.n > 128) tmem_copy_scales(sfb + 4, sm + (1024 >> 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (kb + j >= t.nkb || !ok) break;
              if (!(ok = wait_or_stop(bar, ph, &s_stop))) break;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_e4m3(d, lo + 2 * k, lo + (kABytes >> 4) + 2 * k, idesc + j * ((1u << 4) | (1u << 29)), sfa, sfb,
                         j + k > 0 ? 1u : (uint32_t)kb);
              advance();
            }
            mma_commit_pair(smem_addr(s_sempty + sb), both);
          }
        } else {
          constexpr int ka = MODE == kForward ? 2 : 128, kb_step = MODE == kGradW ? 128 : 2;
          constexpr uint32_t a_atom = MODE == kForward ? 0 : 8192, b_atom = MODE == kGradW ? 8192 : 0;
          for (int kb = 0; kb < t.nkb; ++kb) {
            if (!(ok = wait_or_stop(bar, ph, &s_stop))) break;
            const uint32_t a = lo + ((a_atom >> 4) << 16), b = lo + (kABytes >> 4) + ((b_atom >> 4) << 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_16bit(d, a + ka * k, b + kb_step * k, idesc, k > 0 ? 1u : (uint32_t)kb);
            if (MODE != kForward && terms > 1) {
              const uint32_t b2 = b + (b_bytes >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_16bit(d, a + ka * k, b2 + kb_step * k, idesc, 1u);
            }
            advance();
          }
        }
        mma_commit_pair(smem_addr(s_tfull + as), both);
        ++acc_it;
      }
      if (!ok) {  // products in flight end before tensor memory is freed
        mma_commit_pair(smem_addr(&s_drain), both);
        mbar_wait(smem_addr(&s_drain), 0);
      }
    }
  } else if (MODE == kGradW && warp == 2) {
    // ------------------------------------------- lines past the segment's end
    // The last block of a segment gets zero lines in each of its 64-wide boxes on
    // its way to the products; the others go straight there.
    int at = 0;          // stage of the tile's first block
    uint32_t phase = 0;  // bit s: parity of the next wait on s_raw[s]
    long long blocks = 0;  // of the tiles since the last wait (64 more for each one's epilogue)
    bool ok = true;
    for (Walk k = first(); ok && more(k); step(k)) {
      const Tile t = tile_at(k);
      blocks += t.nkb + 64;
      if (t.nkb > 0 && t.tail < 64) {
        const int s = (at + t.nkb - 1) % stages;
        if (!(ok = warp_wait_or_stop(smem_addr(s_raw + s), (phase >> s) & 1, &s_stop, limit_for(blocks)))) break;
        blocks = 0;
        phase ^= 1u << s;
        // four lines at a time, eight lanes each
        uint8_t* a = ring + s * stage_bytes + (t.tail + (lane >> 3)) * 128 + (lane & 7) * 16;
        const int lines = 64 - t.tail - (lane >> 3), nbox = (t.n / 2 + 63) / 64;
        auto clear = [&](uint8_t* box, int boxes) {
          for (int bx = 0; bx < boxes; ++bx, box += 8192)
            for (int r = 0; r < lines; r += 4) *reinterpret_cast<uint4*>(box + r * 128) = make_uint4(0, 0, 0, 0);
        };
        clear(a, 2);
        for (int term = 0; term < terms; ++term) clear(a + kABytes + term * b_bytes, nbox);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_mapped(map_to_rank(smem_addr(s_full + s), leader));
      }
      at = (at + t.nkb) % stages;
    }
  } else if (FP8 && warp == 2) {
    // ----------------------------------------------------------------- scales
    // Word w of a row holds the exponents of its reduction elements 512 w ..
    // 512 w + 511, one byte per 128. Tensor memory wants row r of a block of
    // 128 at lane r % 32, column r / 32: row r goes to byte 16 (r % 32) +
    // 4 (r / 32) of its block's 512 bytes, by 4-byte asynchronous copies that
    // run up to kScaleBufs words ahead of the products. (Loads through
    // registers wait for the newest load in flight, not for the oldest: 1170
    // cycles a word of a decode batch.) Both CTAs need the words of all rows
    // and of their own weight rows.
    int sf_it = 0;
    bool ok = true;
    const int fstep = p.gated ? 16 : 32;
    for (Walk k = first(); ok && more(k); step(k)) {
      const Tile t = tile_at(k);
      const int f = p.gated ? t.fb * 64 + (lane & 15) : t.fb * 128 + lane;  // this lane's first feature
      const uint32_t* la = p.ws + (int64_t)t.e * p.wrows + (p.gated && (lane & 16) ? p.feats : 0) + f;
      const uint32_t* lb =
          p.xs + (p.cap > 0 ? (int64_t)t.e * p.G4 * p.ld_xs - (int64_t)t.e * p.cap : 0) + t.row0 + lane;
      for (int kb = 0; kb < t.nkb; kb += 4, ++sf_it) {
        const int sb = sf_it % kBufs;
        if (!(ok = warp_wait_or_stop(smem_addr(s_sempty + sb), ((sf_it / kBufs) & 1) ^ 1, &s_stop))) break;
        const uint32_t dst = smem_addr(s_scale + sb * kBufBytes + lane * 16);
        const int64_t word = (t.kb0 + kb) >> 2, wa = word * p.ld_ws, wb = word * p.ld_xs;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (f + i * fstep < p.feats) cp_async4(dst + 4 * i, la + wa + i * fstep);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 32 + lane < t.rows) cp_async4(dst + 512 + (i >> 2) * 512 + 4 * (i & 3), lb + wb + i * 32);
        cp_async_arrive(smem_addr(s_sraw + sb));  // when this lane's copies have landed
      }
    }
    cp_async_wait_all();
  } else if (FP8 && warp == 3) {
    // Makes the words that have landed visible to the asynchronous proxy and hands
    // them to the products. A warp of its own, because the fence waits for the loads
    // its thread has in flight (in warp 2 it exposed their latency).
    if (lane == 0) {
      bool ok = true;
      int sf_it = 0;
      for (Walk k = first(); ok && more(k); step(k)) {
        const int words = (run_nkb + 3) / 4;
        for (int i = 0; i < words; ++i, ++sf_it) {
          const int sb = sf_it % kBufs;
          if (!(ok = wait_or_stop(smem_addr(s_sraw + sb), (sf_it / kBufs) & 1, &s_stop))) break;
          fence_proxy_async_smem();
          mbar_arrive_mapped(map_to_rank(smem_addr(s_sfull + sb), leader));
        }
      }
    }
  } else if (FP4 && warp == 2) {
    // A row's piece of scales is 16 bytes, and those of consecutive rows are
    // contiguous: one bulk copy for the tile's rows and one for its weight rows (gated:
    // the gate rows, then the up rows), up to kBufs pieces ahead. (A copy costs its
    // thread about 60 cycles: the runs of 16 rows that a gated tile interleaves, one by
    // one, took 650 a piece, and 900 from as many lanes.)
    if (elect_one()) {
      int sf_it = 0;
      bool ok = true;
      const uint8_t* ws = reinterpret_cast<const uint8_t*>(p.ws);
      const uint8_t* xs = reinterpret_cast<const uint8_t*>(p.xs);
      for (Walk k = first(); ok && more(k); step(k)) {
        const Tile t = tile_at(k);
        const int f0 = t.fb * fblk, nf = max(min(fblk, p.feats - f0), 0);  // features of the tile
        const uint32_t row_bytes = (uint32_t)t.rows * 16, w_bytes = (uint32_t)nf * 16;
        const uint32_t bytes = row_bytes + (p.gated ? 2 : 1) * w_bytes;
        const uint8_t* xrow = xs + (int64_t)t.row0 * 16;
        const uint8_t* wrow = ws + ((int64_t)t.e * p.wrows + f0) * 16;
        for (int kb = 0; kb < t.nkb; kb += kPerBuf, ++sf_it) {
          const int sb = sf_it % kBufs;
          if (!(ok = wait_or_stop(smem_addr(s_sempty + sb), ((sf_it / kBufs) & 1) ^ 1, &s_stop))) break;
          const uint32_t dst = smem_addr(s_scale + sb * kBufBytes), bar = smem_addr(s_sraw + sb);
          const int64_t piece = (t.kb0 + kb) / kPerBuf;
          mbar_expect_tx(bar, bytes);
          bulk_load_g2s(dst + 2048, xrow + piece * p.ld_xs * 16, row_bytes, bar);
          if (nf > 0) {
            const uint8_t* w = wrow + piece * p.ld_ws * 16;
            bulk_load_g2s(dst, w, w_bytes, bar);
            if (p.gated) bulk_load_g2s(dst + 1024, w + (int64_t)p.feats * 16, w_bytes, bar);
          }
        }
      }
      // whatever ended the walk, no copy outlives the CTA
      for (int i = sf_it > kBufs ? sf_it - kBufs : 0; i < sf_it; ++i)
        if (!mbar_wait(smem_addr(s_sraw + i % kBufs), (i / kBufs) & 1)) break;
    }
  } else if (FP4 && (warp == 3 || warp > 8)) {
    // Tensor memory wants word w of row r of a block of 128 at byte 16 (r % 32) + 4 (r / 32)
    // of the word's 512 bytes; the copies left row r's four words at byte 16 r (gated: the
    // tile's runs of 16 gate rows one after the other, and the up rows 1024 bytes on).
    // Lane l transposes the 4 x 4 words of rows l, 32 + l, 64 + l and 96 + l.
    // A buffer always goes to the same warp: one that had not waited for its last phase
    // could take that for the next.
    static_assert(!FP4 || kBufs % kTransposers == 0, "a buffer's phases are waited for in order");
    // The pieces go round the warps: from a landed copy to the arrival takes one of them
    // about as long as two blocks' products.
    const int turn = warp == 3 ? 0 : warp - 8;
    const int wfirst = !p.gated ? lane : lane < 16 ? lane : 48 + lane, wstep = p.gated ? 16 : 32;
    bool ok = true;
    int sf_it = 0, at_stage = 0;
    for (Walk k = first(); ok && more(k); step(k)) {
      const Tile t = tile_at(k);
      for (int kb = 0; kb < t.nkb; kb += kPerBuf, ++sf_it) {
        const int s0 = at_stage, s1 = s0 + 1 == stages ? 0 : s0 + 1;
        const bool two = kPerBuf > 1 && kb + 1 < t.nkb;
        at_stage = two ? (s1 + 1 == stages ? 0 : s1 + 1) : s1;
        if (sf_it % kTransposers != turn) continue;
        const int sb = sf_it % kBufs;
        if (!(ok = warp_wait_or_stop(smem_addr(s_sraw + sb), (sf_it / kBufs) & 1, &s_stop))) break;
        uint4* at = reinterpret_cast<uint4*>(s_scale + sb * kBufBytes) + lane;
        uint4 r[3][4];
#pragma unroll
        for (int b = 0; b < 3; ++b)
          if (b < 2 || t.n > 128)
#pragma unroll
            for (int i = 0; i < 4; ++i) r[b][i] = b > 0 ? at[b * 128 + i * 32] : at[wfirst - lane + i * wstep];
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 3; ++b)
          if (b < 2 || t.n > 128) {
            at[b * 128] = make_uint4(r[b][0].x, r[b][1].x, r[b][2].x, r[b][3].x);
            at[b * 128 + 32] = make_uint4(r[b][0].y, r[b][1].y, r[b][2].y, r[b][3].y);
            at[b * 128 + 64] = make_uint4(r[b][0].z, r[b][1].z, r[b][2].z, r[b][3].z);
            at[b * 128 + 96] = make_uint4(r[b][0].w, r[b][1].w, r[b][2].w, r[b][3].w);
          }
        fence_proxy_async_smem();
        __syncwarp();  // every lane's words before the arrival
        // The columns are free when the products of the piece before the last are done (before
        // there was any, a buffer's first phase passes at once). Those of the blocks that had
        // these blocks' stages are done then as well (there are at least four stages: launch), so the
        // arrivals count for these.
        const int old = sf_it >= 2 ? sf_it - 2 : sf_it - 2 + kBufs;
        const uint32_t oph = sf_it >= 2 ? (old / kBufs) & 1 : 1;
        if (!(ok = warp_wait_or_stop(smem_addr(s_sempty + old % kBufs), oph, &s_stop))) break;
        if (lane == 0) {
          mbar_arrive_mapped(map_to_rank(smem_addr(s_full + s0), leader));
          if (two) mbar_arrive_mapped(map_to_rank(smem_addr(s_full + s1), leader));
        }
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // --------------------------------------------------------------- epilogue
    const int q = warp & 3;  // this warp's 32 lanes of tensor memory
    const float xscale = FP4 && p.x_tscale != nullptr ? __ldg(p.x_tscale) : 1.0f;
    const bool f16 = p.f16 != 0;
    const Rows16 out = rows16(p.out, p.ldo), pre = rows16(p.pre, p.ld_pre), res = rows16(p.residual, p.ld_res);
    int acc_it = 0;
    for (Walk k = first(); more(k); step(k)) {
      const Tile t = tile_at(k);
      const int as = acc_it & 1;
      // Fragments a and b: lanes 0-15 and 16-31 of this warp's quarter. Gated:
      // gate and up of the same 16 features; else features 0-15 and 16-31. What the
      // tile's features share is on its way while the products are waited for.
      const bool gated = MODE == kForward && p.gated;
      const int f0 = gated ? t.fb * 64 + q * 16 : t.fb * 128 + q * 32;
      const float wscale = FP4 && p.w_tscale != nullptr ? __ldg(p.w_tscale + t.e) : 1.0f;
      float ba[2] = {0.0f, 0.0f}, bb[2] = {0.0f, 0.0f};  // bias of features l / 4 + 8 g
      if (MODE == kForward && p.bias != nullptr) {
        const float* bias = p.bias + (int64_t)t.e * p.wrows;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int f = f0 + (lane >> 2) + 8 * g, f2 = gated ? p.feats + f : f + 16;
          if (f < p.feats) ba[g] = __ldg(bias + f);
          if (gated ? f < p.feats : f2 < p.feats) bb[g] = __ldg(bias + f2);
        }
      }
      if (t.nkb > 0) {
        if (!warp_wait_or_stop(smem_addr(s_tfull + as), (acc_it >> 1) & 1, &s_stop, limit_for(t.nkb))) break;
        tc_fence_after();
      }
      const uint32_t acc = tmem + as * kTileRows + ((uint32_t)(q * 32) << 16);
      if (MODE != kGradW && p.splits > 1) {
        // accumulators of the other runs, [run - 1][32 columns][warp][8][lane] in
        // 16-byte pieces of the fragments, in the first pair's ring
        const uint32_t run_bytes = (uint32_t)((t.rows + 31) / 32) * 16384;
        if (split == 0) {
          if (q == 0 && lane == 0) {
            mbar_expect_tx(smem_addr(&s_recv), (p.splits - 1) * run_bytes);
            for (int i = 1; i < p.splits; ++i) mbar_arrive_mapped(map_to_rank(smem_addr(&s_go), 2 * i + rank));
          }
          if (!warp_wait_or_stop(smem_addr(&s_recv), 0, &s_stop, limit_for(t.nkb))) break;
        } else {
          if (!warp_wait_or_stop(smem_addr(&s_go), 0, &s_stop, limit_for(t.nkb))) break;
          const uint32_t to = map_to_rank(ring_s, rank) + (split - 1) * run_bytes + q * 4096 + lane * 16;
          const uint32_t bar = map_to_rank(smem_addr(&s_recv), rank);
          for (int c0 = 0; c0 < t.rows; c0 += 32) {
            uint32_t ra[16], rb[16];
            tmem_ld_16x32(acc + c0, ra);
            tmem_ld_16x32(acc + c0 + (16u << 16), rb);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              store_async16(to + c0 * 512 + i * 512, ra[4 * i], ra[4 * i + 1], ra[4 * i + 2], ra[4 * i + 3], bar);
              store_async16(to + c0 * 512 + (4 + i) * 512, rb[4 * i], rb[4 * i + 1], rb[4 * i + 2], rb[4 * i + 3], bar);
            }
          }
          break;  // the cluster's only tile
        }
      }
      const int64_t orow = MODE == kGradW ? (int64_t)t.e * p.wrows + t.row0 : t.row0;
      if (MODE == kGradW && p.out_f32) {
        // 32-bit outputs: a lane is a feature, a warp stores 128 bytes of a row
        const int f = t.fb * 128 + q * 32 + lane;
        for (int c0 = 0; c0 < t.rows; c0 += 32) {
          uint32_t raw[32];
          __syncwarp();
          if (t.nkb > 0) {
            tmem_ld_x32(acc + c0, raw);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) raw[j] = 0;
          }
          float* dst = static_cast<float*>(p.out) + (orow + c0) * p.ldo + f;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (f < p.feats && c0 + j < t.rows) dst[j * p.ldo] = __uint_as_float(raw[j]);
        }
      } else {
        uint8_t* st = s_stage + q * 32 * kPitch;
        const float tscale = xscale * wscale;
        for (int c0 = 0; c0 < t.rows; c0 += 32) {
          uint32_t ra[16], rb[16];
          __syncwarp();
          if (t.nkb > 0) {
            tmem_ld_16x32(acc + c0, ra);
            tmem_ld_16x32(acc + c0 + (16u << 16), rb);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) ra[j] = rb[j] = 0;
          }
          float a[16], b[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            a[j] = __uint_as_float(ra[j]);
            b[j] = __uint_as_float(rb[j]);
          }
          if (MODE != kGradW && p.splits > 1) {
            const uint4* from = reinterpret_cast<const uint4*>(ring) + (c0 / 32 * 4 + q) * 256 + lane;
            for (int run = 1; run < p.splits; ++run, from += (t.rows + 31) / 32 * 1024)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4 v = from[i * 32];
                float* dst = (i < 4 ? a : b) + 4 * (i & 3);
                dst[0] += __uint_as_float(v.x);
                dst[1] += __uint_as_float(v.y);
                dst[2] += __uint_as_float(v.z);
                dst[3] += __uint_as_float(v.w);
              }
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            a[j] = FP4 ? fmaf(a[j], tscale, ba[(j >> 1) & 1]) : a[j] + ba[(j >> 1) & 1];
            b[j] = FP4 ? fmaf(b[j], tscale, bb[(j >> 1) & 1]) : b[j] + bb[(j >> 1) & 1];
          }
          const int nr = min(32, t.rows - c0);
          const int64_t row = orow + c0;
          if constexpr (MODE == kForward) {
            if (p.pre != nullptr) {
              if (gated) store_32x32(st, a, b, f16, pre, row, nr, f0, p.feats + f0, p.feats, p.wrows);
              else store_32x32(st, a, b, f16, pre, row, nr, f0, f0 + 16, p.feats, p.feats);
            }
            activate(a, p.act);
            if (gated) {
#pragma unroll
              for (int j = 0; j < 16; ++j) a[j] *= b[j];
              if (p.residual != nullptr) add_rows<false>(st, a, b, f16, res, row, nr, f0, p.feats);
              store_16x32(st, a, f16, out, row, nr, f0, p.feats);
              continue;
            }
            activate(b, p.act);
            if (p.residual != nullptr) add_rows<true>(st, a, b, f16, res, row, nr, f0, p.feats);
          }
          store_32x32(st, a, b, f16, out, row, nr, f0, f0 + 16, p.feats, p.feats);
        }
      }
      if (t.nkb > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_mapped(map_to_rank(smem_addr(s_tempty + as), leader));
        ++acc_it;
      }
    }
  }

  // ---- the end: the other CTA may still arrive on barriers or read this CTA's memory
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && s_stop) set_status(p.status, kStTimeout);
  cluster_sync();
  if (warp == 3) tmem_free(tmem, kTmemCols);
  cluster_sync();  // the pair frees its tensor memory together
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeFn g_encode = nullptr;

void find_encode() {
  void* f = nullptr;
  cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess) {
    (void)cudaGetLastError();
    return;
  }
  g_encode = reinterpret_cast<EncodeFn>(f);
}

// A tensor map over `rank` dimensions (innermost first; strides in bytes of
// dimensions 1..), boxes in the 128-byte swizzle, zeros out of bounds.
bool make_map(CUtensorMap* m, int type, const void* base, int rank, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  const CUtensorMapDataType dt = type == kE4M3 || type >= kE2M1MX ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : type == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return g_encode(m, dt, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_2d(CUtensorMap* m, int type, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_cols,
            int box_rows) {
  const int es = type == kE4M3 || type >= kE2M1MX ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * es)};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  return make_map(m, type, base, 2, dims, strides, box);
}

// The gradient of the pre-activations: [term, R, cols], or one term of any row stride.
bool map_terms(CUtensorMap* m, const MatmulArgs& a, int64_t cols, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)a.R, a.terms == 1 ? 1u : 2u};
  const cuuint64_t strides[2] = {(cuuint64_t)a.ldg * 2, (cuuint64_t)a.R * a.ldg * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  return make_map(m, a.type, a.g, 3, dims, strides, box);
}

template <int MODE, int KIND>
cudaError_t launch(const Maps& maps, Args a, int64_t max_tiles, int num_sms, cudaStream_t s) {
  int optin = 0;
  cudaError_t err = device_attr_cached(cudaDevAttrMaxSharedMemoryPerBlockOptin, &optin);
  if (err != cudaSuccess) return err;
  const size_t smem = (size_t)optin - 1024;  // room for the static arrays
  const size_t lists = (size_t)(4 * a.L + 1) * sizeof(int32_t) + kStageBytes +
                       (KIND != kHalf ? kScaleBufs<KIND> * kScaleBytes<KIND> : 0);
  a.ring_bytes = (int32_t)((smem - 1024 - lists) / 1024 * 1024);
  // the warps that lay out the scales of e2m1 operands count on four stages
  if (is_fp4(KIND) && a.ring_bytes < 4 * (kABytes + box_rows(box_index(kRows<KIND> / 2)) * 128)) return cudaErrorInvalidConfiguration;
  err = opt_in_smem(matmul_kernel<MODE, KIND>, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreadsOf<KIND>);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Runs of the reduction: as many as leave every tile a cluster of its own that
  // is resident, at least eight blocks a run, and accumulators that fit the ring.
  const int64_t blocks = (a.red + (KIND != kHalf ? 127 : 63)) / (KIND != kHalf ? 128 : 64);
  const int64_t tile_rows = a.R < kRows<KIND> ? a.R : kRows<KIND>;
  for (int splits = MODE == kGradW ? 1 : kMaxSplits;; splits /= 2) {
    const int cl = 2 * splits;
    if (splits > 1 && (blocks < 8 * splits || (splits - 1) * ((tile_rows + 31) / 32) * 16384 > a.ring_bytes)) continue;
    attr[0].val.clusterDim.x = (unsigned)cl;
    cfg.gridDim = dim3((unsigned)(num_sms / cl * cl));
    // no more clusters than can be resident at once: one more would start late
    int clusters = 0;
    err = max_clusters_cached(reinterpret_cast<const void*>(matmul_kernel<MODE, KIND>), cfg, cl, &clusters);
    if (err != cudaSuccess) return err;
    if (clusters > num_sms / cl) clusters = num_sms / cl;
    if (splits > 1 && max_tiles > clusters) continue;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    if (clusters > max_tiles) clusters = (int)max_tiles;
    a.splits = splits;
    cfg.gridDim = dim3((unsigned)(clusters * cl));
    return cudaLaunchKernelEx(&cfg, matmul_kernel<MODE, KIND>, maps, a);
  }
}

Args common_args(const MatmulArgs& m) {
  Args a{};
  a.seg_begin = m.seg_begin; a.seg_end = m.seg_end; a.cap = m.cap;
  a.R = (int32_t)m.R; a.L = m.L;
  a.f16 = m.type == kF16 || (m.type != kBF16 && m.out_type == kF16);
  a.terms = m.terms;
  a.status = m.status;
  return a;
}

// Most row tiles any counts can give: every expert's last tile may be short.
int64_t max_row_tiles(const MatmulArgs& m, int tile_rows) {
  const int64_t experts = m.L < m.R ? m.L : m.R;
  return m.R / tile_rows + experts;
}

}  // namespace

cudaError_t launch_matmul(const MatmulArgs& m, int num_sms, cudaStream_t s) {
  std::call_once(g_encode_once, find_encode);
  if (g_encode == nullptr) return cudaErrorNotSupported;
  const bool fp8 = m.type == kE4M3, fp4 = m.type >= kE2M1MX;
  const int es = fp8 || fp4 ? 1 : 2, span = 128 / es;  // elements (e2m1: pairs) per 128-byte line
  const int K = fp4 ? m.K / 2 : m.K;
  Args a = common_args(m);
  a.x_tscale = m.x_tscale; a.w_tscale = m.w_tscale;
  a.red = K; a.feats = m.N; a.wrows = m.gated ? 2 * m.N : m.N;
  a.gated = m.gated; a.act = m.act; a.bias = m.bias; a.residual = m.residual; a.ld_res = m.ld_res;
  a.out = m.out; a.ldo = m.ldo; a.pre = m.pre; a.ld_pre = m.ld_pre;
  a.xs = m.xs; a.ld_xs = m.ld_xs; a.ws = m.ws; a.ld_ws = m.ld_ws; a.G4 = (m.K / 128 + 3) / 4;
  const int fblk = m.gated ? 64 : 128;
  const int nfp = (m.N + 2 * fblk - 1) / (2 * fblk);
  Maps maps;
  const cuuint64_t row = (cuuint64_t)K * es;
  bool ok;
  if (m.gated) {  // (k, 16 features, gate | up, feature / 16, expert)
    const cuuint64_t dims[5] = {(cuuint64_t)K, 16, 2, (cuuint64_t)m.N / 16, (cuuint64_t)m.L};
    const cuuint64_t strides[4] = {row, row * m.N, row * 16, row * 2 * m.N};
    const cuuint32_t box[5] = {(cuuint32_t)span, 16, 2, 4, 1};
    ok = make_map(&maps.a, m.type, m.w, 5, dims, strides, box);
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)m.N, (cuuint64_t)m.L};
    const cuuint64_t strides[2] = {row, row * m.N};
    const cuuint32_t box[3] = {(cuuint32_t)span, 128, 1};
    ok = make_map(&maps.a, m.type, m.w, 3, dims, strides, box);
  }
  for (int i = 0; i < kBoxes; ++i) ok = ok && map_2d(&maps.b[i], m.type, m.x, K, m.R, m.ldx, span, box_rows(i));
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tile_rows = fp4 ? kRows<kFp4Nv> : fp8 ? kRows<kFp8> : kRows<kHalf>;
  const int64_t tiles = max_row_tiles(m, (int)tile_rows) * nfp;
  if (m.type == kE2M1MX) return launch<kForward, kFp4Mx>(maps, a, tiles, num_sms, s);
  if (m.type == kE2M1NV) return launch<kForward, kFp4Nv>(maps, a, tiles, num_sms, s);
  return fp8 ? launch<kForward, kFp8>(maps, a, tiles, num_sms, s) : launch<kForward, kHalf>(maps, a, tiles, num_sms, s);
}

cudaError_t launch_matmul_grad_x(const MatmulArgs& m, int num_sms, cudaStream_t s) {
  std::call_once(g_encode_once, find_encode);
  if (g_encode == nullptr) return cudaErrorNotSupported;
  Args a = common_args(m);
  a.wrows = m.gated ? 2 * m.N : m.N;
  a.red = a.wrows; a.feats = m.K; a.out = m.out; a.ldo = m.ldo;
  const int nfp = (m.K + 255) / 256;
  Maps maps;
  const cuuint64_t row = (cuuint64_t)m.K * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)m.K, (cuuint64_t)a.wrows, (cuuint64_t)m.L};
  const cuuint64_t strides[2] = {row, row * a.wrows};
  const cuuint32_t box[3] = {64, 64, 1};
  bool ok = make_map(&maps.a, m.type, m.w, 3, dims, strides, box);
  for (int i = 0; i < kBoxes; ++i) ok = ok && map_terms(&maps.b[i], m, a.wrows, box_rows(i));
  if (!ok) return cudaErrorInvalidValue;
  return launch<kGradX, kHalf>(maps, a, max_row_tiles(m, kRows<kHalf>) * nfp, num_sms, s);
}

cudaError_t launch_matmul_grad_w(const MatmulArgs& m, int num_sms, cudaStream_t s) {
  std::call_once(g_encode_once, find_encode);
  if (g_encode == nullptr) return cudaErrorNotSupported;
  Args a = common_args(m);
  a.wrows = m.gated ? 2 * m.N : m.N;
  a.feats = m.K; a.out = m.out; a.ldo = m.ldo; a.out_f32 = m.out_type == kF32;
  const int nfp = (m.K + 255) / 256;
  Maps maps;
  bool ok = map_2d(&maps.a, m.type, m.x, m.K, m.R, m.ldx, 64, 64);
  for (int i = 0; i < kBoxes; ++i) ok = ok && map_terms(&maps.b[i], m, a.wrows, 64);
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)m.L * ((a.wrows + 255) / 256) * nfp;
  return launch<kGradW, kHalf>(maps, a, tiles, num_sms, s);
}

}  // namespace moeperm
