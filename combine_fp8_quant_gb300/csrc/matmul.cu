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
//    an expert are cut into equal tiles of at most 256;
//  - a warp's 32 lanes hold neighbouring output elements, so the epilogue
//    stores straight from registers in full 32-byte sectors.
// With a gated activation a tile of 128 weight rows is 64 gate and 64 up rows
// interleaved by 16 (one 5-D tensor map does it), so gate and up of a feature
// are 16 lanes apart in one warp and meet through one shuffle.
//
// A CTA is one of a cluster of two with neighbouring feature blocks and the
// same rows; each loads half of the row tile and multicasts it to both, so a
// 128 x 256 tile costs L2 32 KB per 128 bytes of reduction instead of 48 KB.
// Warp roles: 0 loads (TMA), 1 issues the products, 2 lays out the e4m3 scales,
// 4-7 the epilogue, one warp per 32 lanes of tensor memory; two accumulators
// (columns 0.. and kRows..) let the epilogue of a tile overlap the products of
// the next. The grid is persistent; the tile list is formed on the device from
// the segment ends, so a captured graph can be replayed with other counts.
//
// Rows outside every segment are read at most as columns that are not stored.
// In kGradW rows are the reduction: lines of the last block past the segment's
// end are zeroed in shared memory before the product, so padding rows may hold
// anything (NaN included).
#include <cuda.h>

#include <mutex>

#include "elem.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace moeperm {

namespace {

constexpr int kForward = 0, kGradX = 1, kGradW = 2;
constexpr int kThreads = 256;
constexpr int kMaxStages = 10;
constexpr int kABytes = 16384;            // 128 rows x 128 bytes
constexpr int kTmemCols = 512;
constexpr int kScaleCols = 448;           // e4m3: scale words, 12 columns per buffer
constexpr int kScaleBytes = 512 + 1024;   // of one buffer: 128 + 256 words
constexpr int kBoxes = 7;                 // heights of the row boxes a CTA may load
__host__ __device__ constexpr int box_rows(int i) {
  return i < 3 ? 8 << i : i < 5 ? 32 * (i - 1) : 16 * (i + 2);  // 8 16 32 64 96 112 128
}

// Rows of one tile (the N side): two accumulators fill tensor memory; e4m3
// leaves room for the scale words.
template <bool FP8>
constexpr int kRows = FP8 ? 224 : 256;

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
  int32_t cl;                // CTAs per cluster, 1 or 2
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
  int32_t* status;
};

struct Tile {
  int e, fb;        // expert, feature block of this CTA
  int row0, rows;   // first output row (kGradW: within the expert), rows of the tile
  int n;            // N of the products (rows rounded up to 16)
  int nkb;          // reduction blocks
  int red_row0;     // kGradW: first row of the segment
  int tail;         // kGradW: valid lines of the last block
};

__device__ __forceinline__ int box_index(int half) {  // smallest box of at least `half` rows
  int i = 0;
  while (i < kBoxes - 1 && box_rows(i) < half) ++i;
  return i;
}

// A bounded wait that other roles can cut short.
__device__ __forceinline__ bool wait_or_stop(uint32_t bar, uint32_t parity, volatile int* stop) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if (clock64() - t0 > kWaitCycles) {
      *stop = 1;
      return false;
    }
  }
  return true;
}

// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait_or_stop(uint32_t bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, stop));
}

__device__ __forceinline__ uint16_t to_16bit(float v, bool f16) {
  return (uint16_t)(f16 ? pack_f16x2(v, 0.0f) : pack_bf16x2(v, 0.0f));
}
__device__ __forceinline__ float from_16bit(uint16_t v, bool f16) {
  return f16 ? f16x2_to_float2(v).x : __uint_as_float((uint32_t)v << 16);
}

__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }
// v * (the normal distribution function): no cancellation for negative v
__device__ __forceinline__ float gelu(float v) { return v * normcdff(v); }

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  if (act == kActRelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = v[j] > 0.0f ? v[j] : 0.0f;
  } else if (act == kActSilu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = silu(v[j]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = gelu(v[j]);
  }
}

template <int MODE, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages];
  __shared__ uint64_t s_tfull[2], s_tempty[2], s_sfull[2], s_sempty[2], s_drain;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_stop;
  __shared__ int s_max;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.cl > 1 ? (int)cluster_rank() : 0;
  const int cluster = blockIdx.x / p.cl, nclusters = gridDim.x / p.cl;
  const uint16_t mask = (uint16_t)((1 << p.cl) - 1);
  constexpr int kTileRows = kRows<FP8>;
  constexpr int kRedBlock = FP8 ? 128 : 64;  // reduction elements per stage

  uint8_t* ring = dyn + ((1024 - (smem_addr(dyn) & 1023)) & 1023);
  uint8_t* s_scale = ring + p.ring_bytes;                                 // FP8: two buffers
  int32_t* s_tiles = reinterpret_cast<int32_t*>(s_scale + (FP8 ? 2 * kScaleBytes : 0));  // [L + 1]
  int32_t* s_begin = s_tiles + p.L + 1;
  int32_t* s_count = s_begin + p.L;

  // ---- set-up
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(smem_addr(s_full + i), 1);
      mbar_init(smem_addr(s_empty + i), p.cl);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(s_tfull + i), 1);
      mbar_init(smem_addr(s_tempty + i), 4);
      mbar_init(smem_addr(s_sfull + i), 1);
      mbar_init(smem_addr(s_sempty + i), 1);
    }
    mbar_init(smem_addr(&s_drain), 1);
    mbar_init_fence();
    s_stop = 0;
    s_max = 0;
    prefetch_map(&maps.a);
  }
  if (warp == 3) tmem_alloc(smem_addr(&s_tmem), kTmemCols);
  __syncthreads();
  int mx = 0;
  for (int e = tid; e < p.L; e += kThreads) {
    int64_t b = 0, c = p.R;
    if (p.cap > 0) {
      b = (int64_t)e * p.cap;
      c = __ldg(p.seg_end + e);
    } else if (p.seg_begin != nullptr) {
      b = __ldg(p.seg_begin + e);
      c = (int64_t)__ldg(p.seg_end + e) - b;
    }
    const bool bad = b < 0 || c < 0 || b + c > p.R || (p.cap > 0 && c > p.cap);
    if (bad) {  // nothing of it is read or written
      if (blockIdx.x == 0) set_status(p.status, kStBadLayout);
      b = c = 0;
    }
    s_begin[e] = (int)b;
    s_count[e] = (int)c;
    mx = max(mx, (int)c);
  }
  atomicMax(&s_max, mx);
  __syncthreads();
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
      if (e < p.L) s_tiles[e] = base + incl - v;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_tiles[p.L] = base;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.cl > 1) cluster_sync();  // the peer's barriers are ready before anything arrives on them
  const uint32_t tmem = s_tmem;

  // ---- tile list (the same for every role and both CTAs of the cluster)
  const int fblk = p.gated && MODE == kForward ? 64 : 128;  // features per block
  const int nfc = ((p.feats + fblk - 1) / fblk + p.cl - 1) / p.cl;  // clusters of blocks
  const int nnb = MODE == kGradW ? (p.wrows + 255) / 256 : 0;       // kGradW: row blocks per expert
  const int total = MODE == kGradW ? p.L * nnb * nfc : s_tiles[p.L] * nfc;
  auto tile_at = [&](int w) {
    Tile t;
    t.fb = (w % nfc) * p.cl + rank;
    const int rb = w / nfc;
    if constexpr (MODE == kGradW) {
      t.e = rb / nnb;
      t.row0 = (rb - t.e * nnb) * 256;
      t.rows = min(256, p.wrows - t.row0);
      t.red_row0 = s_begin[t.e];
      t.nkb = (s_count[t.e] + 63) / 64;
      t.tail = s_count[t.e] - (t.nkb - 1) * 64;
    } else {
      int lo = 0, hi = p.L - 1;  // the last expert whose tiles start at or before rb
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tiles[mid] <= rb) lo = mid; else hi = mid - 1;
      }
      t.e = lo;
      const int cnt = s_count[lo], nt = s_tiles[lo + 1] - s_tiles[lo];
      const int per = ((cnt + nt - 1) / nt + 15) / 16 * 16;  // equal tiles
      const int j = rb - s_tiles[lo];
      t.row0 = s_begin[lo] + j * per;
      t.rows = min(per, cnt - j * per);
      t.nkb = (p.red + kRedBlock - 1) / kRedBlock;
      t.red_row0 = t.tail = 0;
    }
    t.n = (t.rows + 15) / 16 * 16;
    return t;
  };

  // ---- ring geometry: as many stages as the largest row tile allows
  const int max_n = MODE == kGradW ? 256 : min(kTileRows, (s_max + 15) / 16 * 16);
  const int b_bytes = MODE == kGradW ? min((p.wrows + 63) / 64, 4) * 8192
                                     : 2 * box_rows(box_index(max_n / 2)) * 128;
  const int stage_bytes = kABytes + b_bytes;
  const int stages = min(kMaxStages, p.ring_bytes / stage_bytes);
  const uint32_t ring_s = smem_addr(ring);

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int w = cluster; w < total && ok; w += nclusters) {
        const Tile t = tile_at(w);
        const int box = MODE == kGradW ? 0 : box_index(t.n / 2);
        const int half = box_rows(box);
        const int nbox = (t.n + 63) / 64;  // kGradW: 64-wide boxes of the row side
        const uint32_t bytes = kABytes + (MODE == kGradW ? nbox * 8192 : 2 * half * 128);
        for (int kb = 0; kb < t.nkb; ++kb, ++it) {
          const int s = it % stages;
          if (!(ok = wait_or_stop(smem_addr(s_empty + s), ((it / stages) & 1) ^ 1, &s_stop))) break;
          const uint32_t full = smem_addr(s_full + s);
          const uint32_t a = ring_s + s * stage_bytes, b = a + kABytes;
          mbar_expect_tx(full, bytes);
          if constexpr (MODE == kForward) {
            if (p.gated) tma_load_5d(a, &maps.a, full, kb * kRedBlock, 0, 0, t.fb * 4, t.e);
            else tma_load_3d(a, &maps.a, full, kb * kRedBlock, t.fb * 128, t.e);
          } else if constexpr (MODE == kGradX) {
            tma_load_3d(a, &maps.a, full, t.fb * 128, kb * 64, t.e);
            tma_load_3d(a + 8192, &maps.a, full, t.fb * 128 + 64, kb * 64, t.e);
          } else {
            tma_load_2d(a, &maps.a, full, t.fb * 128, t.red_row0 + kb * 64);
            tma_load_2d(a + 8192, &maps.a, full, t.fb * 128 + 64, t.red_row0 + kb * 64);
          }
          if constexpr (MODE == kGradW) {
            for (int i = rank; i < nbox; i += p.cl) {
              if (p.cl > 1)
                tma_load_2d_multi(b + i * 8192, &maps.b[0], full, t.row0 + i * 64, t.red_row0 + kb * 64, mask);
              else
                tma_load_2d(b + i * 8192, &maps.b[0], full, t.row0 + i * 64, t.red_row0 + kb * 64);
            }
          } else {
            for (int h = rank; h < 2; h += p.cl) {
              if (p.cl > 1)
                tma_load_2d_multi(b + h * half * 128, &maps.b[box], full, kb * kRedBlock, t.row0 + h * half, mask);
              else
                tma_load_2d(b + h * half * 128, &maps.b[box], full, kb * kRedBlock, t.row0 + h * half);
            }
          }
        }
      }
      if (!ok)  // let the copies in flight land, again with a limit
        for (int i = it > stages ? it - stages : 0; i < it; ++i)
          mbar_wait(smem_addr(s_full + i % stages), (i / stages) & 1);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- products
    // one lane issues; kGradW keeps the warp together to zero the last lines
    int it = 0, acc_it = 0, sf_it = 0;
    bool ok = MODE == kGradW || lane == 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return MODE == kGradW ? warp_wait_or_stop(smem_addr(bar), parity, &s_stop)
                            : wait_or_stop(smem_addr(bar), parity, &s_stop);
    };
    for (int w = cluster; w < total && ok; w += nclusters) {
      const Tile t = tile_at(w);
      if (t.nkb == 0) continue;  // kGradW: an expert without rows; the epilogue writes zeros
      const int as = acc_it & 1;
      if (!(ok = wait(s_tempty + as, ((acc_it >> 1) & 1) ^ 1))) break;
      tc_fence_after();
      const uint32_t d = tmem + as * kTileRows;
      uint32_t idesc = idesc_16bit(!p.f16, MODE != kForward, MODE == kGradW, t.n);
      for (int kb = 0; kb < t.nkb; ++kb, ++it) {
        const int s = it % stages;
        if (!(ok = wait(s_full + s, (it / stages) & 1))) break;
        if constexpr (FP8) {
          if ((kb & 3) == 0 && !(ok = wait(s_sfull + (sf_it & 1), (sf_it >> 1) & 1))) break;
        }
        tc_fence_after();
        uint8_t* a = ring + s * stage_bytes;
        if (MODE == kGradW && kb == t.nkb - 1 && t.tail < 64) {
          // rows past the segment's end: zero lines in every 64-wide box
          const int boxes = 2 + (t.n + 63) / 64;
          for (int i = lane; i < boxes * (64 - t.tail) * 8; i += 32) {
            const int line = i >> 3, bx = line / (64 - t.tail), r = t.tail + line % (64 - t.tail);
            *reinterpret_cast<uint4*>(a + bx * 8192 + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          const uint32_t as_ = smem_addr(a);
          if constexpr (FP8) {
            const int sb = sf_it & 1;
            const uint32_t sfa = tmem + kScaleCols + 12 * sb, sfb = sfa + 4;
            if ((kb & 3) == 0) {
              const uint32_t sm = smem_addr(s_scale + sb * kScaleBytes);
              tmem_copy_scales(sfa, desc_plain16(sm));
              for (int i = 0; i * 128 < t.n; ++i) tmem_copy_scales(sfb + 4 * i, desc_plain16(sm + 512 + 512 * i));
            }
            idesc = idesc_e4m3(t.n, kb & 3);
            const uint64_t da = desc_k_major(as_), db = desc_k_major(as_ + kABytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_e4m3(d, da + 2 * k, db + 2 * k, idesc, sfa, sfb, kb > 0 || k > 0);
            if ((kb & 3) == 3 || kb == t.nkb - 1) mma_commit(smem_addr(s_sempty + sb));
          } else {
            const uint64_t da = MODE == kForward ? desc_k_major(as_) : desc_mn_major(as_, 8192);
            const uint64_t db = MODE == kGradW ? desc_mn_major(as_ + kABytes, 8192) : desc_k_major(as_ + kABytes);
            constexpr int ka = MODE == kForward ? 2 : 128, kb_step = MODE == kGradW ? 128 : 2;
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_16bit(d, da + ka * k, db + kb_step * k, idesc, kb > 0 || k > 0);
          }
          if (p.cl > 1) mma_commit_multi(smem_addr(s_empty + s), mask);
          else mma_commit(smem_addr(s_empty + s));
          if (kb == t.nkb - 1) mma_commit(smem_addr(s_tfull + as));
        }
        if constexpr (MODE == kGradW) __syncwarp();
        if (FP8 && ((kb & 3) == 3 || kb == t.nkb - 1)) ++sf_it;
      }
      ++acc_it;
    }
    if (!ok && lane == 0) {  // products in flight end before tensor memory is freed
      mma_commit(smem_addr(&s_drain));
      mbar_wait(smem_addr(&s_drain), 0);
    }
  } else if (FP8 && warp == 2) {
    // ----------------------------------------------------------------- scales
    // Word w of a row holds the exponents of its reduction elements 512 w ..
    // 512 w + 511, one byte per 128. Tensor memory wants row r of a block of
    // 128 at lane r % 32, column r / 32: lane l stores rows l, l + 32, l + 64
    // and l + 96 as one 16-byte line.
    const int Nw = p.wrows;
    int sf_it = 0;
    bool ok = true;
    for (int w = cluster; w < total && ok; w += nclusters) {
      const Tile t = tile_at(w);
      int64_t arow[4], brow[8];  // word offsets of this lane's rows (-1: none)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int f = t.fb * 128 + i * 32 + lane, wr = f;
        if (p.gated) {
          f = t.fb * 64 + i * 16 + (lane & 15);
          wr = (lane & 16) ? p.feats + f : f;
        }
        arow[i] = f < p.feats ? (int64_t)t.e * Nw + wr : -1;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * 32 + lane;
        const int64_t row = p.cap > 0 ? (int64_t)t.e * p.G4 * p.ld_xs + (t.row0 + r - t.e * p.cap) : t.row0 + r;
        brow[i] = r < t.rows ? row : -1;
      }
      for (int kb = 0; kb < t.nkb; kb += 4, ++sf_it) {
        const int sb = sf_it & 1, word = kb >> 2;
        uint32_t va[4], vb[8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          va[i] = arow[i] >= 0 ? __ldg(p.ws + (int64_t)word * p.ld_ws + arow[i]) : 0x7F7F7F7Fu;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          vb[i] = brow[i] >= 0 ? __ldg(p.xs + (int64_t)word * p.ld_xs + brow[i]) : 0x7F7F7F7Fu;
        if (!(ok = warp_wait_or_stop(smem_addr(s_sempty + sb), ((sf_it >> 1) & 1) ^ 1, &s_stop))) break;
        uint8_t* dst = s_scale + sb * kScaleBytes + lane * 16;
        *reinterpret_cast<uint4*>(dst) = make_uint4(va[0], va[1], va[2], va[3]);
        *reinterpret_cast<uint4*>(dst + 512) = make_uint4(vb[0], vb[1], vb[2], vb[3]);
        *reinterpret_cast<uint4*>(dst + 1024) = make_uint4(vb[4], vb[5], vb[6], vb[7]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(s_sfull + sb));
      }
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------------- epilogue
    const int q = warp & 3;  // this warp's 32 lanes of tensor memory
    const bool f16 = p.f16 != 0;
    int acc_it = 0;
    for (int w = cluster; w < total; w += nclusters) {
      const Tile t = tile_at(w);
      const int as = acc_it & 1;
      if (t.nkb > 0) {
        if (!warp_wait_or_stop(smem_addr(s_tfull + as), (acc_it >> 1) & 1, &s_stop)) break;
        tc_fence_after();
      }
      const uint32_t acc = tmem + as * kTileRows + ((uint32_t)(q * 32) << 16);
      const bool gated = MODE == kForward && p.gated;
      // this lane's feature (gated: lanes 0-15 gate, 16-31 up of the same 16)
      const int f = gated ? t.fb * 64 + q * 16 + (lane & 15) : t.fb * 128 + q * 32 + lane;
      const bool fok = f < p.feats;
      const int wrow = gated && (lane & 16) ? p.feats + f : f;
      float bias = 0.0f;
      if (MODE == kForward && p.bias != nullptr && fok) bias = __ldg(p.bias + (int64_t)t.e * p.wrows + wrow);
      const int64_t orow = MODE == kGradW ? (int64_t)t.e * p.wrows + t.row0 : t.row0;
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
        const int nc = min(32, t.rows - c0);
        if constexpr (MODE == kForward) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) + bias;
          if (p.pre != nullptr && fok) {
            uint16_t* dst = static_cast<uint16_t*>(p.pre) + (orow + c0) * p.ld_pre + wrow;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < nc) dst[j * p.ld_pre] = to_16bit(v[j], f16);
          }
          if (gated) {
            // lanes 0-15 finish the even rows, 16-31 the odd ones: one exchange per pair
            float g[16], u[16];
            const bool upper = (lane & 16) != 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float give = upper ? v[2 * j] : v[2 * j + 1];
              const float got = __shfl_xor_sync(0xffffffffu, give, 16);
              g[j] = upper ? got : v[2 * j];
              u[j] = upper ? v[2 * j + 1] : got;
            }
            activate(g, p.act);
            const int odd = upper ? 1 : 0;
            uint16_t* dst = static_cast<uint16_t*>(p.out) + (orow + c0 + odd) * p.ldo + f;
            const uint16_t* res = static_cast<const uint16_t*>(p.residual) + (orow + c0 + odd) * p.ld_res + f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (!fok || 2 * j + odd >= nc) continue;
              float o = g[j] * u[j];
              if (p.residual != nullptr) o += from_16bit(__ldg(res + 2 * j * p.ld_res), f16);
              dst[2 * j * p.ldo] = to_16bit(o, f16);
            }
          } else {
            activate(v, p.act);
            if (!fok) continue;
            uint16_t* dst = static_cast<uint16_t*>(p.out) + (orow + c0) * p.ldo + f;
            const uint16_t* res = static_cast<const uint16_t*>(p.residual) + (orow + c0) * p.ld_res + f;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (j >= nc) continue;
              if (p.residual != nullptr) v[j] += from_16bit(__ldg(res + j * p.ld_res), f16);
              dst[j * p.ldo] = to_16bit(v[j], f16);
            }
          }
        } else {
          if (!fok) continue;
          if (p.out_f32) {
            float* dst = static_cast<float*>(p.out) + (orow + c0) * p.ldo + f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < nc) dst[j * p.ldo] = __uint_as_float(raw[j]);
          } else {
            uint16_t* dst = static_cast<uint16_t*>(p.out) + (orow + c0) * p.ldo + f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < nc) dst[j * p.ldo] = to_16bit(__uint_as_float(raw[j]), f16);
          }
        }
      }
      if (t.nkb > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(s_tempty + as));
        ++acc_it;
      }
    }
  }

  // ---- the end: nothing of this CTA's peer may still arrive here
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && s_stop) set_status(p.status, kStTimeout);
  if (p.cl > 1) cluster_sync();
  if (warp == 3) tmem_free(tmem, kTmemCols);
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
  const CUtensorMapDataType dt = type == kE4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : type == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return g_encode(m, dt, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_2d(CUtensorMap* m, int type, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_cols,
            int box_rows) {
  const int es = type == kE4M3 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * es)};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  return make_map(m, type, base, 2, dims, strides, box);
}

template <int MODE, bool FP8>
cudaError_t launch(const Maps& maps, Args a, int64_t max_tiles, int num_sms, cudaStream_t s) {
  int optin = 0;
  cudaError_t err = device_attr_cached(cudaDevAttrMaxSharedMemoryPerBlockOptin, &optin);
  if (err != cudaSuccess) return err;
  const size_t smem = (size_t)optin - 1024;  // room for the static arrays
  const size_t lists = (size_t)(3 * a.L + 1) * sizeof(int32_t) + (FP8 ? 2 * kScaleBytes : 0);
  a.ring_bytes = (int32_t)((smem - 1024 - lists) / 1024 * 1024);
  err = opt_in_smem(matmul_kernel<MODE, FP8>, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // as many clusters as can be resident at once: one more would start late
  cfg.gridDim = dim3((unsigned)(num_sms / a.cl * a.cl));
  int clusters = 0;
  err = max_clusters_cached(reinterpret_cast<const void*>(matmul_kernel<MODE, FP8>), cfg, a.cl, &clusters);
  if (err != cudaSuccess) return err;
  if (clusters < 1) return cudaErrorInvalidConfiguration;
  if (clusters > num_sms / a.cl) clusters = num_sms / a.cl;
  if (clusters > max_tiles) clusters = (int)max_tiles;
  cfg.gridDim = dim3((unsigned)(clusters * a.cl));
  return cudaLaunchKernelEx(&cfg, matmul_kernel<MODE, FP8>, maps, a);
}

Args common_args(const MatmulArgs& m) {
  Args a{};
  a.seg_begin = m.seg_begin; a.seg_end = m.seg_end; a.cap = m.cap;
  a.R = (int32_t)m.R; a.L = m.L; a.f16 = m.type == kF16 || (m.type == kE4M3 && m.out_type == kF16);
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
  const bool fp8 = m.type == kE4M3;
  const int es = fp8 ? 1 : 2, span = 128 / es;  // elements per 128-byte line
  Args a = common_args(m);
  a.red = m.K; a.feats = m.N; a.wrows = m.gated ? 2 * m.N : m.N;
  a.gated = m.gated; a.act = m.act; a.bias = m.bias; a.residual = m.residual; a.ld_res = m.ld_res;
  a.out = m.out; a.ldo = m.ldo; a.pre = m.pre; a.ld_pre = m.ld_pre;
  a.xs = m.xs; a.ld_xs = m.ld_xs; a.ws = m.ws; a.ld_ws = m.ld_ws; a.G4 = (m.K / 128 + 3) / 4;
  const int fblk = m.gated ? 64 : 128;
  const int nfb = (m.N + fblk - 1) / fblk;
  a.cl = nfb > 1 ? 2 : 1;
  Maps maps;
  const cuuint64_t row = (cuuint64_t)m.K * es;
  bool ok;
  if (m.gated) {  // (k, 16 features, gate | up, feature / 16, expert)
    const cuuint64_t dims[5] = {(cuuint64_t)m.K, 16, 2, (cuuint64_t)m.N / 16, (cuuint64_t)m.L};
    const cuuint64_t strides[4] = {row, row * m.N, row * 16, row * 2 * m.N};
    const cuuint32_t box[5] = {(cuuint32_t)span, 16, 2, 4, 1};
    ok = make_map(&maps.a, m.type, m.w, 5, dims, strides, box);
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)m.K, (cuuint64_t)m.N, (cuuint64_t)m.L};
    const cuuint64_t strides[2] = {row, row * m.N};
    const cuuint32_t box[3] = {(cuuint32_t)span, 128, 1};
    ok = make_map(&maps.a, m.type, m.w, 3, dims, strides, box);
  }
  for (int i = 0; i < kBoxes; ++i) ok = ok && map_2d(&maps.b[i], m.type, m.x, m.K, m.R, m.ldx, span, box_rows(i));
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tiles = max_row_tiles(m, fp8 ? kRows<true> : kRows<false>) * ((nfb + a.cl - 1) / a.cl);
  return fp8 ? launch<kForward, true>(maps, a, tiles, num_sms, s) : launch<kForward, false>(maps, a, tiles, num_sms, s);
}

cudaError_t launch_matmul_grad_x(const MatmulArgs& m, int num_sms, cudaStream_t s) {
  std::call_once(g_encode_once, find_encode);
  if (g_encode == nullptr) return cudaErrorNotSupported;
  Args a = common_args(m);
  a.wrows = m.gated ? 2 * m.N : m.N;
  a.red = a.wrows; a.feats = m.K; a.out = m.out; a.ldo = m.ldo;
  const int nfb = (m.K + 127) / 128;
  a.cl = nfb > 1 ? 2 : 1;
  Maps maps;
  const cuuint64_t row = (cuuint64_t)m.K * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)m.K, (cuuint64_t)a.wrows, (cuuint64_t)m.L};
  const cuuint64_t strides[2] = {row, row * a.wrows};
  const cuuint32_t box[3] = {64, 64, 1};
  bool ok = make_map(&maps.a, m.type, m.w, 3, dims, strides, box);
  for (int i = 0; i < kBoxes; ++i) ok = ok && map_2d(&maps.b[i], m.type, m.g, a.wrows, m.R, m.ldg, 64, box_rows(i));
  if (!ok) return cudaErrorInvalidValue;
  return launch<kGradX, false>(maps, a, max_row_tiles(m, kRows<false>) * ((nfb + a.cl - 1) / a.cl), num_sms, s);
}

cudaError_t launch_matmul_grad_w(const MatmulArgs& m, int num_sms, cudaStream_t s) {
  std::call_once(g_encode_once, find_encode);
  if (g_encode == nullptr) return cudaErrorNotSupported;
  Args a = common_args(m);
  a.wrows = m.gated ? 2 * m.N : m.N;
  a.feats = m.K; a.out = m.out; a.ldo = m.ldo; a.out_f32 = m.out_type == kF32;
  const int nfb = (m.K + 127) / 128;
  a.cl = nfb > 1 ? 2 : 1;
  Maps maps;
  bool ok = map_2d(&maps.a, m.type, m.x, m.K, m.R, m.ldx, 64, 64);
  for (int i = 0; i < kBoxes; ++i) ok = ok && map_2d(&maps.b[i], m.type, m.g, a.wrows, m.R, m.ldg, 64, 64);
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)m.L * ((a.wrows + 255) / 256) * ((nfb + a.cl - 1) / a.cl);
  return launch<kGradW, false>(maps, a, tiles, num_sms, s);
}

}  // namespace moeperm
