// fp4.cu -- rows to four bits and back (format in fp4.cuh), in place order and as a
// dispatch into the compact layout.
//
// Large batches are bound by HBM: a bf16 row is read once (2 bytes an element) and leaves as
// 0.5 bytes and its scales (1/16 or 1/32): 16384 x 7168 in 48 us with scales per 32 (6.2
// TB/s), 58 with scales per 16 (5.2 TB/s, the division and its correction), the way back in
// 53 and 56 (5.6 and 5.3 TB/s). A lane owns 16 elements, so that a group of
// 16 needs no exchange and one of 32 a single one; a warp covers 512 elements of a row
// at a time, whose scales are one or two whole pieces.
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "layout.cuh"

namespace moeperm {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

template <int TYPE>
constexpr int kChunkBytes = 16 * (TYPE == kF32 ? 4 : 2);  // of 16 elements
// Rows that start on 32 bytes each.
__device__ __forceinline__ bool wide_rows(const void* p, int64_t ld_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uint64_t)ld_bytes) & 31) == 0;
}

// Whether row r is one of those to work on.
__device__ __forceinline__ bool has_row(const Fp4Args& p, int64_t r, int64_t live) {
  if (p.row_ids != nullptr) return __ldg(p.row_ids + r) >= 0;
  if (p.masked_m != nullptr) return (int)(r % p.cap) < __ldg(p.masked_m + r / p.cap);
  return r < live;
}
__device__ __forceinline__ int64_t live_rows(const Fp4Args& p) {
  if (p.d_num_live == nullptr) return p.R;
  int64_t n = __ldg(p.d_num_live);
  if (n > p.R) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, kStLiveOverflow);
    n = p.R;
  }
  return n < 0 ? 0 : n;
}
__device__ __forceinline__ float tensor_scale(const Fp4Args& p, int64_t r) {
  return p.tscale == nullptr ? 1.0f : __ldg(p.tscale + (p.nts == 1 ? 0 : r / (p.R / p.nts)));
}

// A warp takes kAhead slices of 512 elements of a row at a time.
template <int TYPE>
constexpr int kAhead = TYPE == kF32 ? 1 : 2;

template <int TYPE, int FMT>
__global__ void __launch_bounds__(kThreads) quant_fp4_kernel(Fp4Args p) {
  constexpr int kSpan = 32 * kAhead<TYPE>;  // chunks of a unit
  const int lane = threadIdx.x & 31;
  const int nch = p.H / 16, nchp = fp4_pieces(p.H, FMT) * (FMT == kFp4NV ? 16 : 32);  // chunks that have scale bytes
  const int upr = (nchp + kSpan - 1) / kSpan;  // units of a row
  const int64_t live = live_rows(p);
  const int64_t nwarps = (int64_t)gridDim.x * kWarps;
  int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  int64_t r = u / upr;
  int s = (int)(u - r * upr);
  const int64_t dr = nwarps / upr;
  const int ds = (int)(nwarps - dr * upr);
  const bool wide = wide_rows(p.x, p.ldx * (kChunkBytes<TYPE> / 16));
  for (; r < p.R; r += dr, s += ds) {
    if (s >= upr) {
      s -= upr;
      if (++r >= p.R) break;
    }
    if (!has_row(p, r, live)) continue;
    Chunk<TYPE> x[kAhead<TYPE>];
    const int c0 = s * kSpan + lane;
    const uint8_t* src = static_cast<const uint8_t*>(p.x) + r * p.ldx * (kChunkBytes<TYPE> / 16);
#pragma unroll
    for (int i = 0; i < kAhead<TYPE>; ++i) {
      const int c = c0 + 32 * i;
      x[i].load(src + (int64_t)c * kChunkBytes<TYPE>, c < nch, wide);
    }
    const float ts = FMT == kFp4NV ? tensor_scale(p, r) : 1.0f, ts6 = __fmul_rn(6.0f, ts);
#pragma unroll
    for (int i = 0; i < kAhead<TYPE>; ++i) {
      const int c = c0 + 32 * i;
      uint32_t byte;
      const uint2 q = fp4_quant<TYPE, FMT>(x[i], ts, ts6, byte);
      if (c < nch) *reinterpret_cast<uint2*>(p.q + r * (p.H / 2) + (int64_t)c * 8) = q;
      const uint32_t word = fp4_scale_word<FMT>(c < nch ? byte : 0u);
      if (fp4_word_lane<FMT>(lane) && c < nchp)
        *reinterpret_cast<uint32_t*>(p.scales + ((int64_t)fp4_piece_of<FMT>(c) * p.ld + r) * 16 + fp4_byte_of<FMT>(c)) = word;
    }
  }
}

// A lane writes 8 elements at a time (one run of memory for the warp), kUnit times.
constexpr int kUnit = 4;
template <int TYPE, int FMT>
__global__ void __launch_bounds__(kThreads) dequant_fp4_kernel(Fp4Args p) {
  constexpr int kSpan = 32 * kUnit, kBytes = kChunkBytes<TYPE> / 2;
  const int lane = threadIdx.x & 31;
  const int n8 = p.H / 8, upr = (n8 + kSpan - 1) / kSpan;
  const int64_t live = live_rows(p);
  const int64_t nwarps = (int64_t)gridDim.x * kWarps;
  int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  int64_t r = u / upr;
  int s = (int)(u - r * upr);
  const int64_t dr = nwarps / upr;
  const int ds = (int)(nwarps - dr * upr);
  const bool wide = wide_rows(p.x, p.ldx * (kChunkBytes<TYPE> / 16));
  for (; r < p.R; r += dr, s += ds) {
    if (s >= upr) {
      s -= upr;
      if (++r >= p.R) break;
    }
    if (!has_row(p, r, live)) continue;
    uint32_t q[kUnit], byte[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      const int c = s * kSpan + 32 * i + lane;
      if (c < n8) {
        q[i] = __ldg(reinterpret_cast<const uint32_t*>(p.q + r * (p.H / 2)) + c);
        byte[i] = __ldg(p.scales + ((int64_t)fp4_piece_of<FMT>(c / 2) * p.ld + r) * 16 + fp4_byte_of<FMT>(c / 2));
      }
    }
    const float ts = FMT == kFp4NV ? tensor_scale(p, r) : 1.0f;
    uint8_t* dst = static_cast<uint8_t*>(const_cast<void*>(p.x)) + r * p.ldx * (kChunkBytes<TYPE> / 16);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      const int c = s * kSpan + 32 * i + lane;
      if (c >= n8) break;
      const float d = fp4_scale<FMT>(byte[i], ts);
      float f[8];
      e2m1x8_to_floats(q[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], d);
      uint8_t* to = dst + (int64_t)c * kBytes;
      if constexpr (TYPE == kF32) {
        const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
        if (wide) {
          st_v8(to, Vec<TYPE>::pack(lo), Vec<TYPE>::pack(hi));
        } else {
          st_v4(to, Vec<TYPE>::pack(lo));
          st_v4(to + 16, Vec<TYPE>::pack(hi));
        }
      } else {
        st_v4(to, Vec<TYPE>::pack(f));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The dispatch
// ---------------------------------------------------------------------------

// Small problems, one launch: every CTA ranks all slots itself (layout.cuh), then
// quantises its tokens with all its warps and stores every 8 bytes, and every word of
// scales, to each of the token's rows.
template <int TYPE, int FMT, int S>
__global__ void __launch_bounds__(kThreads) dispatch_fp4_small_kernel(DispatchFp4Args p) {
  extern __shared__ int32_t sm[];
  __shared__ int32_t s_wsum[33];
  static_assert(kWarps == kSmallWarps, "small_layout's threads");
  const ScatterArgs& a = p.s;
  const int tid = threadIdx.x, lane = tid & 31;
  const int nch = a.H / 16, nchp = fp4_pieces(a.H, FMT) * (FMT == kFp4NV ? 16 : 32);
  const int n_live = live_count(a.d_num_tokens, a.T, a.status, blockIdx.x == 0 && tid == 0);
  const uint8_t* x = reinterpret_cast<const uint8_t*>(a.x);
  const bool wide = wide_rows(x, p.ldx_bytes);
  Chunk<TYPE> v;  // the first token's first elements load meanwhile
  v.load(x + (int64_t)blockIdx.x * p.ldx_bytes + (int64_t)tid * kChunkBytes<TYPE>, (int)blockIdx.x < n_live && tid < nch, wide);
  const float ts = FMT == kFp4NV && p.tscale != nullptr ? __ldg(p.tscale) : 1.0f, ts6 = __fmul_rn(6.0f, ts);
  small_layout<S>(a, sm, s_wsum, n_live);
  const int32_t* rows_all = small_rows(a, sm);
  for (int t = blockIdx.x; t < n_live; t += gridDim.x) {
    const int32_t* rows = rows_all + (int64_t)t * a.K;
    for (int c = tid; c - lane < nchp; c += kThreads) {
      if (t != (int)blockIdx.x || c >= kThreads)
        v.load(x + (int64_t)t * p.ldx_bytes + (int64_t)c * kChunkBytes<TYPE>, c < nch, wide);
      uint32_t byte;
      const uint2 q = fp4_quant<TYPE, FMT>(v, ts, ts6, byte);
      const uint32_t word = fp4_scale_word<FMT>(c < nch ? byte : 0u);
      const bool has_word = fp4_word_lane<FMT>(lane) && c < nchp;
      for (int k = 0; k < a.K; ++k) {
        const int64_t row = rows[k];
        if (row < 0) continue;
        if (c < nch) *reinterpret_cast<uint2*>(a.xq + row * (a.H / 2) + (int64_t)c * 8) = q;
        if (has_word)
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.scales) +
                                       ((int64_t)fp4_piece_of<FMT>(c) * a.ld_s + row) * 16 + fp4_byte_of<FMT>(c)) = word;
      }
    }
  }
}

// After the route plan. The rows of all tokens of a CTA are found at once; then each warp
// works alone on units of 2048 elements of a token: it quantises them into a staging
// buffer, copies the elements to every row with one bulk copy each (lane k that of slot k)
// and the scales piece by piece. Bound by latencies and
// the layout's prologue: 4096 tokens of 7168, top-8 of 64 experts, 45 us with the route
// plan (191 MB, 4.3 TB/s); whole tokens a warp, one round and an eighth of another, 49.
constexpr int kPart = 128;     // chunks of a unit
constexpr int kStages = 4;     // units in flight a warp
__host__ __device__ constexpr int part_pieces(int fmt) { return kPart / (fmt == kFp4NV ? 16 : 32); }
__host__ __device__ constexpr int stage_bytes(int fmt) { return kPart * 8 + part_pieces(fmt) * 16; }
// Shared memory before the staging buffers: table, starts, ends, rows of the CTA's slots.
__host__ __device__ inline size_t plan_bytes(const ScatterArgs& s, int64_t ntok) {
  const size_t ints = (size_t)s.nchunks * s.L + 2 * (size_t)s.L + (size_t)ntok * s.K;
  return (ints * sizeof(int32_t) + 127) / 128 * 128;
}

template <int TYPE, int FMT>
__global__ void __launch_bounds__(kThreads, TYPE == kF32 ? 2 : 3) dispatch_fp4_kernel(DispatchFp4Args p) {
  extern __shared__ __align__(128) int32_t sm[];
  __shared__ int32_t s_wsum[33];
  const ScatterArgs& a = p.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_live = live_count(a.d_num_tokens, a.T, nullptr, false);  // the route plan flags it
  const int ntok = n_live > (int)blockIdx.x ? (n_live - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  const int nch = a.H / 16, pieces = fp4_pieces(a.H, FMT), row_bytes = a.H / 2;
  constexpr int kPieces = part_pieces(FMT), kStage = stage_bytes(FMT);
  int32_t* st = sm + a.nchunks * a.L;
  int32_t* ps = st + a.L;
  int32_t* rows = ps + a.L;
  uint8_t* stage = reinterpret_cast<uint8_t*>(sm) + plan_bytes(a, ((int64_t)a.T + gridDim.x - 1) / gridDim.x) +
                   (size_t)warp * kStages * kStage;
  const float ts = FMT == kFp4NV && p.tscale != nullptr ? __ldg(p.tscale) : 1.0f, ts6 = __fmul_rn(6.0f, ts);
  pdl_wait_primary();
  layout_prologue(a, sm, st, ps, s_wsum);
  for (int i = tid; i < ntok * a.K; i += kThreads) {
    const int64_t slot = (int64_t)(blockIdx.x + (i / a.K) * gridDim.x) * a.K + i % a.K;
    const int row = slot_row(a, sm, st, slot, __ldg(a.ids + slot), __ldcg(a.src2dst + slot));
    a.src2dst[slot] = row;
    if (row >= 0 && a.row_weights != nullptr) a.row_weights[row] = __ldg(a.w + slot);
    rows[i] = row;
  }
  __syncthreads();
  const bool wide = wide_rows(a.x, p.ldx_bytes);
  const int parts = (nch + kPart - 1) / kPart;
  int buf = 0;
  for (int u = warp; u < ntok * parts; u += kWarps) {
    const int it = u / parts, c0 = (u - it * parts) * kPart;
    const int row = lane < a.K ? rows[it * a.K + lane] : -1;
    if (!__any_sync(0xffffffffu, row >= 0)) continue;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(a.x) + ((int64_t)blockIdx.x + (int64_t)it * gridDim.x) * p.ldx_bytes;
    uint8_t* out = stage + buf * kStage;
    constexpr int kSlices = kPart / 32, kBatch = TYPE == kF32 ? kSlices / 2 : kSlices;
#pragma unroll
    for (int s0 = 0; s0 < kSlices; s0 += kBatch) {
      Chunk<TYPE> x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + 32 * (s0 + i) + lane;
        x[i].load(src + (int64_t)c * kChunkBytes<TYPE>, c < nch, wide);
      }
      if (s0 == 0) {  // the copies that last read this buffer have left it
        bulk_wait_read<kStages - 1>();
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int o = 32 * (s0 + i) + lane, c = c0 + o;
        uint32_t byte;
        const uint2 q = fp4_quant<TYPE, FMT>(x[i], ts, ts6, byte);
        *reinterpret_cast<uint2*>(out + o * 8) = q;
        const uint32_t word = fp4_scale_word<FMT>(c < nch ? byte : 0u);
        if (fp4_word_lane<FMT>(lane))
          *reinterpret_cast<uint32_t*>(out + kPart * 8 + fp4_piece_of<FMT>(o) * 16 + fp4_byte_of<FMT>(o)) = word;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (row >= 0)
      bulk_store_s2g(a.xq + (int64_t)row * row_bytes + c0 * 8, smem_addr(out), (uint32_t)min(kPart, nch - c0) * 8);
    bulk_commit();
    const int first = c0 / (FMT == kFp4NV ? 16 : 32);  // the unit's first piece
    for (int i = lane; i < a.K * kPieces; i += 32) {
      const int c = i % kPieces;
      const int64_t to = rows[it * a.K + i / kPieces];
      if (to >= 0 && first + c < pieces)
        st_v4(static_cast<uint8_t*>(a.scales) + ((int64_t)(first + c) * a.ld_s + to) * 16,
              *reinterpret_cast<const uint4*>(out + kPart * 8 + c * 16));
    }
    buf = buf + 1 == kStages ? 0 : buf + 1;
  }
  // the layout's m_indices while the last copies drain
  fill_m_indices(a, st, ps, tid, kThreads);
  bulk_wait_all();
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

template <typename F>
cudaError_t by_type(int type, int fmt, F f) {
  auto by_fmt = [&](auto ty) -> cudaError_t {
    if (fmt == kFp4NV) return f(ty, std::integral_constant<int, kFp4NV>{});
    if (fmt == kFp4MX) return f(ty, std::integral_constant<int, kFp4MX>{});
    return f(ty, std::integral_constant<int, kFp4E8M0>{});
  };
  if (type == kBF16) return by_fmt(std::integral_constant<int, kBF16>{});
  if (type == kF16) return by_fmt(std::integral_constant<int, kF16>{});
  return by_fmt(std::integral_constant<int, kF32>{});
}

template <typename Kern>
cudaError_t launch_units(Kern kernel, const Fp4Args& a, int64_t units, int num_sms, cudaStream_t s) {
  int per_sm = 0;
  cudaError_t err = occupancy(kernel, kThreads, 0, &per_sm);
  if (err != cudaSuccess) return err;
  const int64_t need = (units + kWarps - 1) / kWarps, most = (int64_t)num_sms * (per_sm < 1 ? 1 : per_sm);
  kernel<<<(unsigned)(need < most ? need : most), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_fp4(const Fp4Args& a, int type, int fmt, int num_sms, cudaStream_t s) {
  return by_type(type, fmt, [&](auto ty, auto f) {
    constexpr int kT = decltype(ty)::value, kF = decltype(f)::value;
    const int nchp = fp4_pieces(a.H, kF) * (kF == kFp4NV ? 16 : 32), span = 32 * kAhead<kT>;
    return launch_units(quant_fp4_kernel<kT, kF>, a, a.R * ((nchp + span - 1) / span), num_sms, s);
  });
}

cudaError_t launch_dequant_fp4(const Fp4Args& a, int type, int fmt, int num_sms, cudaStream_t s) {
  return by_type(type, fmt, [&](auto ty, auto f) {
    return launch_units(dequant_fp4_kernel<decltype(ty)::value, decltype(f)::value>, a, a.R * ((a.H / 8 + 32 * kUnit - 1) / (32 * kUnit)), num_sms, s);
  });
}

cudaError_t launch_dispatch_fp4(const DispatchFp4Args& a0, int type, int fmt, int num_sms, bool after_route_plan,
                                cudaStream_t s) {
  return by_type(type, fmt, [&](auto ty, auto f) -> cudaError_t {
    constexpr int kT = decltype(ty)::value, kF = decltype(f)::value;
    DispatchFp4Args a = a0;
    const int64_t A = (int64_t)a.s.T * a.s.K;
    if (!after_route_plan) {
      if (A > kSmallSlots) return cudaErrorInvalidValue;
      const size_t smem = small_layout_bytes(a.s);
      auto go = [&](auto kernel) -> cudaError_t {
        cudaError_t err = opt_in_smem(kernel, smem);
        if (err != cudaSuccess) return err;
        int per_sm = 0;
        err = occupancy(kernel, kThreads, smem, &per_sm);
        if (err != cudaSuccess) return err;
        int64_t grid = (int64_t)num_sms * (per_sm < 1 ? 1 : per_sm);
        if (grid > a.s.T) grid = a.s.T;
        if (grid < 1) grid = 1;
        kernel<<<(unsigned)grid, kThreads, smem, s>>>(a);
        return cudaGetLastError();
      };
      if (A <= 256) return go(dispatch_fp4_small_kernel<kT, kF, 1>);
      if (A <= 1024) return go(dispatch_fp4_small_kernel<kT, kF, 4>);
      return go(dispatch_fp4_small_kernel<kT, kF, 8>);
    }
    // as many CTAs per SM as registers and shared memory leave room for (the plan's share
    // per CTA shrinks with the number of CTAs)
    auto kernel = dispatch_fp4_kernel<kT, kF>;
    int sm_bytes = 0;
    cudaError_t err = device_attr_cached(cudaDevAttrMaxSharedMemoryPerMultiprocessor, &sm_bytes);
    if (err != cudaSuccess) return err;
    const size_t ring = (size_t)kWarps * kStages * stage_bytes(kF);
    int64_t grid = a.s.T;
    size_t smem = 0;
    for (int per_sm = kT == kF32 ? 2 : 3;; --per_sm) {
      const int64_t g = a.s.T < (int64_t)num_sms * per_sm ? a.s.T : (int64_t)num_sms * per_sm;
      smem = plan_bytes(a.s, (a.s.T + g - 1) / g) + ring;
      if (per_sm == 1 || (smem + 2048) * per_sm <= (size_t)sm_bytes) {
        grid = g;
        break;
      }
    }
    err = opt_in_smem(kernel, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  });
}

}  // namespace moeperm
