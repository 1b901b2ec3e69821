// permute.cu -- tokens sorted by expert: every kept (token, slot) gets a copy
// of its token's row, unquantised, in the compact layout of the dispatch
// (same row order, m_indices, src2dst, counts, starts, psum, total).
//
//   xs[row(t,k)] = x[t],  row(t,k) = starts[e] + rank of the slot among e's
//
// No arithmetic, so no registers: one warp per CTA moves the rows with bulk
// copies, a ring of row pieces in shared memory (global -> shared once per
// token, shared -> global once per kept slot, each slot's copy issued by the
// lane that holds its row). The first pieces are loaded before the layout is
// known; a later token without a kept slot is not read. The other warps fill
// m_indices meanwhile. Bound by HBM writes (top-8: eight rows written per row
// read): 8192 x 7168 bf16, 1.06 GB in 176 us after the 5 us route plan, 6.0 TB/s;
// rings of 3 to 8 pieces and eviction hints on the rows measured within 1%.
//
// Like the quantising dispatch: up to kSmallSlots slots one launch in which
// every CTA ranks all slots itself, above that the route plan and this launch,
// started early with programmatic dependent launch.
#include "common.cuh"
#include "kernels.h"
#include "layout.cuh"

namespace moeperm {

namespace {

constexpr int kThreads = kSmallWarps * 32;
constexpr int kMaxStages = 4;

// One warp's stream of row pieces through the ring. Tokens of the CTA are
// it = 0 .. ntok-1 (token blockIdx.x + it * gridDim.x); rows + it * stride
// holds token it's K rows once they are known.
struct Mover {
  const PermuteArgs& p;
  uint8_t* ring;
  uint64_t* bars;
  int* desc;             // [stages] (it * units + part) of the piece in each slot
  int ntok, lane;
  int lit = 0, lpart = 0;  // next piece to load
  int issued = 0, done = 0;

  __device__ Mover(const PermuteArgs& p_, uint8_t* ring_, uint64_t* bars_, int* desc_, int ntok_, int lane_)
      : p(p_), ring(ring_), bars(bars_), desc(desc_), ntok(ntok_), lane(lane_) {
    if (lane == 0) {
      for (int i = 0; i < p.stages; ++i) mbar_init(smem_addr(bars + i), 1);
      mbar_init_fence();
    }
    __syncwarp();
  }
  __device__ int piece_bytes(int part) const {
    return min(p.unit_bytes, p.row_bytes - part * p.unit_bytes);
  }
  __device__ void load_next() {
    const int slot = issued % p.stages;
    if (lane == 0) {
      const int64_t t = (int64_t)blockIdx.x + (int64_t)lit * gridDim.x;
      const uint32_t bytes = (uint32_t)piece_bytes(lpart);
      const uint32_t bar = smem_addr(bars + slot);
      mbar_expect_tx(bar, bytes);
      bulk_load_g2s(smem_addr(ring + (size_t)slot * p.unit_bytes),
                    reinterpret_cast<const uint8_t*>(p.s.x) + t * p.ldx_bytes + (int64_t)lpart * p.unit_bytes,
                    bytes, bar);
      desc[slot] = lit * p.units + lpart;
    }
    __syncwarp();
    ++issued;
    if (++lpart == p.units) {
      lpart = 0;
      ++lit;
    }
  }
  __device__ void preload() {
    while (issued < p.stages && lit < ntok) load_next();
  }
  // Loads the next piece of a token that has a kept slot, if there is one.
  __device__ void refill(const int* rows, int stride) {
    if (lpart == 0)
      while (lit < ntok &&
             !__any_sync(0xffffffffu, lane < p.s.K && rows[(int64_t)lit * stride + lane] >= 0))
        ++lit;
    if (lit < ntok) load_next();
  }
  __device__ void run(const int* rows, int stride) {
    while (done < issued) {
      const int slot = done % p.stages;
      const bool landed = mbar_wait(smem_addr(bars + slot), (uint32_t)(done / p.stages) & 1u);
      if (!__all_sync(0xffffffffu, landed)) {  // the same answer in every lane
        if (lane == 0) set_status(p.s.status, kStTimeout);
        for (; done < issued; ++done)  // its own loads still in flight, again with a limit
          mbar_wait(smem_addr(bars + done % p.stages), (uint32_t)(done / p.stages) & 1u);
        break;
      }
      const int u = desc[slot];
      const int it = u / p.units, part = u - it * p.units;
      const int row = lane < p.s.K ? rows[(int64_t)it * stride + lane] : -1;
      if (row >= 0)
        bulk_store_s2g(p.s.xq + (int64_t)row * p.row_bytes + (int64_t)part * p.unit_bytes,
                       smem_addr(ring + (size_t)slot * p.unit_bytes), (uint32_t)piece_bytes(part));
      bulk_commit();
      ++done;
      if (issued - done <= p.stages - 2) {
        bulk_wait_read<1>();  // the copies of every piece but the last have left their slots
        __syncwarp();
        refill(rows, stride);
      }
    }
    bulk_wait_all();
  }
};

__host__ __device__ inline size_t plan_bytes(const ScatterArgs& s, int64_t ntok) {
  const size_t ints = (size_t)s.nchunks * s.L + 2 * (size_t)s.L + (size_t)ntok * s.K;
  return (ints * sizeof(int32_t) + 127) / 128 * 128;
}

__device__ __forceinline__ int own_tokens(int n_live) {
  return n_live > (int)blockIdx.x ? (n_live - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
}

// After the route plan (programmatic dependent launch).
__global__ void __launch_bounds__(kThreads) permute_kernel(PermuteArgs p) {
  extern __shared__ int32_t sm[];
  __shared__ int32_t s_wsum[33];
  __shared__ uint64_t s_bars[kMaxStages];
  __shared__ int s_desc[kMaxStages];
  const ScatterArgs& s = p.s;
  const int tid = threadIdx.x, lane = tid & 31;
  const int n_live = live_count(s.d_num_tokens, s.T, nullptr, false);  // the route plan flags it
  const int ntok = own_tokens(n_live);
  uint8_t* ring = reinterpret_cast<uint8_t*>(sm) + plan_bytes(s, ((int64_t)s.T + gridDim.x - 1) / gridDim.x);
  Mover mv(p, ring, s_bars, s_desc, tid < 32 ? ntok : 0, tid < 32 ? lane : -1);
  if (tid < 32) mv.preload();
  pdl_wait_primary();
  int32_t* st = sm + s.nchunks * s.L;
  int32_t* ps = st + s.L;
  int32_t* rows = ps + s.L;
  layout_prologue(s, sm, st, ps, s_wsum);
  for (int i = tid; i < ntok * s.K; i += kThreads) {
    const int64_t a = (int64_t)(blockIdx.x + (i / s.K) * gridDim.x) * s.K + (i % s.K);
    const int row = slot_row(s, sm, st, a, __ldg(s.ids + a), __ldcg(s.src2dst + a));
    s.src2dst[a] = row;
    if (row >= 0 && s.row_weights != nullptr) s.row_weights[row] = __ldg(s.w + a);
    rows[i] = row;
  }
  __syncthreads();
  if (tid < 32) mv.run(rows, s.K);
  else fill_m_indices(s, st, ps, tid - 32, kThreads - 32);
}

// Small problems: every CTA ranks all slots itself.
template <int S>
__global__ void __launch_bounds__(kThreads) permute_small_kernel(PermuteArgs p) {
  extern __shared__ int32_t sm[];
  __shared__ int32_t s_wsum[33];
  __shared__ uint64_t s_bars[kMaxStages];
  __shared__ int s_desc[kMaxStages];
  const ScatterArgs& s = p.s;
  const int tid = threadIdx.x, lane = tid & 31;
  const int n_live = live_count(s.d_num_tokens, s.T, s.status, blockIdx.x == 0 && tid == 0);
  uint8_t* ring = reinterpret_cast<uint8_t*>(sm) + (small_layout_bytes(s) + 127) / 128 * 128;
  Mover mv(p, ring, s_bars, s_desc, tid < 32 ? own_tokens(n_live) : 0, tid < 32 ? lane : -1);
  if (tid < 32) mv.preload();
  small_layout<S>(s, sm, s_wsum, n_live);
  if (tid < 32) mv.run(small_rows(s, sm) + (int64_t)blockIdx.x * s.K, (int)gridDim.x * s.K);
}

template <typename Kern>
cudaError_t launch_ring(Kern kernel, PermuteArgs a, size_t plan, int64_t grid, bool pdl, cudaStream_t s) {
  const size_t smem = plan + (size_t)a.stages * a.unit_bytes;
  cudaError_t err = opt_in_smem(kernel, smem);
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
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_permute(const PermuteArgs& a0, int num_sms, bool after_route_plan, cudaStream_t s) {
  PermuteArgs a = a0;
  a.stages = kMaxStages;
  int64_t grid = a.s.T < 1 ? 1 : a.s.T;
  if (!after_route_plan) {
    const int64_t A = (int64_t)a.s.T * a.s.K;
    if (A > kSmallSlots) return cudaErrorInvalidValue;
    if (grid > 2 * num_sms) grid = 2 * num_sms;
    const size_t plan = (small_layout_bytes(a.s) + 127) / 128 * 128;
    if (A <= 256) return launch_ring(permute_small_kernel<1>, a, plan, grid, false, s);
    if (A <= 1024) return launch_ring(permute_small_kernel<4>, a, plan, grid, false, s);
    return launch_ring(permute_small_kernel<8>, a, plan, grid, false, s);
  }
  // as many CTAs per SM as the plan and the ring leave room for (the plan's
  // share per CTA shrinks with the number of CTAs)
  int sm_bytes = 0;
  cudaError_t err = device_attr_cached(cudaDevAttrMaxSharedMemoryPerMultiprocessor, &sm_bytes);
  if (err != cudaSuccess) return err;
  int per_sm = 4;
  size_t plan = 0;
  for (;; --per_sm) {
    const int64_t g = grid < (int64_t)num_sms * per_sm ? grid : (int64_t)num_sms * per_sm;
    plan = plan_bytes(a.s, (a.s.T + g - 1) / g);
    if (per_sm == 1 || (plan + (size_t)a.stages * a.unit_bytes + 2048) * per_sm <= (size_t)sm_bytes) {
      grid = g;
      break;
    }
  }
  return launch_ring(permute_kernel, a, plan, grid, true, s);
}

}  // namespace moeperm
