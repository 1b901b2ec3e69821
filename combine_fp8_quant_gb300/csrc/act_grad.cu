// act_grad.cu -- gradient of the experts' activation and gate, with the bias
// gradient:
//
//   P = x W^T + b, out = act(P)              dP = dout * act'(P)
//   gated: out = act(P[:N]) * P[N:]          dP[:N] = dout * P[N:] * act'(P[:N])
//                                            dP[N:] = dout * act(P[:N])
//   db_e = sum over the rows of e of dP      (fp32, of dP before its rounding)
//
// One CTA takes a strip of 128 columns of an expert's rows (one of `splits`
// equal runs of them); 16 threads cover the strip with 16-byte vectors and 16
// rows go at once. Each thread keeps its columns' sums in registers; with
// splits > 1 the partial sums go to the workspace and a second launch adds them
// in a fixed order. dP is rounded to the rows' 16-bit type because the two
// products that follow take 16-bit operands; with few rows, or for a weight gradient
// in fp32, what the rounding left over follows as a second term. Bound by HBM (reads
// dout and P, writes dP): 16382 rows of 1408 gated features, 230 MB in 40 us, 5.8 TB/s
// (52 us with loads straight to registers). Without an activation dP = dout and only
// the sums are formed.
#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "segments.cuh"

namespace moeperm {

namespace {

constexpr int kThreads = 256, kStrip = 128, kCols = kStrip / 8, kRowLanes = kThreads / kCols;
constexpr int kSlots = 3;  // rows of a thread in flight and in work

// (act(v), act'(v))
__device__ __forceinline__ float2 act_and_slope(float v, int act) {
  if (act == kActRelu) return v <= 0.0f ? make_float2(0.0f, 0.0f) : make_float2(v, 1.0f);  // NaN: (NaN, 1)
  if (act == kActSilu) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-v));
    return make_float2(v * s, s * (1.0f + v * (1.0f - s)));
  }
  if (act == kActGelu) {
    const float c = normcdff(v);
    return make_float2(v * c, c + v * 0.3989422804014327f * __expf(-0.5f * v * v));
  }
  return make_float2(v, 1.0f);
}

// Eight rounded values and, `rest` elements on (0: not at all), the rounding of
// what that left over.
template <int TYPE>
__device__ __forceinline__ void put(uint16_t* dst, const float (&v)[8], int64_t rest) {
  const uint4 q = Vec<TYPE>::pack(v);
  st_v4(dst, q);
  if (rest == 0) return;
  float f[8];
  Vec<TYPE>::unpack(q, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = isfinite(f[j]) ? v[j] - f[j] : 0.0f;  // nothing is left over of an overflow
  st_v4(dst + rest, Vec<TYPE>::pack(f));
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 3) act_grad_kernel(ActGradArgs p) {
  __shared__ uint4 s_ring[kSlots][3][kThreads];
  __shared__ float s_sum[kRowLanes][kStrip + 4];
  __shared__ int s_held[kThreads / 32];
  const int tid = threadIdx.x, rl = tid / kCols, col = blockIdx.x * kStrip + (tid % kCols) * 8;
  const int e = blockIdx.y, Nw = p.gated ? 2 * p.N : p.N;
  int64_t b, c;
  bool bad = !segment(p, e, b, c);
  const int64_t lo = b + c * blockIdx.z / p.splits;
  int64_t hi = b + c * (blockIdx.z + 1) / p.splits;
  const uint16_t* dout = static_cast<const uint16_t*>(p.dout);
  const uint16_t* pre = static_cast<const uint16_t*>(p.pre);
  uint16_t* dpre = static_cast<uint16_t*>(p.dpre);
  float s0[8], s1[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s0[j] = s1[j] = 0.0f;
  // this thread's vectors of the next kSlots - 1 rows are in flight while it works
  // on one (the slots are private to the thread: no barrier)
  const bool has_act = dpre != nullptr;
  auto fetch = [&](int64_t r, int slot) {
    if (r < hi) {
      cp_async16(&s_ring[slot][0][tid], dout + r * p.ldd + col);
      if (has_act) cp_async16(&s_ring[slot][1][tid], pre + r * p.ld_pre + col);
      if (p.gated) cp_async16(&s_ring[slot][2][tid], pre + r * p.ld_pre + p.N + col);
    }
    cp_async_commit();
  };
  if (col < p.N) {
#pragma unroll
    for (int i = 0; i + 1 < kSlots; ++i) fetch(lo + rl + i * kRowLanes, i);
  }
  // A segment that shares rows with an earlier one counts as empty, as it does for the
  // products. Its rows' dP is the same from either, so only the sums need to know.
  const bool sums = p.dbias != nullptr && p.seg_begin != nullptr, count = p.terms == kTermsByRows;
  int terms = p.terms;
  if (sums || count) {
    bool hit = false;
    int held = 0;
    for (int f = tid; f < (count ? p.L : e); f += kThreads) {
      int64_t bf, cf;
      segment(p, f, bf, cf);
      held += rows_held(cf);
      hit |= sums && f < e && share_rows(b, c, bf, cf);
    }
    held = __reduce_add_sync(0xffffffffu, held);
    if (tid % 32 == 0) s_held[tid / 32] = held;
    bad |= __syncthreads_or(hit) != 0;
    if (count) {
      held = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) held += s_held[i];
      terms = terms_of(held, p.L);
    }
  }
  const int64_t rest = terms > 1 ? p.R * Nw : 0;
  if (bad) {
    if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0) set_status(p.status, kStBadLayout);
    cp_async_wait_all();
    hi = lo;
  }
  if (col < p.N) {
    int64_t r = lo + rl;
    int slot = 0;
    for (; r < hi; r += kRowLanes) {
      fetch(r + (kSlots - 1) * kRowLanes, slot == 0 ? kSlots - 1 : slot - 1);
      cp_async_wait_group<kSlots - 1>();
      float d[8];
      Vec<TYPE>::unpack(s_ring[slot][0][tid], d);
      if (!has_act) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s0[j] += d[j];
      } else {
        float v[8], u[8];
        Vec<TYPE>::unpack(s_ring[slot][1][tid], v);
        if (p.gated) Vec<TYPE>::unpack(s_ring[slot][2][tid], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 a = act_and_slope(v[j], p.act);
          v[j] = p.gated ? d[j] * u[j] * a.y : d[j] * a.y;
          u[j] = d[j] * a.x;
          s0[j] += v[j];
          s1[j] += u[j];
        }
        put<TYPE>(dpre + r * Nw + col, v, rest);
        if (p.gated) put<TYPE>(dpre + r * Nw + p.N + col, u, rest);
      }
      if (++slot == kSlots) slot = 0;
    }
  }
  if (p.dbias == nullptr) return;  // uniform over the grid
  float* dst = (p.splits > 1 ? p.ws + (int64_t)blockIdx.z * p.L * Nw : p.dbias) + (int64_t)e * Nw;
  for (int half = 0; half < (p.gated ? 2 : 1); ++half) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sum[rl][(tid % kCols) * 8 + j] = half ? s1[j] : s0[j];
    __syncthreads();
    const int h = blockIdx.x * kStrip + tid;
    if (tid < kStrip && h < p.N) {
      float acc = 0.0f;
#pragma unroll
      for (int i = 0; i < kRowLanes; ++i) acc += s_sum[i][tid];
      dst[half * p.N + h] = acc;
    }
  }
}

__global__ void bias_sum_kernel(const float* ws, float* dbias, int64_t n, int splits) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float acc = 0.0f;
  for (int s = 0; s < splits; ++s) acc += __ldcg(ws + (int64_t)s * n + i);
  dbias[i] = acc;
}

}  // namespace

// Runs per expert: enough CTAs for the GPU (eight per SM at 152 SMs) from
// host-known sizes, at least 64 rows each on average and at most kActGradSplits.
int act_grad_splits(int64_t R, int32_t L, int32_t N) {
  const int64_t strips = (N + kStrip - 1) / kStrip;
  int64_t s = (8 * 152 + L * strips - 1) / (L * strips);
  const int64_t most = R / L / 64;
  if (s > most) s = most;
  if (s > kActGradSplits) s = kActGradSplits;
  return s < 1 ? 1 : (int)s;
}

cudaError_t launch_act_grad(const ActGradArgs& a, int type, cudaStream_t s) {
  const dim3 grid((a.N + kStrip - 1) / kStrip, a.L, a.splits);
  if (type == kF16) act_grad_kernel<kF16><<<grid, kThreads, 0, s>>>(a);
  else act_grad_kernel<kBF16><<<grid, kThreads, 0, s>>>(a);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || a.dbias == nullptr || a.splits == 1) return err;
  const int64_t n = (int64_t)a.L * (a.gated ? 2 * a.N : a.N);
  bias_sum_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a.ws, a.dbias, n, a.splits);
  return cudaGetLastError();
}

}  // namespace moeperm
