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
// products that follow take 16-bit operands. Bound by HBM (reads dout and P,
// writes dP). Without an activation dP = dout and only the sums are formed.
#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"

namespace moeperm {

namespace {

constexpr int kThreads = 256, kStrip = 128, kRowLanes = kThreads / 16, kRows = 2;

// (act(v), act'(v))
__device__ __forceinline__ float2 act_and_slope(float v, int act) {
  if (act == kActRelu) return v > 0.0f ? make_float2(v, 1.0f) : make_float2(0.0f, 0.0f);
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

template <int TYPE>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(ActGradArgs p) {
  __shared__ float s_sum[kRowLanes][kStrip + 4];
  const int tid = threadIdx.x, rl = tid >> 4, col = blockIdx.x * kStrip + (tid & 15) * 8;
  const int e = blockIdx.y, Nw = p.gated ? 2 * p.N : p.N;
  int64_t b = 0, c = p.R;
  if (p.cap > 0) {
    b = (int64_t)e * p.cap;
    c = __ldg(p.seg_end + e);
  } else if (p.seg_begin != nullptr) {
    b = __ldg(p.seg_begin + e);
    c = (int64_t)__ldg(p.seg_end + e) - b;
  }
  if (b < 0 || c < 0 || b + c > p.R || (p.cap > 0 && c > p.cap)) {
    if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0) set_status(p.status, kStBadLayout);
    b = c = 0;
  }
  const int64_t lo = b + c * blockIdx.z / p.splits, hi = b + c * (blockIdx.z + 1) / p.splits;
  const uint16_t* dout = static_cast<const uint16_t*>(p.dout);
  const uint16_t* pre = static_cast<const uint16_t*>(p.pre);
  uint16_t* dpre = static_cast<uint16_t*>(p.dpre);
  float s0[8], s1[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s0[j] = s1[j] = 0.0f;
  // kRows rows at once, their loads issued before the arithmetic
  for (int64_t r0 = lo + rl; r0 < hi && col < p.N; r0 += kRows * kRowLanes) {
    uint4 dv[kRows], pv[kRows], uv[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = r0 + i * kRowLanes;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const bool in = r < hi;
      dv[i] = in ? ld_nc_v4(dout + r * p.ldd + col) : zero;
      pv[i] = in && dpre != nullptr ? ld_nc_v4(pre + r * p.ld_pre + col) : zero;
      uv[i] = in && p.gated ? ld_nc_v4(pre + r * p.ld_pre + p.N + col) : zero;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = r0 + i * kRowLanes;
      if (r >= hi) break;
      float d[8];
      Vec<TYPE>::unpack(dv[i], d);
      if (dpre == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s0[j] += d[j];
        continue;
      }
      float v[8], u[8];
      Vec<TYPE>::unpack(pv[i], v);
      Vec<TYPE>::unpack(uv[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 a = act_and_slope(v[j], p.act);
        v[j] = p.gated ? d[j] * u[j] * a.y : d[j] * a.y;
        u[j] = d[j] * a.x;
        s0[j] += v[j];
        s1[j] += u[j];
      }
      st_v4(dpre + r * Nw + col, Vec<TYPE>::pack(v));
      if (p.gated) st_v4(dpre + r * Nw + p.N + col, Vec<TYPE>::pack(u));
    }
  }
  if (p.dbias == nullptr) return;  // uniform over the grid
  float* dst = (p.splits > 1 ? p.ws + (int64_t)blockIdx.z * p.L * Nw : p.dbias) + (int64_t)e * Nw;
  for (int half = 0; half < (p.gated ? 2 : 1); ++half) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sum[rl][(tid & 15) * 8 + j] = half ? s1[j] : s0[j];
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
