// combine_grad.cu -- gradients of the weighted combine.
//
//   out[t] = sum_k w[t,k] * y[row(t,k)]     (combine.cu)
//   dy[row(t,k)] = w[t,k] * dout[t]
//   dw[t,k]      = sum_h dout[t,h] * y[row(t,k),h]      (fp32)
//
// Each kept row belongs to one slot, so both gradients are written by the CTA
// that owns the token and nothing is accumulated across CTAs: the result does
// not depend on the launch.
//
// One CTA walks a token at a time, each thread a column of 16-byte chunks. A
// token's slots go in batches of kBatch rows: their loads are all issued
// before the first product, and dout stays in L1 for the batches after the
// first. The dot products are summed in fp32 per thread, per warp by shuffles
// and per token through shared memory (double buffered: one barrier a token).
// CTAs of at most 256 threads, four to an SM, keep each other's reductions covered
// (fp32, 1777 x 2048, top-6: 28 us, against 47 with 512 threads). Bound by HBM:
// T*H + kept*H elements read, kept*H written; 8192 x 7168 bf16, top-8: 1.99 GB in
// 304 us, 6.6 TB/s.
#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"

namespace moeperm {

namespace {

constexpr int kBatch = 4;    // rows in flight per thread and chunk
constexpr int kMaxSlots = 32;
constexpr int kMaxThreads = 256;

template <int TYPE>
__global__ void __launch_bounds__(kMaxThreads, 4) combine_grad_kernel(CombineGradArgs p) {
  constexpr int N = Vec<TYPE>::kN;
  __shared__ float s_part[2][kMaxSlots][kMaxThreads / 32 + 1];  // [slot][warp], padded
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bd = blockDim.x, nw = bd >> 5;
  const int nch = p.H / N;
  const int n_live = live_count(p.d_num_tokens, p.T, p.status, blockIdx.x == 0 && tid == 0);
  const uint8_t* dout = static_cast<const uint8_t*>(p.dout);
  const uint8_t* y = static_cast<const uint8_t*>(p.y);
  uint8_t* dy = static_cast<uint8_t*>(p.dy);
  const int64_t ldd = p.ldd * Vec<TYPE>::kBytes, ldy = p.ldy * Vec<TYPE>::kBytes;
  const int64_t lddy = p.lddy * Vec<TYPE>::kBytes;
  const bool need_dw = p.dw != nullptr;
  int buf = 0;
  for (int t = blockIdx.x; t < n_live; t += gridDim.x, buf ^= 1) {
    // lane k holds slot k (every warp reads them: K <= 32 words, in L1)
    int myrow = -1;
    float myw = 0.0f;
    if (lane < p.K) {
      const int64_t a = (int64_t)t * p.K + lane;
      myrow = __ldg(p.src2dst + a);
      if (myrow >= 0 && (int64_t)myrow >= p.R) {
        if (warp == 0) set_status(p.status, kStBadLayout);
        myrow = -1;
      }
      myw = p.w != nullptr ? __ldg(p.w + a) : 1.0f;
    }
    const uint8_t* drow = dout + (int64_t)t * ldd;
    for (int k0 = 0; k0 < p.K; k0 += kBatch) {
      int row[kBatch];
      float w[kBatch], acc[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int k = k0 + j;
        const int r = __shfl_sync(0xffffffffu, myrow, k & 31);
        w[j] = __shfl_sync(0xffffffffu, myw, k & 31);
        row[j] = k < p.K ? r : -1;
        acc[j] = 0.0f;
      }
      for (int c = tid; c < nch; c += bd) {
        const uint4 gv = *reinterpret_cast<const uint4*>(drow + (int64_t)c * 16);
        uint4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          v[j] = (need_dw && row[j] >= 0) ? ld_nc_v4(y + (int64_t)row[j] * ldy + (int64_t)c * 16)
                                          : make_uint4(0, 0, 0, 0);
        float g[N];
        Vec<TYPE>::unpack(gv, g);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (row[j] < 0) continue;
          float f[N];
          if (need_dw) {
            Vec<TYPE>::unpack(v[j], f);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[j] = __fmaf_rn(g[i], f[i], acc[j]);
          }
          if (dy != nullptr) {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = __fmul_rn(w[j], g[i]);
            st_v4(dy + (int64_t)row[j] * lddy + (int64_t)c * 16, Vec<TYPE>::pack(f));
          }
        }
      }
      if (need_dw) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], off);
          if (lane == 0 && k0 + j < p.K) s_part[buf][k0 + j][warp] = acc[j];
        }
      }
    }
    if (need_dw) {
      __syncthreads();
      // the other buffer is free again once this barrier has been passed
      if (tid < p.K) {
        float sum = 0.0f;
        for (int i = 0; i < nw; ++i) sum += s_part[buf][tid][i];
        p.dw[(int64_t)t * p.K + tid] = sum;
      }
    }
  }
}

template <int TYPE>
cudaError_t launch_type(const CombineGradArgs& a, int num_sms, cudaStream_t s) {
  const int nch = a.H / Vec<TYPE>::kN;
  const int per_thread = (nch + kMaxThreads - 1) / kMaxThreads;  // chunks per thread, of equal count
  int bd = ((nch + per_thread - 1) / per_thread + 31) / 32 * 32;
  int per_sm = 0;
  cudaError_t err = occupancy(combine_grad_kernel<TYPE>, bd, 0, &per_sm);
  if (err != cudaSuccess) return err;
  if (per_sm < 1) per_sm = 1;
  int64_t grid = (int64_t)num_sms * per_sm;
  if (grid > a.T) grid = a.T;
  combine_grad_kernel<TYPE><<<(unsigned)grid, bd, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_combine_grad(const CombineGradArgs& a, int type, int num_sms, cudaStream_t s) {
  if (type == kF16) return launch_type<kF16>(a, num_sms, s);
  if (type == kF32) return launch_type<kF32>(a, num_sms, s);
  return launch_type<kBF16>(a, num_sms, s);
}

}  // namespace moeperm
