// block_norm.cu -- the norms before and after a block, fused with the block's
// gate, residual scale and residual sum, and their gradients.
//
//   n  = rms(y) * w_post            rms(v) = v * rstd(v), rstd(v) = (mean_h v^2 + eps)^-1/2
//   x' = x + scale * gate * n       gate per channel [H], per token [T], or 1
//   h  = rms(x') * w_pre            the next block's input
//
// (no y: x' = x; no w_post: n = y; no w_pre: no h). Gradients, for dx' and dh:
//
//   t  = dh * w_pre,  xh = x' * rstd_pre
//   g  = dx' + rstd_pre * (t - xh * mean(t * xh));   dx = g;   dw_pre = sum_t dh * xh
//   yh = y * rstd_post, n = yh * w_post, u = scale * gate * g
//   dgate = sum over t (or h) of scale * g * n;      dw_post = sum_t u * yh
//   dy = rstd_post * (u * w_post - yh * mean(u * w_post * yh))     (no w_post: dy = u)
//
// Both kernels read every tensor once and are bound by HBM. One CTA holds a
// row in registers, VPT 16-byte vectors per thread, so the two sums a row
// needs are the only synchronisation. All sums are in fp32; h is computed
// from x' before its rounding to the element type. The backward CTAs walk rows
// strided by the grid and keep the sums over tokens of their columns in
// registers; each CTA writes one row of partial sums per weight and a second
// small launch adds the rows in a fixed order, so results do not depend on
// timing.
#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"

namespace moeperm {

namespace {

// Sum over the CTA, in every thread; s: [2][32] floats, buf alternates between
// consecutive calls so that one barrier per call suffices.
template <int M>
__device__ __forceinline__ void block_sum(float (&v)[M], float (*s)[M][32], int buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int m = 0; m < M; ++m) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v[m] += __shfl_xor_sync(0xffffffffu, v[m], off);
    if (lane == 0) s[buf][m][warp] = v[m];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) {
    v[m] = lane < nw ? s[buf][m][lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v[m] += __shfl_xor_sync(0xffffffffu, v[m], off);
  }
}

template <int N>
__device__ __forceinline__ void load_f(float (&f)[N], const float* p) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(p + i));
    f[i] = q.x; f[i + 1] = q.y; f[i + 2] = q.z; f[i + 3] = q.w;
  }
}

template <int TYPE, int VPT>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs p) {
  using V = Vec<TYPE>;
  constexpr int N = V::kN;
  __shared__ float s_sum[2][1][32];
  const int tid = threadIdx.x, bd = blockDim.x;
  const int nv = p.H / N;
  const float inv_h = 1.0f / (float)p.H;
  const uint8_t* x = static_cast<const uint8_t*>(p.x);
  const uint8_t* y = static_cast<const uint8_t*>(p.y);
  const bool has_y = y != nullptr;
  int buf = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    float xf[VPT][N];
    uint4 yv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * bd + tid;
      uint4 v = make_uint4(0, 0, 0, 0);
      yv[i] = v;
      if (c < nv) {
        v = ld_nc_v4(x + (t * p.ldx + (int64_t)c * N) * V::kBytes);
        if (has_y) yv[i] = ld_nc_v4(y + (t * p.ldy + (int64_t)c * N) * V::kBytes);
      }
      V::unpack(v, xf[i]);
    }
    if (has_y) {
      float ry = 1.0f;
      if (p.w_post != nullptr) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          float f[N];
          V::unpack(yv[i], f);
#pragma unroll
          for (int j = 0; j < N; ++j) s[0] = __fmaf_rn(f[j], f[j], s[0]);
        }
        block_sum<1>(s, s_sum, buf);
        buf ^= 1;
        ry = rsqrtf(s[0] * inv_h + p.eps);
        if (tid == 0 && p.rstd_post != nullptr) p.rstd_post[t] = ry;
      }
      float sc = p.scale * ry;
      if (p.gate_mode == kGateToken) sc *= __ldg(p.gate + t);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = i * bd + tid;
        if (c >= nv) continue;
        float f[N];
        V::unpack(yv[i], f);
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] *= sc;
        if (p.w_post != nullptr) {
          float w[N];
          load_f(w, p.w_post + (int64_t)c * N);
#pragma unroll
          for (int j = 0; j < N; ++j) f[j] *= w[j];
        }
        if (p.gate_mode == kGateChannel) {
          float w[N];
          load_f(w, p.gate + (int64_t)c * N);
#pragma unroll
          for (int j = 0; j < N; ++j) f[j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) xf[i][j] += f[j];
        st_v4(static_cast<uint8_t*>(p.x_out) + (t * p.H + (int64_t)c * N) * V::kBytes, V::pack(xf[i]));
      }
    }
    if (p.w_pre != nullptr) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) s[0] = __fmaf_rn(xf[i][j], xf[i][j], s[0]);
      block_sum<1>(s, s_sum, buf);
      buf ^= 1;
      const float rx = rsqrtf(s[0] * inv_h + p.eps);
      if (tid == 0 && p.rstd_pre != nullptr) p.rstd_pre[t] = rx;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = i * bd + tid;
        if (c >= nv) continue;
        float w[N];
        load_f(w, p.w_pre + (int64_t)c * N);
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] *= xf[i][j] * rx;
        st_v4(static_cast<uint8_t*>(p.h) + (t * p.H + (int64_t)c * N) * V::kBytes, V::pack(w));
      }
    }
  }
}

template <int TYPE, int VPT>
__global__ void __launch_bounds__(512) norm_grad_kernel(NormArgs p) {
  using V = Vec<TYPE>;
  constexpr int N = V::kN;
  __shared__ float s_sum[2][2][32];
  const int tid = threadIdx.x, bd = blockDim.x;
  const int nv = p.H / N;
  const float inv_h = 1.0f / (float)p.H;
  const bool has_y = p.y != nullptr, post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  const bool gate_c = p.gate_mode == kGateChannel, gate_t = p.gate_mode == kGateToken;
  float a_pre[VPT][N], a_post[VPT][N], a_gate[VPT][N];  // sums over this CTA's tokens
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) a_pre[i][j] = a_post[i][j] = a_gate[i][j] = 0.0f;
  int buf = 0;
  auto row_ptr = [](const void* base, int64_t t, int64_t ld) {
    return static_cast<const uint8_t*>(base) + t * ld * V::kBytes;
  };
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 gv[VPT], xv[VPT], hv[VPT], yv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * bd + tid;
      const bool in = c < nv;
      gv[i] = in && p.dxo != nullptr ? ld_nc_v4(row_ptr(p.dxo, t, p.ld_dxo) + (int64_t)c * 16) : zero;
      xv[i] = in && pre ? ld_nc_v4(row_ptr(p.x, t, p.ldx) + (int64_t)c * 16) : zero;
      hv[i] = in && pre ? ld_nc_v4(row_ptr(p.dh, t, p.ld_dh) + (int64_t)c * 16) : zero;
      yv[i] = in && has_y ? ld_nc_v4(row_ptr(p.y, t, p.ldy) + (int64_t)c * 16) : zero;
    }
    float rx = 0.0f, m1 = 0.0f;
    if (pre) {
      rx = __ldg(p.rstd_pre + t);
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = i * bd + tid;
        if (c >= nv) continue;
        float x[N], d[N], w[N];
        V::unpack(xv[i], x);
        V::unpack(hv[i], d);
        load_f(w, p.w_pre + (int64_t)c * N);
#pragma unroll
        for (int j = 0; j < N; ++j) s[0] = __fmaf_rn(d[j] * w[j], x[j] * rx, s[0]);
      }
      block_sum<2>(s, s_sum, buf);
      buf ^= 1;
      m1 = s[0] * inv_h;
    }
    const float ry = post ? __ldg(p.rstd_post + t) : 1.0f;
    const float gt = has_y ? (gate_t ? __ldg(p.gate + t) : 1.0f) * p.scale : 0.0f;
    float u[VPT][N];                 // scale * gate * g, then u * w_post
    float s[2] = {0.0f, 0.0f};       // sum of u * w_post * yh; sum of scale * g * n
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * bd + tid;
      if (c >= nv) {
#pragma unroll
        for (int j = 0; j < N; ++j) u[i][j] = 0.0f;
        continue;
      }
      float g[N], f[N], w[N];
      V::unpack(gv[i], g);
      if (pre) {
        float d[N];
        V::unpack(xv[i], f);
        V::unpack(hv[i], d);
        load_f(w, p.w_pre + (int64_t)c * N);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float xh = f[j] * rx;
          g[j] = __fmaf_rn(rx, d[j] * w[j] - xh * m1, g[j]);
          a_pre[i][j] = __fmaf_rn(d[j], xh, a_pre[i][j]);
        }
      }
      st_v4(static_cast<uint8_t*>(p.dx) + (t * p.H + (int64_t)c * N) * V::kBytes, V::pack(g));
      if (!has_y) continue;
      float wp[N], gc[N];
      if (post) load_f(wp, p.w_post + (int64_t)c * N);
      if (gate_c) load_f(gc, p.gate + (int64_t)c * N);
      V::unpack(yv[i], f);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float yh = f[j] * ry;
        const float n = post ? yh * wp[j] : yh;
        const float sg = p.scale * g[j];
        if (gate_c) a_gate[i][j] = __fmaf_rn(sg, n, a_gate[i][j]);
        s[1] = __fmaf_rn(sg, n, s[1]);
        float v = gate_c ? sg * gc[j] : gt * g[j];
        if (post) {
          a_post[i][j] = __fmaf_rn(v, yh, a_post[i][j]);
          v *= wp[j];
          s[0] = __fmaf_rn(v, yh, s[0]);
        }
        u[i][j] = v;
      }
    }
    if (!has_y) continue;
    float m2 = 0.0f;
    if (post || gate_t) {
      block_sum<2>(s, s_sum, buf);
      buf ^= 1;
      m2 = post ? s[0] * inv_h : 0.0f;
      if (gate_t && tid == 0) p.dgate[t] = s[1];
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * bd + tid;
      if (c >= nv) continue;
      float f[N];
      V::unpack(yv[i], f);
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = ry * (u[i][j] - f[j] * ry * m2);
      st_v4(static_cast<uint8_t*>(p.dy) + (t * p.H + (int64_t)c * N) * V::kBytes, V::pack(f));
    }
  }
  auto put = [&](int which, const float (&a)[VPT][N]) {
    float* dst = p.ws + ((int64_t)which * p.parts + blockIdx.x) * p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * bd + tid;
      if (c < nv)
#pragma unroll
        for (int j = 0; j < N; j += 4)
          *reinterpret_cast<float4*>(dst + (int64_t)c * N + j) =
              make_float4(a[i][j], a[i][j + 1], a[i][j + 2], a[i][j + 3]);
    }
  };
  if (pre) put(0, a_pre);
  if (post) put(1, a_post);
  if (gate_c) put(2, a_gate);
}

constexpr int kSumCols = 32, kSumRows = 8;  // columns per CTA, row groups per column

// out[h] = sum over the partial rows, in a fixed order; blockIdx.y: which weight.
__global__ void __launch_bounds__(kSumCols * kSumRows) norm_sum_kernel(NormArgs p, int used) {
  __shared__ float s[kSumRows][kSumCols];
  const int col = threadIdx.x % kSumCols, grp = threadIdx.x / kSumCols;
  const int h = blockIdx.x * kSumCols + col;
  float* outs[3] = {p.w_pre != nullptr ? p.dw_pre : nullptr, p.w_post != nullptr ? p.dw_post : nullptr,
                    p.gate_mode == kGateChannel ? p.dgate : nullptr};
  float* out = outs[blockIdx.y];
  if (out == nullptr) return;  // uniform over the CTA
  const float* src = p.ws + (int64_t)blockIdx.y * p.parts * p.H + h;
  float acc = 0.0f;
  if (h < p.H)
#pragma unroll 8
    for (int r = grp; r < used; r += kSumRows) acc += __ldcg(src + (int64_t)r * p.H);
  s[grp][col] = acc;
  __syncthreads();
  if (grp == 0 && h < p.H) {
    for (int i = 1; i < kSumRows; ++i) acc += s[i][col];
    out[h] = acc;
  }
}

template <int TYPE, int VPT>
cudaError_t launch_vpt(const NormArgs& a, bool grad, int num_sms, cudaStream_t s) {
  const int nv = a.H / Vec<TYPE>::kN;
  const int bd = ((nv + VPT - 1) / VPT + 31) / 32 * 32;
  int per_sm = 0;
  cudaError_t err = grad ? occupancy(norm_grad_kernel<TYPE, VPT>, bd, 0, &per_sm)
                         : occupancy(norm_kernel<TYPE, VPT>, bd, 0, &per_sm);
  if (err != cudaSuccess) return err;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  int64_t grid = (int64_t)num_sms * per_sm;
  if (!grad) {
    if (grid > a.T) grid = a.T;
    norm_kernel<TYPE, VPT><<<(unsigned)grid, bd, 0, s>>>(a);
    return cudaGetLastError();
  }
  if (grid > a.parts) grid = a.parts;
  if (grid > a.T) grid = a.T;
  if (grid < 1) grid = 1;  // no rows: the sums are still written (zeros)
  norm_grad_kernel<TYPE, VPT><<<(unsigned)grid, bd, 0, s>>>(a);
  err = cudaGetLastError();
  if (err != cudaSuccess || (a.w_pre == nullptr && a.w_post == nullptr && a.gate_mode != kGateChannel)) return err;
  norm_sum_kernel<<<dim3((a.H + kSumCols - 1) / kSumCols, 3), kSumCols * kSumRows, 0, s>>>(a, (int)grid);
  return cudaGetLastError();
}

// Vectors per thread: the fewest that keep a row within 512 threads. Rows of up
// to 2048 vectors (16384 elements of 16 bits, 8192 of 32) are accepted.
template <int TYPE>
cudaError_t launch_type(const NormArgs& a, bool grad, int num_sms, cudaStream_t s) {
  const int nv = a.H / Vec<TYPE>::kN;
  if (nv <= 512) return launch_vpt<TYPE, 1>(a, grad, num_sms, s);
  if (nv <= 1024) return launch_vpt<TYPE, 2>(a, grad, num_sms, s);
  if (nv <= 2048) return launch_vpt<TYPE, 4>(a, grad, num_sms, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch(const NormArgs& a, int type, bool grad, int num_sms, cudaStream_t s) {
  if (type == kF16) return launch_type<kF16>(a, grad, num_sms, s);
  if (type == kF32) return launch_type<kF32>(a, grad, num_sms, s);
  return launch_type<kBF16>(a, grad, num_sms, s);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int type, int num_sms, cudaStream_t s) {
  return launch(a, type, false, num_sms, s);
}
cudaError_t launch_block_norm_grad(const NormArgs& a, int type, int num_sms, cudaStream_t s) {
  return launch(a, type, true, num_sms, s);
}

}  // namespace moeperm
