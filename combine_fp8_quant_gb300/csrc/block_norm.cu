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
// Both kernels read every tensor once. Forward is bound by HBM (8192 x 7168 in bf16:
// 470 MB in 83 us, 5.7 TB/s); backward (705 MB in 136 us, 5.2 TB/s) HBM is busy 62% and
// issue 45% of the time, and a row's reduction and barrier with one CTA on an SM are
// what it waits for. One CTA holds a row, 8
// (or 16) elements per thread, and walks rows strided by the grid. The rows to
// come arrive by asynchronous copies in a ring of shared memory whose slots are
// private to each thread (a thread copies and reads its own vectors), so loads
// stay in flight across the row's sums without a barrier of their own; weights
// of a thread's columns stay in registers for all rows.
//
// The arithmetic is packed (fma.rn.f32x2: two 32-bit multiply-adds an issue slot).
// Backward, the two sums of a row become one reduction: with c = scale * gate *
// w_post, P = sum t * x', B = sum c * y * (dx' + rstd_pre * t), C = sum c * y * x',
//   sum over h of u * w_post * y = B - (rstd_pre^3 * P / H) * C
// And since gate and w_post of a column do not depend on the token,
// Q = sum_t scale * g * yh gives both dw_post = gate * Q and dgate = w_post * Q.
// The sums over tokens stay in registers; each CTA writes one row of partial
// sums and a second small launch adds the rows in a fixed order, so results do
// not depend on timing. All sums are in fp32; h is computed from x' before its
// rounding to the element type.
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

// The ring: `slots` rows, each of nt tensors of VPT vectors per thread.
constexpr int kMaxSlots = 3;
__device__ __forceinline__ void wait_slots(int slots) {  // the oldest of `slots` groups has landed
  switch (slots) {
    case 1: cp_async_wait_group<0>(); break;
    case 2: cp_async_wait_group<1>(); break;
    default: cp_async_wait_group<2>(); break;
  }
}

// Column weights of this thread as pairs: w[i][j], 1 where p is null.
template <int N, int VPT>
__device__ __forceinline__ void load_cols(f32x2 (&w)[VPT][N / 2], const float* p, int nv) {
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      w[i][j] = pair(1.0f, 1.0f);
      if (p != nullptr && c < nv) {
        const float2 q = __ldg(reinterpret_cast<const float2*>(p + (int64_t)c * N) + j);
        w[i][j] = pair(q.x, q.y);
      }
    }
  }
}
// c = scale * gate (per channel) * w_post of this thread's columns.
template <int N, int VPT>
__device__ __forceinline__ void load_post(f32x2 (&c)[VPT][N / 2], const NormArgs& p, int nv) {
  f32x2 g[VPT][N / 2];
  load_cols<N>(c, p.w_post, nv);
  load_cols<N>(g, p.gate_mode == kGateChannel ? p.gate : nullptr, nv);
  const f32x2 s = pair(p.scale, p.scale);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N / 2; ++j) c[i][j] = mul2(mul2(c[i][j], s), g[i][j]);
}
__device__ __forceinline__ float sum_halves(f32x2 v) {
  const float2 h = halves(v);
  return h.x + h.y;
}

// One tensor's rows on their way through the ring: the global address of this
// thread's first vector in the next row to fetch.
struct Stream {
  const uint8_t* p;
  int64_t step;  // bytes from one of this CTA's rows to the next
};
template <int TYPE>
__device__ __forceinline__ Stream stream(const void* base, int64_t ld) {
  return {static_cast<const uint8_t*>(base) + ((int64_t)blockIdx.x * ld + (int64_t)threadIdx.x * Vec<TYPE>::kN) * Vec<TYPE>::kBytes,
          (int64_t)gridDim.x * ld * Vec<TYPE>::kBytes};
}
template <int VPT>
__device__ __forceinline__ void fetch(Stream& s, uint4* slot, int nv) {  // and move on to the next row
  const int bd = blockDim.x;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (i * bd + (int)threadIdx.x < nv) cp_async16(slot + i * bd, s.p + (int64_t)i * bd * 16);
  s.p += s.step;
}

// kAll: y, w_post and w_pre are all given (the kernel then has no tests for them).
// kForwardRows rows go through the two reductions together: half the barriers
// per row, and two independent chains between them.
constexpr int kForwardRows = 2;
template <int TYPE, int VPT, int MAXT, bool kAll>
__global__ void __launch_bounds__(MAXT) norm_kernel(NormArgs p, int slots) {
  using V = Vec<TYPE>;
  constexpr int N = V::kN, P = V::kP, R = kForwardRows;
  extern __shared__ uint4 s_ring[];
  __shared__ float s_sum[2][R][32];
  const int tid = threadIdx.x, bd = blockDim.x;
  const int nv = p.H / N;
  const float inv_h = 1.0f / (float)p.H;
  const bool has_y = kAll || p.y != nullptr, post = kAll || p.w_post != nullptr, pre = kAll || p.w_pre != nullptr;
  const int oy = VPT * bd, row_vecs = (has_y ? 2 : 1) * VPT * bd, slot_vecs = R * row_vecs;  // in vectors of the ring
  Stream sx = stream<TYPE>(p.x, p.ldx), sy = stream<TYPE>(p.y, p.ldy);
  uint4* const ring = s_ring + tid;
  const int64_t step = gridDim.x;
  auto fetch_rows = [&](int64_t t, int slot) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (t + r * step < p.T) {
        uint4* row = ring + slot * slot_vecs + r * row_vecs;
        fetch<VPT>(sx, row, nv);
        if (has_y) fetch<VPT>(sy, row + oy, nv);
      }
    cp_async_commit();
  };
  int64_t t = blockIdx.x;
  for (int i = 0; i + 1 < slots; ++i) fetch_rows(t + i * R * step, i);
  f32x2 cw[VPT][P], wp[VPT][P];
  load_post<N>(cw, p, nv);
  load_cols<N>(wp, p.w_pre, nv);
  int buf = 0, slot = 0;
  for (; t < p.T; t += R * step) {
    fetch_rows(t + (slots - 1) * R * step, slot == 0 ? slots - 1 : slot - 1);  // over the rows before these
    wait_slots(slots);
    const uint4* row = ring + slot * slot_vecs;
    if (++slot == slots) slot = 0;
    f32x2 x[R][VPT][P];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i * bd + tid < nv) v = row[r * row_vecs + i * bd];
        V::unpack2(v, x[r][i]);
      }
    if (has_y) {
      f32x2 y[R][VPT][P];
      float s[R], q[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        f32x2 a2 = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (i * bd + tid < nv) v = row[r * row_vecs + oy + i * bd];
          V::unpack2(v, y[r][i]);
#pragma unroll
          for (int j = 0; j < P; ++j) a2 = fma2(y[r][i][j], y[r][i][j], a2);
        }
        s[r] = sum_halves(a2);
      }
      if (post) {
        block_sum<R>(s, s_sum, buf);
        buf ^= 1;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t tr = t + r * step;
        q[r] = post ? rsqrtf(s[r] * inv_h + p.eps) : 1.0f;
        if (tid == 0 && post && p.rstd_post != nullptr && tr < p.T) p.rstd_post[tr] = q[r];
        if (p.gate_mode == kGateToken && tr < p.T) q[r] *= __ldg(p.gate + tr);
        const f32x2 q2 = pair(q[r], q[r]);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
          for (int j = 0; j < P; ++j) x[r][i][j] = fma2(mul2(y[r][i][j], q2), cw[i][j], x[r][i][j]);
          if (i * bd + tid < nv && tr < p.T)
            st_v4(static_cast<uint8_t*>(p.x_out) + (tr * nv + i * bd + tid) * 16, V::pack2(x[r][i]));
        }
      }
    }
    if (pre) {
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        f32x2 a2 = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int j = 0; j < P; ++j) a2 = fma2(x[r][i][j], x[r][i][j], a2);
        s[r] = sum_halves(a2);
      }
      block_sum<R>(s, s_sum, buf);
      buf ^= 1;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t tr = t + r * step;
        const float q = rsqrtf(s[r] * inv_h + p.eps);
        if (tr >= p.T) continue;
        if (tid == 0 && p.rstd_pre != nullptr) p.rstd_pre[tr] = q;
        const f32x2 q2 = pair(q, q);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
          for (int j = 0; j < P; ++j) x[r][i][j] = mul2(x[r][i][j], mul2(q2, wp[i][j]));
          if (i * bd + tid < nv)
            st_v4(static_cast<uint8_t*>(p.h) + (tr * nv + i * bd + tid) * 16, V::pack2(x[r][i]));
        }
      }
    }
  }
}

// kAll: dx', y, w_post and w_pre are all given.
template <int TYPE, int VPT, int MAXT, bool kAll>
__global__ void __launch_bounds__(MAXT) norm_grad_kernel(NormArgs p, int slots) {
  using V = Vec<TYPE>;
  constexpr int N = V::kN, P = V::kP;
  extern __shared__ uint4 s_ring[];
  __shared__ float s_sum[2][3][32];
  const int tid = threadIdx.x, bd = blockDim.x;
  const int nv = p.H / N;
  const float inv_h = 1.0f / (float)p.H;
  const bool has_g = kAll || p.dxo != nullptr, has_y = kAll || p.y != nullptr;
  const bool post = kAll || p.w_post != nullptr, pre = kAll || p.w_pre != nullptr;
  const bool gate_t = p.gate_mode == kGateToken;
  // tensors of a row in the ring, in vectors: dx', y, x', dh
  const int oy = has_g ? VPT * bd : 0, ox = oy + (has_y ? VPT * bd : 0), od = ox + VPT * bd;
  const int row_vecs = ox + (pre ? 2 * VPT * bd : 0);
  Stream sg = stream<TYPE>(p.dxo, p.ld_dxo), sy = stream<TYPE>(p.y, p.ldy), sx = stream<TYPE>(p.x, p.ldx),
         sd = stream<TYPE>(p.dh, p.ld_dh);
  uint4* const ring = s_ring + tid;
  auto fetch_row = [&](int64_t t, int slot) {
    if (t < p.T) {
      uint4* row = ring + slot * row_vecs;
      if (has_g) fetch<VPT>(sg, row, nv);
      if (has_y) fetch<VPT>(sy, row + oy, nv);
      if (pre) {
        fetch<VPT>(sx, row + ox, nv);
        fetch<VPT>(sd, row + od, nv);
      }
    }
    cp_async_commit();
  };
  const int64_t step = gridDim.x;
  int64_t t = blockIdx.x;
  for (int i = 0; i + 1 < slots; ++i) fetch_row(t + i * step, i);
  f32x2 cw[VPT][P], wp[VPT][P], a_pre[VPT][P], a_q[VPT][P];
  load_post<N>(cw, p, nv);
  load_cols<N>(wp, p.w_pre, nv);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) a_pre[i][j] = a_q[i][j] = 0;
  int buf = 0, slot = 0;
  for (; t < p.T; t += step) {
    fetch_row(t + (slots - 1) * step, slot == 0 ? slots - 1 : slot - 1);  // over the row before this one
    const float rx = pre ? __ldg(p.rstd_pre + t) : 0.0f;
    const float ry = post ? __ldg(p.rstd_post + t) : 1.0f;
    const float gt = gate_t ? __ldg(p.gate + t) : 1.0f;
    wait_slots(slots);
    const uint4* row = ring + slot * row_vecs;
    if (++slot == slots) slot = 0;
    const f32x2 rx2 = pair(rx, rx);
    f32x2 s0 = 0, s1 = 0, s2 = 0;  // P, B, C
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (pre || post || gate_t) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * bd + tid >= nv) continue;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        f32x2 g[P], y[P];
        V::unpack2(has_g ? row[i * bd] : zero, g);
        V::unpack2(has_y ? row[oy + i * bd] : zero, y);
        if (pre) {
          f32x2 x[P], d[P];
          V::unpack2(row[ox + i * bd], x);
          V::unpack2(row[od + i * bd], d);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const f32x2 tt = mul2(d[j], wp[i][j]), e = mul2(cw[i][j], y[j]);
            s0 = fma2(tt, x[j], s0);
            s1 = fma2(e, fma2(rx2, tt, g[j]), s1);
            s2 = fma2(e, x[j], s2);
          }
        } else {
#pragma unroll
          for (int j = 0; j < P; ++j) s1 = fma2(mul2(cw[i][j], y[j]), g[j], s1);
        }
      }
      s[0] = sum_halves(s0);
      s[1] = sum_halves(s1);
      s[2] = sum_halves(s2);
      block_sum<3>(s, s_sum, buf);
      buf ^= 1;
    }
    // The sums first, then one rstd after the other: rstd^3 alone leaves the range of
    // fp32 for rows of 1e-13 and of 1e15, whose gradients are ordinary numbers.
    const float k1 = rx * s[0] * inv_h * rx * rx;  // g = dx' + rx * t - k1 * x'
    const float dot = s[1] - k1 * s[2];            // sum of scale * gate_c * w_post * y * g
    if (gate_t && has_y && tid == 0) p.dgate[t] = dot * ry;
    const float k2 = post ? ry * dot * inv_h * ry : 0.0f;  // dy = gt * ry * (c * g - k2 * y)
    const float gry = gt * ry, kq = p.scale * gry;
    const f32x2 nk1 = pair(-k1, -k1), nk2 = pair(-k2, -k2), gry2 = pair(gry, gry), kq2 = pair(kq, kq);
    const int64_t out0 = (t * nv + tid) * 16;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (i * bd + tid >= nv) continue;
      f32x2 g[P];
      V::unpack2(has_g ? row[i * bd] : make_uint4(0, 0, 0, 0), g);
      if (pre) {
        f32x2 x[P], d[P];
        V::unpack2(row[ox + i * bd], x);
        V::unpack2(row[od + i * bd], d);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const f32x2 dr = mul2(d[j], rx2);
          g[j] = fma2(nk1, x[j], fma2(dr, wp[i][j], g[j]));
          a_pre[i][j] = fma2(dr, x[j], a_pre[i][j]);
        }
      }
      st_v4(static_cast<uint8_t*>(p.dx) + out0 + (int64_t)i * bd * 16, V::pack2(g));
      if (!has_y) continue;
      f32x2 y[P];
      V::unpack2(row[oy + i * bd], y);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        a_q[i][j] = fma2(mul2(kq2, g[j]), y[j], a_q[i][j]);
        y[j] = mul2(gry2, fma2(nk2, y[j], mul2(cw[i][j], g[j])));
      }
      st_v4(static_cast<uint8_t*>(p.dy) + out0 + (int64_t)i * bd * 16, V::pack2(y));
    }
  }
  auto put = [&](int which, const f32x2 (&a)[VPT][P]) {
    float* dst = p.ws + ((int64_t)which * p.parts + blockIdx.x) * p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * bd + tid;
      if (c < nv)
#pragma unroll
        for (int j = 0; j < P; ++j) reinterpret_cast<float2*>(dst + (int64_t)c * N)[j] = halves(a[i][j]);
    }
  };
  if (pre) put(0, a_pre);
  if (post || p.gate_mode == kGateChannel) put(1, a_q);
}

constexpr int kSumCols = 32, kSumRows = 16;  // columns per CTA, row groups per column

// Column sums of the partial rows in a fixed order. blockIdx.y = 0: dw_pre;
// 1: Q, which gives dw_post and the gate's gradient per channel.
__global__ void __launch_bounds__(kSumCols * kSumRows) norm_sum_kernel(NormArgs p, int used) {
  __shared__ float s[kSumRows][kSumCols];
  const bool q = blockIdx.y == 1, gate_c = p.gate_mode == kGateChannel;
  if (q ? (p.w_post == nullptr && !gate_c) : p.w_pre == nullptr) return;  // uniform over the CTA
  const int col = threadIdx.x % kSumCols, grp = threadIdx.x / kSumCols;
  const int h = blockIdx.x * kSumCols + col;
  const float* src = p.ws + (int64_t)blockIdx.y * p.parts * p.H + h;
  float acc = 0.0f;
  if (h < p.H)
#pragma unroll 10
    for (int r = grp; r < used; r += kSumRows) acc += __ldcg(src + (int64_t)r * p.H);
  s[grp][col] = acc;
  __syncthreads();
  if (grp != 0 || h >= p.H) return;
  for (int i = 1; i < kSumRows; ++i) acc += s[i][col];
  if (!q) {
    p.dw_pre[h] = acc;
    return;
  }
  if (p.w_post != nullptr) p.dw_post[h] = gate_c ? acc * __ldg(p.gate + h) : acc;
  if (gate_c) p.dgate[h] = p.w_post != nullptr ? acc * __ldg(p.w_post + h) : acc;
}

template <typename Kern>
cudaError_t launch_ring(Kern kernel, const NormArgs& a, int bd, int nt, int vpt, int64_t grid_max, int num_sms,
                        cudaStream_t s, int* grid_out) {
  int optin = 0;
  cudaError_t err = device_attr_cached(cudaDevAttrMaxSharedMemoryPerBlockOptin, &optin);
  if (err != cudaSuccess) return err;
  const size_t slot = (size_t)nt * vpt * bd * 16;
  int slots = (int)(((size_t)optin - 1024) / slot);  // rows of any accepted size leave room for one
  if (slots < 1) return cudaErrorInvalidConfiguration;
  if (slots > kMaxSlots) slots = kMaxSlots;
  const size_t smem = slots * slot;
  err = opt_in_smem(kernel, smem);
  if (err != cudaSuccess) return err;
  int per_sm = 0;
  err = occupancy(kernel, bd, smem, &per_sm);
  if (err != cudaSuccess) return err;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  int64_t grid = (int64_t)num_sms * per_sm;
  if (grid > grid_max) grid = grid_max;
  if (grid < 1) grid = 1;  // no rows: the sums over tokens are still written (zeros)
  *grid_out = (int)grid;
  kernel<<<(unsigned)grid, bd, smem, s>>>(a, slots);
  return cudaGetLastError();
}

// EPT: elements per thread; MAXT: threads the kernel is compiled for.
template <int TYPE, int EPT, int MAXT>
cudaError_t launch_forward(const NormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int VPT = EPT / Vec<TYPE>::kN;
  const int nv = a.H / Vec<TYPE>::kN;
  const int bd = ((nv + VPT - 1) / VPT + 31) / 32 * 32;
  const int nt = kForwardRows * (a.y != nullptr ? 2 : 1);
  int grid = 0;
  if (a.y != nullptr && a.w_post != nullptr && a.w_pre != nullptr)
    return launch_ring(norm_kernel<TYPE, VPT, MAXT, true>, a, bd, nt, VPT, a.T, num_sms, s, &grid);
  return launch_ring(norm_kernel<TYPE, VPT, MAXT, false>, a, bd, nt, VPT, a.T, num_sms, s, &grid);
}

template <int TYPE, int EPT, int MAXT>
cudaError_t launch_backward(const NormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int VPT = EPT / Vec<TYPE>::kN;
  const int nv = a.H / Vec<TYPE>::kN;
  const int bd = ((nv + VPT - 1) / VPT + 31) / 32 * 32;
  const bool all = a.y != nullptr && a.w_post != nullptr && a.w_pre != nullptr && a.dxo != nullptr;
  int grid = 0;
  const int nt = (a.dxo != nullptr) + (a.y != nullptr) + (a.w_pre != nullptr ? 2 : 0);
  const int64_t rows = a.T < a.parts ? a.T : a.parts;
  cudaError_t err =
      all ? launch_ring(norm_grad_kernel<TYPE, VPT, MAXT, true>, a, bd, 4, VPT, rows, num_sms, s, &grid)
          : launch_ring(norm_grad_kernel<TYPE, VPT, MAXT, false>, a, bd, nt < 1 ? 1 : nt, VPT, rows, num_sms, s, &grid);
  if (err != cudaSuccess || (a.w_pre == nullptr && a.w_post == nullptr && a.gate_mode != kGateChannel)) return err;
  norm_sum_kernel<<<dim3((a.H + kSumCols - 1) / kSumCols, 2), kSumCols * kSumRows, 0, s>>>(a, grid);
  return cudaGetLastError();
}

// Elements per thread. Forward: 8 while a CTA's threads can hold a row, compiled for
// 896 threads (72 registers hold the weights of 8 columns and two rows) or for 1024
// (64, which spill a little). Backward: 16, up to 512 threads (128 registers, weights
// and sums of 16 columns): half the warps repeat the row's reduction and scalars.
// Longer rows take 16 and up to 1024 threads. Measured in bf16 (us):
//   forward, 8 elements, 896 / 1024 threads     16384 x 4096  86 / 96   40000 x 2048  119 / 121
//                                               8192 x 7168 without y   41 / 47
//   forward, 8 elements / 16, 1024 threads      8192 x 7176   88 / 142  8192 x 8192    89 / 147
//   backward, 8 / 16 elements                   8192 x 7168  158 / 152
template <int TYPE>
cudaError_t launch_type(const NormArgs& a, bool grad, int num_sms, cudaStream_t s) {
  if (grad) {
    if (a.H <= 16 * 512) return launch_backward<TYPE, 16, 512>(a, num_sms, s);
    return launch_backward<TYPE, 16, 1024>(a, num_sms, s);
  }
  if (a.H <= 8 * 896) return launch_forward<TYPE, 8, 896>(a, num_sms, s);
  if (a.H <= 8 * 1024) return launch_forward<TYPE, 8, 1024>(a, num_sms, s);
  return launch_forward<TYPE, 16, 1024>(a, num_sms, s);
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
