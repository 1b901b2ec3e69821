// fp4_few_rows.cu -- the four-bit product for one or two rows of one dense matrix of
// moderate size, the step of a single token.
//
//   P[r, f] = sum over groups g of s_w[f, g] * sum_{k in g} x[r, k] * w[f, k]
//
// Every weight is used once or a few times, so the tensor cores have nothing to do and
// their set-up (tensor maps, tensor memory, clusters) is most of the time. Here a warp
// takes two weight rows (gated: the gate and the up row of a feature), a lane 32
// elements at a time; the rows of x lie in shared memory as bf16, which holds an element
// times its group's scale exactly (six significant bits at most). Products and sums are
// in fp32. Bound by latencies (the launch, one read of x, one of the weights) for a
// short reduction, by the conversions of the weights for a long one.
#include "activation.cuh"
#include "fp4.cuh"
#include "kernels.h"

namespace moeperm {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

struct FewArgs {
  const uint8_t* x;
  int64_t ldx;
  const uint8_t* xs;
  int64_t ld_xs;
  const uint8_t* w;
  const uint8_t* ws;
  int64_t ld_ws;
  const float* x_tscale;
  const float* w_tscale;
  int32_t R, K, N, gated, act, f16;
  const float* bias;
  const void* residual;
  int64_t ld_res;
  void* out;
  int64_t ldo;
};

// 32 elements and their group scales.
template <int FMT>
struct Run {
  uint4 q;
  uint32_t byte[2];  // of the first and the second half
  __device__ __forceinline__ void load(const uint8_t* row, const uint8_t* scales, int64_t ld, int64_t r, int c, bool valid) {
    q = make_uint4(0, 0, 0, 0);
    byte[0] = byte[1] = 0;
    if (!valid) return;
    q = ld_nc_v4(row + (int64_t)c * 16);
    if constexpr (FMT == kFp4NV) {  // groups 2 c and 2 c + 1
      const uint32_t v = __ldg(reinterpret_cast<const uint16_t*>(scales + ((int64_t)(c >> 3) * ld + r) * 16 + 2 * (c & 7)));
      byte[0] = v & 0xFF;
      byte[1] = v >> 8;
    } else {  // group c
      byte[0] = byte[1] = __ldg(scales + ((int64_t)(c >> 4) * ld + r) * 16 + (c & 15));
    }
  }
};

__device__ __forceinline__ float value16(const void* p, int64_t i, bool f16) {
  const uint32_t w = __ldg(static_cast<const uint16_t*>(p) + i);
  return f16 ? f16x2_to_float2(w).x : __uint_as_float(w << 16);
}

template <int FMT, int ROWS>
__global__ void __launch_bounds__(kThreads) few_rows_kernel(FewArgs p) {
  extern __shared__ uint4 s_x[];  // [row][step][4][lane]: 8 elements each
  const int tid = threadIdx.x, lane = tid & 31;
  const int runs = p.K / 32, steps = (runs + 31) / 32;
  const int units = p.gated ? p.N : p.N / 2, nwarps = gridDim.x * kWarps;
  int u = blockIdx.x * kWarps + (tid >> 5);
  // weight rows of unit u: 2 u and 2 u + 1, or u and N + u
  auto first_row = [&](int unit) { return (int64_t)(p.gated ? unit : 2 * unit); };
  const int64_t second = p.gated ? p.N : 1;
  const int64_t wbytes = p.K / 2;
  if (u < units) {  // the weights set out while x is prepared
    const uint8_t* w = p.w + first_row(u) * wbytes;
    for (int64_t o = lane * 128; o < wbytes; o += 32 * 128) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(w + o));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(w + second * wbytes + o));
    }
  }
  for (int i = tid; i < ROWS * steps * 32; i += kThreads) {
    const int r = i / (steps * 32), c = i - r * steps * 32;
    Run<FMT> x;
    x.load(p.x + r * p.ldx, p.xs, p.ld_xs, r, c, c < runs && r < p.R);
    const uint32_t q[4] = {x.q.x, x.q.y, x.q.z, x.q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
      e2m1x8_to_floats(q[j], f);
      const float d = fp4_scale<FMT>(x.byte[j / 2], 1.0f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= d;
      s_x[((r * steps + c / 32) * 4 + j) * 32 + c % 32] = Vec<kBF16>::pack(f);
    }
  }
  __syncthreads();
  float alpha = 1.0f;
  if (p.x_tscale != nullptr) alpha = __ldg(p.x_tscale);
  if (p.w_tscale != nullptr) alpha *= __ldg(p.w_tscale);
  for (; u < units; u += nwarps) {
    const int64_t row0 = first_row(u);
    float acc[2][ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) acc[0][r] = acc[1][r] = 0.0f;
#pragma unroll 2
    for (int s = 0; s < steps; ++s) {
      const int c = s * 32 + lane;
      Run<FMT> w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[h].load(p.w + (row0 + h * second) * wbytes, p.ws, p.ld_ws, row0 + h * second, c, c < runs);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float part[2][ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) part[0][r] = part[1][r] = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float wv[2][8];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            e2m1x8_to_floats(half ? (j ? w[h].q.w : w[h].q.z) : (j ? w[h].q.y : w[h].q.x), wv[h]);
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            float xv[8];
            Vec<kBF16>::unpack(s_x[((r * steps + s) * 4 + half * 2 + j) * 32 + lane], xv);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              part[0][r] = fmaf(wv[0][k], xv[k], part[0][r]);
              part[1][r] = fmaf(wv[1][k], xv[k], part[1][r]);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float d = fp4_scale<FMT>(w[h].byte[half], 1.0f);
#pragma unroll
          for (int r = 0; r < ROWS; ++r) acc[h][r] = c < runs ? fmaf(part[h][r], d, acc[h][r]) : acc[h][r];
        }
      }
    }
    // lane r (r < ROWS) keeps row r's sums
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = acc[h][r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == r) sum[h] = v;
      }
    if (lane < p.R) {
      float v[2] = {sum[0] * alpha, sum[1] * alpha};
      if (p.bias != nullptr) {
        v[0] += __ldg(p.bias + row0);
        v[1] += __ldg(p.bias + row0 + second);
      }
      const bool f16 = p.f16 != 0;
      uint16_t* out = static_cast<uint16_t*>(p.out) + lane * p.ldo;
      if (p.gated) {
        float a[1] = {v[0]};
        activate(a, p.act);
        a[0] *= v[1];
        if (p.residual != nullptr) a[0] += value16(p.residual, lane * p.ld_res + u, f16);
        out[u] = (uint16_t)(f16 ? pack_f16x2(a[0], 0.0f) : pack_bf16x2(a[0], 0.0f));
      } else {
        activate(v, p.act);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (p.residual != nullptr) v[h] += value16(p.residual, lane * p.ld_res + row0 + h, f16);
          out[row0 + h] = (uint16_t)(f16 ? pack_f16x2(v[h], 0.0f) : pack_bf16x2(v[h], 0.0f));
        }
      }
    }
  }
}

// A warp's step takes two weight rows 32 elements a lane: the time is that of the launch and of
// x, which grows with K, and about 0.25 us for each 1024 steps of all weight rows (two rows of
// x: 0.35). The tensor cores take 9 us and then the weights' time from HBM. Measured, matrices in
// turn so that they come from HBM, here against there in us (scales per 16; those per 32 lie
// within 0.8):
//   one row    2048 -> 7168 4.9 / 9.3, 4096 -> 8192 10.3 / 11.5, 7168 -> 4096 11.0 / 12.2, 8192 -> 4096
//              12.3 / 12.3; beyond: 4096 -> 10240 12.1 / 11.7, 7168 -> 6144 13.6 / 13.0, 10240 -> 2048
//              11.8 / 11.5, 24576 -> 512 19.2 / 14.4, 8192 -> 28672 41 / 30, 64 -> 262144 55 / 19
//   two rows   2048 -> 7168 6.0 / 9.2, 2048 -> 12288 9.7 / 10.0, 6144 -> 4096 11.6 / 11.3, 8192 -> 2048
//              10.8 / 10.8; beyond: 2048 -> 14336 10.7 / 10.2, 7168 -> 4096 13.0 / 12.3, 10240 -> 1024
//              12.9 / 11.2
constexpr int kMostRows = 2, kMostLength = 8192;
constexpr int64_t kMostSteps[kMostRows + 1] = {0, 32768, 24576};  // weight rows times steps of 1024 elements
size_t smem_bytes(int K, int rows) { return (size_t)rows * ((K / 32 + 31) / 32) * 4 * 32 * 16; }
static_assert(kMostRows * kMostLength * 2 <= 46 * 1024, "x fits the shared memory that needs no opt-in");

}  // namespace

bool few_rows_fp4(const MatmulArgs& a) {
  if (a.seg_end != nullptr || a.R > kMostRows || a.K > kMostLength) return false;
  return (a.gated ? 2 : 1) * (int64_t)a.N * ((a.K + 1023) / 1024) <= kMostSteps[a.R];
}

cudaError_t launch_matmul_few_rows(const MatmulArgs& m, int num_sms, cudaStream_t s) {
  FewArgs a{};
  a.x = static_cast<const uint8_t*>(m.x); a.ldx = m.ldx; a.xs = reinterpret_cast<const uint8_t*>(m.xs); a.ld_xs = m.ld_xs;
  a.w = static_cast<const uint8_t*>(m.w); a.ws = reinterpret_cast<const uint8_t*>(m.ws); a.ld_ws = m.ld_ws;
  a.x_tscale = m.x_tscale; a.w_tscale = m.w_tscale;
  a.R = (int32_t)m.R; a.K = m.K; a.N = m.N; a.gated = m.gated; a.act = m.act; a.f16 = m.out_type == kF16;
  a.bias = m.bias; a.residual = m.residual; a.ld_res = m.ld_res; a.out = m.out; a.ldo = m.ldo;
  auto go = [&](auto kernel, int rows) -> cudaError_t {
    const size_t smem = smem_bytes(m.K, rows);
    int per_sm = 0;
    cudaError_t err = occupancy(kernel, kThreads, smem, &per_sm);
    if (err != cudaSuccess) return err;
    const int64_t units = m.gated ? m.N : m.N / 2, need = (units + kWarps - 1) / kWarps;
    const int64_t most = (int64_t)num_sms * (per_sm < 1 ? 1 : per_sm);
    kernel<<<(unsigned)(need < most ? need : most), kThreads, smem, s>>>(a);
    return cudaGetLastError();
  };
  if (m.type == kE2M1NV) return m.R == 1 ? go(few_rows_kernel<kFp4NV, 1>, 1) : go(few_rows_kernel<kFp4NV, 2>, 2);
  return m.R == 1 ? go(few_rows_kernel<kFp4MX, 1>, 1) : go(few_rows_kernel<kFp4MX, 2>, 2);
}

}  // namespace moeperm
