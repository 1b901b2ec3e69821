// api_fp4.cu -- the C ABI of the four-bit calls (include/moeperm.h): argument
// validation and launches only.
#include "../../include/moeperm.h"
#include "api_util.h"
#include "kernels.h"

using namespace moeperm;

namespace {

cudaStream_t cu(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool fmt_ok(int fmt) { return fmt >= MOE_FP4_E8M0 && fmt <= MOE_FP4_NV; }
bool width_ok(int32_t H) { return H > 0 && H % 64 == 0; }
// Tensor scales only where the format has them; rows in n equal blocks.
bool tscale_ok(int fmt, const float* ts, int32_t n, int64_t R) {
  if (ts == nullptr) return true;
  return fmt == MOE_FP4_NV && n >= 1 && R % n == 0 && aligned_to(ts, 4);
}
// At most one of the ways to name the rows.
bool rows_named_ok(const int32_t* live, const int32_t* ids, const int32_t* masked_m, int32_t cap, int64_t R) {
  if ((live != nullptr) + (ids != nullptr) + (masked_m != nullptr) > 1) return false;
  if (masked_m != nullptr && (cap < 1 || R % cap)) return false;
  return words_ok({live, ids, masked_m});
}

}  // namespace

extern "C" {

size_t moe_fp4_scale_bytes(int64_t ld, int32_t H, moe_fp4_t fmt) {
  if (ld < 0 || !width_ok(H) || !fmt_ok(fmt)) return 0;
  const int64_t groups = H / (fmt == MOE_FP4_NV ? 16 : 32);
  return (size_t)((groups + 15) / 16) * (size_t)ld * 16;
}

moe_status_t moe_quant_fp4(const void* x, int64_t ldx, moe_elem_t type, int64_t R, int32_t H, moe_fp4_t fmt,
                           const float* tensor_scale, int32_t n_scales, const int32_t* d_num_live,
                           const int32_t* m_indices, const int32_t* masked_m, int32_t cap, void* xq, void* scales,
                           int64_t ld_s, int32_t* d_status, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (es == 0 || R < 0 || R >= (int64_t(1) << 31) || !width_ok(H) || !fmt_ok(fmt)) return MOE_ERR_INVALID_ARG;
  if (!tscale_ok(fmt, tensor_scale, n_scales, R) || !rows_named_ok(d_num_live, m_indices, masked_m, cap, R) ||
      !words_ok({d_status}))
    return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!rows_ok(x, ldx, H, es) || !xq || !aligned16(xq) || !scales || !aligned16(scales) || ld_s < R)
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  Fp4Args a{};
  a.x = x; a.ldx = ldx; a.R = R; a.H = H; a.tscale = tensor_scale; a.nts = n_scales;
  a.d_num_live = d_num_live; a.row_ids = m_indices; a.masked_m = masked_m; a.cap = cap;
  a.q = static_cast<uint8_t*>(xq); a.scales = static_cast<uint8_t*>(scales); a.ld = ld_s; a.status = d_status;
  return cuda_status(launch_quant_fp4(a, (int)type, (int)fmt, sms, cu(stream)));
}

moe_status_t moe_dequant_fp4(const void* xq, const void* scales, int64_t ld_s, int64_t R, int32_t H, moe_fp4_t fmt,
                             const float* tensor_scale, int32_t n_scales, const int32_t* d_num_live,
                             const int32_t* m_indices, const int32_t* masked_m, int32_t cap, void* x, int64_t ldx,
                             moe_elem_t type, int32_t* d_status, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (es == 0 || R < 0 || R >= (int64_t(1) << 31) || !width_ok(H) || !fmt_ok(fmt)) return MOE_ERR_INVALID_ARG;
  if (!tscale_ok(fmt, tensor_scale, n_scales, R) || !rows_named_ok(d_num_live, m_indices, masked_m, cap, R) ||
      !words_ok({d_status}))
    return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!rows_ok(x, ldx, H, es) || !xq || !aligned16(xq) || !scales || !aligned16(scales) || ld_s < R)
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  Fp4Args a{};
  a.x = x; a.ldx = ldx; a.R = R; a.H = H; a.tscale = tensor_scale; a.nts = n_scales;
  a.d_num_live = d_num_live; a.row_ids = m_indices; a.masked_m = masked_m; a.cap = cap;
  a.q = static_cast<uint8_t*>(const_cast<void*>(xq)); a.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  a.ld = ld_s; a.status = d_status;
  return cuda_status(launch_dequant_fp4(a, (int)type, (int)fmt, sms, cu(stream)));
}

moe_status_t moe_dispatch_fp4(const void* x, int64_t ldx, moe_elem_t type, int32_t T, const int32_t* d_num_tokens,
                              int32_t H, const int32_t* topk_ids, const float* topk_weights, int32_t K, int32_t E,
                              int32_t L, int32_t block_e, moe_fp4_t fmt, const float* tensor_scale, void* xq,
                              void* scales, int64_t ld_s, int32_t* m_indices, int64_t bound, int32_t* src2dst,
                              int32_t* counts, int32_t* starts, int32_t* psum, int32_t* total, float* row_weights,
                              void* workspace, size_t workspace_bytes, int32_t* d_status, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (es == 0 || T < 0 || !width_ok(H) || H > kMaxHidden || !fmt_ok(fmt)) return MOE_ERR_INVALID_ARG;
  if (!tscale_ok(fmt, tensor_scale, 1, T)) return MOE_ERR_INVALID_ARG;
  if (K < 1 || K > kMaxK || L < 1 || L > kMaxL || E < L || block_e < 1) return MOE_ERR_INVALID_ARG;
  const int64_t A = (int64_t)T * K;
  if (A > kMaxAssignments) return MOE_ERR_INVALID_ARG;
  const RouteGeom geom = route_geometry(A, L, route_table_pref(H, L));
  if (geom.S == 0) return MOE_ERR_INVALID_ARG;
  if (bound < moe_compact_bound(A, L, block_e) || bound >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!rows_ok(x, ldx, H, es) || !topk_ids || !src2dst)) return MOE_ERR_INVALID_ARG;
  if (bound > 0 && (!m_indices || !xq || !aligned16(xq) || !scales || !aligned16(scales) || ld_s < bound))
    return MOE_ERR_INVALID_ARG;
  if (!counts || !starts || !psum || !total || (row_weights && !topk_weights)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({d_num_tokens, topk_ids, topk_weights, m_indices, src2dst, counts, starts, psum, total, row_weights, d_status}))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < moe_workspace_bytes(T, K, L))
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;

  DispatchFp4Args a{};
  ScatterArgs& s = a.s;
  s.x = static_cast<const uint16_t*>(x); s.T = T; s.d_num_tokens = d_num_tokens; s.H = H;
  s.ids = topk_ids; s.w = topk_weights; s.K = K; s.L = L; s.E = E; s.mode = kModeCompact;
  s.block_e = block_e; s.xq = static_cast<uint8_t*>(xq); s.scales = scales; s.ld_s = ld_s; s.src2dst = src2dst;
  s.row_weights = row_weights; s.m_indices = m_indices; s.bound = bound; s.counts = counts;
  s.starts = starts; s.psum = psum; s.total = total; s.status = d_status;
  a.ldx_bytes = ldx * es;
  a.tscale = tensor_scale;
  if (A > kSmallSlots) {
    s.chunk = geom.chunk;
    s.nchunks = (int32_t)geom.nchunks;
    s.table = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + kWsHeader);
    RoutePlanArgs rp{};
    rp.ids = topk_ids; rp.d_num_tokens = d_num_tokens; rp.T = T; rp.K = K; rp.L = L;
    rp.chunk = s.chunk; rp.nchunks = s.nchunks; rp.lrank = src2dst;
    rp.table = const_cast<int32_t*>(s.table); rp.status = d_status;
    if (launch_route_plan(rp, geom, cu(stream)) != cudaSuccess) return MOE_ERR_CUDA;
  }
  return cuda_status(launch_dispatch_fp4(a, (int)type, (int)fmt, sms, /*after_route_plan=*/A > kSmallSlots, cu(stream)));
}

moe_status_t moe_expert_matmul_fp4(const void* x, int64_t ldx, const void* x_scales, int64_t ld_xs,
                                   const float* x_tscale, int64_t R, int32_t K, const void* w, const void* w_scales,
                                   int64_t ld_ws, const float* w_tscale, moe_fp4_t fmt, int32_t L, int32_t N,
                                   int32_t gated, moe_act_t act, const float* bias, const int32_t* seg_begin,
                                   const int32_t* seg_end, int32_t cap, const void* residual, int64_t ld_res, void* out,
                                   int64_t ldo, moe_elem_t out_type, int32_t* d_status, moe_stream_t stream) {
  if (!fmt_ok(fmt) || (out_type != MOE_BF16 && out_type != MOE_F16)) return MOE_ERR_INVALID_ARG;
  if (L < 1 || L > kMaxL || R < 0 || R >= (int64_t(1) << 31) || cap < 0) return MOE_ERR_INVALID_ARG;
  if (cap > 0 ? (seg_begin != nullptr || seg_end == nullptr || R != (int64_t)L * cap)
              : ((seg_begin == nullptr) != (seg_end == nullptr) || (seg_begin == nullptr && L != 1)))
    return MOE_ERR_INVALID_ARG;
  if ((gated != 0 && gated != 1) || N < 1 || N % (gated ? 16 : 8) || act < MOE_ACT_NONE || act > MOE_ACT_GELU)
    return MOE_ERR_INVALID_ARG;
  const int64_t Nw = gated ? 2 * (int64_t)N : N;
  if (L * Nw >= (int64_t(1) << 31) || !width_ok(K)) return MOE_ERR_INVALID_ARG;
  if (!w || !aligned16(w) || !w_scales || !aligned16(w_scales) || ld_ws < L * Nw) return MOE_ERR_INVALID_ARG;
  if ((x_tscale || w_tscale) && fmt != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
  if (!words_ok({seg_begin, seg_end, d_status, x_tscale, w_tscale, bias})) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!rows_ok(x, ldx, K / 2, 1) || !x_scales || !aligned16(x_scales) || ld_xs < R) return MOE_ERR_INVALID_ARG;
  if (!out || ldo < N || (residual && ld_res < N) || !aligned_to(out, 2) || !aligned_to(residual, 2))
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  MatmulArgs m{};
  m.x = x; m.ldx = ldx; m.terms = 1; m.w = w; m.R = R; m.K = K; m.L = L; m.N = N;
  m.type = fmt == MOE_FP4_NV ? kE2M1NV : kE2M1MX;
  m.out_type = (int)out_type; m.gated = gated; m.act = (int)act; m.seg_begin = seg_begin;
  m.seg_end = seg_end; m.cap = cap; m.bias = bias; m.residual = residual; m.ld_res = ld_res;
  m.out = out; m.ldo = ldo;
  m.xs = static_cast<const uint32_t*>(x_scales); m.ld_xs = ld_xs;
  m.ws = static_cast<const uint32_t*>(w_scales); m.ld_ws = ld_ws;
  m.x_tscale = x_tscale; m.w_tscale = w_tscale; m.status = d_status;
  return cuda_status(few_rows_fp4(m) ? launch_matmul_few_rows(m, sms, cu(stream)) : launch_matmul(m, sms, cu(stream)));
}

}  // extern "C"
