// api_block.cu -- the C ABI of the calls around the dispatch (include/moeperm.h):
// plain permute, combine for every type, their gradients, and the norms around
// a block. Host-side argument validation and launches only.
#include "../../include/moeperm.h"
#include "api_util.h"
#include "kernels.h"

using namespace moeperm;

namespace {

cudaStream_t cu(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Which parts a norm call has: a block output or a pre norm, and a post norm or
// a gate only with a block output. Without rows the block output and a gate per
// token may be NULL (they are empty); a gate per channel may not, since the
// gradient still reads it for its sums over no tokens. Kernels read a gate per
// channel in vectors, one per token a float at a time.
bool norm_parts_ok(int32_t T, const void* y, const float* w_post, const float* gate, int mode,
                   const float* w_pre) {
  if (mode != MOE_GATE_NONE && mode != MOE_GATE_CHANNEL && mode != MOE_GATE_TOKEN) return false;
  if (mode == MOE_GATE_CHANNEL && (!gate || !aligned16(gate))) return false;
  if (T <= 0) return true;
  if (!y && (!w_pre || w_post || mode != MOE_GATE_NONE)) return false;
  return mode != MOE_GATE_TOKEN || (gate && aligned_to(gate, 4));
}

// Rows of a norm: at most 2048 16-byte vectors.
bool norm_shape_ok(int32_t T, int32_t H, int es) {
  return es != 0 && T >= 0 && H > 0 && (int64_t)H * es % 16 == 0 && (int64_t)H * es <= 2048 * 16;
}

// Where the rows of the experts are: segments, slabs or one dense matrix.
bool segments_ok(int64_t R, int32_t L, const int32_t* begin, const int32_t* end, int32_t cap) {
  if (L < 1 || L > kMaxL || R < 0 || R >= (int64_t(1) << 31) || cap < 0) return false;
  if (cap > 0) return begin == nullptr && end != nullptr && R == (int64_t)L * cap;
  if ((begin == nullptr) != (end == nullptr)) return false;
  return begin != nullptr || L == 1;
}
bool act_ok(int act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_GELU; }
// Output features, and weight rows within 32 bits.
bool feats_ok(int32_t N, int32_t L, int32_t gated) {
  if (N < 1 || N % (gated ? 16 : 8) || (gated != 0 && gated != 1)) return false;
  return (int64_t)L * N * (gated ? 2 : 1) < (int64_t(1) << 31);
}

// Room for the gradient of the pre-activations in two terms: the rows held decide
// whether both are used, and they may be few in any buffer.
size_t dpre_bytes(int64_t R, int32_t Nw) { return ((size_t)2 * R * Nw * 2 + 255) / 256 * 256; }

}  // namespace

extern "C" {

moe_status_t moe_permute(const void* x, int64_t ldx, moe_elem_t type, int32_t T,
                         const int32_t* d_num_tokens, int32_t H, const int32_t* topk_ids,
                         const float* topk_weights, int32_t K, int32_t E, int32_t L, int32_t block_e,
                         void* xs, int32_t* m_indices, int64_t bound, int32_t* src2dst, int32_t* counts,
                         int32_t* starts, int32_t* psum, int32_t* total, float* row_weights,
                         void* workspace, size_t workspace_bytes, int32_t* d_status, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (es == 0 || T < 0 || H <= 0 || H > kMaxHidden || (int64_t)H * es % 16) return MOE_ERR_INVALID_ARG;
  if (K < 1 || K > kMaxK || L < 1 || L > kMaxL || E < L || block_e < 1) return MOE_ERR_INVALID_ARG;
  const int64_t A = (int64_t)T * K;
  if (A > kMaxAssignments) return MOE_ERR_INVALID_ARG;
  const RouteGeom geom = route_geometry(A, L, route_table_pref(H, L));
  if (geom.S == 0) return MOE_ERR_INVALID_ARG;
  if (bound < moe_compact_bound(A, L, block_e) || bound >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!rows_ok(x, ldx, H, es) || !topk_ids || !src2dst)) return MOE_ERR_INVALID_ARG;
  if (bound > 0 && (!m_indices || !xs || !aligned16(xs))) return MOE_ERR_INVALID_ARG;
  if (!counts || !starts || !psum || !total || (row_weights && !topk_weights)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({d_num_tokens, topk_ids, topk_weights, m_indices, src2dst, counts, starts, psum, total, row_weights, d_status}))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < moe_workspace_bytes(T, K, L))
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;

  PermuteArgs a{};
  ScatterArgs& s = a.s;
  s.x = static_cast<const uint16_t*>(x); s.T = T; s.d_num_tokens = d_num_tokens; s.H = H;
  s.ids = topk_ids; s.w = topk_weights; s.K = K; s.L = L; s.E = E; s.mode = kModeCompact;
  s.block_e = block_e; s.xq = static_cast<uint8_t*>(xs); s.src2dst = src2dst;
  s.row_weights = row_weights; s.m_indices = m_indices; s.bound = bound; s.counts = counts;
  s.starts = starts; s.psum = psum; s.total = total; s.status = d_status;
  a.ldx_bytes = ldx * es;
  a.row_bytes = H * es;
  constexpr int kPiece = 16384;  // largest piece of a row moved at once
  a.units = (a.row_bytes + kPiece - 1) / kPiece;
  a.unit_bytes = ((a.row_bytes + a.units - 1) / a.units + 15) / 16 * 16;
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
  return cuda_status(launch_permute(a, sms, /*after_route_plan=*/A > kSmallSlots, cu(stream)));
}

moe_status_t moe_combine_ex(const void* y, int64_t ldy, moe_elem_t type, int64_t R,
                            const int32_t* src2dst, const float* w, int32_t T,
                            const int32_t* d_num_tokens, int32_t K, int32_t H, void* out,
                            int32_t* d_status, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (es == 0 || T < 0 || K < 1 || K > kMaxK || H <= 0 || (int64_t)H * es % 16 || R < 0)
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!src2dst || !out || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({src2dst, w, d_num_tokens, d_status})) return MOE_ERR_INVALID_ARG;
  if (R > 0 && !rows_ok(y, ldy, H, es)) return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  CombineArgs a{};
  a.y = y; a.ldy = ldy; a.R = R; a.src2dst = src2dst; a.w = w; a.T = T;
  a.d_num_tokens = d_num_tokens; a.K = K; a.H = H; a.out = out; a.status = d_status;
  return cuda_status(launch_combine(a, (int)type, sms, cu(stream)));
}

moe_status_t moe_combine_grad(const void* dout, int64_t ldd, const void* y, int64_t ldy, moe_elem_t type,
                              int64_t R, const int32_t* src2dst, const float* w, int32_t T,
                              const int32_t* d_num_tokens, int32_t K, int32_t H, void* dy, int64_t lddy,
                              float* dw, int32_t* d_status, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (es == 0 || T < 0 || K < 1 || K > kMaxK || H <= 0 || (int64_t)H * es % 16 || R < 0)
    return MOE_ERR_INVALID_ARG;
  if (!dy && !dw) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!src2dst || !rows_ok(dout, ldd, H, es)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({src2dst, w, d_num_tokens, dw, d_status})) return MOE_ERR_INVALID_ARG;
  if (R > 0 && dw && !rows_ok(y, ldy, H, es)) return MOE_ERR_INVALID_ARG;
  if (R > 0 && dy && !rows_ok(dy, lddy, H, es)) return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  CombineGradArgs a{};
  a.dout = dout; a.ldd = ldd; a.y = y; a.ldy = ldy; a.R = R; a.src2dst = src2dst; a.w = w; a.T = T;
  a.d_num_tokens = d_num_tokens; a.K = K; a.H = H; a.dy = dy; a.lddy = lddy; a.dw = dw; a.status = d_status;
  return cuda_status(launch_combine_grad(a, (int)type, sms, cu(stream)));
}

moe_status_t moe_block_norm(const void* x, int64_t ldx, const void* y, int64_t ldy, moe_elem_t type,
                            int32_t T, int32_t H, const float* w_post, const float* gate,
                            moe_gate_t gate_mode, float scale, const float* w_pre, float eps, void* x_out,
                            void* h, float* rstd_post, float* rstd_pre, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (!norm_shape_ok(T, H, es) || !norm_parts_ok(T, y, w_post, gate, gate_mode, w_pre))
    return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !aligned16(w_post) || !aligned16(w_pre)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({rstd_post, rstd_pre})) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!rows_ok(x, ldx, H, es) || (y && (!rows_ok(y, ldy, H, es) || !x_out || !aligned16(x_out))) ||
      (w_pre && (!h || !aligned16(h))))
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  NormArgs a{};
  a.x = x; a.ldx = ldx; a.y = y; a.ldy = ldy; a.T = T; a.H = H; a.w_post = w_post; a.gate = gate;
  a.gate_mode = gate_mode; a.scale = scale; a.w_pre = w_pre; a.eps = eps; a.x_out = x_out; a.h = h;
  a.rstd_post = rstd_post; a.rstd_pre = rstd_pre;
  return cuda_status(launch_block_norm(a, (int)type, sms, cu(stream)));
}

size_t moe_block_norm_workspace_bytes(int32_t T, int32_t H) {
  if (T < 0 || H < 1) return 0;
  const int64_t parts = T < 1 ? 1 : T < kNormParts ? T : kNormParts;
  return (size_t)2 * parts * H * sizeof(float);
}

moe_status_t moe_block_norm_grad(const void* dx_out, int64_t ld_dxo, const void* dh, int64_t ld_dh,
                                 const void* x_out, int64_t ldx, const void* y, int64_t ldy,
                                 moe_elem_t type, int32_t T, int32_t H, const float* w_post,
                                 const float* gate, moe_gate_t gate_mode, float scale, const float* w_pre,
                                 const float* rstd_post, const float* rstd_pre, void* dx, void* dy,
                                 float* dw_post, float* dgate, float* dw_pre, void* workspace,
                                 size_t workspace_bytes, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (!norm_shape_ok(T, H, es) || !norm_parts_ok(T, y, w_post, gate, gate_mode, w_pre))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(w_post) || !aligned16(w_pre)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({rstd_post, rstd_pre, dw_post, dgate, dw_pre})) return MOE_ERR_INVALID_ARG;
  if ((w_post && !dw_post) || (w_pre && !dw_pre)) return MOE_ERR_INVALID_ARG;
  if (gate_mode == MOE_GATE_CHANNEL && !dgate) return MOE_ERR_INVALID_ARG;
  if ((w_post || w_pre || gate_mode == MOE_GATE_CHANNEL) &&
      (!workspace || !aligned16(workspace) || workspace_bytes < moe_block_norm_workspace_bytes(T, H)))
    return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    if (dx_out && !rows_ok(dx_out, ld_dxo, H, es)) return MOE_ERR_INVALID_ARG;
    if (w_pre && (!rows_ok(dh, ld_dh, H, es) || !rows_ok(x_out, ldx, H, es) || !rstd_pre))
      return MOE_ERR_INVALID_ARG;
    if (y && (!rows_ok(y, ldy, H, es) || !dy || !aligned16(dy))) return MOE_ERR_INVALID_ARG;
    if (w_post && !rstd_post) return MOE_ERR_INVALID_ARG;
    if (gate_mode == MOE_GATE_TOKEN && !dgate) return MOE_ERR_INVALID_ARG;
    if (!dx || !aligned16(dx)) return MOE_ERR_INVALID_ARG;
  }
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  NormArgs a{};
  a.x = x_out; a.ldx = ldx; a.y = y; a.ldy = ldy; a.T = T; a.H = H; a.w_post = w_post; a.gate = gate;
  a.gate_mode = gate_mode; a.scale = scale; a.w_pre = w_pre;
  a.rstd_post = const_cast<float*>(rstd_post); a.rstd_pre = const_cast<float*>(rstd_pre);
  a.dxo = dx_out; a.ld_dxo = ld_dxo; a.dh = dh; a.ld_dh = ld_dh; a.dx = dx; a.dy = dy;
  a.dw_post = dw_post; a.dgate = dgate; a.dw_pre = dw_pre; a.ws = static_cast<float*>(workspace);
  a.parts = T < 1 ? 1 : T < kNormParts ? T : kNormParts;
  return cuda_status(launch_block_norm_grad(a, (int)type, sms, cu(stream)));
}

moe_status_t moe_expert_matmul(const void* x, int64_t ldx, moe_elem_t type, const void* x_scales,
                               int64_t ld_xs, int64_t R, int32_t K, const void* w, const void* w_scales,
                               int64_t ld_ws, int32_t L, int32_t N, int32_t gated, moe_act_t act,
                               const float* bias, const int32_t* seg_begin, const int32_t* seg_end,
                               int32_t cap, const void* residual, int64_t ld_res, void* out, int64_t ldo,
                               moe_elem_t out_type, void* pre, int64_t ld_pre, int32_t* d_status,
                               moe_stream_t stream) {
  const bool fp8 = type == MOE_E4M3;
  const int es = fp8 ? 1 : 2;
  if (type != MOE_BF16 && type != MOE_F16 && !fp8) return MOE_ERR_INVALID_ARG;
  if (out_type != MOE_BF16 && out_type != MOE_F16) return MOE_ERR_INVALID_ARG;
  if (!fp8 && out_type != type) return MOE_ERR_INVALID_ARG;
  if (!segments_ok(R, L, seg_begin, seg_end, cap) || !feats_ok(N, L, gated) || !act_ok(act))
    return MOE_ERR_INVALID_ARG;
  if (K < 1 || K % (fp8 ? 128 : 8) || (fp8 && pre)) return MOE_ERR_INVALID_ARG;
  if (!w || !aligned16(w)) return MOE_ERR_INVALID_ARG;
  const int32_t Nw = gated ? 2 * N : N;
  if (fp8 && (!w_scales || !aligned16(w_scales) || ld_ws < (int64_t)L * Nw || ld_ws % 4)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({seg_begin, seg_end, d_status})) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!rows_ok(x, ldx, K, es) || !out || ldo < N || (residual && ld_res < N) || (pre && ld_pre < Nw))
    return MOE_ERR_INVALID_ARG;
  if (!aligned_to(out, 2) || !aligned_to(residual, 2) || !aligned_to(pre, 2) || !aligned_to(bias, 4))
    return MOE_ERR_INVALID_ARG;
  if (fp8 && (!x_scales || !aligned16(x_scales) || ld_xs < (cap > 0 ? cap : R) || ld_xs % 4))
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  MatmulArgs m{};
  m.x = x; m.ldx = ldx; m.terms = 1; m.w = w; m.R = R; m.K = K; m.L = L; m.N = N; m.type = (int)type;
  m.out_type = (int)out_type; m.gated = gated; m.act = (int)act; m.seg_begin = seg_begin;
  m.seg_end = seg_end; m.cap = cap; m.bias = bias; m.residual = residual; m.ld_res = ld_res;
  m.out = out; m.ldo = ldo; m.pre = pre; m.ld_pre = ld_pre;
  m.xs = static_cast<const uint32_t*>(x_scales); m.ld_xs = ld_xs;
  m.ws = static_cast<const uint32_t*>(w_scales); m.ld_ws = ld_ws; m.status = d_status;
  return cuda_status(launch_matmul(m, sms, cu(stream)));
}

size_t moe_expert_matmul_grad_workspace_bytes(int64_t R, int32_t L, int32_t Nw) {
  if (R < 0 || L < 1 || Nw < 1) return 0;
  // the split count depends on N; a gated N is half of Nw and gives the larger one
  const int splits = act_grad_splits(R, L, Nw < 2 ? 1 : Nw / 2);
  return dpre_bytes(R, Nw) + (splits > 1 ? (size_t)splits * L * Nw * sizeof(float) : 0);
}

moe_status_t moe_expert_matmul_grad(const void* dout, int64_t ldd, const void* x, int64_t ldx,
                                    moe_elem_t type, int64_t R, int32_t K, const void* w, int32_t L,
                                    int32_t N, int32_t gated, moe_act_t act, const void* pre, int64_t ld_pre,
                                    const int32_t* seg_begin, const int32_t* seg_end, int32_t cap, void* dx,
                                    int64_t ld_dx, void* dw, moe_elem_t dw_type, float* dbias,
                                    void* workspace, size_t workspace_bytes, int32_t* d_status,
                                    moe_stream_t stream) {
  if (type != MOE_BF16 && type != MOE_F16) return MOE_ERR_INVALID_ARG;
  if (!segments_ok(R, L, seg_begin, seg_end, cap) || !feats_ok(N, L, gated) || !act_ok(act))
    return MOE_ERR_INVALID_ARG;
  if (K < 1 || K % 8 || (!dx && !dw && !dbias)) return MOE_ERR_INVALID_ARG;
  if (dw && (dw_type != type && dw_type != MOE_F32)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({seg_begin, seg_end, d_status})) return MOE_ERR_INVALID_ARG;
  const int32_t Nw = gated ? 2 * N : N;
  const size_t dw_bytes = (size_t)L * Nw * K * (dw_type == MOE_F32 ? 4 : 2);
  cudaStream_t s = cu(stream);
  if (R == 0) {  // no rows: the sums are zero
    if (dw && cudaMemsetAsync(dw, 0, dw_bytes, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, (size_t)L * Nw * 4, s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const bool has_act = act != MOE_ACT_NONE || gated;
  const int terms = grad_terms(R, L, /*dense=*/seg_end == nullptr);
  const int dw_terms = dw && dw_type == MOE_F32 ? 2 : terms;  // (dx does not depend on what dw is)
  if (!rows_ok(dout, ldd, N, 2)) return MOE_ERR_INVALID_ARG;
  if (has_act && !rows_ok(pre, ld_pre, Nw, 2)) return MOE_ERR_INVALID_ARG;
  if (dw && !rows_ok(x, ldx, K, 2)) return MOE_ERR_INVALID_ARG;
  if (dx && (!w || !aligned16(w) || ld_dx < K)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(dx, 2) || !aligned_to(dw, dw_type == MOE_F32 ? 4 : 2) || !aligned_to(dbias, 4))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < moe_expert_matmul_grad_workspace_bytes(R, L, Nw))
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  if (has_act || dbias) {
    ActGradArgs a{};
    a.dout = dout; a.ldd = ldd; a.pre = pre; a.ld_pre = ld_pre; a.R = R; a.L = L; a.N = N; a.gated = gated;
    a.act = (int)act; a.seg_begin = seg_begin; a.seg_end = seg_end; a.cap = cap;
    a.dpre = has_act ? workspace : nullptr;
    a.terms = dw_terms;
    a.dbias = dbias;
    a.ws = reinterpret_cast<float*>(static_cast<char*>(workspace) + dpre_bytes(R, Nw));
    a.splits = act_grad_splits(R, L, N);
    a.status = d_status;
    if (launch_act_grad(a, (int)type, s) != cudaSuccess) return MOE_ERR_CUDA;
  }
  MatmulArgs m{};
  m.x = x; m.ldx = ldx; m.g = has_act ? workspace : dout; m.ldg = has_act ? Nw : ldd;
  m.terms = has_act ? terms : 1;
  m.w = w; m.R = R; m.K = K; m.L = L; m.N = N; m.type = (int)type; m.gated = gated;
  m.seg_begin = seg_begin; m.seg_end = seg_end; m.cap = cap; m.status = d_status;
  if (dx) {
    m.out = dx; m.ldo = ld_dx; m.out_type = (int)type;
    if (launch_matmul_grad_x(m, sms, s) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (dw) {
    m.out = dw; m.ldo = K; m.out_type = (int)dw_type; m.terms = has_act ? dw_terms : 1;
    if (launch_matmul_grad_w(m, sms, s) != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
