// api_router.cu -- the C ABI of the router's calls (include/moeperm.h): argument
// validation and launches only.
#include "../../include/moeperm.h"
#include "api_util.h"
#include "kernels.h"

using namespace moeperm;

namespace {

cudaStream_t cu(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Logits [T, ld] of a type, and a choice of K of E experts.
bool logits_ok(const void* logits, int64_t ld, int es, int32_t T, int32_t E, int32_t K) {
  if (es == 0 || T < 0 || T > (1 << 30) || E < 1 || E > kMaxRouted || K < 1 || K > kMaxK || K > E) return false;
  return T == 0 || (logits != nullptr && aligned_to(logits, es) && ld >= E);
}
bool score_ok(int s) { return s == MOE_SCORE_SOFTMAX || s == MOE_SCORE_SIGMOID; }

// Groups: both ends of each, or one group of all tokens.
bool groups_ok(const int32_t* begin, const int32_t* end, int32_t Q) {
  if (Q < 1 || Q > kMaxGroups || (begin == nullptr) != (end == nullptr)) return false;
  return (begin != nullptr || Q == 1) && words_ok({begin, end});
}

}  // namespace

extern "C" {

moe_status_t moe_route(const void* logits, int64_t ldl, moe_elem_t type, int32_t T, const int32_t* d_num_tokens,
                       int32_t E, int32_t K, moe_score_t score, const float* bias, int32_t renorm, float scale,
                       int32_t* topk_ids, float* topk_weights, int32_t* d_status, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (!logits_ok(logits, ldl, es, T, E, K) || !score_ok(score) || (renorm != 0 && renorm != 1)) return MOE_ERR_INVALID_ARG;
  if (!words_ok({d_num_tokens, bias, topk_ids, topk_weights, d_status})) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!topk_ids || !topk_weights) return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  RouteArgs a{};
  a.logits = logits; a.ld = ldl; a.T = T; a.d_num_tokens = d_num_tokens; a.E = E; a.K = K;
  a.sigmoid = score == MOE_SCORE_SIGMOID; a.renorm = renorm; a.bias = bias; a.scale = scale;
  a.ids = topk_ids; a.weights = topk_weights; a.status = d_status;
  return cuda_status(launch_route(a, (int)type, sms, cu(stream)));
}

size_t moe_balance_loss_workspace_bytes(int32_t E, int32_t Q) {
  if (E < 1 || E > kMaxRouted || Q < 1 || Q > kMaxGroups) return 0;
  return balance_ws_bytes(E, Q);
}

moe_status_t moe_balance_loss(const void* logits, int64_t ldl, moe_elem_t type, int32_t T, const int32_t* d_num_tokens,
                              int32_t E, const int32_t* topk_ids, int32_t K, moe_score_t score, const int32_t* seq_begin,
                              const int32_t* seq_end, int32_t Q, float* loss, int32_t* counts, float* prob_sums,
                              void* workspace, size_t workspace_bytes, int32_t* d_status, moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (!logits_ok(logits, ldl, es, T, E, K) || !score_ok(score) || !groups_ok(seq_begin, seq_end, Q))
    return MOE_ERR_INVALID_ARG;
  if (!words_ok({d_num_tokens, topk_ids, loss, counts, prob_sums, d_status})) return MOE_ERR_INVALID_ARG;
  if ((T > 0 && !topk_ids) || !loss || !counts || !prob_sums) return MOE_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < balance_ws_bytes(E, Q)) return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  BalanceArgs a{};
  a.logits = logits; a.ld = ldl; a.T = T; a.d_num_tokens = d_num_tokens; a.E = E; a.K = K;
  a.sigmoid = score == MOE_SCORE_SIGMOID; a.ids = topk_ids;
  a.g.begin = seq_begin; a.g.end = seq_end; a.g.Q = Q;
  a.loss = loss; a.counts = counts; a.prob_sums = prob_sums; a.ws = static_cast<float*>(workspace); a.status = d_status;
  return cuda_status(launch_balance(a, (int)type, sms, cu(stream)));
}

moe_status_t moe_route_grad(const void* logits, int64_t ldl, moe_elem_t type, int32_t T, const int32_t* d_num_tokens,
                            int32_t E, const int32_t* topk_ids, int32_t K, moe_score_t score, int32_t renorm, float scale,
                            const float* dweights, const float* dloss, const int32_t* counts, const int32_t* seq_begin,
                            const int32_t* seq_end, int32_t Q, void* dlogits, int64_t ldd, int32_t* d_status,
                            moe_stream_t stream) {
  const int es = elem_bytes(type);
  if (!logits_ok(logits, ldl, es, T, E, K) || !score_ok(score) || !groups_ok(seq_begin, seq_end, Q) ||
      (renorm != 0 && renorm != 1))
    return MOE_ERR_INVALID_ARG;
  if (!words_ok({d_num_tokens, topk_ids, dweights, dloss, counts, d_status})) return MOE_ERR_INVALID_ARG;
  if ((!dweights && !dloss) || (dloss && !counts)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!dlogits || !aligned_to(dlogits, es) || ldd < E || (dweights && !topk_ids)) return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_cached();
  if (sms <= 0) return MOE_ERR_CUDA;
  RouteGradArgs a{};
  a.logits = logits; a.ld = ldl; a.T = T; a.d_num_tokens = d_num_tokens; a.E = E; a.K = K;
  a.sigmoid = score == MOE_SCORE_SIGMOID; a.renorm = renorm; a.scale = scale; a.ids = topk_ids;
  a.dweights = dweights; a.dloss = dloss; a.counts = counts;
  a.g.begin = seq_begin; a.g.end = seq_end; a.g.Q = Q;
  a.dlogits = dlogits; a.ldd = ldd; a.status = d_status;
  return cuda_status(launch_route_grad(a, (int)type, sms, cu(stream)));
}

}  // extern "C"
