// C ABI of the block operators: routing with groups, combine gradient, block
// norms and the linear layer. Argument checks and launch sequences.
#include <cmath>

#include "api_util.cuh"
#include "common.cuh"
#include "kernels_block.cuh"

namespace moe {
namespace {

moe_status check_norm(const moe_norm_desc* d) {
  if (!d || d->T < 0 || d->H < 1) return MOE_ERR_INVALID_ARG;
  if (d->dtype != MOE_F32 && d->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (d->gate < MOE_GATE_NONE || d->gate > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->alpha))
    return MOE_ERR_INVALID_ARG;
  const int n = d->dtype == MOE_BF16 ? 8 : 4;
  if (d->H % n || d->H / n > 2048 || d->T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_linear(const moe_linear_desc* d) {
  if (!d || d->T < 0 || d->in < 1 || d->out < 1) return MOE_ERR_INVALID_ARG;
  if (d->dtype != MOE_F32 && d->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  const int n = d->dtype == MOE_BF16 ? 8 : 4;
  if (d->in % n || d->out % n) return MOE_ERR_UNSUPPORTED;
  if (d->T > (1 << 21) || d->in > (1 << 18) || d->out > (1 << 18)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool bad_ptr(const void* p) { return p && !aligned16(p); }

// Workspace of the linear layer: header, arrival counters, then the partial
// sums of shared tiles (one product at a time), dz and the column sums.
struct LinearLayout {
  size_t hdr, arrivals, partials, dz, parts, total;
  LinearPlan fwd, dx, dw;
};

LinearLayout linear_layout(const moe_linear_desc& d) {
  LinearLayout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) & ~size_t(255);
    return at;
  };
  L.hdr = take(sizeof(WsHeader));
  L.arrivals = take(sizeof(int) * 2 * kMaxSharedTiles);
  static_assert(sizeof(WsHeader) + sizeof(int) * 2 * kMaxSharedTiles <= MOE_LINEAR_WS_HEAD,
                "what has to be zero is in the head");
  size_t most = 0;
  if (d.dtype == MOE_BF16 && d.T > 0) {
    L.fwd = linear_plan(d.T, d.out, d.in, false, false, kPlanSms);
    L.dx = linear_plan(d.T, d.in, d.out, false, true, kPlanSms);
    L.dw = linear_plan(d.out, d.in, d.T, true, true, kPlanSms);
    most = std::max({L.fwd.partial_bytes, L.dx.partial_bytes, L.dw.partial_bytes});
  }
  L.partials = take(most);
  L.dz = take(d.act != MOE_ACT_NONE ? dtype_size(d.dtype) * d.T * d.out : 0);
  L.parts = take(sizeof(float) * ((d.T + kGradRows - 1) / kGradRows) * d.out);
  L.total = o;
  return L;
}

moe_status linear_product(const moe_linear_desc& d, const LinearLayout& L, const LinearPlan& plan,
                          char* ws, int M, int N, int K, const void* A, bool a_mn, const void* B,
                          bool b_mn, const LinearEpilogue& epi, cudaStream_t st) {
  if (d.dtype == MOE_BF16)
    MOE_CUDA_TRY(launch_linear_tc(plan, M, N, K, A, a_mn, B, b_mn, epi,
                                  reinterpret_cast<float*>(ws + L.partials),
                                  reinterpret_cast<int*>(ws + L.arrivals),
                                  &reinterpret_cast<WsHeader*>(ws + L.hdr)->status, st));
  else
    MOE_CUDA_TRY(launch_linear_simt(M, N, K, static_cast<const float*>(A), a_mn,
                                    static_cast<const float*>(B), b_mn, epi, st));
  return MOE_OK;
}

}  // namespace

moe_status check_route(const moe_route_desc* d) {
  if (!d || d->T < 0 || d->E < 1 || d->K < 1) return MOE_ERR_INVALID_ARG;
  if (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (d->groups < 1 || d->E % d->groups) return MOE_ERR_INVALID_ARG;
  if (d->topk_groups < 1 || d->topk_groups > d->groups) return MOE_ERR_INVALID_ARG;
  const int size = d->E / d->groups;
  if (d->group_top < 1 || d->group_top > 2 || d->group_top > size) return MOE_ERR_INVALID_ARG;
  if (d->K > d->topk_groups * size) return MOE_ERR_INVALID_ARG;
  if (d->renorm != 0 && d->renorm != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(d->scale)) return MOE_ERR_INVALID_ARG;
  if (d->K > kMaxK || d->E > kMaxE || d->groups > 32) return MOE_ERR_UNSUPPORTED;
  if ((long long)d->T * d->K > (1LL << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route(const moe_route_desc* desc, const float* logits, const float* bias,
                     int32_t* topk_idx, float* topk_w, moe_stream stream) {
  MOE_TRY(check_route(desc));
  if (desc->T == 0) return MOE_OK;
  MOE_TRY(check_ptrs({logits, topk_idx, topk_w}));
  if (bad_ptr(bias)) return MOE_ERR_INVALID_ARG;
  MOE_CUDA_TRY(launch_route(*desc, logits, 1, 0, bias, topk_idx, topk_w, nullptr,
                            static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

moe_status moe_route_backward(const moe_route_desc* desc, const float* logits,
                              const int32_t* topk_idx, const float* d_topk_w, float* d_logits,
                              moe_stream stream) {
  MOE_TRY(check_route(desc));
  if (desc->T == 0) return MOE_OK;
  MOE_TRY(check_ptrs({logits, topk_idx, d_topk_w, d_logits}));
  MOE_CUDA_TRY(launch_route_backward(*desc, logits, topk_idx, d_topk_w, d_logits,
                                     static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

size_t moe_norm_workspace_size(const moe_norm_desc* desc) {
  if (check_norm(desc) != MOE_OK) return 0;
  const size_t n = sizeof(float) * 3 * desc->H * block_norm_backward_grid(*desc, kPlanSms);
  return std::max<size_t>(256, (n + 255) & ~size_t(255));
}

moe_status moe_block_norm(const moe_norm_desc* desc, const void* h, const void* y,
                          const void* w_post, const void* gate, const void* w_pre, void* h_out,
                          void* x, moe_stream stream) {
  MOE_TRY(check_norm(desc));
  const moe_norm_desc& d = *desc;
  if (d.T == 0) return MOE_OK;
  if (!y && (w_post || gate || h_out || d.gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((gate != nullptr) != (d.gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((w_pre != nullptr) != (x != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!h_out && !x) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ptrs({h}));
  for (const void* p : {y, w_post, gate, w_pre, (const void*)h_out, (const void*)x})
    if (bad_ptr(p)) return MOE_ERR_INVALID_ARG;
  MOE_CUDA_TRY(launch_block_norm(d, h, y, w_post, gate, w_pre, h_out, x, num_sms(),
                                 static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

moe_status moe_block_norm_backward(const moe_norm_desc* desc, const void* d_h_out,
                                   const void* d_x, const void* h_out, const void* y,
                                   const void* w_post, const void* gate, const void* w_pre,
                                   void* d_h, void* d_y, float* d_w_post, void* d_gate,
                                   float* d_w_pre, void* ws, size_t ws_bytes, moe_stream stream) {
  MOE_TRY(check_norm(desc));
  const moe_norm_desc& d = *desc;
  if ((d_w_post && !w_post) || (d_gate && d.gate == MOE_GATE_NONE) || (d_w_pre && !w_pre))
    return MOE_ERR_INVALID_ARG;
  for (const void* p : {d_h_out, d_x, h_out, y, w_post, gate, w_pre, (const void*)d_h,
                        (const void*)d_y, (const void*)d_w_post, (const void*)d_gate,
                        (const void*)d_w_pre})
    if (bad_ptr(p)) return MOE_ERR_INVALID_ARG;
  if (d.T > 0) {
    if (!y && (w_post || gate || d.gate != MOE_GATE_NONE || d_y)) return MOE_ERR_INVALID_ARG;
    if ((gate != nullptr) != (d.gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if (w_pre && (!d_x || !h_out)) return MOE_ERR_INVALID_ARG;
    if (!w_pre && d_x) return MOE_ERR_INVALID_ARG;
  }
  if (!ws || !aligned16(ws) || ws_bytes < moe_norm_workspace_size(desc))
    return MOE_ERR_WORKSPACE;
  MOE_CUDA_TRY(launch_block_norm_backward(d, d_h_out, d_x, h_out, y, w_post, gate, w_pre, d_h,
                                          d_y, d_w_post, d_gate, d_w_pre,
                                          static_cast<float*>(ws), kPlanSms,
                                          static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

size_t moe_linear_workspace_size(const moe_linear_desc* desc) {
  if (check_linear(desc) != MOE_OK) return 0;
  return linear_layout(*desc).total;
}

moe_status moe_linear(const moe_linear_desc* desc, const void* x, const void* w, const void* bias,
                      const void* residual, void* pre, void* y, void* ws, size_t ws_bytes,
                      moe_stream stream) {
  MOE_TRY(check_linear(desc));
  const moe_linear_desc& d = *desc;
  const LinearLayout L = linear_layout(d);
  if (!ws || !aligned16(ws) || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (d.T == 0) return MOE_OK;
  MOE_TRY(check_ptrs({x, w, y}));
  if (bad_ptr(bias) || bad_ptr(residual) || bad_ptr(pre)) return MOE_ERR_INVALID_ARG;
  const LinearEpilogue epi{y, bias, residual, pre, d.act};
  if (linear_few_tokens(d)) {
    MOE_CUDA_TRY(launch_linear_few(d, x, w, epi, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
  }
  return linear_product(d, L, L.fwd, static_cast<char*>(ws), d.T, d.out, d.in, x, false, w, false,
                        epi, static_cast<cudaStream_t>(stream));
}

moe_status moe_linear_backward(const moe_linear_desc* desc, const void* dy, const void* x,
                               const void* w, const void* pre, void* dx, void* dw, float* d_bias,
                               void* ws, size_t ws_bytes, moe_stream stream) {
  MOE_TRY(check_linear(desc));
  const moe_linear_desc& d = *desc;
  const LinearLayout L = linear_layout(d);
  if (!ws || !aligned16(ws) || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  for (const void* p : {dy, x, w, pre, (const void*)dx, (const void*)dw, (const void*)d_bias})
    if (bad_ptr(p)) return MOE_ERR_INVALID_ARG;
  if (d.T > 0 && (!dy || (dw && !x) || (dx && !w) || (d.act != MOE_ACT_NONE && !pre)))
    return MOE_ERR_INVALID_ARG;
  if (d.act == MOE_ACT_NONE && pre) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(ws);
  if (d.T == 0) {   // sums over no tokens
    if (dw) MOE_CUDA_TRY(cudaMemsetAsync(dw, 0, dtype_size(d.dtype) * d.in * d.out, st));
    if (d_bias) MOE_CUDA_TRY(cudaMemsetAsync(d_bias, 0, sizeof(float) * d.out, st));
    return MOE_OK;
  }
  const void* dz = dy;
  float* parts = d_bias ? reinterpret_cast<float*>(base + L.parts) : nullptr;
  if (d.act != MOE_ACT_NONE || d_bias) {
    void* out = d.act != MOE_ACT_NONE ? base + L.dz : nullptr;
    MOE_CUDA_TRY(launch_linear_act_grad(d, dy, pre, out, parts, st));
    if (out) dz = out;
  }
  if (d_bias) {
    ColumnSums o{};
    o.out[0] = d_bias;
    MOE_CUDA_TRY(launch_column_sums(parts, (d.T + kGradRows - 1) / kGradRows, 1, d.out, o, st));
  }
  if (dx)
    MOE_TRY(linear_product(d, L, L.dx, base, d.T, d.in, d.out, dz, false, w, true,
                           LinearEpilogue{dx, nullptr, nullptr, nullptr, MOE_ACT_NONE}, st));
  if (dw)
    MOE_TRY(linear_product(d, L, L.dw, base, d.out, d.in, d.T, dz, true, x, true,
                           LinearEpilogue{dw, nullptr, nullptr, nullptr, MOE_ACT_NONE}, st));
  return MOE_OK;
}

}  // extern "C"
