// C entry points of the few-token layer and of the 4-bit expert weights:
// argument checks and launches.  The kernels are in few_tokens.cu and
// quantize_w4.cu.
#include <nvtx3/nvToolsExt.h>

#include <type_traits>

#include "abi_checks.cuh"
#include "few_tokens.cuh"

namespace {

using moe::abi::aligned16;
using moe::abi::check_routing_shape;
using moe::abi::check_width;
using moe::abi::cuda_status;

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

bool group_ok(int64_t g) { return g == 32 || g == 64 || g == 128; }

// E matrices of K x N in the 4-bit form.
int check_w4(int64_t E, int64_t K, int64_t N, int64_t group) {
  if (E < 1 || E > 65535) return MOE_ERR_INVALID_ARG;
  int st = check_width(K);
  if (st != MOE_OK) return st;
  if ((st = check_width(N)) != MOE_OK) return st;
  if (E * K * N >= (int64_t(1) << 40)) return MOE_ERR_INVALID_ARG;
  return group_ok(group) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int few_shape(int64_t T, int64_t d, int64_t E, int64_t k, int64_t f, double cf) {
  int st = check_routing_shape(T, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_width(d)) != MOE_OK) return st;
  if ((st = check_width(f)) != MOE_OK) return st;
  if (moe_capacity(T, E, k, cf) < 0) return MOE_ERR_INVALID_ARG;
  return T > MOE_FEW_MAX_TOKENS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// The call behind both entry points; group 0: bf16 weights.
int few_layer(const char* name, const void* x, const float* w_router, const float* bias,
              const void* const (&w)[3], const void* const (&s)[3], int64_t T, int64_t d,
              int64_t E, int64_t k, int64_t f, double cf, int64_t group, void* y, float* logits,
              int32_t* topk_idx, float* topk_w, int32_t* slot, int32_t* counts, void* ws,
              size_t ws_bytes, void* stream) {
  int st = few_shape(T, d, E, k, f, cf);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !y || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(y) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (!w[i] || !aligned16(w[i])) return MOE_ERR_INVALID_ARG;
    if (group && (!s[i] || !aligned16(s[i]))) return MOE_ERR_INVALID_ARG;
  }
  if (ws_bytes < moe_workspace_size_few(T, d, E, k, f)) return MOE_ERR_WORKSPACE;
  moe::FewArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.w_router = w_router;
  a.bias = bias;
  auto matrix = [&](int i, int64_t K, int64_t N) {
    return moe::FewMatrix{w[i], static_cast<const __nv_bfloat16*>(s[i]), (int)K, (int)N,
                          (int)group};
  };
  a.gate = matrix(0, d, f);
  a.up = matrix(1, d, f);
  a.down = matrix(2, f, d);
  a.T = (int)T;
  a.d = (int)d;
  a.E = (int)E;
  a.k = (int)k;
  a.f = (int)f;
  const int64_t C = moe_capacity(T, E, k, cf);
  a.C = (int)(C < T ? C : T);                  // a slot never reaches T
  a.y = static_cast<__nv_bfloat16*>(y);
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.slot = slot;
  a.counts = counts;
  nvtxRangePushA(name);
  bool map_failed = false;
  const cudaError_t err = moe::launch_few(a, ws, as_stream(stream), &map_failed);
  nvtxRangePop();
  if (map_failed) return MOE_ERR_CUDA;
  return cuda_status(err);
}

}  // namespace

extern "C" {

int moe_quantize_weights_w4(const void* w, int64_t E, int64_t K, int64_t N, int64_t group,
                            uint8_t* q, void* scale, void* stream) {
  const int st = check_w4(E, K, N, group);
  if (st != MOE_OK) return st;
  if (!w || !q || !scale || !aligned16(w) || !aligned16(q) || !aligned16(scale))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(moe::launch_quantize_w4(static_cast<const __nv_bfloat16*>(w), (int)E, (int)K,
                                             (int)N, (int)group, q,
                                             static_cast<__nv_bfloat16*>(scale),
                                             as_stream(stream)));
}

int moe_dequantize_weights_w4(const uint8_t* q, const void* scale, int64_t E, int64_t K,
                              int64_t N, int64_t group, void* w, void* stream) {
  const int st = check_w4(E, K, N, group);
  if (st != MOE_OK) return st;
  if (!w || !q || !scale || !aligned16(w) || !aligned16(q) || !aligned16(scale))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(moe::launch_dequantize_w4(q, static_cast<const __nv_bfloat16*>(scale), (int)E,
                                               (int)K, (int)N, (int)group,
                                               static_cast<__nv_bfloat16*>(w),
                                               as_stream(stream)));
}

size_t moe_workspace_size_few(int64_t T, int64_t d, int64_t E, int64_t k, int64_t f) {
  if (few_shape(T, d, E, k, f, 0.0) != MOE_OK) return 0;
  return moe::few_workspace_bytes(T, d, E, k, f);
}

int moe_layer_forward_few(const void* x, const float* w_router, const float* bias,
                          const void* w_gate, const void* w_up, const void* w_down, int64_t T,
                          int64_t d, int64_t E, int64_t k, int64_t f, double cf, void* y,
                          float* logits_out, int32_t* topk_idx_out, float* topk_w_out,
                          int32_t* slot_out, int32_t* counts_out, void* ws, size_t ws_bytes,
                          void* stream) {
  return few_layer("moe_layer_forward_few", x, w_router, bias, {w_gate, w_up, w_down},
                   {nullptr, nullptr, nullptr}, T, d, E, k, f, cf, 0, y, logits_out, topk_idx_out,
                   topk_w_out, slot_out, counts_out, ws, ws_bytes, stream);
}

int moe_layer_forward_few_w4(const void* x, const float* w_router, const float* bias,
                             const uint8_t* q_gate, const void* s_gate, const uint8_t* q_up,
                             const void* s_up, const uint8_t* q_down, const void* s_down,
                             int64_t T, int64_t d, int64_t E, int64_t k, int64_t f, double cf,
                             int64_t group, void* y, float* logits_out, int32_t* topk_idx_out,
                             float* topk_w_out, int32_t* slot_out, int32_t* counts_out, void* ws,
                             size_t ws_bytes, void* stream) {
  if (!group_ok(group)) return MOE_ERR_UNSUPPORTED;
  return few_layer("moe_layer_forward_few_w4", x, w_router, bias, {q_gate, q_up, q_down},
                   {s_gate, s_up, s_down}, T, d, E, k, f, cf, group, y, logits_out, topk_idx_out,
                   topk_w_out, slot_out, counts_out, ws, ws_bytes, stream);
}

}  // extern "C"
