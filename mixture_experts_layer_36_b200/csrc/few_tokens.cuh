// Arguments of the few-token layer, shared by its kernel and its C entry points.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// One expert matrix [E, K, N]: bf16 (group 0), or 4-bit codes with scales.
struct FewMatrix {
  const void* w;
  const __nv_bfloat16* scale;
  int K, N, group;
};

struct FewArgs {
  const __nv_bfloat16* x;       // [T, d]
  const float* w_router;        // [d, E]
  const float* bias;            // [E] or null
  FewMatrix gate, up, down;
  int T, d, E, k, f, C;         // C: capacity (at most T)
  __nv_bfloat16* y;             // [T, d]
  float* logits;                // [T, E]
  int32_t* topk_idx;            // [T, k]
  float* topk_w;                // [T, k]
  int32_t* slot;                // [T, k]
  int32_t* counts;              // [E]
  int32_t* status;
  uint32_t* sync;               // grid-wide counters (few_tokens.cu)
  double* rpart;                // router partial sums
  float* part;                  // sums of the chunks of G, then of D
  uint8_t* xq;                  // codes: x as digits, [T, ceil(d/128), 3, 144]
  uint8_t* hq;                  // codes: h as digits, [T*k, ceil(f/128), 3, 144]
  __nv_bfloat16* h;             // bf16: [T*k, 2, f], h as two bf16 terms
  int CW, CG, KS;               // router split: columns a block, column groups, row splits
};

// silu in fp32 to within a few ulp (the fast intrinsics' 2^-21 would show next
// to an h that is not rounded)
__device__ __forceinline__ float few_silu(float z) { return z / (1.0f + expf(-z)); }

size_t few_workspace_bytes(int64_t T, int64_t d, int64_t E, int64_t k, int64_t f);
cudaError_t launch_few(FewArgs a, void* ws, cudaStream_t s, bool* map_failed);
cudaError_t launch_quantize_w4(const __nv_bfloat16* w, int E, int K, int N, int G, uint8_t* q,
                               __nv_bfloat16* scale, cudaStream_t s);
cudaError_t launch_dequantize_w4(const uint8_t* q, const __nv_bfloat16* scale, int E, int K, int N,
                                 int G, __nv_bfloat16* w, cudaStream_t s);

}  // namespace moe
