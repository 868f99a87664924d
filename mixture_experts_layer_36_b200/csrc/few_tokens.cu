// The MoE layer for a few tokens (a decode step), on bf16 experts or on 4-bit
// codes with group scales.  Simple form: one kernel per step, one thread per
// column, every sum in a fixed order.
#include "abi_checks.cuh"
#include "common.cuh"
#include "host_util.cuh"
#include "few_tokens.cuh"
#include "w4.cuh"

namespace moe {

__global__ void __launch_bounds__(256)
    few_route_kernel(FewArgs a) {
  __shared__ float l[256];
  const int t = blockIdx.x, e = threadIdx.x;
  if (e < a.E) {
    double acc = 0.0;
    for (int i = 0; i < a.d; ++i)
      acc += (double)__bfloat162float(a.x[(size_t)t * a.d + i]) * (double)a.w_router[(size_t)i * a.E + e];
    if (a.bias) acc += (double)a.bias[e];
    l[e] = (float)acc;
    a.logits[(size_t)t * a.E + e] = l[e];
  }
  __syncthreads();
  if (e == 0) {
    uint64_t used[4] = {0, 0, 0, 0};
    float v[8], p[8], sum = 0.f;
    int id[8];
    for (int j = 0; j < a.k; ++j) {
      int best = -1;
      for (int c = 0; c < a.E; ++c) {
        if (used[c / 64] >> (c % 64) & 1) continue;
        if (best < 0 || few_order(l[c]) > few_order(l[best])) best = c;
      }
      used[best / 64] |= 1ull << (best % 64);
      v[j] = l[best];
      id[j] = best;
    }
    for (int j = 0; j < a.k; ++j) sum += p[j] = expf(v[j] - v[0]);
    for (int j = 0; j < a.k; ++j) {
      a.topk_idx[t * a.k + j] = id[j];
      a.topk_w[t * a.k + j] = p[j] / sum;
    }
  }
}

__global__ void __launch_bounds__(256) few_slot_kernel(FewArgs a) {
  const int e = threadIdx.x;
  if (e >= a.E) return;
  int n = 0;
  for (int p = 0; p < a.T * a.k; ++p)
    if (a.topk_idx[p] == e) {
      a.slot[p] = n < a.C ? n : -1;
      ++n;
    }
  a.counts[e] = min(n, a.C);
}

__device__ float few_weight(const FewMatrix& m, int e, int kk, int n) {
  if (m.group == 0)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(m.w)[((size_t)e * m.K + kk) * m.N + n]);
  const W4Place p = w4_place(kk, n, m.K / 64, m.N / 64);
  const uint32_t word = static_cast<const uint32_t*>(m.w)[(size_t)e * m.K * m.N / 8 + p.word];
  const int groups = (m.K + m.group - 1) / m.group;
  const float s = __bfloat162float(m.scale[((size_t)e * groups + kk / m.group) * m.N + n]);
  return (float)((int)((word >> (4 * p.nibble)) & 15) - 8) * s;
}

__global__ void __launch_bounds__(64) few_gate_up_kernel(FewArgs a) {
  const int p = blockIdx.y, t = p / a.k, n = blockIdx.x * 64 + threadIdx.x;
  if (a.slot[p] < 0) return;
  const int e = a.topk_idx[p];
  float g = 0.f, u = 0.f;
  for (int i = 0; i < a.d; ++i) {
    const float x = __bfloat162float(a.x[(size_t)t * a.d + i]);
    g += x * few_weight(a.gate, e, i, n);
    u += x * few_weight(a.up, e, i, n);
  }
  a.h[(size_t)p * a.f + n] = few_silu(g) * u;
}

__global__ void __launch_bounds__(64) few_down_kernel(FewArgs a) {
  const int t = blockIdx.y, n = blockIdx.x * 64 + threadIdx.x;
  float y = 0.f;
  bool any = false;
  for (int j = 0; j < a.k; ++j) {
    const int p = t * a.k + j;
    if (a.slot[p] < 0) continue;
    any = true;
    float o = 0.f;
    for (int i = 0; i < a.f; ++i) o += a.h[(size_t)p * a.f + i] * few_weight(a.down, a.topk_idx[p], i, n);
    y += a.topk_w[p] * o;
  }
  a.y[(size_t)t * a.d + n] = any ? __float2bfloat16(y) : a.x[(size_t)t * a.d + n];
}

size_t few_workspace_bytes(int64_t T, int64_t d, int64_t E, int64_t k, int64_t f) {
  (void)d;
  return few_header_bytes(T, E, k) + (size_t)(T * k * f) * 4;
}

cudaError_t launch_few(FewArgs a, void* ws, cudaStream_t s, bool* map_failed) {
  *map_failed = false;
  cudaError_t err = cudaMemsetAsync(ws, 0, 4, s);
  if (err != cudaSuccess) return err;
  few_place_header(&a, ws);
  a.h = reinterpret_cast<float*>(static_cast<char*>(ws) + few_header_bytes(a.T, a.E, a.k));
  few_route_kernel<<<a.T, 256, 0, s>>>(a);
  few_slot_kernel<<<1, 256, 0, s>>>(a);
  few_gate_up_kernel<<<dim3(a.f / 64, a.T * a.k), 64, 0, s>>>(a);
  few_down_kernel<<<dim3(a.d / 64, a.T), 64, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
