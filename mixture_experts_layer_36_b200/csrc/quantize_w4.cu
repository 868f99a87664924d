// 4-bit expert weights with group scales: quantization and its inverse
// (inferensys.com "Expert Parallelism" glossary, quantization entry).
//
// A group of G rows of one column shares s = bf16(max |v| / 7) (1 where that is
// 0; non-finite where the group holds a NaN or an infinity); the code of v is
// u = 8 + rne(v / s) clamped to 1..15, 8 where v / s is not finite, and stands
// for (u - 8) * s.  The scale is rounded to bf16 (2 bytes a group, 3 % of the
// codes at G = 128 instead of 6 % in fp32) before the codes are taken from it,
// so that rounding adds nothing to the codes' own error of half a step.
#include "common.cuh"
#include "w4.cuh"

namespace moe {

// one thread per (column, group)
__global__ void __launch_bounds__(128)
    w4_quantize_kernel(const __nv_bfloat16* __restrict__ w, int K, int N, int G,
                       uint8_t* __restrict__ q, __nv_bfloat16* __restrict__ scale) {
  const int n = blockIdx.x * 128 + threadIdx.x;
  const int g = blockIdx.y;
  const size_t e = blockIdx.z;
  if (n >= N) return;
  const int k0 = g * G, k1 = min(K, k0 + G);
  const __nv_bfloat16* src = w + e * K * N + n;
  float mx = 0.f;
  for (int k = k0; k < k1; ++k) mx = w4_max(mx, __bfloat162float(src[(size_t)k * N]));
  const __nv_bfloat16 sb = w4_scale(mx);
  const float s = __bfloat162float(sb);
  scale[(e * gridDim.y + g) * N + n] = sb;
  uint32_t* dst = reinterpret_cast<uint32_t*>(q);
  for (int k = k0; k < k1; ++k) {
    const uint32_t u = w4_code(__bfloat162float(src[(size_t)k * N]), s);
    const W4Place p = w4_place(k, n, K / 64, N / 64);
    atomicOr(dst + e * ((size_t)K * N / 8) + p.word, u << (4 * p.nibble));
  }
}

__global__ void __launch_bounds__(128)
    w4_dequantize_kernel(const uint8_t* __restrict__ q, const __nv_bfloat16* __restrict__ scale,
                         int K, int N, int G, __nv_bfloat16* __restrict__ w) {
  const int n = blockIdx.x * 128 + threadIdx.x;
  const int g = blockIdx.y;
  const size_t e = blockIdx.z;
  if (n >= N) return;
  const int k0 = g * G, k1 = min(K, k0 + G);
  const float s = __bfloat162float(scale[(e * gridDim.y + g) * N + n]);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(q) + e * ((size_t)K * N / 8);
  for (int k = k0; k < k1; ++k) {
    const W4Place p = w4_place(k, n, K / 64, N / 64);
    const int u = (src[p.word] >> (4 * p.nibble)) & 15;
    w[(e * K + k) * N + n] = __float2bfloat16(static_cast<float>(u - 8) * s);
  }
}

cudaError_t launch_quantize_w4(const __nv_bfloat16* w, int E, int K, int N, int G, uint8_t* q,
                               __nv_bfloat16* scale, cudaStream_t s) {
  cudaError_t err = cudaMemsetAsync(q, 0, (size_t)E * K * N / 2, s);
  if (err != cudaSuccess) return err;
  w4_quantize_kernel<<<dim3((N + 127) / 128, (K + G - 1) / G, E), 128, 0, s>>>(w, K, N, G, q,
                                                                               scale);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_w4(const uint8_t* q, const __nv_bfloat16* scale, int E, int K,
                                 int N, int G, __nv_bfloat16* w, cudaStream_t s) {
  w4_dequantize_kernel<<<dim3((N + 127) / 128, (K + G - 1) / G, E), 128, 0, s>>>(q, scale, K, N,
                                                                                 G, w);
  return cudaGetLastError();
}

}  // namespace moe
