// 4-bit expert weights with group scales: quantization and its inverse
// (inferensys.com "Expert Parallelism" glossary, quantization entry).
//
// A group of G rows of one column shares s = bf16(max |v| / 7) (1 where that is
// 0; non-finite where the group holds a NaN or an infinity); the code of v is
// u = 8 + rne(v / s) clamped to 1..15, 8 where v / s is not finite, and stands
// for (u - 8) * s.  The scale is rounded to bf16 (2 bytes a group, 3 % of the
// codes at G = 128 instead of 6 % in fp32) before the codes are taken from it,
// so that rounding adds nothing to the codes' own error of half a step.
//
// Both kernels move 2 + 0.5 bytes a weight once, so HBM bounds them.  One warp
// takes 16 columns by 128 rows, all in registers: lane -> (row lane / 2 of 16,
// 8 columns), eight 16-byte loads in flight.  A packed word holds 8 codes of 2
// columns and 4 rows where a lane has 8 columns of one row: an 8 x 8 transposition
// of 4-bit codes among 8 lanes, in three shuffles, with no shared memory.
#include "common.cuh"
#include "w4.cuh"

namespace moe {

constexpr int kW4Warps = 4;           // of a block: 64 adjacent columns

// Exchange bit B of the code index with lane bit LB: in a word and its
// partner's, the codes whose index has that bit trade places.
template <int LB, int B>
__device__ __forceinline__ uint32_t w4_swap(uint32_t x) {
  constexpr uint32_t kLow = B == 0 ? 0x0F0F0F0Fu : (B == 1 ? 0x00FF00FFu : 0x0000FFFFu);
  constexpr int kShift = 4 << B;
  const uint32_t y = __shfl_xor_sync(0xffffffffu, x, 1 << LB);
  return (threadIdx.x >> LB) & 1 ? (x & ~kLow) | ((y & ~kLow) >> kShift)
                                 : (x & kLow) | ((y & kLow) << kShift);
}
// From 8 columns of row lane / 2 (columns 8 (lane % 2) ..) to the packed word of
// lane w4_lane(), or back.
__device__ __forceinline__ uint32_t w4_transpose(uint32_t x) {
  return w4_swap<1, 2>(w4_swap<4, 1>(w4_swap<0, 0>(x)));
}
// Where this lane's word lies in a block of 16 columns: 4 g + c.
__device__ __forceinline__ int w4_lane() {
  const int l = threadIdx.x % 32;
  const int g = (l & 1) | (l >> 4 & 1) << 1 | (l >> 1 & 1) << 2;
  return 4 * g + (l >> 2 & 3);
}

// One warp's tile: expert, first column, first row; false past the matrix.
struct W4Tile {
  size_t e;
  int n0, k0, blocks;                 // blocks of 16 rows, 8 or 4
  __device__ W4Tile(int K) {
    e = blockIdx.z;
    n0 = (blockIdx.x * kW4Warps + threadIdx.x / 32) * 16;
    k0 = blockIdx.y * 128;
    blocks = min(128, K - k0) / 16;
  }
};

template <int G>
__global__ void __launch_bounds__(32 * kW4Warps)
    w4_quantize_kernel(const __nv_bfloat16* __restrict__ w, int K, int N, uint8_t* __restrict__ q,
                       __nv_bfloat16* __restrict__ scale) {
  const W4Tile t(K);
  const int lane = threadIdx.x % 32;
  const __nv_bfloat16* src = w + (t.e * K + t.k0 + lane / 2) * (size_t)N + t.n0 + 8 * (lane % 2);
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = i < t.blocks ? __ldcs(reinterpret_cast<const uint4*>(src + (size_t)i * 16 * N))
                        : make_uint4(0, 0, 0, 0);
  const size_t groups = (K + G - 1) / G;
  uint4* out = reinterpret_cast<uint4*>(
      q + ((t.e * (N / 64) + t.n0 / 64) * (K / 64) + t.k0 / 64) * 2048 + (t.n0 % 64) * 32) +
      w4_lane();
  uint32_t words[4];
#pragma unroll
  for (int g = 0; g < 128 / G; ++g) {
    constexpr int kPer = G / 16;                           // blocks of a group
    // largest magnitude by column: as integers |NaN| > |inf| > |finite|
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = g * kPer; i < (g + 1) * kPer; ++i) {
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) m[c] = __vmaxu2(m[c], x[c] & 0x7FFF7FFFu);
    }
    // over the 16 rows: the first two steps also part the columns, so that a
    // lane ends with two of them (2 c, 2 c + 1) and works out their scales only
    const bool b1 = lane & 2, b2 = lane & 4;
    uint32_t h[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
      h[c] = __vmaxu2(b1 ? m[2 + c] : m[c],
                      __shfl_xor_sync(0xffffffffu, b1 ? m[c] : m[2 + c], 2));
    uint32_t mx = __vmaxu2(b2 ? h[1] : h[0], __shfl_xor_sync(0xffffffffu, b2 ? h[0] : h[1], 4));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    const __nv_bfloat16 sa = w4_scale(__uint_as_float(mx << 16));
    const __nv_bfloat16 sb = w4_scale(__uint_as_float(mx & 0xFFFF0000u));
    const float s0 = __bfloat162float(sa), s1 = __bfloat162float(sb);
    const float i0 = __fdividef(1.0f, s0), i1 = __fdividef(1.0f, s1);
    const bool plain = __all_sync(0xffffffffu, w4_scale_plain(s0) && w4_scale_plain(s1));
    if (lane < 8 && g * kPer < t.blocks)
      *reinterpret_cast<uint32_t*>(scale + (t.e * groups + t.k0 / G + g) * N + t.n0 +
                                   8 * (lane % 2) + 4 * b1 + 2 * b2) =
          (uint32_t)__bfloat16_as_ushort(sa) | (uint32_t)__bfloat16_as_ushort(sb) << 16;
    float inv[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int from = (lane & ~6) | (c & 2) | (c & 1) << 2;
      inv[2 * c] = __shfl_sync(0xffffffffu, i0, from);
      inv[2 * c + 1] = __shfl_sync(0xffffffffu, i1, from);
    }
#pragma unroll
    for (int i = g * kPer; i < (g + 1) * kPer; ++i) {
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t codes = 0;
      if (plain) {
        // sum of (kW4Bits + u) 16^column, less what the bits add up to
#pragma unroll
        for (int c = 3; c >= 0; --c) {
          codes = codes * 16 + w4_code_bits(__uint_as_float(x[c] & 0xFFFF0000u), inv[2 * c + 1]);
          codes = codes * 16 + w4_code_bits(__uint_as_float(x[c] << 16), inv[2 * c]);
        }
        codes -= kW4Bits * 0x11111111u;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int from = (lane & ~6) | (c & 2) | (c & 1) << 2;
          const float t0 = __shfl_sync(0xffffffffu, s0, from);
          const float t1 = __shfl_sync(0xffffffffu, s1, from);
          codes |= w4_code(__uint_as_float(x[c] << 16), t0) << (8 * c);
          codes |= w4_code(__uint_as_float(x[c] & 0xFFFF0000u), t1) << (8 * c + 4);
        }
      }
      words[i % 4] = w4_transpose(codes);
      if (i % 4 == 3 && i < t.blocks)
        out[(i / 4) * 128] = make_uint4(words[0], words[1], words[2], words[3]);
    }
  }
}

template <int G>
__global__ void __launch_bounds__(32 * kW4Warps)
    w4_dequantize_kernel(const uint8_t* __restrict__ q, const __nv_bfloat16* __restrict__ scale,
                         int K, int N, __nv_bfloat16* __restrict__ w) {
  const W4Tile t(K);
  const int lane = threadIdx.x % 32;
  const uint4* src = reinterpret_cast<const uint4*>(
      q + ((t.e * (N / 64) + t.n0 / 64) * (K / 64) + t.k0 / 64) * 2048 + (t.n0 % 64) * 32) +
      w4_lane();
  const size_t groups = (K + G - 1) / G;
  const __nv_bfloat16* sc = scale + (t.e * groups + t.k0 / G) * N + t.n0 + 8 * (lane % 2);
  __nv_bfloat16* dst = w + (t.e * K + t.k0 + lane / 2) * (size_t)N + t.n0 + 8 * (lane % 2);
  uint4 v[2];
  uint4 s4[128 / G];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (4 * i < t.blocks) v[i] = __ldcs(src + i * 128);
#pragma unroll
  for (int g = 0; g < 128 / G; ++g)
    if (g * (G / 16) < t.blocks) s4[g] = __ldg(reinterpret_cast<const uint4*>(sc + (size_t)g * N));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= t.blocks) break;
    const uint32_t words[4] = {v[i / 4].x, v[i / 4].y, v[i / 4].z, v[i / 4].w};
    const uint4 sg = s4[i * 16 / G];
    const uint32_t s[4] = {sg.x, sg.y, sg.z, sg.w};
    const uint32_t codes = w4_transpose(words[i % 4]);
    uint32_t o[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float lo = static_cast<float>((int)(codes >> (8 * c) & 15) - 8);
      const float hi = static_cast<float>((int)(codes >> (8 * c + 4) & 15) - 8);
      o[c] = pack_bf16x2(lo * __uint_as_float(s[c] << 16),
                         hi * __uint_as_float(s[c] & 0xFFFF0000u));
    }
    __stcs(reinterpret_cast<uint4*>(dst + (size_t)i * 16 * N), make_uint4(o[0], o[1], o[2], o[3]));
  }
}

static dim3 w4_grid(int E, int K, int N) { return dim3(N / (16 * kW4Warps), (K + 127) / 128, E); }

cudaError_t launch_quantize_w4(const __nv_bfloat16* w, int E, int K, int N, int G, uint8_t* q,
                               __nv_bfloat16* scale, cudaStream_t s) {
  const dim3 grid = w4_grid(E, K, N);
  if (G == 128)
    w4_quantize_kernel<128><<<grid, 32 * kW4Warps, 0, s>>>(w, K, N, q, scale);
  else if (G == 64)
    w4_quantize_kernel<64><<<grid, 32 * kW4Warps, 0, s>>>(w, K, N, q, scale);
  else
    w4_quantize_kernel<32><<<grid, 32 * kW4Warps, 0, s>>>(w, K, N, q, scale);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_w4(const uint8_t* q, const __nv_bfloat16* scale, int E, int K,
                                 int N, int G, __nv_bfloat16* w, cudaStream_t s) {
  const dim3 grid = w4_grid(E, K, N);
  if (G == 128)
    w4_dequantize_kernel<128><<<grid, 32 * kW4Warps, 0, s>>>(q, scale, K, N, w);
  else if (G == 64)
    w4_dequantize_kernel<64><<<grid, 32 * kW4Warps, 0, s>>>(q, scale, K, N, w);
  else
    w4_dequantize_kernel<32><<<grid, 32 * kW4Warps, 0, s>>>(q, scale, K, N, w);
  return cudaGetLastError();
}

}  // namespace moe
