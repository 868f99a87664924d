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
// Both kernels move 2 + 0.5 bytes a weight once, so HBM bounds them: 8 x 4096 x
// 14336 quantized in 199, 214 and 239 us with groups of 128, 64 and 32, read back
// in 187 (180 us of bytes at the rate of a copy; groups of 32 take four times the
// maxima, scales and reciprocals).  One warp
// takes 16 columns by 128 rows, all in registers: lane -> (row lane / 2 of 16,
// 8 columns), eight 16-byte loads in flight.  A packed word holds 8 codes of 2
// columns and 4 rows where a lane has 8 columns of one row: an 8 x 8 transposition
// of 4-bit codes among 8 lanes, in three shuffles, with no shared memory.
#include "common.cuh"
#include "w4.cuh"

namespace moe {

constexpr int kW4Warps = 4;           // of a block: 64 adjacent columns

// The transposition of 8 codes: three times a bit of the code's index trades
// places with a lane bit (index bits 0, 1, 2 with lane bits 0, 4, 1), codes whose
// index has that bit going one way between two lanes.  Selections that depend on
// the lane alone are made once.
struct W4Transpose {
  uint32_t keep, turn, bytes, halves;
  __device__ W4Transpose() {
    const int l = threadIdx.x % 32;
    keep = l & 1 ? 0xF0F0F0F0u : 0x0F0F0F0Fu;
    turn = l & 1 ? 28 : 4;
    bytes = l & 16 ? 0x3715u : 0x6240u;
    halves = l & 2 ? 0x3276u : 0x5410u;
  }
  // From 8 columns of row lane / 2 (columns 8 (lane % 2) ..) to the packed word of
  // lane w4_lane(), or back.
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, 1);
    x = (x & keep) | (__funnelshift_l(y, y, turn) & ~keep);
    x = __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 16), bytes);
    return __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 2), halves);
  }
};
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
  const W4Transpose transpose;
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
  constexpr int kG = 128 / G, kPer = G / 16;               // groups; blocks of one
  // Largest magnitudes by group and column: as integers |NaN| > |inf| > |finite|.
  uint32_t m[kG][4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) m[i / kPer][c] = __vmaxu2(m[i / kPer][c], x[c] & 0x7FFF7FFFu);
  }
  // Over the 16 rows in four steps, which also part columns and groups among the
  // lanes, so that a lane ends with two columns (2 c, 2 c + 1) of one group.
  const bool b1 = lane & 2, b2 = lane & 4, b3 = lane & 8, b4 = lane & 16;
  auto part = [&](bool up, uint32_t lo, uint32_t hi, int mask) {
    return __vmaxu2(up ? hi : lo, __shfl_xor_sync(0xffffffffu, up ? lo : hi, mask));
  };
  uint32_t top[kG];
#pragma unroll
  for (int g = 0; g < kG; ++g)
    top[g] = part(b2, part(b1, m[g][0], m[g][2], 2), part(b1, m[g][1], m[g][3], 2), 4);
  uint32_t mx;
  int group = 0;                                           // this lane's
  if constexpr (kG == 4) {
    mx = part(b4, part(b3, top[0], top[2], 8), part(b3, top[1], top[3], 8), 16);
    group = 2 * b3 + b4;
  } else if constexpr (kG == 2) {
    mx = part(b3, top[0], top[1], 8);
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    group = b3;
  } else {
    mx = __vmaxu2(top[0], __shfl_xor_sync(0xffffffffu, top[0], 8));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
  }
  const __nv_bfloat16 sa = w4_scale(__uint_as_float(mx << 16));
  const __nv_bfloat16 sb = w4_scale(__uint_as_float(mx & 0xFFFF0000u));
  const float s0 = __bfloat162float(sa), s1 = __bfloat162float(sb);
  const float i0 = __fdividef(1.0f, s0), i1 = __fdividef(1.0f, s1);
  const bool plain = __all_sync(0xffffffffu, w4_scale_plain(s0) && w4_scale_plain(s1));
  if ((kG == 4 || !b4) && (kG >= 2 || !b3) && group * kPer < t.blocks)
    *reinterpret_cast<uint32_t*>(scale + (t.e * groups + t.k0 / G + group) * N + t.n0 +
                                 8 * (lane % 2) + 4 * b1 + 2 * b2) =
        (uint32_t)__bfloat16_as_ushort(sa) | (uint32_t)__bfloat16_as_ushort(sb) << 16;
  // the lane that holds columns 2 c, 2 c + 1 of group g (and this lane's half)
  auto holder = [&](int g, int c) {
    const int rest = kG == 4 ? (g & 2) << 2 | (g & 1) << 4 : (kG == 2 ? g << 3 : 0);
    return (lane & 1) | (c & 2) | (c & 1) << 2 | rest;
  };
  uint32_t words[4];
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    float inv[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      inv[2 * c] = __shfl_sync(0xffffffffu, i0, holder(g, c));
      inv[2 * c + 1] = __shfl_sync(0xffffffffu, i1, holder(g, c));
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
          const float t0 = __shfl_sync(0xffffffffu, s0, holder(g, c));
          const float t1 = __shfl_sync(0xffffffffu, s1, holder(g, c));
          codes |= w4_code(__uint_as_float(x[c] << 16), t0) << (8 * c);
          codes |= w4_code(__uint_as_float(x[c] & 0xFFFF0000u), t1) << (8 * c + 4);
        }
      }
      words[i % 4] = transpose(codes);
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
  const W4Transpose transpose;
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
    const uint32_t codes = transpose(words[i % 4]);
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
