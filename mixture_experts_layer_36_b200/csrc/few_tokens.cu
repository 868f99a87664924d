// The MoE layer for a few tokens (a decode step) as one persistent kernel, on
// bf16 experts or on 4-bit codes with group scales.
//
// With T tokens and A distinct experts chosen, the layer reads 3 A d f weights
// and takes 2 operations per weight and token: for T <= 32 the time is the
// weights' bytes at the HBM rate, plus whatever keeps the memory idle.  So the
// kernel is one stream of weights: one CTA per SM, which takes chunks of the
// matrices' blocks from a counter, a ring of shared-memory stages that a producer
// warp fills by TMA, and the dependencies between the steps taken inside the
// kernel (a cooperative launch), where the ring stays full across them:
//   R  router: every CTA sums its rows of x Wr in fp64 (the choice of experts
//      must not hang on the order of a sum); the CTA of token t adds the
//      partial sums, rounds once to fp32, and one warp picks the top k;
//   G  gate/up: units of (expert, 128 columns of f, all of d) are cut into
//      chunks of a few blocks, which CTAs take from a counter (SMs see up to a
//      tenth more or less of the memory's rate, so equal shares leave the fast
//      ones idle); each chunk leaves fp32 sums in the workspace;
//   H  the chunks of a unit are added in order and h = silu(g) u is stored for
//      the next products (bf16 weights: as two bf16 terms, hi + lo, 2^-16);
//   D  down: the same over (expert, 256 columns of d, all of f); its first
//      weights are in flight while H runs;
//   Y  the weighted sums of each token's k rows.
// The cuts follow from the shapes and the routing alone and sums are added in
// a fixed order, so results do not depend on which CTA took what.
//
// Measured (in brackets the bytes at the rate of a copy, 6.55 TB/s), on several
// boxes: 256 experts of 7168 x 2048, k = 8, one token 121 to 123 us on bf16 (109) and
// 52 to 55 on codes of groups of 128 (29), 32 tokens 2022 to 2146 (2196) and 623 to
// 657 (567); 8 experts of 4096 x 14336, k = 2, groups of 64, 8 tokens 123 to 157 (86
// to 114 for 6 to 8 experts chosen).  What is above the bytes is some 25 us of
// router, tables, grid-wide waits and first blocks; on codes of few experts with
// many tokens each also the products themselves (32 tokens 227 to 275, groups of
// 128, of 111).
//
// The products run on mma.sync with the weights as the 16-row operand and the
// tokens as the 8 columns: bf16 m16n8k16 on bf16 weights, s8 m16n8k32 on codes
// (8 clocks an SM sub-partition each).  An SM gets 23 bytes of weights a clock
// from HBM, for which one 8-column block keeps that unit a tenth (bf16) or a
// fifth (codes) busy; tcgen05 would want the codes back in shared memory.
#include <type_traits>

#include "abi_checks.cuh"
#include "common.cuh"
#include "few_tokens.cuh"
#include "host_util.cuh"

namespace moe {

// A team: 8 consumer warps with two 16-column strips of a tile each, a thread
// that issues the weights' copies and a warp that loads token rows, with a ring
// of stages and a row of chunks of its own.  bf16 blocks leave one team idle
// half the time; on codes two teams hide one another's latencies (8 warps: 480
// clocks a block at one token block, 680 at three; 2 x 8: 330 and 630), although
// 640 threads leave 96 registers each and the forms on codes then spill 40 to 220
// bytes (the bf16 ones, 320 threads of up to 168, 8 at most).  One team for
// units of more than 8 tokens, with registers for them, is not tried.
constexpr int kTeamWarps = 8;
constexpr int kFewMaxPairs = MOE_FEW_MAX_TOKENS * 8;
constexpr int kFewRouterRows = 384;                // router rows staged at once
constexpr int kFewMaxSplits = 32;
constexpr int kFewMaxStages = 10;
constexpr int kDigitBytes = 3 * 144;               // 128 values of a token as int8 digits
constexpr float kCodesUnit = 2048.f;               // of the sums that chunks of codes leave

// The chunks of a phase keep sums of at most T*k*tiles + few_part_rows(T) tile
// rows (1 KB each): room for 2560 chunks, 8 or more a team, of 4 tokens.
inline __host__ __device__ int few_part_rows(int T) { return 2560 * (T < 4 ? T : 4); }

// grid-wide counters, zeroed by the call, each on its own line: arrivals of the
// router's partial sums, of the tokens' routing, of the CTAs that finished G,
// H and D; the next chunk of G and of D.
constexpr int kSyncRouter = 0, kSyncRouted = 32, kSyncG = 64, kSyncH = 96, kSyncY = 128,
              kSyncNext = 160, kSyncWords = 224;

// KIND 0: bf16; 1, 2, 3: codes with groups of 128, 64, 32 rows.
// Tokens enter the products as bf16 rows (KIND 0: x, and h as two terms), or
// as three rows of int8 digits (codes; few_digits below).
template <int KIND, int NBT>
struct FewCfg {
  static constexpr int kTeams = KIND == 0 ? 1 : 2;
  static constexpr int kWorkers = 32 * kTeamWarps * kTeams;      // consumer threads
  static constexpr int kThreads = kWorkers + 64 * kTeams;
  static constexpr int KB = KIND == 0 ? 64 : 128;         // rows of a block
  static constexpr int G = 256 >> KIND;                   // rows of a group (codes)
  static constexpr int kWBytes = KIND == 0 ? 32768 : 16384;
  static constexpr int kScaleBytes = KIND == 0 ? 0 : KB / G * 512;
  // a token row: 128 bytes of values, 16 of padding, which keep ldmatrix free
  // of bank conflicts (and hold the scale of the digits)
  static constexpr int kPitch = 144;
  // tokens of a unit: with codes, an expert with more has several units, whose
  // chunks run side by side and find the weights in L2 (a block's time grows
  // with its tokens there, and two teams leave 96 registers a thread)
  static constexpr int kUnitTokens = KIND != 0 ? 8 : 8 * NBT;
  static constexpr int kRows = (KIND == 0 ? 2 : 3) * kUnitTokens;
  static constexpr int kColsG = (KIND == 0 ? 1 : 3) * kUnitTokens / 8;   // most 8-column blocks
  static constexpr int kColsD = (KIND == 0 ? 2 : 3) * kUnitTokens / 8;
  static constexpr int kStageBytes =
      (kWBytes + kScaleBytes + kRows * kPitch + 1023) / 1024 * 1024;
  static constexpr int kFit = 224256 / kStageBytes / kTeams;
  static constexpr int kStages = kFit > kFewMaxStages / 2 * (3 - kTeams)
                                     ? kFewMaxStages / 2 * (3 - kTeams) : kFit;   // of a team
  static constexpr int kSmemBytes = kTeams * kStages * kStageBytes + 1024;
  // the router's staging uses the same memory: x (fp64), then W rows
  static constexpr int kXsBytes = (8 * NBT + 2) * kFewRouterRows * 8;
  static_assert(kXsBytes + kFewRouterRows * 32 * 4 < kSmemBytes - 1024, "router staging");
  static_assert(kWorkers * 8 * NBT * 8 < kSmemBytes - 1024, "router reduction");
};

// The chunk whose first block a stage holds (len 0: the phase is over).
struct alignas(16) ChunkInfo {
  int len, kb0, a, c;                 // blocks, the first one; active expert, column tile
  int n, row0, e, sums;               // its rows and expert; where its sums go (1 KB each)
};

// How a phase is cut: column tiles, blocks of a unit, blocks of a chunk, chunks
// of a unit, of the phase.
struct Phase {
  int nct, nkb, len, q, chunks;
  // Where the sums of chunk 0 of a unit lie, in tokens of 256 floats (1 KB); the
  // next chunk's are n further.
  __device__ int tile_at(int row0, int n, int c) const { return (row0 * nct + c * n) * q; }
};

struct FewShared {
  uint64_t full[kFewMaxStages];       // weights, token rows and scales have landed
  uint64_t empty[kFewMaxStages];      // all consumer warps are done with the stage
  uint64_t ready[kFewMaxStages];      // the weights' copy is issued, info is written
  ChunkInfo info[kFewMaxStages];
  int abort_flag, never, ok;
  uint32_t mask[256];                 // tokens that chose expert e
  uint16_t row0[257];                 // first kept row of active expert a (with codes: of
                                      // at most 8 rows of one; so for all a below)
  uint8_t expert[256];                // active expert a -> e
  uint8_t active[256];                // e -> its first a
  uint8_t part0[256], parts[256];     // a -> the first a of its expert, and their number
  uint8_t row_tok[kFewMaxPairs];      // kept row -> token
  uint8_t row_a[kFewMaxPairs];        // kept row -> active expert
  int16_t pair_row[kFewMaxPairs];     // pair -> kept row, -1 dropped
  float pair_w[kFewMaxPairs];
  int pick_e[16];                     // experts of the tokens routed by this CTA
  float logit[2][256];
  uint32_t warp_sum[8];
  int A;                              // active experts
  Phase phase[2];                     // G, D
};

// ---------------------------------------------------------------- small pieces
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release(uint32_t* p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}
// order this thread's and (through barriers) other threads' generic accesses
// with asynchronous copies of the same memory
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}
// c = products + (first ? init : c)
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1, bool first,
                                       int init) {
  if (first)
    asm(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(init));
  else
    asm(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (w & m) ^ c in one instruction
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t m, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(m), "r"(c));
  return r;
}
// The weights pass through L2 as its first lines to go: what the phases hand on,
// the tokens and the kernel's code stay (with other memory read in between, 8
// experts of 4096 x 14336, 32 tokens, bf16: 465 -> 442 us; fine-grained, one token,
// codes: 64.4 -> 62.6).
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------- digits
// Products with 4-bit codes are taken in integers: a code is an int8 operand
// after a mask and an xor (16 (u - 8); the bf16 operand takes four times the
// instructions, which made that form issue-bound at 38 % of the HBM rate), and
// s8 m16n8k32 does twice the products of bf16 m16n8k16 in the same 8 clocks.
// 128 values of a token are held as v = rint(x 2^(22 - e)), 2^(e-1) <= max|x| <
// 2^e, in three balanced base-256 digits: fixed point with 23 bits and sign
// relative to the largest of the 128, exact for a bf16 x down to 2^-14 of it
// (the last bit of an 8-bit significand at 2^(e-15) is the unit 2^(e-22)).
// Every digit is a token column of the product; sums of 128 rows are at most
// 2^21 (digit -128, code 0) and exact.
struct DigitScale {
  float inv;        // 2^(22 - e)
  float unit;       // 2^(e - 22) / 16, NaN if the largest is not finite
};
__device__ __forceinline__ DigitScale digit_scale(float mx) {
  int e = (int)((__float_as_uint(mx) >> 23) & 255) - 126;
  const bool bad = e > 128;
  e = max(-100, min(e, 128));
  DigitScale s;
  s.inv = bad ? 0.f : __uint_as_float((uint32_t)(22 - e + 127) << 23);
  s.unit = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(e - 26 + 127) << 23);
  return s;
}
// the digits of x, lowest first, as bytes 0..2
__device__ __forceinline__ uint32_t digits_of(float x, const DigitScale& s) {
  const int v = s.inv == 0.f ? 0 : __float2int_rn(x * s.inv);
  const int d0 = (int)(int8_t)(v & 255);
  const int v1 = (v - d0) >> 8;
  const int d1 = (int)(int8_t)(v1 & 255);
  const int d2 = (v1 - d1) >> 8;
  return (uint32_t)(d0 & 255) | (uint32_t)(d1 & 255) << 8 | (uint32_t)(d2 & 255) << 16;
}

// Wait until the counter reaches `target`; false after kWaitLimitNs, or when
// another role of this CTA gave up.
__device__ __forceinline__ bool wait_count(const uint32_t* c, uint32_t target,
                                           volatile int* abort) {
  if (ld_acquire(c) >= target) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ld_acquire(c) >= target) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
}

__device__ __forceinline__ int few_tiles(int width, int tile) { return (width + tile - 1) / tile; }

__device__ __forceinline__ ChunkInfo chunk_info(const FewShared& sh, const Phase& ph, int id) {
  // an expert's units take turns, so that they read the same weights together
  const int f = sh.part0[id / (ph.q * ph.nct)], m = sh.parts[f];
  const int in = id - f * ph.nct * ph.q, chunk = in / m, a = f + in - chunk * m;
  ChunkInfo i;
  i.a = a;
  i.c = chunk / ph.q;
  const int qi = chunk - i.c * ph.q;
  i.kb0 = qi * ph.len;
  i.len = min(ph.len, ph.nkb - i.kb0);
  i.row0 = sh.row0[a];
  i.n = sh.row0[a + 1] - i.row0;
  i.e = sh.expert[a];
  i.sums = ph.tile_at(i.row0, i.n, i.c) + qi * i.n;
  return i;
}

// The cut of a phase, by one warp: each lane weighs two chunk lengths by the
// time of the team with the most chunks, in sixteenths of a block's time, a chunk
// costing kChunkCost on top of its blocks; on codes, half a chunk more for teams
// that take their last one late.  Short chunks cost starts and sums to add, long
// ones leave teams idle at the end.  Measured in us at a cost of 8 (10 on codes),
// 32, 96: 8 experts of 4096 x 14336, one token, bf16 122.0, 120.0, 121.0; 64 of
// 7168 x 2048, one token, bf16 121.5, 121.0, 122.9, codes 56.1, 54.6, 53.8; codes
// of the 8 experts at 8 tokens 135.9, 137.0, 139.5, and 141.9 without the half.
constexpr int kChunkCost = 32;
__device__ void few_cut(const FewArgs& p, FewShared& sh, int which, int nct, int nkb, bool codes) {
  const int lane = threadIdx.x % 32;
  const unsigned teams = gridDim.x * (codes ? 2 : 1);
  const int units = sh.A * nct, rows = sh.row0[sh.A] * nct;
  const int q_max = (p.T * p.k * nct + few_part_rows(p.T)) / rows;     // 1 or more
  unsigned best = 0xFFFFFFFFu;
  int best_len = nkb;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // lengths of 1 to 32 blocks, and units cut in 1 to 32
    const int len = min(nkb, i ? (nkb + lane) / (lane + 1) : lane + 1);
    const int q = (nkb + len - 1) / len;
    const unsigned rounds = ((unsigned)units * q + teams - 1) / teams;
    const unsigned long long cost =
        (unsigned long long)rounds * (16u * len + kChunkCost) +
        (codes ? 8u * len : 0u);
    const unsigned c = q > q_max || cost > 0x7FFFFFFFull ? 0xFFFFFFFEu : (unsigned)cost;
    if (c < best) {
      best = c;
      best_len = len;
    }
  }
  const unsigned least = __reduce_min_sync(0xffffffffu, best);
  const unsigned len = __reduce_max_sync(0xffffffffu, best == least ? (unsigned)best_len : 0u);
  if (lane == 0) {
    // no candidate within bounds (units longer than 32 q_max blocks): whole units
    const int l = least >= 0xFFFFFFFEu ? nkb : (int)len, q = (nkb + l - 1) / l;
    sh.phase[which] = Phase{nct, nkb, l, q, units * q};
  }
}

// ---------------------------------------------------------------- R: router
// Partial sums of this CTA's rows and columns for all tokens, in fp64.
template <int NBT, int kWorkers>
__device__ void few_router_rows(const FewArgs& p, uint8_t* smem) {
  constexpr int RR = kFewRouterRows, TT = 8 * NBT, TP = TT + 2;   // padded: no bank conflicts
  const int tid = threadIdx.x;
  const bool worker = tid < kWorkers;
  const int cg = blockIdx.x % p.CG, ks = blockIdx.x / p.CG;
  const int c = tid % p.CW, rg = tid / p.CW, nrg = kWorkers / p.CW;
  const int col0 = cg * p.CW, cols = min(p.CW, p.E - col0);
  const int k0 = (int)((long long)p.d * ks / p.KS), k1 = (int)((long long)p.d * (ks + 1) / p.KS);
  double* xs = reinterpret_cast<double*>(smem);                    // [RR][TP]
  float* wsm = reinterpret_cast<float*>(smem + TP * RR * 8);       // [RR][CW]
  double acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.0;
  for (int base = k0; base < k1; base += RR) {
    const int len = min(RR, k1 - base);
    if (base != k0) __syncthreads();
    if (worker) {
      const float* src = p.w_router + (size_t)base * p.E + col0;
      if (p.E % 4 == 0) {
        const int lg = __ffs(p.CW) - 3;                     // CW / 4 of 16 bytes a row
#pragma unroll 4
        for (int i = tid; i < len << lg; i += kWorkers) {
          const int r = i >> lg, v = i - (r << lg);
          if (4 * v < cols)
            cp_async16(smem_u32(wsm + r * p.CW + 4 * v), src + (size_t)r * p.E + 4 * v);
        }
      } else {
        for (int i = tid; i < len * p.CW; i += kWorkers) {
          const int r = i / p.CW, v = i % p.CW;
          if (v < cols) cp_async4(smem_u32(wsm + r * p.CW + v), src + (size_t)r * p.E + v);
        }
      }
      // x as fp64, a row's tokens together: two a load below
      if (NBT == 1) {
        for (int r = tid; r < len; r += kWorkers) {
#pragma unroll 8
          for (int t = 0; t < p.T; ++t)
            xs[r * TP + t] = (double)__bfloat162float(p.x[(size_t)t * p.d + base + r]);
        }
      } else {                                    // a warp for each token
        for (int t = tid / 32; t < p.T; t += kWorkers / 32) {
          const __nv_bfloat16* x = p.x + (size_t)t * p.d + base;
#pragma unroll 8
          for (int r = tid % 32; r < len; r += 32) xs[r * TP + t] = (double)__bfloat162float(x[r]);
        }
      }
      cp_async_wait();
    }
    __syncthreads();
    if (worker && c < cols) {
      if (NBT == 1 && p.T == 1) {                // one token: four chains of sums
#pragma unroll 2
        for (int r = rg; r < len; r += 4 * nrg)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (r + i * nrg < len)
              acc[i] = fma((double)wsm[(r + i * nrg) * p.CW + c], xs[(r + i * nrg) * TP], acc[i]);
      } else {
#pragma unroll 2
        for (int r = rg; r < len; r += nrg) {
          const double w = (double)wsm[r * p.CW + c];
          const double2* x = reinterpret_cast<const double2*>(xs + r * TP);
#pragma unroll
          for (int t = 0; t < TT / 2; ++t) {
            const double2 v = x[t];
            acc[2 * t] = fma(w, v.x, acc[2 * t]);
            acc[2 * t + 1] = fma(w, v.y, acc[2 * t + 1]);
          }
        }
      }
    }
  }
  if (NBT == 1 && p.T == 1) acc[0] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  __syncthreads();
  double* red = reinterpret_cast<double*>(smem);                   // [T][kWorkers]
  if (worker) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
      if (t < p.T) red[t * kWorkers + tid] = acc[t];
  }
  __syncthreads();
  if (worker) {
    for (int i = tid; i < p.T * p.CW; i += kWorkers) {
      const int t = i / p.CW, cc = i % p.CW;
      if (cc >= cols) continue;
      double s = 0.0;
#pragma unroll 8
      for (int g = 0; g < nrg; ++g) s += red[t * kWorkers + g * p.CW + cc];
      p.rpart[((size_t)ks * p.T + t) * p.E + col0 + cc] = s;
    }
  }
}

// The digits of 128 values of a token, by one warp.  Row r of 16 lies at byte 4 c
// + 2 h + v, r = 8 v + 2 c + h, the order of the codes' rows in a word: lane has
// rows 2 c, 8 + 2 c, 2 c + 1, 9 + 2 c of 16, c = lane % 4.
__device__ __forceinline__ void put_digits(uint8_t* out, const float (&x)[4]) {
  const int lane = threadIdx.x % 32;
  // as integers, |NaN| > |inf| > |finite|
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  m = __reduce_max_sync(0xffffffffu, m);
  const DigitScale s = digit_scale(__uint_as_float(m));
  uint32_t d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] = digits_of(x[j], s);
#pragma unroll
  for (int l = 0; l < 3; ++l) {
    const uint32_t sel = 0x0040u + 0x0011u * l;              // byte l of two words
    const uint32_t w = __byte_perm(__byte_perm(d[0], d[1], sel), __byte_perm(d[2], d[3], sel),
                                   0x5410);
    *reinterpret_cast<uint32_t*>(out + l * 144 + 4 * lane) = w;
    if (lane < 4)
      *reinterpret_cast<float*>(out + l * 144 + 128 + 4 * lane) =
          lane == 0 ? s.unit * (float)(1 << (8 * l)) : 0.f;
  }
}

// The digits of the tokens.
__device__ void few_digits(const FewArgs& p) {
  const int lane = threadIdx.x % 32, nkb = (p.d + 127) / 128;
  for (int i = threadIdx.x / 32 * gridDim.x + blockIdx.x; i < p.T * nkb;
       i += blockDim.x / 32 * gridDim.x) {
    const int t = i / nkb, kb = i - t * nkb;
    const int at = kb * 128 + (lane / 4) * 16 + 2 * (lane % 4);
    uint32_t lo = 0, hi = 0;
    if (at < p.d) {
      const __nv_bfloat16* src = p.x + (size_t)t * p.d + at;
      lo = __ldg(reinterpret_cast<const uint32_t*>(src));
      hi = __ldg(reinterpret_cast<const uint32_t*>(src + 8));
    }
    const float x[4] = {__uint_as_float(lo << 16), __uint_as_float(hi << 16),
                        __uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi & 0xFFFF0000u)};
    put_digits(p.xq + (size_t)i * kDigitBytes, x);
  }
}

// Logits, top-k and gate weights of tokens t0, t0 + 1, .. (one for every 256
// worker threads; all threads of the CTA come here), into shared memory and,
// where `write` is set, to the results.
template <int kWorkers>
__device__ void few_route(const FewArgs& p, FewShared& sh, int t0, bool write) {
  const int tid = threadIdx.x % 256, which = threadIdx.x / 256, t = t0 + which;
  const bool mine = threadIdx.x < kWorkers && t < p.T;
  if (mine && tid < p.E) {
    double v[kFewMaxSplits];
#pragma unroll
    for (int i = 0; i < kFewMaxSplits; ++i)
      v[i] = i < p.KS ? __ldcg(p.rpart + ((size_t)i * p.T + t) * p.E + tid) : 0.0;
    double s[4] = {p.bias ? (double)__ldg(p.bias + tid) : 0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kFewMaxSplits; ++i) s[i % 4] += v[i];
    const float l = (float)((s[0] + s[1]) + (s[2] + s[3]));
    sh.logit[which][tid] = l;
    if (write) p.logits[(size_t)t * p.E + tid] = l;
  }
  __syncthreads();
  if (mine && tid < 32) {
    const float* logit = sh.logit[which];
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = tid + 32 * i;
      key[i] = e < p.E ? logit_key(logit[e]) : 0u;          // no number has key 0
    }
    int own_e = 0;
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = 0, be = 256;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (key[i] > best) {
          best = key[i];
          be = tid + 32 * i;
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? be : 256u);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e == tid + 32u * i) key[i] = 0u;
      if (tid == j) own_e = (int)e;
    }
    const float v = logit[own_e], v0 = __shfl_sync(0xffffffffu, v, 0);
    const float own = tid < p.k ? expf(v - v0) : 0.f;
    float sum = own;                                        // lanes 0..7 hold the k
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (tid < p.k) {
      sh.pick_e[which * p.k + tid] = own_e;
      sh.pair_w[which * p.k + tid] = own / sum;
      if (write) {
        p.topk_idx[t * p.k + tid] = own_e;
        p.topk_w[t * p.k + tid] = own / sum;
      }
    }
  }
}

// Which experts run and on which tokens: every CTA builds the same tables.
template <int kUnitTokens>
__device__ void few_tables(const FewArgs& p, FewShared& sh, bool local) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int pairs = p.T * p.k;
  int e = 0, t = 0;
  if (tid < pairs) {
    if (local) {
      e = sh.pick_e[tid];
    } else {
      e = __ldcg(p.topk_idx + tid);
      sh.pair_w[tid] = __ldcg(p.topk_w + tid);
    }
    t = tid / p.k;
    atomicOr(&sh.mask[e], 1u << t);                // k distinct experts a token
  }
  __syncthreads();
  uint32_t n = 0, v = 0, incl = 0;
  if (tid < 256) {
    n = min(__popc(sh.mask[tid]), p.C);
    v = n | (n + kUnitTokens - 1) / kUnitTokens << 16;
    incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
  }
  __syncthreads();
  if (tid < 256) {
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
    const uint32_t excl = before + incl - v;
    if (n) {
      const int a = (int)(excl >> 16);
      sh.active[tid] = (uint8_t)a;
      const int parts = ((int)n + kUnitTokens - 1) / kUnitTokens;
      for (int i = 0; i < parts; ++i) {
        sh.part0[a + i] = (uint8_t)a;
        sh.parts[a + i] = (uint8_t)parts;
        sh.expert[a + i] = (uint8_t)tid;
        sh.row0[a + i] = (uint16_t)((excl & 0xFFFF) + i * kUnitTokens);
      }
    }
    if (tid == 255) {
      const uint32_t all = before + incl;
      sh.A = (int)(all >> 16);
      sh.row0[all >> 16] = (uint16_t)(all & 0xFFFF);
    }
    if (blockIdx.x == 0 && tid < p.E) p.counts[tid] = (int)n;
  }
  __syncthreads();
  if (tid < pairs) {
    const int slot = __popc(sh.mask[e] & ((1u << t) - 1));
    const bool kept = slot < p.C;
    const int row = kept ? sh.row0[sh.active[e]] + slot : -1;
    sh.pair_row[tid] = (int16_t)row;
    if (kept) {
      sh.row_tok[row] = (uint8_t)t;
      sh.row_a[row] = (uint8_t)(sh.active[e] + slot / kUnitTokens);
    }
    if (blockIdx.x == 0) p.slot[tid] = kept ? slot : -1;
  }
}

// ---------------------------------------------------------------- producers
// A team's ring: stages base .. base + stages - 1.
template <int S>
struct Ring {
  int base, st, n = 0;
  uint32_t ph = 0;
  __device__ explicit Ring(int team) : base(team * S), st(team * S) {}
  __device__ void next() {
    ++n;
    if (++st == base + S) {
      st = base;
      ph ^= 1;
    }
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// One thread takes chunks and issues the weights' copies, one TMA box a matrix
// and block.  It runs into phase D on its own: nothing it reads depends on G.
template <int KIND, int NBT>
__device__ void few_weights(const FewArgs& p, FewShared& sh, uint8_t* smem, int team,
                            const CUtensorMap* tmG, const CUtensorMap* tmU,
                            const CUtensorMap* tmD) {
  using Cfg = FewCfg<KIND, NBT>;
  constexpr int S = Cfg::kStages;
  volatile int* abort_flag = &sh.abort_flag;
  constexpr int kAt = KIND == 0 ? 64 : 4;      // box rows: 64 of bf16, 4 KB chunks of codes
  const uint64_t policy = policy_evict_first();
  Ring<S> r(team);
  bool ok = true;
#pragma unroll 1
  for (int down = 0; ok && down < 2; ++down) {
    const Phase ph = sh.phase[down];
    uint32_t* counter = p.sync + kSyncNext + 32 * down;
    int id = blockIdx.x + team * gridDim.x;
    while (ok && id < ph.chunks) {
      const ChunkInfo info = chunk_info(sh, ph, id);
      id = Cfg::kTeams * gridDim.x + (int)atomicAdd(counter, 1u);    // used when this chunk is issued
      const int e = info.e, col = info.c * (down ? 4 : 2);
#pragma unroll 1
      for (int i = 0; i < info.len; ++i) {
        if (!(ok = mbar_wait(&sh.empty[r.st], r.ph ^ 1, abort_flag))) break;
        uint64_t* bar = &sh.full[r.st];
        uint8_t* stage = smem + r.st * Cfg::kStageBytes;
        if (i == 0) sh.info[r.st] = info;
        mbar_arrive(&sh.ready[r.st]);
        mbar_arrive_expect_tx(bar, Cfg::kWBytes);
        const int at = (info.kb0 + i) * kAt;
        if (down) {
          tma_load_4d(stage, tmD, bar, 0, at, col, e, policy);
        } else {
          tma_load_4d(stage, tmG, bar, 0, at, col, e, policy);
          tma_load_4d(stage + Cfg::kWBytes / 2, tmU, bar, 0, at, col, e, policy);
        }
        r.next();
      }
    }
    // the phase is over
    if (ok && (ok = mbar_wait(&sh.empty[r.st], r.ph ^ 1, abort_flag))) {
      sh.info[r.st].len = 0;
      mbar_arrive(&sh.ready[r.st]);
      mbar_arrive(&sh.full[r.st]);
      r.next();
    }
  }
  if (!ok) {
    *abort_flag = 1;
    report(p.status, kDevErrWaitTimeout);
  }
  // every copy has landed before the CTA may exit
  for (int back = 1; back <= S && back <= r.n; ++back) {
    const int it = r.n - back;
    if (!mbar_wait(&sh.full[r.base + it % S], (it / S) & 1, &sh.never)) break;
  }
}

// One warp adds the token rows and the scales, by 16-byte cp.async of all
// lanes: their pieces are small, and a bulk copy each took 150 clocks to issue,
// which bound the stream at 60 % of the HBM rate.
template <int KIND, int NBT, bool DOWN>
__device__ bool few_tokens_phase(const FewArgs& p, FewShared& sh, uint8_t* smem,
                                 Ring<FewCfg<KIND, NBT>::kStages>& r) {
  using Cfg = FewCfg<KIND, NBT>;
  constexpr int kTile = DOWN ? 256 : 128;
  constexpr int kScaleRows = KIND ? Cfg::KB / Cfg::G : 0;
  constexpr int kStep = KIND ? kDigitBytes : 128;           // bytes of a token row's block
  constexpr int kChunks = kStep / 16;
  const int lane = threadIdx.x % 32;
  const int K = DOWN ? p.f : p.d, N = DOWN ? p.d : p.f;
  const int row_bytes = KIND ? few_tiles(K, 128) * kDigitBytes : K * 2;
  const uint8_t* rows_at = KIND ? (DOWN ? p.hq : p.xq)
                                : reinterpret_cast<const uint8_t*>(DOWN ? p.h : p.x);
  bool waited = !DOWN;
  while (true) {
    bool ok = mbar_wait(&sh.ready[r.st], r.ph, &sh.abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return false;
    const ChunkInfo info = sh.info[r.st];
    if (info.len == 0) {
      mbar_arrive(&sh.full[r.st]);
      r.next();
      return true;
    }
    if (!waited) {                                          // h of all tokens is there
      ok = wait_count(p.sync + kSyncH, gridDim.x, &sh.abort_flag);
      if (!__all_sync(0xffffffffu, ok)) return false;
      waited = true;
    }
    const int c = info.c, row0 = info.row0, n = info.n;
    const int chunks = (DOWN && KIND == 0 ? 2 * n : n) * kChunks;
    // 16 bytes i of the rows: row, and place in its block
    auto src = [&](int i) {
      const int t = i / kChunks, o = (i - t * kChunks) * 16;
      const int row = DOWN ? (KIND == 0 ? 2 * row0 + t : row0 + t) : sh.row_tok[row0 + t];
      return rows_at + (size_t)row * row_bytes + o;
    };
    auto dst = [&](int i) {
      return KIND ? i * 16 : (i / kChunks) * Cfg::kPitch + (i % kChunks) * 16;
    };
    const uint8_t* mine = src(lane < chunks ? lane : 0) + (size_t)info.kb0 * kStep;
    const uint32_t mine_to = Cfg::kWBytes + Cfg::kScaleBytes + dst(lane);
    const __nv_bfloat16* scale = nullptr;
    if constexpr (KIND != 0) {
      // lane -> 8 columns: of the tile, or of gate (0..15) and up (16..31)
      const int n0 = c * kTile + 8 * (DOWN ? lane : lane % 16);
      const FewMatrix& w = DOWN ? p.down : (lane / 16 ? p.up : p.gate);
      if (n0 < N)
        scale = w.scale + ((size_t)info.e * few_tiles(K, Cfg::G) +
                           (size_t)info.kb0 * kScaleRows) * N + n0;
    }
#pragma unroll 1
    for (int i = 0; i < info.len; ++i) {
      if (i) {
        ok = mbar_wait(&sh.ready[r.st], r.ph, &sh.abort_flag);
        if (!__all_sync(0xffffffffu, ok)) return false;
      }
      const uint32_t stage = smem_u32(smem + r.st * Cfg::kStageBytes);
      if constexpr (KIND != 0) {
        if (scale) {
          // rows past the last group (zero digits) take its scales
          const int last = few_tiles(K - (info.kb0 + i) * Cfg::KB, Cfg::G) - 1;
#pragma unroll
          for (int g = 0; g < kScaleRows; ++g)
            cp_async16(stage + Cfg::kWBytes + g * 512 + lane * 16,
                       scale + (size_t)min(g, last) * N);
          scale += (size_t)kScaleRows * N;
        }
      }
      if (lane < chunks) cp_async16(stage + mine_to, mine);
      for (int j = lane + 32; j < chunks; j += 32)
        cp_async16(stage + Cfg::kWBytes + Cfg::kScaleBytes + dst(j),
                   src(j) + (size_t)(info.kb0 + i) * kStep);
      mine += kStep;
      // this lane's arrival, when its copies have landed
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                       smem_u32(&sh.full[r.st]))
                   : "memory");
      r.next();
    }
  }
}

template <int KIND, int NBT>
__device__ void few_tokens(const FewArgs& p, FewShared& sh, uint8_t* smem, int team) {
  Ring<FewCfg<KIND, NBT>::kStages> r(team);
  bool ok = few_tokens_phase<KIND, NBT, false>(p, sh, smem, r);
  ok = ok && few_tokens_phase<KIND, NBT, true>(p, sh, smem, r);
  if (!ok && threadIdx.x % 32 == 0) {
    *static_cast<volatile int*>(&sh.abort_flag) = 1;
    report(p.status, kDevErrWaitTimeout);
  }
  cp_async_wait();
}

// ---------------------------------------------------------------- consumers
// acc[m][j] += the weights of this warp's strip m times token block j.  A
// warp's strips are columns 16 w .. 16 w + 15 of the tile's two halves (gate and
// up).  NBL: token blocks.  Rows past the matrix's end hold zero weights (bf16)
// or zero digits, columns past it give sums that nobody stores: no block needs
// a branch (conditions on either cost a thousand bytes of register spills).
template <int NBT, int NBL>
__device__ __forceinline__ void few_block_bf16(const uint8_t* stage, float (&acc)[2][NBL][4]) {
  using Cfg = FewCfg<0, NBT>;
  const int warp = threadIdx.x / 32 % kTeamWarps, lane = threadIdx.x % 32;
  const uint32_t rows =
      smem_u32(stage + Cfg::kWBytes) + (lane % 8) * Cfg::kPitch + (lane / 8) * 16;
  const int chunk = 2 * (warp % 4) + ((lane / 8) & 1);
  // row k of a swizzled tile: 128 k, its 16-byte chunk c at c ^ (k % 8)
  const uint32_t at = smem_u32(stage) + (warp / 4) * 8192 + ((lane / 16) * 8 + lane % 8) * 128 +
                      ((chunk ^ (lane % 8)) << 4);
#pragma unroll
  for (int s2 = 0; s2 < 2; ++s2) {
    uint32_t b[NBL][4];
#pragma unroll
    for (int j = 0; j < NBL; ++j) ldsm4(b[j], rows + j * 8 * Cfg::kPitch + s2 * 64);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t a[4];
        ldsm4_trans(a, at + m * 16384 + (2 * s2 + s) * 2048);
#pragma unroll
        for (int j = 0; j < NBL; ++j) mma_bf16(acc[m][j], a, b[j][2 * s], b[j][2 * s + 1]);
      }
  }
}

// Two fp32 values at a time (one instruction each on sm_100a).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pack2(int lo, int hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The same on codes; acc[m][j][i]: row half i (columns g, g + 8 of the strip),
// two token columns.  A block's sums are integers, which scale and join the fp32
// sums group by group: that arithmetic, not the products, was half of a block's
// time before it was done two values an instruction (8 warps, one token block:
// 430 clocks a block with groups of 128, 590 with 64, of the 720 that HBM
// leaves).  All of it is held times 2^-11 until H and Y read the sums: 128
// products with the top digit, times its unit, reach 2^138, also where the
// group's scale brings them back into range.  That costs nothing (the integers
// are read as such multiples) and changes no bits but of results below 2^-115.
template <int KIND, int NBT, int NBL>
__device__ __forceinline__ void few_block_codes(const uint8_t* stage, uint64_t (&acc)[2][NBL][2]) {
  using Cfg = FewCfg<KIND, NBT>;
  constexpr int kMagicBits = 0x45C00000;                // 1.5 2^12: sums start as its bits
  constexpr int kGroups = Cfg::KB / Cfg::G, kPer = 4 / kGroups;      // groups; k32 steps of one
  constexpr int kRowsAt = Cfg::kWBytes + Cfg::kScaleBytes;
  const int warp = threadIdx.x / 32 % kTeamWarps, lane = threadIdx.x % 32;
  const uint8_t* codes = stage + (warp / 4) * 4096 + (warp % 4) * 512 + lane * 16;
  const uint32_t rows = smem_u32(stage + kRowsAt) + (lane % 8) * Cfg::kPitch + (lane / 8) * 16;
  const uint8_t* units = stage + kRowsAt + 128 + (lane % 4) * 2 * Cfg::kPitch;
  const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(stage + Cfg::kWBytes) +
                            16 * warp + lane / 4;
  const uint64_t minus_magic = pack2(-6144.f, -6144.f);
  uint4 w4[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
      w4[m][sub] = *reinterpret_cast<const uint4*>(codes + m * 8192 + sub * 2048);
  uint32_t b[NBL][2][4];
  uint64_t u[NBL];
#pragma unroll
  for (int j = 0; j < NBL; ++j) {
    const int at = j * 8 * Cfg::kPitch;
    ldsm4(b[j][0], rows + at);
    ldsm4(b[j][1], rows + at + 64);
    u[j] = pack2(*reinterpret_cast<const float*>(units + at),
                 *reinterpret_cast<const float*>(units + at + Cfg::kPitch));
  }
  int t[2][NBL][4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint4& w = w4[m][h / 2];
      const uint32_t lo = h % 2 ? w.z : w.x, hi = h % 2 ? w.w : w.y;
      // even nibbles: column g; odd ones: column g + 8; 16 (u - 8) as int8
      const uint32_t a0 = and_xor(lo << 4, 0xF0F0F0F0u, 0x80808080u);
      const uint32_t a1 = and_xor(lo, 0xF0F0F0F0u, 0x80808080u);
      const uint32_t a2 = and_xor(hi << 4, 0xF0F0F0F0u, 0x80808080u);
      const uint32_t a3 = and_xor(hi, 0xF0F0F0F0u, 0x80808080u);
#pragma unroll
      for (int j = 0; j < NBL; ++j)
        mma_s8(t[m][j], a0, a1, a2, a3, b[j][h / 2][h % 2 * 2], b[j][h / 2][h % 2 * 2 + 1],
               h % kPer == 0, kMagicBits);
    }
    if (h % kPer != kPer - 1) continue;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int at = (kGroups == 1 ? 0 : h / kPer) * 256 + m * 128;
      const float s0 = __bfloat162float(sc[at]), s1 = __bfloat162float(sc[at + 8]);
      const uint64_t ss[2] = {pack2(s0, s0), pack2(s1, s1)};
#pragma unroll
      for (int j = 0; j < NBL; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t sum = add2(pack2(t[m][j][2 * i], t[m][j][2 * i + 1]), minus_magic);
          acc[m][j][i] = fma2(mul2(sum, u[j]), ss[i], acc[m][j][i]);
        }
    }
  }
}

// One chunk, NBL token blocks wide: its blocks, then this warp's two strips of
// its sums.  False when a wait gave up.
template <int KIND, int NBT, int NBL, bool DOWN>
__device__ __forceinline__ bool few_chunk(const FewArgs& p, FewShared& sh, const uint8_t* smem,
                                          Ring<FewCfg<KIND, NBT>::kStages>& r,
                                          const ChunkInfo& info) {
  using Cfg = FewCfg<KIND, NBT>;
  const int warp = threadIdx.x / 32 % kTeamWarps, lane = threadIdx.x % 32;
  const int len = info.len, n = info.n;
  // strips past the matrix's width have nothing to store
  const int c64 = (DOWN ? p.d : p.f) / 64 - info.c * (DOWN ? 4 : 2) - warp / 4;
  float* const sums = p.part + (size_t)info.sums * 256 + 16 * warp;
  float acc[2][NBL][4] = {};
  auto landed = [&](const auto& at) {
    return __all_sync(0xffffffffu, mbar_wait(&sh.full[at.st], at.ph, &sh.abort_flag)) != 0;
  };
  auto done = [&] {
    if (lane == 0) mbar_arrive(&sh.empty[r.st]);
    r.next();
  };
  [[maybe_unused]] uint64_t acc2[2][NBL][2] = {};         // codes: pairs of sums
#pragma unroll 1
  for (int i = 0; i < len; ++i) {
    if (i && !landed(r)) return false;
    const uint8_t* stage = smem + r.st * Cfg::kStageBytes;
    if constexpr (KIND == 0)
      few_block_bf16<NBT, NBL>(stage, acc);
    else
      few_block_codes<KIND, NBT, NBL>(stage, acc2);
    __syncwarp();
    done();
  }
  if constexpr (KIND != 0) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NBL; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 v = unpack2(acc2[m][j][i]);
          acc[m][j][2 * i] = v.x;
          acc[m][j][2 * i + 1] = v.y;
        }
  }
  const int g = lane / 4, q = lane % 4;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    if (c64 <= (DOWN ? 2 * m : 0)) continue;
    float* to = sums + m * 128;
    if constexpr (KIND == 0 && !DOWN) {
#pragma unroll
      for (int j = 0; j < NBL; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 8 * j + 2 * q + (i & 1);
          if (tok < n) __stcg(to + tok * 256 + g + 8 * (i >> 1), acc[m][j][i]);
        }
    } else if constexpr (KIND == 0) {        // a token's two columns: the two terms of h
#pragma unroll
      for (int j = 0; j < NBL; ++j) {
        const int tok = 4 * j + q;
        if (tok < n) {
          __stcg(to + tok * 256 + g, acc[m][j][0] + acc[m][j][1]);
          __stcg(to + tok * 256 + g + 8, acc[m][j][2] + acc[m][j][3]);
        }
      }
    } else {
      // a token's three columns: its digits.  Column pairs P = 4 j + q: token
      // 2 e has pair 3 e and the first of pair 3 e + 1, token 2 e + 1 the rest
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float after[NBL], before[NBL];                    // of the next, of the previous pair
        const int quad = lane & ~3;
#pragma unroll
        for (int j = 0; j < NBL; ++j) {
          after[j] = __shfl_sync(0xffffffffu, acc[m][j][2 * i], quad | ((q + 1) & 3));
          before[j] = __shfl_sync(0xffffffffu, acc[m][j][2 * i + 1], quad | ((q + 3) & 3));
        }
#pragma unroll
        for (int j = 0; j < NBL; ++j) {
          const float c0 = acc[m][j][2 * i], c1 = acc[m][j][2 * i + 1];
          const int P = 4 * j + q, e = P / 3, kind = P - 3 * e;
          const float next = q < 3 || j + 1 == NBL ? after[j] : after[j + 1 < NBL ? j + 1 : j];
          const float prev = q > 0 || j == 0 ? before[j] : before[j > 0 ? j - 1 : 0];
          const int tok = 2 * e + (kind == 2);
          const float v = kind == 0 ? next + (c1 + c0) : c1 + (c0 + prev);
          if (kind != 1 && tok < n) __stcg(to + tok * 256 + g + 8 * i, v);
        }
      }
    }
  }
  return true;
}

// All chunks of a phase that this team takes.
template <int KIND, int NBT, bool DOWN>
__device__ __forceinline__ bool few_phase(const FewArgs& p, FewShared& sh, const uint8_t* smem,
                                          Ring<FewCfg<KIND, NBT>::kStages>& r) {
  using Cfg = FewCfg<KIND, NBT>;
  constexpr int NB = DOWN ? Cfg::kColsD : Cfg::kColsG;
  constexpr int kPerToken = KIND ? 3 : (DOWN ? 2 : 1), kMid = KIND ? 3 : 4;
#pragma unroll 1
  while (true) {
    if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[r.st], r.ph, &sh.abort_flag))) return false;
    const ChunkInfo info = sh.info[r.st];
    if (info.len == 0) {
      __syncwarp();
      if (threadIdx.x % 32 == 0) mbar_arrive(&sh.empty[r.st]);
      r.next();
      return true;
    }
    const int nb = (info.n * kPerToken + 7) / 8;
    bool ok;
    // as wide as needed: 1, 2, 4, 8 blocks (bf16), 1, 2, 3 (digits)
    if (nb == 1) {
      ok = few_chunk<KIND, NBT, 1, DOWN>(p, sh, smem, r, info);
    } else if (NB == 2 || (NB > 2 && nb == 2)) {
      ok = few_chunk<KIND, NBT, (NB < 2 ? 1 : 2), DOWN>(p, sh, smem, r, info);
    } else if (NB == kMid || (NB > kMid && nb <= kMid)) {
      ok = few_chunk<KIND, NBT, (NB < kMid ? 1 : kMid), DOWN>(p, sh, smem, r, info);
    } else if (NB == 2 * kMid || (NB > 2 * kMid && nb <= 2 * kMid)) {
      ok = few_chunk<KIND, NBT, (NB < 2 * kMid ? 1 : 2 * kMid), DOWN>(p, sh, smem, r, info);
    } else {
      ok = few_chunk<KIND, NBT, (NB > 2 * kMid ? NB : 1), DOWN>(p, sh, smem, r, info);
    }
    if (!ok) return false;
  }
}

// The sums of row r's unit in column tile c: where they start, and how far apart
// the chunks' are, in tokens of 256 floats.
__device__ __forceinline__ int2 few_sums(const FewShared& sh, const Phase& ph, int r, int c) {
  const int a = sh.row_a[r], row0 = sh.row0[a], n = sh.row0[a + 1] - row0;
  return make_int2(ph.tile_at(row0, n, c) + r - row0, n);
}

constexpr float kBf16Max = 3.38953139e38f;             // (2 - 2^-7) 2^127

// h of one row in one tile of 128 columns, by one warp: lane -> columns 2 c,
// 2 c + 1, 8 + 2 c, 9 + 2 c of 16 (the order of the digits).
template <int KIND>
__device__ void few_h(const FewArgs& p, const FewShared& sh, const Phase& ph, int row, int c) {
  const int lane = threadIdx.x % 32;
  const int at = (lane / 4) * 16 + 2 * (lane % 4);
  const bool valid = c * 128 + at < p.f;
  const int2 s = few_sums(sh, ph, row, c);
  const float* src = p.part + (size_t)s.x * 256 + at;
  const size_t step = (size_t)s.y * 256;
  float g[4] = {}, u[4] = {};
  if (valid) {
#pragma unroll 8
    for (int i = 0; i < ph.q; ++i, src += step) {
      const float2 g0 = __ldcg(reinterpret_cast<const float2*>(src));
      const float2 g1 = __ldcg(reinterpret_cast<const float2*>(src + 8));
      const float2 u0 = __ldcg(reinterpret_cast<const float2*>(src + 128));
      const float2 u1 = __ldcg(reinterpret_cast<const float2*>(src + 136));
      g[0] += g0.x, g[1] += g0.y, g[2] += g1.x, g[3] += g1.y;
      u[0] += u0.x, u[1] += u0.y, u[2] += u1.x, u[3] += u1.y;
    }
  }
  float h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (KIND != 0) g[i] *= kCodesUnit, u[i] *= kCodesUnit;
    h[i] = few_silu(g[i]) * u[i];
  }
  if constexpr (KIND == 0) {
    if (!valid) return;
    float lo[4];
    __nv_bfloat162 hi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // an infinite or NaN h has no second term; a finite one past the largest bf16
      // value has that as its first
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float x = h[2 * i + j];
        f[j] = fabsf(x) < INFINITY ? fminf(fmaxf(x, -kBf16Max), kBf16Max) : x;
      }
      hi[i] = __floats2bfloat162_rn(f[0], f[1]);
      const float f0 = __low2float(hi[i]), f1 = __high2float(hi[i]);
      lo[2 * i] = fabsf(f0) <= kBf16Max ? h[2 * i] - f0 : 0.f;
      lo[2 * i + 1] = fabsf(f1) <= kBf16Max ? h[2 * i + 1] - f1 : 0.f;
    }
    __nv_bfloat16* out = p.h + (size_t)(2 * row) * p.f + c * 128 + at;
    *reinterpret_cast<__nv_bfloat162*>(out) = hi[0];
    *reinterpret_cast<__nv_bfloat162*>(out + 8) = hi[1];
    *reinterpret_cast<uint32_t*>(out + p.f) = pack_bf16x2(lo[0], lo[1]);
    *reinterpret_cast<uint32_t*>(out + p.f + 8) = pack_bf16x2(lo[2], lo[3]);
  } else {
    const float x[4] = {h[0], h[2], h[1], h[3]};
    put_digits(p.hq + ((size_t)row * ph.nct + c) * kDigitBytes, x);
  }
}

// y of 32 columns of token t by one warp: lane -> (columns 4 (lane % 8), every
// fourth of the chunks of the token's rows, row after row); the four lanes'
// weighted sums are added last.
template <int KIND>
__device__ void few_combine(const FewArgs& p, const FewShared& sh, const Phase& ph, int t,
                            int col32) {
  constexpr int kBatch = 8;                  // loads in flight
  const int lane = threadIdx.x % 32;
  const int col = 32 * col32 + 4 * (lane % 8);
  const int c = col / 256;
  // lane j < k: row j of the token
  const int row = lane < p.k ? sh.pair_row[t * p.k + lane] : -1;
  const float weight =
      lane < p.k ? sh.pair_w[t * p.k + lane] * (KIND ? kCodesUnit : 1.f) : 0.f;
  const int2 at = row >= 0 ? few_sums(sh, ph, row, c) : make_int2(0, 0);
  const bool any = __any_sync(0xffffffffu, row >= 0);
  const float* base = p.part + col % 256;
  const int terms = p.k * ph.q;
  const float inv_q = 1.0f / (float)ph.q;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = lane / 8; i0 - lane / 8 < terms; i0 += 4 * kBatch) {
    float4 v[kBatch];
    float w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 4 * u;
      const int j = (int)(((float)i + 0.5f) * inv_q);        // i / q: exact, i < 2^16
      const int r = __shfl_sync(0xffffffffu, row, j % 32);
      const int x = __shfl_sync(0xffffffffu, at.x, j % 32);
      const int n = __shfl_sync(0xffffffffu, at.y, j % 32);
      w[u] = __shfl_sync(0xffffffffu, weight, j % 32);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < terms && r >= 0)
        v[u] = __ldcg(reinterpret_cast<const float4*>(
            base + (size_t)(x + (i - j * ph.q) * n) * 256));
      else
        w[u] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      y.x = fmaf(w[u], v[u].x, y.x);
      y.y = fmaf(w[u], v[u].y, y.y);
      y.z = fmaf(w[u], v[u].z, y.z);
      y.w = fmaf(w[u], v[u].w, y.w);
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
    y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
    y.z += __shfl_xor_sync(0xffffffffu, y.z, o);
    y.w += __shfl_xor_sync(0xffffffffu, y.w, o);
  }
  if (lane >= 8) return;
  const size_t out = (size_t)t * p.d + col;
  *reinterpret_cast<uint2*>(p.y + out) =
      any ? make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w))
          : __ldg(reinterpret_cast<const uint2*>(p.x + out));
}

// All N consumer threads of this CTA are done with a phase: counted, once its
// results are visible (the add's release covers what the barrier ordered).
template <int N>
__device__ __forceinline__ void few_arrive(const FewShared& sh, uint32_t* counter) {
  consumer_sync<N>();
  if (threadIdx.x == 0 && !*static_cast<const volatile int*>(&sh.abort_flag)) red_release(counter);
}
// ... and all CTAs are.
template <int N>
__device__ __forceinline__ bool few_await(FewShared& sh, const uint32_t* counter) {
  if (threadIdx.x == 0) sh.ok = wait_count(counter, gridDim.x, &sh.abort_flag);
  consumer_sync<N>();
  const bool ok = sh.ok;
  consumer_sync<N>();
  return ok;
}

template <int KIND, int NBT>
__device__ void few_consumer(const FewArgs& p, FewShared& sh, uint8_t* smem) {
  using Cfg = FewCfg<KIND, NBT>;
  constexpr int N = Cfg::kWorkers, kWarps = N / 32;
  const int warp = threadIdx.x / 32;
  Ring<Cfg::kStages> r(warp / kTeamWarps);
  const Phase up = sh.phase[0], down = sh.phase[1];
  bool ok = few_phase<KIND, NBT, false>(p, sh, smem, r);
  if (!ok) *static_cast<volatile int*>(&sh.abort_flag) = 1;
  few_arrive<N>(sh, p.sync + kSyncG);

  const int rows = sh.row0[sh.A];
  if ((int)blockIdx.x < rows * up.nct) {     // (row, tile) to warps, CTA by CTA
    ok = few_await<N>(sh, p.sync + kSyncG) && ok;
    if (ok)
      for (int i = warp * gridDim.x + blockIdx.x; i < rows * up.nct; i += kWarps * gridDim.x)
        few_h<KIND>(p, sh, up, i / up.nct, i % up.nct);
  }
  few_arrive<N>(sh, p.sync + kSyncH);

  ok = ok && few_phase<KIND, NBT, true>(p, sh, smem, r);
  if (!ok) *static_cast<volatile int*>(&sh.abort_flag) = 1;
  few_arrive<N>(sh, p.sync + kSyncY);

  const int items = p.d / 32 * p.T;          // (token, 32 columns) to warps
  if ((int)blockIdx.x < items) {
    ok = few_await<N>(sh, p.sync + kSyncY) && ok;
    if (ok)
      for (int i = warp * gridDim.x + blockIdx.x; i < items; i += kWarps * gridDim.x) {
        const int t = i / (p.d / 32);
        few_combine<KIND>(p, sh, down, t, i - t * (p.d / 32));
      }
  }
  if (!ok && threadIdx.x % 32 == 0) report(p.status, kDevErrWaitTimeout);
}

// Zeroes the workspace header (status word and counters).  The layer's kernel
// is launched as its dependent and reads the router's weights while this one
// and the launch itself pass: a memset in its place left 3 us between the two.
__global__ void few_header_kernel(uint32_t* header, int words) {
  grid_dep_launch();
  for (int i = threadIdx.x; i < words; i += blockDim.x) header[i] = 0;
}

template <int KIND, int NBT>
__global__ void __launch_bounds__(FewCfg<KIND, NBT>::kThreads, 1)
    few_kernel(const __grid_constant__ FewArgs p, const __grid_constant__ CUtensorMap tmG,
               const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmD) {
  using Cfg = FewCfg<KIND, NBT>;
  extern __shared__ uint8_t dsmem_raw[];
  __shared__ FewShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x;
  volatile int* abort_flag = &sh.abort_flag;
  if (tid < 256) sh.mask[tid] = 0;
  if (tid == 0) {
    for (int s = 0; s < Cfg::kTeams * Cfg::kStages; ++s) {
      mbar_init(&sh.full[s], 1 + 32);        // the weights' thread, and each token lane
      mbar_init(&sh.ready[s], 1);
      mbar_init(&sh.empty[s], kTeamWarps);
    }
    sh.abort_flag = 0;
    sh.never = 0;
    fence_barrier_init();
  }
  __syncthreads();

  // ---- R: router, top-k, tables
  if constexpr (KIND != 0) few_digits(p);
  if ((int)blockIdx.x < p.KS * p.CG) few_router_rows<NBT, Cfg::kWorkers>(p, smem);
  grid_dep_wait();                       // the counters are zero from here on
  __syncthreads();
  if (tid == 0) red_release(p.sync + kSyncRouter);
  // One or two tokens are routed by every CTA for itself, which takes one wait
  // less than routing each by one CTA and handing on the result (1.5 us).
  const bool local = p.T <= Cfg::kWorkers / 256;
  if (local || (int)blockIdx.x < p.T) {
    if (tid == 0) sh.ok = wait_count(p.sync + kSyncRouter, gridDim.x, abort_flag);
    __syncthreads();
    if (sh.ok && local) {
      few_route<Cfg::kWorkers>(p, sh, 0, blockIdx.x == 0);
    } else if (sh.ok) {
      for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        few_route<256>(p, sh, t, true);
        __syncthreads();
        if (tid == 0) red_release(p.sync + kSyncRouted);
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    if (!local) sh.ok = wait_count(p.sync + kSyncRouted, p.T, abort_flag);
    if (!sh.ok) report(p.status, kDevErrWaitTimeout);
  }
  fence_proxy_async_all();               // the router's staging becomes the ring
  __syncthreads();
  if (!sh.ok) return;
  few_tables<Cfg::kUnitTokens>(p, sh, local);
  // by warps that have no pairs
  const int extra = tid / 32 - Cfg::kWorkers / 32;
  if (sh.A && extra >= 0 && extra < 2)
    few_cut(p, sh, extra, few_tiles(extra ? p.d : p.f, extra ? 256 : 128),
            few_tiles(extra ? p.f : p.d, Cfg::KB), KIND != 0);
  __syncthreads();
  if (sh.A == 0) {                       // a capacity of 0: every token passes through
    for (size_t i = (size_t)blockIdx.x * Cfg::kThreads + tid; i < (size_t)p.T * p.d;
         i += (size_t)gridDim.x * Cfg::kThreads)
      p.y[i] = p.x[i];
    return;
  }

  // ---- G and D
  if (extra < 0) {
    few_consumer<KIND, NBT>(p, sh, smem);
  } else if (extra < Cfg::kTeams) {
    if (elect_one()) few_weights<KIND, NBT>(p, sh, smem, extra, &tmG, &tmU, &tmD);
  } else {
    few_tokens<KIND, NBT>(p, sh, smem, extra - Cfg::kTeams);
  }
}

// ---------------------------------------------------------------- host side
namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Byte sizes of the workspace, in order: the counters (with the status word
// first), the routing results, then what the phases hand on.
struct FewLayout {
  size_t sync, logits, idx, w, slot, counts, rpart, part, xq, h;
  FewLayout(int64_t T, int64_t d, int64_t E, int64_t k, int64_t f) {
    const size_t dt = (size_t)(d + 255) / 256, ft = (size_t)(f + 127) / 128;
    sync = up256(256 + kSyncWords * 4);
    logits = up256(size_t(T * E) * 4);
    idx = w = slot = up256(size_t(T * k) * 4);
    counts = up256(size_t(E) * 4);
    rpart = up256(size_t(kFewMaxSplits * T * E) * 8);
    // G's sums are read before D's are written
    part = (size_t(T * k) * (ft > dt ? ft : dt) + few_part_rows((int)T)) * 1024;
    xq = up256(size_t(T) * ((d + 127) / 128) * kDigitBytes);
    // two bf16 terms, or digits
    h = up256(size_t(T * k) * (ft * kDigitBytes > size_t(f) * 4 ? ft * kDigitBytes : size_t(f) * 4));
  }
  size_t total() const {
    return sync + logits + idx + w + slot + counts + rpart + part + xq + h;
  }
};

// One matrix as a 4-D tensor, a box being `groups` 64-column groups of one
// block, each group's bytes together: bf16 as (64 columns, K rows, N/64 groups,
// E), 128-byte swizzle, 64 rows a box; codes as (1 KB, 1 KB chunks of a group,
// N/64 groups, E), 4 chunks (128 rows) a box.  Boxes that reach past K or N
// read zeros there.
bool map_few(CUtensorMap* m, const FewMatrix& w, uint64_t E, uint32_t groups) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const uint64_t K = w.K, N = w.N;
  const bool codes = w.group != 0;
  cuuint64_t dims[4] = {64, K, N / 64, E};
  cuuint64_t strides[3] = {N * 2, 128, K * N * 2};
  cuuint32_t box[4] = {64, 64, groups, 1};
  if (codes) {
    dims[0] = 256;
    dims[1] = K / 32;
    strides[0] = 1024;
    strides[1] = K * 32;
    strides[2] = K * N / 2;
    box[0] = 256;
    box[1] = 4;
  }
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(w.w), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int KIND, int NBT>
cudaError_t launch_few_t(const FewArgs& a, int grid, const CUtensorMap& g, const CUtensorMap& u,
                         const CUtensorMap& dn, DeviceInfo* di, cudaStream_t s) {
  using Cfg = FewCfg<KIND, NBT>;
  auto kern = few_kernel<KIND, NBT>;
  const int slot = kFewAttrSlot + 3 * KIND + (NBT == 1 ? 0 : NBT == 2 ? 1 : 2);
  if (!di->attr_set[slot]) {
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           Cfg::kSmemBytes);
    if (err != cudaSuccess) return err;
    di->attr_set[slot] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = s;
  // cooperative: the CTAs wait for one another, so all of them run or none
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, g, u, dn);
}

// Token blocks by T: accumulators, stages and the router's sums are sized by
// them.  One token in the kernel of four blocks: 64 experts of 7168 x 2048 131.0
// us instead of 121.0 on bf16, 63.8 instead of 54.6 on codes.
template <int KIND>
cudaError_t launch_few_kind(const FewArgs& a, int grid, const CUtensorMap& g, const CUtensorMap& u,
                            const CUtensorMap& dn, DeviceInfo* di, cudaStream_t s) {
  if (a.T <= 8) return launch_few_t<KIND, 1>(a, grid, g, u, dn, di, s);
  if (a.T <= 16) return launch_few_t<KIND, 2>(a, grid, g, u, dn, di, s);
  return launch_few_t<KIND, 4>(a, grid, g, u, dn, di, s);
}

}  // namespace

size_t few_workspace_bytes(int64_t T, int64_t d, int64_t E, int64_t k, int64_t f) {
  return FewLayout(T, d, E, k, f).total();
}

cudaError_t launch_few(FewArgs a, void* ws, cudaStream_t s, bool* map_failed) {
  *map_failed = false;
  DeviceInfo* di = nullptr;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const int grid = di->sms;

  const FewLayout lay(a.T, a.d, a.E, a.k, a.f);
  char* at = static_cast<char*>(ws);
  a.status = reinterpret_cast<int32_t*>(at);
  a.sync = reinterpret_cast<uint32_t*>(at + 256);
  at += lay.sync;
  auto take = [&](auto*& p, size_t bytes) {
    using P = std::remove_reference_t<decltype(p)>;
    if (!p) p = reinterpret_cast<P>(at);       // a caller's buffer takes the field's place
    at += bytes;
  };
  take(a.logits, lay.logits);
  take(a.topk_idx, lay.idx);
  take(a.topk_w, lay.w);
  take(a.slot, lay.slot);
  take(a.counts, lay.counts);
  take(a.rpart, lay.rpart);
  take(a.part, lay.part);
  take(a.xq, lay.xq);
  a.h = reinterpret_cast<__nv_bfloat16*>(at);
  a.hq = reinterpret_cast<uint8_t*>(at);

  // the router's split: 32 columns (or all of a few experts', as the lanes past
  // the last expert would idle: 8 experts, 32 tokens, bf16 460 us, 464 at 32
  // columns) by as many row ranges as there are CTAs for, at most kFewMaxSplits
  // (a token's CTA adds them)
  a.CW = a.E <= 8 ? 8 : (a.E <= 16 ? 16 : 32);
  a.CG = (a.E + a.CW - 1) / a.CW;
  a.KS = grid / a.CG;
  if (a.KS < 1) return cudaErrorInvalidConfiguration;
  if (a.KS > kFewMaxSplits) a.KS = kFewMaxSplits;

  CUtensorMap g{}, u{}, dn{};
  if (!map_few(&g, a.gate, a.E, 2) || !map_few(&u, a.up, a.E, 2) || !map_few(&dn, a.down, a.E, 4)) {
    *map_failed = true;
    return cudaSuccess;
  }
  few_header_kernel<<<1, 320, 0, s>>>(static_cast<uint32_t*>(ws), (int)(lay.sync / 4));
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  if (a.gate.group == 0) return launch_few_kind<0>(a, grid, g, u, dn, di, s);
  if (a.gate.group == 64) return launch_few_kind<2>(a, grid, g, u, dn, di, s);
  if (a.gate.group == 32) return launch_few_kind<3>(a, grid, g, u, dn, di, s);
  return launch_few_kind<1>(a, grid, g, u, dn, di, s);
}

}  // namespace moe
