// The MoE layer for a few tokens (a decode step) as one persistent kernel, on
// bf16 experts or on 4-bit codes with group scales.
//
// With T tokens and A distinct experts chosen, the layer reads 3 A d f weights
// and takes 2 operations per weight and token: for T <= 32 the time is the
// weights' bytes at the HBM rate, plus whatever keeps the memory idle.  So the
// kernel is one stream of weights: one CTA per SM, each with an equal share of
// the blocks of all matrices, a ring of shared-memory stages that a producer
// warp fills by TMA, and the dependencies between the steps taken inside the
// kernel (a cooperative launch), where the ring stays full across them:
//   R  router: every CTA sums its rows of x Wr in fp64 (the choice of experts
//      must not hang on the order of a sum); the CTA of token t adds the
//      partial sums, rounds once to fp32, and one warp picks the top k;
//   G  gate/up: the blocks (expert, 128 columns of f, KB rows) of all chosen
//      experts lie on one line that is cut into gridDim equal pieces.  A tile
//      cut between CTAs goes to the workspace as fp32 partial sums, and the
//      warp that arrives last adds them in CTA order, so no sum depends on
//      timing.  h = silu(g) u is stored as two bf16 terms (hi + lo: 2^-16);
//   D  down: the same over (expert, 256 columns of d, KB rows of f); its first
//      weights are in flight before the last CTA has finished G.  The warp
//      that completes a column tile of all experts adds the k weighted rows of
//      each token in j order and writes y.
//
// The products run on mma.sync (m16n8k16) with the weights as the 16-row
// operand and the tokens as the 8 columns: an SM gets 23 bytes of weights a
// clock, 12 bf16 values, which times 8 columns is a tenth of that unit's rate,
// and the 4-bit codes become bf16 operands in registers, which tcgen05 would
// want back in shared memory (four times the bytes the codes take there).
#include <type_traits>

#include "abi_checks.cuh"
#include "common.cuh"
#include "few_tokens.cuh"
#include "host_util.cuh"
#include "w4.cuh"

namespace moe {

constexpr int kFewWarps = 8;                       // consumer warps
constexpr int kFewThreads = 32 * kFewWarps + 32;   // and the producer warp
constexpr int kFewMaxCtas = 256;                   // sizes the workspace
constexpr int kFewMaxPairs = MOE_FEW_MAX_TOKENS * 8;
constexpr int kFewRouterRows = 512;                // router rows staged at once
constexpr int kFewMaxSplits = 32;

// grid-wide counters, zeroed by the call: arrivals of the router's partial
// sums, of the tokens' routing and of the CTAs that finished G; then for each
// cut gate/up tile (by the CTA that holds its first piece) and for each down
// column tile, per warp, the blocks that are summed.
constexpr int kSyncRouter = 0, kSyncRouted = 32, kSyncH = 64, kSyncTiles = 96;

// KIND 0: bf16; 1: codes with groups of 64 or 128 rows; 2: groups of 32.
template <int KIND, int NBT>
struct FewCfg {
  static constexpr int KB = KIND == 0 ? 64 : 128;         // rows of a block
  static constexpr int kWBytes = KIND == 0 ? 32768 : 16384;
  static constexpr int kScaleBytes = KIND == 0 ? 0 : (KIND == 1 ? 2 : 4) * 512;
  // token rows: 16 bytes of padding keep ldmatrix free of bank conflicts
  static constexpr int kPitch = KB * 2 + 16;
  static constexpr int kRows = 16 * NBT;                  // D: hi and lo of 8 NBT tokens
  static constexpr int kStageBytes =
      (kWBytes + kScaleBytes + kRows * kPitch + 1023) / 1024 * 1024;
  static constexpr int kFit = 215040 / kStageBytes;
  static constexpr int kStages = kFit > 9 ? 9 : kFit;
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024;
  // the router's staging uses the same memory: x (fp64), then W rows
  static constexpr int kXsBytes = 8 * NBT * kFewRouterRows * 8;
  static_assert(kXsBytes + kFewRouterRows * 32 * 4 <= kStages * kStageBytes, "router staging");
  static_assert(256 * 8 * NBT * 8 <= kStages * kStageBytes, "router reduction");
};

struct FewShared {
  uint64_t full[9], empty[9];
  int abort_flag, never, ok;
  uint32_t mask[256];                 // tokens that chose expert e
  uint16_t row0[257];                 // first kept row of active expert a
  uint8_t expert[256];                // active expert a -> e
  uint8_t active[256];                // e -> a
  uint8_t row_tok[kFewMaxPairs];      // kept row -> token
  int16_t pair_row[kFewMaxPairs];     // pair -> kept row, -1 dropped
  float pair_w[kFewMaxPairs];
  float logit[256];
  uint32_t warp_sum[8];
  int A;                              // active experts
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
  asm volatile(
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
// order this thread's and (through barriers) other threads' generic accesses
// with asynchronous copies of the same memory
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory");
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

// The blocks of a phase on one line: units (expert a, column tile c) of nkb
// blocks each, cut into `parts` pieces of equal length (one block or more, so
// that every piece between a unit's first and last one holds blocks of it).
struct Line {
  int nct, nkb, parts;
  long long total;
  __device__ Line(int A, int nct_, int nkb_)
      : nct(nct_), nkb(nkb_), parts(gridDim.x), total((long long)A * nct_ * nkb_) {
    if (total < parts) parts = (int)total;
  }
  __device__ long long begin(int b) const { return b < parts ? total * b / parts : total; }
  // the piece that holds block i
  __device__ int piece(long long i) const {
    return (int)(((i + 1) * parts + total - 1) / total) - 1;
  }
};
// A walk over one piece, block by block.
struct Walk {
  long long i, end;
  int a, c, kb;
  __device__ Walk(const Line& l, int b) : i(l.begin(b)), end(l.begin(b + 1)), a(0), c(0), kb(0) {
    if (i < end) {
      const long long u = i / l.nkb;
      kb = (int)(i - u * l.nkb);
      a = (int)(u / l.nct);
      c = (int)(u - (long long)a * l.nct);
    }
  }
  __device__ bool more() const { return i < end; }
  __device__ void next(const Line& l) {
    ++i;
    if (++kb == l.nkb) {
      kb = 0;
      if (++c == l.nct) {
        c = 0;
        ++a;
      }
    }
  }
};

// Float offset of the partial tile of unit (a, c) in CTA b: each 256 x n_a,
// apart for every (unit, CTA) since n_a <= T.
__device__ __forceinline__ size_t part_at(const FewShared& sh, int a, int c, int nct, int b, int T) {
  const int n = sh.row0[a + 1] - sh.row0[a];
  return 256 * ((size_t)sh.row0[a] * nct + (size_t)c * n + (size_t)b * T);
}

// ---------------------------------------------------------------- R: router
// Partial sums of this CTA's rows and columns for all tokens, in fp64.
template <int NBT>
__device__ void few_router_rows(const FewArgs& p, uint8_t* smem) {
  constexpr int RR = kFewRouterRows;
  const int tid = threadIdx.x;
  const bool worker = tid < 256;
  const int cg = blockIdx.x % p.CG, ks = blockIdx.x / p.CG;
  const int c = tid % p.CW, rg = tid / p.CW, nrg = 256 / p.CW;
  const int col0 = cg * p.CW, cols = min(p.CW, p.E - col0);
  const int k0 = (int)((long long)p.d * ks / p.KS), k1 = (int)((long long)p.d * (ks + 1) / p.KS);
  double* xs = reinterpret_cast<double*>(smem);                    // [T][RR]
  float* wsm = reinterpret_cast<float*>(smem + 8 * NBT * RR * 8);  // [RR][CW]
  double acc[8 * NBT];
#pragma unroll
  for (int t = 0; t < 8 * NBT; ++t) acc[t] = 0.0;
  for (int base = k0; base < k1; base += RR) {
    const int len = min(RR, k1 - base);
    if (base != k0) __syncthreads();
    if (worker) {
      const float* src = p.w_router + (size_t)base * p.E + col0;
      if (p.E % 4 == 0) {
        const int q = p.CW / 4;
        for (int i = tid; i < len * q; i += 256) {
          const int r = i / q, v = i % q;
          if (4 * v < cols) cp_async16(smem_u32(wsm + r * p.CW + 4 * v), src + (size_t)r * p.E + 4 * v);
        }
      } else {
        for (int i = tid; i < len * p.CW; i += 256) {
          const int r = i / p.CW, v = i % p.CW;
          if (v < cols) cp_async4(smem_u32(wsm + r * p.CW + v), src + (size_t)r * p.E + v);
        }
      }
      for (int i = tid; i < p.T * RR; i += 256) {
        const int t = i / RR, r = i % RR;
        if (r < len) xs[i] = (double)__bfloat162float(p.x[(size_t)t * p.d + base + r]);
      }
      cp_async_wait();
    }
    __syncthreads();
    if (worker && c < cols) {
      for (int r = rg; r < len; r += nrg) {
        const double w = (double)wsm[r * p.CW + c];
#pragma unroll
        for (int t = 0; t < 8 * NBT; ++t)
          if (t < p.T) acc[t] = fma(w, xs[t * RR + r], acc[t]);
      }
    }
  }
  __syncthreads();
  double* red = reinterpret_cast<double*>(smem);                   // [T][256]
  if (worker) {
#pragma unroll
    for (int t = 0; t < 8 * NBT; ++t)
      if (t < p.T) red[t * 256 + tid] = acc[t];
  }
  __syncthreads();
  if (worker) {
    for (int i = tid; i < p.T * p.CW; i += 256) {
      const int t = i / p.CW, cc = i % p.CW;
      if (cc >= cols) continue;
      double s = 0.0;
      for (int g = 0; g < nrg; ++g) s += red[t * 256 + g * p.CW + cc];
      p.rpart[((size_t)ks * p.T + t) * p.E + col0 + cc] = s;
    }
  }
}

// Logits, top-k and gate weights of token t (all threads of one CTA).
__device__ void few_route_token(const FewArgs& p, FewShared& sh, int t) {
  const int tid = threadIdx.x;
  if (tid < p.E) {
    double s = 0.0;
#pragma unroll 8
    for (int ks = 0; ks < p.KS; ++ks) s += __ldcg(p.rpart + ((size_t)ks * p.T + t) * p.E + tid);
    if (p.bias) s += (double)__ldg(p.bias + tid);
    const float l = (float)s;
    sh.logit[tid] = l;
    p.logits[(size_t)t * p.E + tid] = l;
  }
  __syncthreads();
  if (tid < 32) {
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = tid + 32 * i;
      key[i] = e < p.E ? few_order(sh.logit[e]) : 0u;       // no number has key 0
    }
    float v0 = 0.f, mine = 0.f, sum = 0.f;
    int my_e = 0;
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
      const float v = sh.logit[e];
      if (j == 0) v0 = v;
      const float pj = expf(v - v0);
      sum += pj;
      if (tid == j) {
        mine = pj;
        my_e = (int)e;
      }
    }
    if (tid < p.k) {
      p.topk_idx[t * p.k + tid] = my_e;
      p.topk_w[t * p.k + tid] = mine / sum;
    }
    __threadfence();
    __syncwarp();
    if (tid == 0) atomicAdd(p.sync + kSyncRouted, 1u);
  }
  __syncthreads();
}

// Which experts run and on which tokens: every CTA builds the same tables.
__device__ void few_tables(const FewArgs& p, FewShared& sh) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int pairs = p.T * p.k;
  if (tid < 256) sh.mask[tid] = 0;
  int e = 0, t = 0;
  __syncthreads();
  if (tid < pairs) {
    e = __ldcg(p.topk_idx + tid);
    sh.pair_w[tid] = __ldcg(p.topk_w + tid);
    t = tid / p.k;
    atomicOr(&sh.mask[e], 1u << t);                // k distinct experts a token
  }
  __syncthreads();
  uint32_t n = 0, v = 0, incl = 0;
  if (tid < 256) {
    n = min(__popc(sh.mask[tid]), p.C);
    v = n | (n ? 1u << 16 : 0u);
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
      sh.expert[a] = (uint8_t)tid;
      sh.active[tid] = (uint8_t)a;
      sh.row0[a] = (uint16_t)(excl & 0xFFFF);
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
    if (kept) sh.row_tok[row] = (uint8_t)t;
    if (blockIdx.x == 0) p.slot[tid] = kept ? slot : -1;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- producer
// One stage of a block: the weights of `boxes` 64-column groups and (tokens)
// the token rows.  Returns after issuing; `what` 1: weights, 2: token rows.
template <int KIND, int NBT, bool DOWN>
__device__ __forceinline__ void few_fill(const FewArgs& p, const FewShared& sh,
                                         const CUtensorMap* tm0, const CUtensorMap* tm1,
                                         uint8_t* stage, uint64_t* bar, int a, int c, int kb,
                                         int what) {
  using Cfg = FewCfg<KIND, NBT>;
  const int lane = threadIdx.x % 32;
  const int K = DOWN ? p.f : p.d, N = DOWN ? p.d : p.f;
  const int klen = min(Cfg::KB, K - kb * Cfg::KB);
  const int n = sh.row0[a + 1] - sh.row0[a];
  const int rows = DOWN ? 2 * n : n;
  const int e = sh.expert[a];
  const int group = p.gate.group;
  // 64-column groups of this tile: per matrix in G, of the one matrix in D
  const int boxes = min(DOWN ? 4 : 2, N / 64 - c * (DOWN ? 4 : 2));
  const int mats = DOWN ? 1 : 2;
  const int grows = KIND == 0 ? 0 : (klen + group - 1) / group;
  if (what & 1) {
    if (lane == 0) {
      const uint32_t wbytes = KIND == 0 ? 8192u : 32u * klen;
      mbar_arrive_expect_tx(bar, mats * boxes * (wbytes + grows * 128u) + rows * klen * 2u);
    }
    __syncwarp();
    if constexpr (KIND == 0) {
      if (lane < mats * boxes) {
        const int m = lane / boxes, b = lane % boxes;
        tma_load_3d(stage + (2 * m + b) * 8192, m ? tm1 : tm0, bar,
                    (c * (DOWN ? 4 : 2) + b) * 64, kb * 64, e);
      }
    } else {
      if (lane < mats * boxes) {
        const int m = lane / boxes, b = lane % boxes;
        const FewMatrix& w = DOWN ? p.down : (m ? p.up : p.gate);
        const size_t tile = ((size_t)e * (N / 64) + c * (DOWN ? 4 : 2) + b) * (K / 64) + kb * 2;
        bulk_load(stage + (2 * m + b) * 4096, static_cast<const uint8_t*>(w.w) + tile * 2048,
                  32 * klen, bar);
      }
      if (lane < mats * grows) {
        const int m = lane / grows, g = lane % grows;
        const FewMatrix& w = DOWN ? p.down : (m ? p.up : p.gate);
        const size_t groups = (K + group - 1) / group;
        bulk_load(stage + Cfg::kWBytes + g * 512 + m * 256,
                  w.scale + ((size_t)e * groups + (size_t)kb * Cfg::KB / group + g) * N +
                      c * (DOWN ? 256 : 128),
                  boxes * 128, bar);
      }
    }
  }
  if (what & 2) {
    uint8_t* rowbuf = stage + Cfg::kWBytes + Cfg::kScaleBytes;
    for (int i = lane; i < rows; i += 32) {
      const __nv_bfloat16* src =
          DOWN ? p.h + (size_t)(2 * sh.row0[a] + i) * p.f
               : p.x + (size_t)sh.row_tok[sh.row0[a] + i] * p.d;
      bulk_load(rowbuf + i * Cfg::kPitch, src + kb * Cfg::KB, klen * 2, bar);
    }
  }
}

struct Ring {
  int st = 0, n = 0;
  uint32_t ph = 0;
  __device__ void next(int stages) {
    ++n;
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
  }
};

template <int KIND, int NBT>
__device__ void few_producer(const FewArgs& p, FewShared& sh, uint8_t* smem,
                             const CUtensorMap* tmG, const CUtensorMap* tmU,
                             const CUtensorMap* tmD) {
  using Cfg = FewCfg<KIND, NBT>;
  constexpr int S = Cfg::kStages;
  volatile int* abort_flag = &sh.abort_flag;
  const int lane = threadIdx.x % 32;
  Ring r;
  bool ok = true;
  auto stage = [&](int s) { return smem + s * Cfg::kStageBytes; };
  {
    const Line line(sh.A, (p.f + 127) / 128, (p.d + Cfg::KB - 1) / Cfg::KB);
    for (Walk w(line, blockIdx.x); ok && w.more(); w.next(line)) {
      ok = mbar_wait(&sh.empty[r.st], r.ph ^ 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) ok = false;
      if (!ok) break;
      few_fill<KIND, NBT, false>(p, sh, tmG, tmU, stage(r.st), &sh.full[r.st], w.a, w.c, w.kb, 3);
      r.next(S);
    }
  }
  {
    const Line line(sh.A, (p.d + 255) / 256, (p.f + Cfg::KB - 1) / Cfg::KB);
    Walk w(line, blockIdx.x);
    Walk w0 = w;
    Ring r0 = r;
    int ahead = 0;                       // stages that hold weights but no rows yet
    for (; ok && w.more() && ahead < S; w.next(line), ++ahead) {
      ok = mbar_wait(&sh.empty[r.st], r.ph ^ 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) ok = false;
      if (!ok) break;
      few_fill<KIND, NBT, true>(p, sh, tmD, nullptr, stage(r.st), &sh.full[r.st], w.a, w.c, w.kb,
                                1);
      r.next(S);
    }
    if (ok && ahead) {
      ok = wait_count(p.sync + kSyncH, gridDim.x, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) ok = false;
    }
    fence_proxy_async_all();             // h was written through the generic proxy
    for (; ok && ahead; --ahead, w0.next(line), r0.next(S))
      few_fill<KIND, NBT, true>(p, sh, tmD, nullptr, stage(r0.st), &sh.full[r0.st], w0.a, w0.c,
                                w0.kb, 2);
    for (; ok && w.more(); w.next(line)) {
      ok = mbar_wait(&sh.empty[r.st], r.ph ^ 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) ok = false;
      if (!ok) break;
      few_fill<KIND, NBT, true>(p, sh, tmD, nullptr, stage(r.st), &sh.full[r.st], w.a, w.c, w.kb,
                                3);
      r.next(S);
    }
  }
  if (!ok && lane == 0) {
    *abort_flag = 1;
    report(p.status, kDevErrWaitTimeout);
  }
  __syncwarp();
  // every copy has landed before the CTA may exit
  if (lane == 0) {
    for (int back = 1; back <= S && back <= r.n; ++back) {
      const int it = r.n - back;
      if (!mbar_wait(&sh.full[it % S], (it / S) & 1, &sh.never)) break;
    }
  }
}

// ---------------------------------------------------------------- consumers
// acc[m][j] += weights of matrix m (16 columns of this warp) times token block j
template <int KIND, int NBT, int NB>
__device__ __forceinline__ void few_block(const uint8_t* stage, int klen, int group, int nb,
                                          const bool (&valid)[2], float (&acc)[2][NB][4]) {
  using Cfg = FewCfg<KIND, NBT>;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rows = smem_u32(stage + Cfg::kWBytes + Cfg::kScaleBytes) +
                        (lane % 8) * Cfg::kPitch + (lane / 8) * 16;
  if constexpr (KIND == 0) {
    const uint32_t base = smem_u32(stage) + (warp / 4) * 8192;
    const int chunk = 2 * (warp % 4) + ((lane / 8) & 1);
#pragma unroll
    for (int s2 = 0; s2 < 2; ++s2) {
      uint32_t b[NB][4];
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (j < nb) ldsm4(b[j], rows + j * 8 * Cfg::kPitch + s2 * 64);
#pragma unroll
      for (int s1 = 0; s1 < 2; ++s1) {
        const int k = (2 * s2 + s1) * 16 + (lane / 16) * 8 + lane % 8;
        const uint32_t at = k * 128 + ((chunk ^ (k & 7)) << 4);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (!valid[m]) continue;
          uint32_t a[4];
          ldsm4_trans(a, base + m * 16384 + at);
#pragma unroll
          for (int j = 0; j < NB; ++j)
            if (j < nb) mma_bf16(acc[m][j], a, b[j][2 * s1], b[j][2 * s1 + 1]);
        }
      }
    }
  } else {
    const int subs = klen / 64;
    const uint8_t* codes = stage + (warp / 4) * 4096 + (warp % 4) * 512 + lane * 16;
    const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(stage + Cfg::kWBytes) +
                              16 * warp + lane / 4;
    const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
    for (int sub = 0; sub < subs; ++sub) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (!valid[m]) continue;
        const uint4 w4 = *reinterpret_cast<const uint4*>(codes + m * 8192 + sub * 2048);
        const uint32_t words[4] = {w4.x, w4.y, w4.z, w4.w};
        uint32_t a[4][4];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // 0x4300 | u is the bf16 value 128 + u
            uint32_t v = ((words[s] >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
            const __nv_bfloat162 z = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), off);
            a[s][i] = *reinterpret_cast<const uint32_t*>(&z);
          }
        constexpr int GS = KIND == 1 ? 4 : 2;              // k16 steps between scalings
#pragma unroll
        for (int g = 0; g < 4 / GS; ++g) {
          const int grow = (sub * 64 + g * 32) / group;
          const float s0 = __bfloat162float(sc[grow * 256 + m * 128]);
          const float s1 = __bfloat162float(sc[grow * 256 + m * 128 + 8]);
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            if (j >= nb) continue;
            float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < GS / 2; ++h) {
              uint32_t b[4];
              ldsm4(b, rows + j * 8 * Cfg::kPitch + sub * 128 + (g * GS / 2 + h) * 64);
              mma_bf16(t, a[g * GS + 2 * h], b[0], b[1]);
              mma_bf16(t, a[g * GS + 2 * h + 1], b[2], b[3]);
            }
            acc[m][j][0] = fmaf(s0, t[0], acc[m][j][0]);
            acc[m][j][1] = fmaf(s0, t[1], acc[m][j][1]);
            acc[m][j][2] = fmaf(s1, t[2], acc[m][j][2]);
            acc[m][j][3] = fmaf(s1, t[3], acc[m][j][3]);
          }
        }
      }
    }
  }
}

__device__ __forceinline__ void store_h(const FewArgs& p, int row, int col, float g, float u) {
  const float h = few_silu(g) * u;
  const __nv_bfloat16 hi = __float2bfloat16(h);
  const float hf = __bfloat162float(hi);
  // an infinite or NaN h has no second term
  const __nv_bfloat16 lo = __float2bfloat16(fabsf(hf) <= 3.4e38f ? h - hf : 0.f);
  p.h[(size_t)(2 * row) * p.f + col] = hi;
  p.h[(size_t)(2 * row + 1) * p.f + col] = lo;
}

// The end of a gate/up piece: h if the tile is whole, else partial sums, and h
// by the warp whose piece completes the tile.
template <int NB>
__device__ void few_gate_up_end(const FewArgs& p, const FewShared& sh, const Line& line, int a,
                                int c, int blocks, bool valid, const float (&acc)[2][NB][4]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, q = lane % 4;
  const int n = sh.row0[a + 1] - sh.row0[a];
  const int col = 16 * warp + g;
  if (!valid) return;
  if (blocks == line.nkb) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 8 * j + 2 * q + (i & 1);
        if (tok < n)
          store_h(p, sh.row0[a] + tok, c * 128 + col + 8 * (i >> 1), acc[0][j][i], acc[1][j][i]);
      }
    return;
  }
  float* part = p.gpart + part_at(sh, a, c, line.nct, blockIdx.x, p.T);
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 8 * j + 2 * q + (i & 1);
      if (tok < n) {
        __stcg(part + tok * 256 + col + 8 * (i >> 1), acc[0][j][i]);
        __stcg(part + tok * 256 + 128 + col + 8 * (i >> 1), acc[1][j][i]);
      }
    }
  const long long u = (long long)a * line.nct + c;
  const int first = line.piece(u * line.nkb), last = line.piece((u + 1) * line.nkb - 1);
  __threadfence();
  __syncwarp();
  uint32_t old = 0;
  if (lane == 0) old = atomicAdd(p.sync + kSyncTiles + first * kFewWarps + warp, (uint32_t)blocks);
  old = __shfl_sync(0xffffffffu, old, 0);
  if (old + blocks != (uint32_t)line.nkb) return;
  __threadfence();
  for (int i = lane; i < 16 * n; i += 32) {
    const int tok = i / 16, cc = 16 * warp + i % 16;
    float gs = 0.f, us = 0.f;
    for (int b = first; b <= last; ++b) {
      const float* src = p.gpart + part_at(sh, a, c, line.nct, b, p.T) + tok * 256 + cc;
      gs += __ldcg(src);
      us += __ldcg(src + 128);
    }
    store_h(p, sh.row0[a] + tok, c * 128 + cc, gs, us);
  }
}

// y of this warp's columns of tile c (lane 0..15: matrix half 0, 16..31: half
// 1) for all tokens: the weighted rows in j order, their pieces in CTA order.
__device__ void few_combine(const FewArgs& p, const FewShared& sh, const Line& line, int c,
                            bool valid) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cc = (lane / 16) * 128 + 16 * warp + lane % 16;
  for (int t = 0; t < p.T; ++t) {
    int row = -1, first = 0, last = -1;
    uint32_t at = 0;
    if (lane < p.k) {
      row = sh.pair_row[t * p.k + lane];
      if (row >= 0) {
        int a = 0;                          // the active expert that holds the row
        for (int step = 128; step; step >>= 1)
          if (a + step < sh.A && sh.row0[a + step] <= row) a += step;
        const long long u = (long long)a * line.nct + c;
        first = line.piece(u * line.nkb);
        last = line.piece((u + 1) * line.nkb - 1);
        at = (uint32_t)(part_at(sh, a, c, line.nct, first, p.T) / 256) + (row - sh.row0[a]);
      }
    }
    float y = 0.f;
    bool any = false;
    for (int j = 0; j < p.k; ++j) {
      if (__shfl_sync(0xffffffffu, row, j) < 0) continue;
      any = true;
      const int pieces = __shfl_sync(0xffffffffu, last - first, j);
      const float* src = p.dpart + (size_t)__shfl_sync(0xffffffffu, at, j) * 256 + cc;
      float o = 0.f;
      if (valid)
        for (int b = 0; b <= pieces; ++b) o += __ldcg(src + (size_t)b * p.T * 256);
      y = fmaf(sh.pair_w[t * p.k + j], o, y);
    }
    if (valid) {
      const size_t out = (size_t)t * p.d + c * 256 + cc;
      p.y[out] = any ? __float2bfloat16(y) : p.x[out];
    }
  }
}

// The end of a down piece: its partial sums (a token's two columns, from the
// two terms of h, added), and y by the warp that completes the column tile.
template <int NB>
__device__ void few_down_end(const FewArgs& p, const FewShared& sh, const Line& line, int a, int c,
                             int blocks, const bool (&valid)[2], const float (&acc)[2][NB][4]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, q = lane % 4;
  const int n = sh.row0[a + 1] - sh.row0[a];
  if (!valid[0]) return;                 // half 1 is valid only if half 0 is
  float* part = p.dpart + part_at(sh, a, c, line.nct, blockIdx.x, p.T);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int tok = 4 * j + q;
      if (tok < n && valid[m]) {
        __stcg(part + tok * 256 + m * 128 + 16 * warp + g, acc[m][j][0] + acc[m][j][1]);
        __stcg(part + tok * 256 + m * 128 + 16 * warp + g + 8, acc[m][j][2] + acc[m][j][3]);
      }
    }
  __threadfence();
  __syncwarp();
  uint32_t old = 0;
  if (lane == 0)
    old = atomicAdd(p.sync + kSyncTiles + kFewWarps * (kFewMaxCtas + c) + warp, (uint32_t)blocks);
  old = __shfl_sync(0xffffffffu, old, 0);
  if (old + blocks != (uint32_t)sh.A * line.nkb) return;
  __threadfence();
  few_combine(p, sh, line, c, lane < 16 || valid[1]);
}

template <int KIND, int NBT>
__device__ void few_consumer(const FewArgs& p, FewShared& sh, uint8_t* smem) {
  using Cfg = FewCfg<KIND, NBT>;
  constexpr int S = Cfg::kStages;
  volatile int* abort_flag = &sh.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  Ring r;
  bool ok = true;
  {
    const Line line(sh.A, (p.f + 127) / 128, (p.d + Cfg::KB - 1) / Cfg::KB);
    Walk w(line, blockIdx.x);
    while (ok && w.more()) {
      float acc[2][NBT][4] = {};
      const int a = w.a, c = w.c;
      const int nb = (sh.row0[a + 1] - sh.row0[a] + 7) / 8;
      const bool v = c * 2 + warp / 4 < p.f / 64;
      const bool valid[2] = {v, v};
      int blocks = 0;
      while (w.more() && w.a == a && w.c == c) {
        ok = mbar_wait(&sh.full[r.st], r.ph, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) ok = false;
        if (!ok) break;
        few_block<KIND, NBT, NBT>(smem + r.st * Cfg::kStageBytes,
                                  min(Cfg::KB, p.d - w.kb * Cfg::KB), p.gate.group, nb, valid, acc);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[r.st]);
        r.next(S);
        w.next(line);
        ++blocks;
      }
      if (ok) few_gate_up_end<NBT>(p, sh, line, a, c, blocks, v, acc);
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report(p.status, kDevErrWaitTimeout);
    }
  }
  fence_proxy_async_all();               // h is read by asynchronous copies
  __threadfence();
  consumer_sync();
  if (threadIdx.x == 0 && !*abort_flag) {
    __threadfence();
    atomicAdd(p.sync + kSyncH, 1u);
  }
  {
    const Line line(sh.A, (p.d + 255) / 256, (p.f + Cfg::KB - 1) / Cfg::KB);
    Walk w(line, blockIdx.x);
    while (ok && w.more()) {
      float acc[2][2 * NBT][4] = {};
      const int a = w.a, c = w.c;
      const int nb = (2 * (sh.row0[a + 1] - sh.row0[a]) + 7) / 8;
      const bool valid[2] = {c * 4 + warp / 4 < p.d / 64, c * 4 + 2 + warp / 4 < p.d / 64};
      int blocks = 0;
      while (w.more() && w.a == a && w.c == c) {
        ok = mbar_wait(&sh.full[r.st], r.ph, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) ok = false;
        if (!ok) break;
        few_block<KIND, NBT, 2 * NBT>(smem + r.st * Cfg::kStageBytes,
                                      min(Cfg::KB, p.f - w.kb * Cfg::KB), p.gate.group, nb, valid,
                                      acc);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[r.st]);
        r.next(S);
        w.next(line);
        ++blocks;
      }
      if (ok) few_down_end<2 * NBT>(p, sh, line, a, c, blocks, valid, acc);
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report(p.status, kDevErrWaitTimeout);
    }
  }
}

template <int KIND, int NBT>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ FewArgs p, const __grid_constant__ CUtensorMap tmG,
               const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmD) {
  using Cfg = FewCfg<KIND, NBT>;
  extern __shared__ uint8_t dsmem_raw[];
  __shared__ FewShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x;
  volatile int* abort_flag = &sh.abort_flag;
  if (tid == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kFewWarps);
    }
    sh.abort_flag = 0;
    sh.never = 0;
    fence_barrier_init();
  }
  __syncthreads();

  // ---- R: router, top-k, tables
  if ((int)blockIdx.x < p.KS * p.CG) {
    few_router_rows<NBT>(p, smem);
    __threadfence();
    __syncthreads();
    if (tid == 0) atomicAdd(p.sync + kSyncRouter, 1u);
  }
  if ((int)blockIdx.x < p.T) {
    if (tid == 0) sh.ok = wait_count(p.sync + kSyncRouter, p.KS * p.CG, abort_flag);
    __syncthreads();
    if (sh.ok)
      for (int t = blockIdx.x; t < p.T; t += gridDim.x) few_route_token(p, sh, t);
  }
  __syncthreads();
  if (tid == 0) {
    sh.ok = wait_count(p.sync + kSyncRouted, p.T, abort_flag);
    if (!sh.ok) report(p.status, kDevErrWaitTimeout);
  }
  fence_proxy_async_smem();              // the router's staging becomes the ring
  __syncthreads();
  if (!sh.ok) return;
  few_tables(p, sh);
  if (sh.A == 0) {                       // a capacity of 0: every token passes through
    for (size_t i = (size_t)blockIdx.x * kFewThreads + tid; i < (size_t)p.T * p.d;
         i += (size_t)gridDim.x * kFewThreads)
      p.y[i] = p.x[i];
    return;
  }

  // ---- G and D
  if (tid < 32 * kFewWarps)
    few_consumer<KIND, NBT>(p, sh, smem);
  else
    few_producer<KIND, NBT>(p, sh, smem, &tmG, &tmU, &tmD);
}

// ---------------------------------------------------------------- host side
namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Byte sizes of the workspace, in order: the counters (with the status word
// first), the routing results, then what the phases hand on.
struct FewLayout {
  size_t sync, logits, idx, w, slot, counts, rpart, gpart, dpart, h;
  FewLayout(int64_t T, int64_t d, int64_t E, int64_t k, int64_t f) {
    const size_t dt = (size_t)(d + 255) / 256, ft = (size_t)(f + 127) / 128;
    sync = up256(256 + (kSyncTiles + kFewWarps * (kFewMaxCtas + dt)) * 4);
    logits = up256(size_t(T * E) * 4);
    idx = w = slot = up256(size_t(T * k) * 4);
    counts = up256(size_t(E) * 4);
    rpart = up256(size_t(kFewMaxSplits * T * E) * 8);
    gpart = (size_t(T * k) * ft + size_t(kFewMaxCtas) * T) * 1024;
    dpart = (size_t(T * k) * dt + size_t(kFewMaxCtas) * T) * 1024;
    h = up256(size_t(T * k * f) * 4);
  }
  size_t total() const {
    return sync + logits + idx + w + slot + counts + rpart + gpart + dpart + h;
  }
};

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
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = s;
  // cooperative: the CTAs wait for one another, so all of them run or none
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, g, u, dn);
}

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
  const int grid = di->sms < kFewMaxCtas ? di->sms : kFewMaxCtas;

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
  take(a.gpart, lay.gpart);
  take(a.dpart, lay.dpart);
  take(a.h, lay.h);

  // the router's split: 32 columns (or all of a few experts') by as many row
  // ranges as there are CTAs for, at most kFewMaxSplits (a token's CTA adds them)
  a.CW = a.E <= 8 ? 8 : (a.E <= 16 ? 16 : 32);
  a.CG = (a.E + a.CW - 1) / a.CW;
  a.KS = grid / a.CG;
  if (a.KS < 1) return cudaErrorInvalidConfiguration;
  if (a.KS > kFewMaxSplits) a.KS = kFewMaxSplits;

  CUtensorMap g{}, u{}, dn{};
  if (a.gate.group == 0 &&
      (!map_weights(&g, a.gate.w, a.E, a.d, a.f) || !map_weights(&u, a.up.w, a.E, a.d, a.f) ||
       !map_weights(&dn, a.down.w, a.E, a.f, a.d))) {
    *map_failed = true;
    return cudaSuccess;
  }
  if ((err = cudaMemsetAsync(ws, 0, lay.sync, s)) != cudaSuccess) return err;
  if (a.gate.group == 0) return launch_few_kind<0>(a, grid, g, u, dn, di, s);
  if (a.gate.group == 32) return launch_few_kind<2>(a, grid, g, u, dn, di, s);
  return launch_few_kind<1>(a, grid, g, u, dn, di, s);
}

}  // namespace moe
