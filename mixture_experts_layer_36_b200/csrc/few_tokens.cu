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
//      weights are in flight before the last CTA has finished G.  When all are
//      done, the k weighted rows of each token are added in j order.
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

constexpr int kColWarps = 8;                       // 16 columns of each half tile a warp
constexpr int kFewWarps = 2 * kColWarps;           // consumers: one a 16-column strip
constexpr int kWorkers = 32 * kFewWarps;
constexpr int kFewThreads = kWorkers + 32;         // and the producer warp
constexpr int kFewMaxCtas = 256;                   // sizes the workspace
constexpr int kFewMaxPairs = MOE_FEW_MAX_TOKENS * 8;
constexpr int kFewRouterRows = 384;                // router rows staged at once
constexpr int kFewMaxSplits = 32;

// grid-wide counters, zeroed by the call: arrivals of the router's partial
// sums, of the tokens' routing, of the CTAs that finished G and D; then for
// each cut gate/up tile (by the CTA that holds its first piece), per column
// warp, the blocks that are summed.
constexpr int kSyncRouter = 0, kSyncRouted = 32, kSyncH = 64, kSyncY = 96, kSyncTiles = 128;
constexpr int kSyncWords = kSyncTiles + kColWarps * kFewMaxCtas;

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
  static constexpr int kMergeBytes = kColWarps * 32 * 16; // gate and up sums meet here
  static constexpr int kFit = (224256 - kMergeBytes) / kStageBytes;
  static constexpr int kStages = kFit > 9 ? 9 : kFit;
  static constexpr int kSmemBytes = kStages * kStageBytes + kMergeBytes + 1024;
  // the router's staging uses the same memory: x (fp64), then W rows
  static constexpr int kXsBytes = 8 * NBT * kFewRouterRows * 8;
  static_assert(kXsBytes + kFewRouterRows * 32 * 4 <= kStages * kStageBytes, "router staging");
  static_assert(kWorkers * 8 * NBT * 8 <= kStages * kStageBytes, "router reduction");
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
  asm volatile("bar.sync 1, %0;" ::"n"(kWorkers) : "memory");
}
// the two warps that hold gate and up of the same columns
__device__ __forceinline__ void pair_sync(int col_warp) {
  asm volatile("bar.sync %0, 64;" ::"r"(2 + col_warp) : "memory");
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
  // the piece that holds block i: the last b with begin(b) <= i, which is
  // total * b < (i + 1) * parts; the quotient in fp32 is at most 1 off
  __device__ int piece(long long i) const {
    const long long lim = (i + 1) * parts;
    int b = (int)((float)lim / (float)total);
    while (b > 0 && total * b >= lim) --b;
    while (total * (b + 1) < lim) ++b;
    return b;
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
  // over `n` blocks of one unit
  __device__ void skip(const Line& l, int n) {
    i += n;
    kb += n;
    if (kb == l.nkb) {
      kb = 0;
      if (++c == l.nct) {
        c = 0;
        ++a;
      }
    }
  }
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
  const bool worker = tid < kWorkers;
  const int cg = blockIdx.x % p.CG, ks = blockIdx.x / p.CG;
  const int c = tid % p.CW, rg = tid / p.CW, nrg = kWorkers / p.CW;
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
        for (int i = tid; i < len * q; i += kWorkers) {
          const int r = i / q, v = i % q;
          if (4 * v < cols) cp_async16(smem_u32(wsm + r * p.CW + 4 * v), src + (size_t)r * p.E + 4 * v);
        }
      } else {
        for (int i = tid; i < len * p.CW; i += kWorkers) {
          const int r = i / p.CW, v = i % p.CW;
          if (v < cols) cp_async4(smem_u32(wsm + r * p.CW + v), src + (size_t)r * p.E + v);
        }
      }
      for (int i = tid; i < p.T * RR; i += kWorkers) {
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
  double* red = reinterpret_cast<double*>(smem);                   // [T][kWorkers]
  if (worker) {
#pragma unroll
    for (int t = 0; t < 8 * NBT; ++t)
      if (t < p.T) red[t * kWorkers + tid] = acc[t];
  }
  __syncthreads();
  if (worker) {
    for (int i = tid; i < p.T * p.CW; i += kWorkers) {
      const int t = i / p.CW, cc = i % p.CW;
      if (cc >= cols) continue;
      double s = 0.0;
      for (int g = 0; g < nrg; ++g) s += red[t * kWorkers + g * p.CW + cc];
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
// Fills stages with blocks of one phase.  unit() computes once for a tile what
// its blocks share, one copy (two token rows) a lane; the block index only
// moves the addresses.
template <int KIND, int NBT, bool DOWN>
struct Filler {
  using Cfg = FewCfg<KIND, NBT>;
  static constexpr int kTile = DOWN ? 4 : 2;    // 64-column groups of a full tile, per matrix
  const CUtensorMap* map;
  const uint8_t* code;
  const __nv_bfloat16* scale;
  const __nv_bfloat16 *row_a, *row_b;
  int K, lg, lane, jobs, mats, boxes, rows, e, dst, col, sdst, sjob;
  size_t scale_step;                            // scales from one block to the next

  __device__ Filler(const FewArgs& p)
      : K(DOWN ? p.f : p.d), lg(p.lg), lane(threadIdx.x % 32),
        mats(DOWN ? 1 : 2), scale_step((size_t)(KIND ? (Cfg::KB >> lg) : 0) * (DOWN ? p.d : p.f)) {}

  __device__ void unit(const FewArgs& p, const FewShared& sh, const CUtensorMap* tm0,
                       const CUtensorMap* tm1, int a, int c) {
    const int N = DOWN ? p.d : p.f;
    const int n = sh.row0[a + 1] - sh.row0[a];
    rows = DOWN ? 2 * n : n;
    e = sh.expert[a];
    boxes = min(kTile, N / 64 - c * kTile);
    jobs = mats * boxes;
    const int m = DOWN ? 0 : (lane >= boxes);
    const int b = lane - (m ? boxes : 0);
    col = (c * kTile + b) * 64;
    if constexpr (KIND == 0) {
      map = m ? tm1 : tm0;
      dst = (2 * m + b) * 8192;
    } else {
      const FewMatrix& w = DOWN ? p.down : (m ? p.up : p.gate);
      dst = (2 * m + b) * 4096;
      if (lane < jobs)
        code = static_cast<const uint8_t*>(w.w) +
               ((size_t)e * (N / 64) + c * kTile + b) * (K / 64) * 2048;
      // scale rows: a lane's matrix and group of the block (at most 2 x 4)
      const int per = Cfg::KB >> lg;
      const int sm = DOWN ? 0 : (lane >= per);
      const int sg = lane - (sm ? per : 0);
      const FewMatrix& sw = DOWN ? p.down : (sm ? p.up : p.gate);
      const int groups = (K + (1 << lg) - 1) >> lg;
      sjob = lane < mats * per ? sg : 1 << 20;
      sdst = Cfg::kWBytes + sg * 512 + sm * 256;
      scale = sw.scale + ((size_t)e * groups + sg) * N + c * (kTile * 64);
    }
    auto row = [&](int i) {
      return DOWN ? p.h + (size_t)(2 * sh.row0[a] + i) * p.f
                  : p.x + (size_t)sh.row_tok[sh.row0[a] + i] * p.d;
    };
    if (lane < rows) row_a = row(lane);
    if (lane + 32 < rows) row_b = row(lane + 32);
  }
  __device__ void weights(uint8_t* stage, uint64_t* bar, int kb) const {
    const int klen = min(Cfg::KB, K - kb * Cfg::KB);
    const int grows = KIND ? (klen + (1 << lg) - 1) >> lg : 0;
    const uint32_t wbytes = KIND == 0 ? 8192u : 32u * klen;
    if (lane == 0)
      mbar_arrive_expect_tx(bar, jobs * (wbytes + grows * 128u) + rows * klen * 2u);
    __syncwarp();
    if constexpr (KIND == 0) {
      if (lane < jobs) tma_load_3d(stage + dst, map, bar, col, kb * 64, e);
    } else {
      if (lane < jobs) bulk_load(stage + dst, code + (size_t)kb * 4096, wbytes, bar);
      if (sjob < grows) bulk_load(stage + sdst, scale + kb * scale_step, boxes * 128, bar);
    }
  }
  __device__ void tokens(uint8_t* stage, uint64_t* bar, int kb) const {
    const int klen = min(Cfg::KB, K - kb * Cfg::KB);
    uint8_t* to = stage + Cfg::kWBytes + Cfg::kScaleBytes + lane * Cfg::kPitch;
    if (lane < rows) bulk_load(to, row_a + kb * Cfg::KB, klen * 2, bar);
    if (lane + 32 < rows) bulk_load(to + 32 * Cfg::kPitch, row_b + kb * Cfg::KB, klen * 2, bar);
  }
};

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
  auto empty = [&] {
    return __all_sync(0xffffffffu, mbar_wait(&sh.empty[r.st], r.ph ^ 1, abort_flag)) != 0;
  };
  {
    const Line line(sh.A, (p.f + 127) / 128, (p.d + Cfg::KB - 1) / Cfg::KB);
    Filler<KIND, NBT, false> fill(p);
    bool fresh = true;
    for (Walk w(line, blockIdx.x); w.more(); w.next(line)) {
      if (fresh || w.kb == 0) fill.unit(p, sh, tmG, tmU, w.a, w.c);
      fresh = false;
      if (!(ok = empty())) break;
      fill.weights(stage(r.st), &sh.full[r.st], w.kb);
      fill.tokens(stage(r.st), &sh.full[r.st], w.kb);
      r.next(S);
    }
  }
  if (ok) {
    const Line line(sh.A, (p.d + 255) / 256, (p.f + Cfg::KB - 1) / Cfg::KB);
    Filler<KIND, NBT, true> fill(p);
    Walk w(line, blockIdx.x);
    Walk w0 = w;
    Ring r0 = r;
    bool fresh = true;
    int ahead = 0;                       // stages that hold weights but no rows yet
    for (; w.more() && ahead < S; w.next(line), ++ahead) {
      if (fresh || w.kb == 0) fill.unit(p, sh, tmD, tmD, w.a, w.c);
      fresh = false;
      if (!(ok = empty())) break;
      fill.weights(stage(r.st), &sh.full[r.st], w.kb);
      r.next(S);
    }
    if (ok && ahead)
      ok = __all_sync(0xffffffffu, wait_count(p.sync + kSyncH, gridDim.x, abort_flag)) != 0;
    fence_proxy_async_all();             // h was written through the generic proxy
    fresh = true;
    for (; ok && ahead; --ahead, w0.next(line), r0.next(S)) {
      if (fresh || w0.kb == 0) fill.unit(p, sh, tmD, tmD, w0.a, w0.c);
      fresh = false;
      fill.tokens(stage(r0.st), &sh.full[r0.st], w0.kb);
    }
    for (; ok && w.more(); w.next(line)) {
      if (w.kb == 0) fill.unit(p, sh, tmD, tmD, w.a, w.c);
      if (!(ok = empty())) break;
      fill.weights(stage(r.st), &sh.full[r.st], w.kb);
      fill.tokens(stage(r.st), &sh.full[r.st], w.kb);
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
// acc[j] += the weights of this warp's 16 columns times token block j.  Warps
// 0..7 hold the first half of the tile (gate), 8..15 the second (up).  NBL:
// token blocks.
template <int KIND, int NBT, int NBL, int NB>
__device__ __forceinline__ void few_block(const uint8_t* stage, int klen, int lg,
                                          float (&acc)[NB][4]) {
  using Cfg = FewCfg<KIND, NBT>;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rows = smem_u32(stage + Cfg::kWBytes + Cfg::kScaleBytes) +
                        (lane % 8) * Cfg::kPitch + (lane / 8) * 16;
  if constexpr (KIND == 0) {
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
      for (int s = 0; s < 2; ++s) {
        uint32_t a[4];
        ldsm4_trans(a, at + (2 * s2 + s) * 2048);
#pragma unroll
        for (int j = 0; j < NBL; ++j) mma_bf16(acc[j], a, b[j][2 * s], b[j][2 * s + 1]);
      }
    }
  } else {
    const uint8_t* codes = stage + (warp / 4) * 4096 + (warp % 4) * 512 + lane * 16;
    const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(stage + Cfg::kWBytes) +
                              16 * warp + lane / 4;
    const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      if (sub * 64 >= klen) break;
      const uint4 w4 = *reinterpret_cast<const uint4*>(codes + sub * 2048);
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
        const int grow = KIND == 1 ? (sub * 64) >> lg : 2 * sub + g;
        const float s0 = __bfloat162float(sc[grow * 256]);
        const float s1 = __bfloat162float(sc[grow * 256 + 8]);
#pragma unroll
        for (int j = 0; j < NBL; ++j) {
          float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < GS / 2; ++h) {
            uint32_t b[4];
            ldsm4(b, rows + j * 8 * Cfg::kPitch + sub * 128 + (g * GS / 2 + h) * 64);
            mma_bf16(t, a[g * GS + 2 * h], b[0], b[1]);
            mma_bf16(t, a[g * GS + 2 * h + 1], b[2], b[3]);
          }
          acc[j][0] = fmaf(s0, t[0], acc[j][0]);
          acc[j][1] = fmaf(s0, t[1], acc[j][1]);
          acc[j][2] = fmaf(s1, t[2], acc[j][2]);
          acc[j][3] = fmaf(s1, t[3], acc[j][3]);
        }
      }
    }
  }
}

// The blocks of one unit that lie in this CTA's piece, NBL token blocks wide;
// returns how many.  A warp whose wait gave up (ok = false) still walks all
// units, without waiting or computing: warps of a pair meet after each.
template <int KIND, int NBT, int NBL, int NB>
__device__ __forceinline__ int few_unit(FewShared& sh, const uint8_t* smem, int K, int lg,
                                        const Line& line, Walk& w, Ring& r, bool valid, bool& ok,
                                        float (&acc)[NB][4]) {
  using Cfg = FewCfg<KIND, NBT>;
  const int lane = threadIdx.x % 32;
  const int blocks = (int)min((long long)(line.nkb - w.kb), w.end - w.i);
  int left = K - w.kb * Cfg::KB;
  for (int i = 0; ok && i < blocks; ++i, left -= Cfg::KB) {
    if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[r.st], r.ph, &sh.abort_flag))) {
      ok = false;
      break;
    }
    if (valid) few_block<KIND, NBT, NBL, NB>(smem + r.st * Cfg::kStageBytes, left, lg, acc);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[r.st]);
    r.next(Cfg::kStages);
  }
  w.skip(line, blocks);
  return blocks;
}

template <int KIND, int NBT, int NB>
__device__ __forceinline__ int few_unit_n(FewShared& sh, const uint8_t* smem, int K, int lg,
                                          const Line& line, Walk& w, Ring& r, int nb, bool valid, bool& ok,
                                          float (&acc)[NB][4]) {
  if constexpr (NB >= 8)
    if (nb > 4) return few_unit<KIND, NBT, 8, NB>(sh, smem, K, lg, line, w, r, valid, ok, acc);
  if constexpr (NB >= 4)
    if (nb > 2) return few_unit<KIND, NBT, 4, NB>(sh, smem, K, lg, line, w, r, valid, ok, acc);
  if constexpr (NB >= 2)
    if (nb > 1) return few_unit<KIND, NBT, 2, NB>(sh, smem, K, lg, line, w, r, valid, ok, acc);
  return few_unit<KIND, NBT, 1, NB>(sh, smem, K, lg, line, w, r, valid, ok, acc);
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
// by the warp whose piece completes the tile.  Called by both warps of a pair;
// the second one hands its sums (up) to the first.
template <int NB>
__device__ void few_gate_up_end(const FewArgs& p, const FewShared& sh, float* merge,
                                const Line& line, int a, int c, int blocks,
                                const float (&acc)[NB][4]) {
  const int warp = threadIdx.x / 32 % kColWarps, lane = threadIdx.x % 32;
  const bool up = threadIdx.x / 32 >= kColWarps;
  const int g = lane / 4, q = lane % 4;
  const int n = sh.row0[a + 1] - sh.row0[a];
  const int col = 16 * warp + g;
  const bool whole = blocks == line.nkb;
  float* part = p.gpart + part_at(sh, a, c, line.nct, blockIdx.x, p.T);
  float4* slot = reinterpret_cast<float4*>(merge) + warp * 32 + lane;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    if (8 * j >= n) break;
    if (up) *slot = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    pair_sync(warp);
    if (!up) {
      const float4 o = *slot;
      const float us[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 8 * j + 2 * q + (i & 1), cc = col + 8 * (i >> 1);
        if (tok >= n) continue;
        if (whole) {
          store_h(p, sh.row0[a] + tok, c * 128 + cc, acc[j][i], us[i]);
        } else {
          __stcg(part + tok * 256 + cc, acc[j][i]);
          __stcg(part + tok * 256 + 128 + cc, us[i]);
        }
      }
    }
    pair_sync(warp);
  }
  if (whole || up) return;
  const long long u = (long long)a * line.nct + c;
  const int first = line.piece(u * line.nkb), last = line.piece((u + 1) * line.nkb - 1);
  __threadfence();
  __syncwarp();
  uint32_t old = 0;
  if (lane == 0) old = atomicAdd(p.sync + kSyncTiles + first * kColWarps + warp, (uint32_t)blocks);
  old = __shfl_sync(0xffffffffu, old, 0);
  if (old + blocks != (uint32_t)line.nkb) return;
  __threadfence();
  for (int i = lane; i < 16 * n; i += 32) {
    const int tok = i / 16, cc = 16 * warp + i % 16;
    const float* src = p.gpart + part_at(sh, a, c, line.nct, first, p.T) + tok * 256 + cc;
    float gs = 0.f, us = 0.f;
    for (int b = first; b <= last; ++b, src += (size_t)p.T * 256) {
      gs += __ldcg(src);
      us += __ldcg(src + 128);
    }
    store_h(p, sh.row0[a] + tok, c * 128 + cc, gs, us);
  }
}

// The end of a down piece: its partial sums (a token's two columns, from the
// two terms of h, added).
template <int NB>
__device__ void few_down_end(const FewArgs& p, const FewShared& sh, const Line& line, int a, int c,
                             const float (&acc)[NB][4]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, q = lane % 4;
  const int n = sh.row0[a + 1] - sh.row0[a];
  float* part = p.dpart + part_at(sh, a, c, line.nct, blockIdx.x, p.T) + 16 * warp + g;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int tok = 4 * j + q;
    if (tok < n) {
      __stcg(part + tok * 256, acc[j][0] + acc[j][1]);
      __stcg(part + tok * 256 + 8, acc[j][2] + acc[j][3]);
    }
  }
}

// y of 128 columns (half m of tile c, 4 a lane) of token t by one warp: the
// weighted rows in j order, the pieces of each in CTA order.
__device__ void few_combine(const FewArgs& p, const FewShared& sh, const Line& line, int t, int c,
                            int m) {
  const int lane = threadIdx.x % 32;
  const int col = c * 256 + m * 128 + 4 * lane;
  int pieces = -1;
  uint32_t at = 0;
  if (lane < p.k) {
    const int row = sh.pair_row[t * p.k + lane];
    if (row >= 0) {
      int a = 0;                          // the active expert that holds the row
      for (int step = 128; step; step >>= 1)
        if (a + step < sh.A && sh.row0[a + step] <= row) a += step;
      const long long u = (long long)a * line.nct + c;
      const int first = line.piece(u * line.nkb);
      pieces = line.piece((u + 1) * line.nkb - 1) - first;
      at = (uint32_t)(part_at(sh, a, c, line.nct, first, p.T) / 256) + (row - sh.row0[a]);
    }
  }
  const bool valid = col < p.d;
  float4 v[8];
  int extra[8];
  const float* src[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    extra[j] = __shfl_sync(0xffffffffu, pieces, j);
    src[j] = p.dpart + (size_t)__shfl_sync(0xffffffffu, at, j) * 256 + m * 128 + 4 * lane;
    v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (extra[j] >= 0 && valid) v[j] = __ldcg(reinterpret_cast<const float4*>(src[j]));
  }
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  bool any = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (extra[j] < 0) continue;
    any = true;
    for (int b = 1; b <= extra[j] && valid; ++b) {
      const float4 o = __ldcg(reinterpret_cast<const float4*>(src[j] + (size_t)b * p.T * 256));
      v[j].x += o.x;
      v[j].y += o.y;
      v[j].z += o.z;
      v[j].w += o.w;
    }
    const float w = sh.pair_w[t * p.k + j];
    y.x = fmaf(w, v[j].x, y.x);
    y.y = fmaf(w, v[j].y, y.y);
    y.z = fmaf(w, v[j].z, y.z);
    y.w = fmaf(w, v[j].w, y.w);
  }
  if (!valid) return;
  const size_t out = (size_t)t * p.d + col;
  *reinterpret_cast<uint2*>(p.y + out) =
      any ? make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w))
          : __ldg(reinterpret_cast<const uint2*>(p.x + out));
}

// All consumer warps of this CTA are done with a phase: its results are
// visible, then counted.
__device__ __forceinline__ void few_arrive(const FewShared& sh, uint32_t* counter) {
  __threadfence();
  consumer_sync();
  if (threadIdx.x == 0 && !*static_cast<const volatile int*>(&sh.abort_flag)) {
    __threadfence();
    atomicAdd(counter, 1u);
  }
}

template <int KIND, int NBT>
__device__ void few_consumer(const FewArgs& p, FewShared& sh, uint8_t* smem) {
  using Cfg = FewCfg<KIND, NBT>;
  volatile int* abort_flag = &sh.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float* merge = reinterpret_cast<float*>(smem + Cfg::kStages * Cfg::kStageBytes);
  Ring r;
  bool ok = true;
  {
    const Line line(sh.A, (p.f + 127) / 128, (p.d + Cfg::KB - 1) / Cfg::KB);
    Walk w(line, blockIdx.x);
    while (w.more()) {
      float acc[NBT][4] = {};
      const int a = w.a, c = w.c;
      const int nb = (sh.row0[a + 1] - sh.row0[a] + 7) / 8;
      const bool valid = c * 2 + warp % kColWarps / 4 < p.f / 64;
      const int blocks =
          few_unit_n<KIND, NBT, NBT>(sh, smem, p.d, p.lg, line, w, r, nb, valid, ok, acc);
      if (valid) few_gate_up_end<NBT>(p, sh, merge, line, a, c, ok ? blocks : 0, acc);
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report(p.status, kDevErrWaitTimeout);
    }
  }
  fence_proxy_async_all();               // h is read by asynchronous copies
  few_arrive(sh, p.sync + kSyncH);
  const Line line(sh.A, (p.d + 255) / 256, (p.f + Cfg::KB - 1) / Cfg::KB);
  Walk w(line, blockIdx.x);
  while (ok && w.more()) {
    float acc[2 * NBT][4] = {};
    const int a = w.a, c = w.c;
    const int nb = (2 * (sh.row0[a + 1] - sh.row0[a]) + 7) / 8;
    const bool valid = c * 4 + warp / 4 < p.d / 64;
    few_unit_n<KIND, NBT, 2 * NBT>(sh, smem, p.f, p.lg, line, w, r, nb, valid, ok, acc);
    if (ok && valid) few_down_end<2 * NBT>(p, sh, line, a, c, acc);
  }
  if (!ok && lane == 0) {
    *abort_flag = 1;
    report(p.status, kDevErrWaitTimeout);
  }
  few_arrive(sh, p.sync + kSyncY);

  // ---- combine: (tile half, token) to warps, CTA by CTA
  const int items = 2 * line.nct * p.T;
  if ((int)blockIdx.x >= items) return;
  if (threadIdx.x == 0) {
    sh.ok = !*abort_flag && wait_count(p.sync + kSyncY, gridDim.x, abort_flag);
    if (!sh.ok) report(p.status, kDevErrWaitTimeout);
  }
  consumer_sync();
  if (!sh.ok) return;
  for (int i = threadIdx.x / 32 * gridDim.x + blockIdx.x; i < items; i += kFewWarps * gridDim.x) {
    const int t = i / (2 * line.nct), x = i - t * 2 * line.nct;
    few_combine(p, sh, line, t, x / 2, x % 2);
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
  if (tid < kWorkers)
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
    sync = up256(256 + kSyncWords * 4);
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

  a.lg = a.gate.group == 128 ? 7 : (a.gate.group == 64 ? 6 : 5);

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
