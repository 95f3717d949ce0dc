// Sampled acceptance of speculative drafts: each drafted token is verified
// against the target model's probabilities, with the caller's random numbers.
//
// Request b's nodes are logits rows qo_indptr[b] ..; p_v = softmax(logits[v] /
// T_b).  From the root, the children c_1 < c_2 < ... of node v are tried in
// index order, x_j the token of c_j and q the distribution it was drawn from:
//   r_0 = p_v;  c_j is accepted iff u_j q(x_j) < r_{j-1}(x_j), else
//   r_j = (r_{j-1} - q)+ / sum (r_{j-1} - q)+
// (speculative sampling, Leviathan et al. 2023, one residual per rejected
// sibling as in SpecInfer, Miao et al. 2024).  The residuals have the closed
// form r_j = (p - A_j q)+ / B_j with A_0 = 0, B_0 = 1, A_{j+1} = A_j + B_j and
// B_{j+1} = sum_x (p(x) - A_{j+1} q(x))+, since ((p - A q)+ - B q)+ =
// (p - (A + B) q)+: two numbers stand for r_j, and a rejection costs a sum over
// the row only when another sibling follows.  Without draft distributions q is
// the indicator of x_j: r_j is p with the rejected tokens taken out and B_j
// what is left of it.  When no child is accepted the bonus token is drawn from
// r by a race of exponentials, argmax_x r(x) / e(x) with e(x) ~ Exp(1) given:
// a maximum, so neither a prefix sum over the vocabulary nor the order of the
// reduction enters the result.
//
// One cluster of CTAs per request walks its tree, each CTA on its slice of
// the vocabulary.  A pass reads the rows of the current node and of its first
// child, that one's first child and so on (kRows of them at most), since a walk
// is a chain of dependent steps -- load, reduce, exchange, decide -- whose
// latency and not its bytes sets the time: the rows of a pass share one
// exchange through distributed shared memory, and a warp for each decides about
// its children at the same time.  The walk then follows the decisions as far as
// they lead along those rows.  Rows further off are read only when the walk
// gets there, so a 64-node tree whose path is two nodes long reads four rows.
//
// On one GB300 in a CUDA graph: a chain of 4 drafts over 32,016 tokens 7.7 us,
// 8 trees of 64 nodes over 128,256 tokens 13.4 us (latency both), 64 ragged
// chains of up to 8 nodes over 128,256 tokens, fp32 drafts, 39.9 us (103 MB of
// HBM: 38 % of its rate; 1.7 waves of CTAs of some 15 us, a pass bound by HBM and
// by the exponentials, 16 a cycle and SM, the steps between by latency).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/verify_attn.h"
#include "va_device.cuh"
#include "va_kernels.h"
#include "va_tc.cuh"

namespace va {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kRows = 8;        // rows of a pass at most
constexpr int kChildList = 64;  // children's tokens kept in shared memory (further ones are searched)
constexpr int kMarks = 32;
constexpr int kGroups = 16;     // groups of eight entries a thread keeps bounds of
constexpr int kVectors = 8;     // 16-byte loads of a thread in flight
static_assert(kWarps == 2 * kRows, "a warp that decides and one that prefetches for each row");
constexpr int kNodes = 128;     // a tree of at most so many nodes is kept in shared memory

__device__ __forceinline__ uint64_t race_key(float v, uint32_t idx) {  // v >= 0
  return ((uint64_t)(__float_as_uint(v) | 0x80000000u) << 32) | (uint64_t)(0xffffffffu - idx);
}
__device__ __forceinline__ uint64_t logit_key(float v, uint32_t idx) {
  const uint32_t u = __float_as_uint(v);
  return ((uint64_t)((u & 0x80000000u) ? ~u : (u | 0x80000000u)) << 32) | (uint64_t)(0xffffffffu - idx);
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Store 16 bytes at shared address `addr` (of this CTA) in the shared memory
// of CTA `cta` of the cluster, counted there by the mbarrier at `bar`.
__device__ __forceinline__ void cluster_store(uint32_t addr, uint32_t bar, uint32_t cta, uint64_t x, uint64_t y) {
  uint32_t a, m;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(cta));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(m) : "r"(bar), "r"(cta));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(a),
               "l"(x), "l"(y), "r"(m)
               : "memory");
}
__device__ __forceinline__ bool cluster_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Ask for [p, p + bytes) to be brought into L2, rounded inwards to 16 bytes:
// one instruction, by one thread.
__device__ __forceinline__ void prefetch_l2(const void* p, int64_t bytes) {
  const uintptr_t a = (reinterpret_cast<uintptr_t>(p) + 15) & ~(uintptr_t)15,
                  z = (reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes) & ~(uintptr_t)15;
  if (z > a)   // (at most 1 GB, far more than L2 holds)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a),
                 "r"((uint32_t)(z - a < (1u << 30) ? z - a : (1u << 30)))
                 : "memory");
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// An element as it lies in memory, and its value: apart, since whatever is
// done to a loaded word waits for it.
template <bool BF16>
__device__ __forceinline__ uint32_t load_bits(const void* row, int64_t i) {
  uint32_t w;   // (a 16-bit load into a 32-bit register: no conversion behind it)
  if constexpr (BF16)
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(w) : "l"(static_cast<const uint16_t*>(row) + i));
  else
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w) : "l"(static_cast<const uint32_t*>(row) + i));
  return w;
}
template <bool BF16>
__device__ __forceinline__ float bits_value(uint32_t w) {
  return __uint_as_float(BF16 ? w << 16 : w);
}
template <bool BF16>
__device__ __forceinline__ float load_elem(const void* row, int64_t i) {
  return bits_value<BF16>(load_bits<BF16>(row, i));
}

// Eight consecutive elements from element i (16-byte aligned there).
template <bool BF16>
__device__ __forceinline__ void load8(const void* row, int64_t i, float* x) {
  if constexpr (BF16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(u[k] << 16);
      x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + i));
    const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + i) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

// What is known of one row of a pass.
struct RowState {
  // Maximum; its weights 2^((x - m) log2(e) / T) but the maximum's own 1; their
  // sum, 1 + tail; A after the children tried so far, times the sum.
  float m, tail, sf, as;
  float x;                  // logit of the accepted child's token
  int am, dead;             // first argmax (T = 0); nothing of the row is possible
  int n_child;
  int kid[32];              // the children now in the lanes of the row's warp
  uint32_t marks[kMarks];   // bit (x >> 3) mod 32 kMarks for every child's token x
  int child_tok[kChildList];
};
// What a CTA tells the others of the cluster about a row: a tail, a residual's
// sum or a key; a maximum (low half) and where its walk stands (high half).
struct alignas(16) Message {
  uint64_t a, b;
};
struct Shared {
  uint64_t part[kRows][kWarps];        // the warps' parts of a row: tail and maximum, or a key or sum
  float beat[kWarps];
  Message ex[2][kRows][kMaxCluster];   // the cluster's exchange, two phases
  uint64_t ex_bar[2];
  alignas(16) int keys[kThreads];   // of every request: the larger, the sooner it is taken
  int b, o, L;                      // this cluster's request, its first row, its nodes
  RowState row[kRows];
  // each row's node; the accepted child, or -1; whether a residual's sum is wanted first
  int node[kRows], next[kRows], more[kRows];
  int par[kNodes], tok[kNodes], first[kNodes], kids[kNodes];  // parents, tokens, first children, their number
  float u[kNodes];
  float lx[kNodes], lm[kNodes], lt[kNodes];     // emitted tokens' logits and their rows' maxima and tails
  float c_hi, c_lo;
  // the request's temperature, read again where fp64 needs it: kept in a
  // register, its conversion would be hoisted and done by every thread, on a
  // pipe of two lanes a cycle
  volatile float temp;
};

// Sums cross threads as integers: adding them is exact, takes the integer pipe
// (fp64 adds run at a 64th of its rate here) and needs no order.  A warp reduces
// with redux, whose 32-bit words a 64-bit sum is cut into: 27 bits of 32 lanes
// stay below 2^32.  (A step of a walk is a dozen short dependent pieces of one
// warp; with five rounds of shuffles for each of its reductions a chain of 4
// drafts took 1.5 us longer.)  Residuals are in units of 2^-50; terms of a tail,
// which may be as small as they like, in the unit that gives the largest of them 27 bits.
__device__ __forceinline__ uint64_t warp_add64(uint64_t v) {
  constexpr uint32_t kLimb = (1u << 27) - 1;
  const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)v & kLimb),
                 b = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27) & kLimb),
                 c = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 54));
  return (uint64_t)a + ((uint64_t)b << 27) + ((uint64_t)c << 54);
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The lanes' terms >= 0 added, each rounded to 2^-27 of the largest or less.
__device__ __forceinline__ float warp_add(float v) {
  const int e = max(__float_as_int(warp_max(v)) >> 23, 27);   // (below 2^-100 the unit stays)
  const uint32_t sum = __reduce_add_sync(0xffffffffu, __float2uint_rn(v * __int_as_float((280 - e) << 23)));
  return __uint2float_rn(sum) * __int_as_float((e - 26) << 23);
}

// (x - m) c ln 2 - log(1 + tail) in fp32 pairs (fp64 took 1.2 us of a request's
// end): c = c_hi + c_lo is log2(e) / T.  Of the likeliest token the first term
// is 0 and the second keeps the tail's digits, however small it is.
__device__ __forceinline__ float log_prob(float x, float m, float c_hi, float c_lo, float tail) {
  const float d = x - m, dv = d - x, d_lo = (x - (d - dv)) - (m + dv);   // x - m = d + d_lo
  const float y = d * c_hi;
  if (!(y > -3e38f)) return -INFINITY;
  const float y_lo = fmaf(d, c_hi, -y) + fmaf(d, c_lo, d_lo * c_hi);
  const float r = y * 0.693147182464599609f;
  // ln 2 less its rounding to fp32: -1.9046543e-9
  const float r_lo = fmaf(y, 0.693147182464599609f, -r) + fmaf(y, -1.9046543e-9f, y_lo * 0.693147182464599609f);
  const float l = log1pf(tail);
  const float t = r - l, tv = t - r;
  return t + ((r - (t - tv)) - (l + tv) + r_lo);
}

// LB: logits bf16 (else fp32).  QT: draft distributions: 0 none, 1 bf16, 2 fp32.
template <bool LB, int QT>
__global__ void __launch_bounds__(kThreads, 1) accept_sample_kernel(const SampleParams p) {
  __shared__ Shared sh;
  __shared__ float bounds[QT ? kGroups : 1][kThreads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = p.cluster;
  const int rank = (int)cluster_rank(), place = blockIdx.x / C;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.ex_bar[i]), 1);
    mbar_fence_init();
    for (int i = 0; i < 2; ++i) mbar_expect_tx(smem_u32(&sh.ex_bar[i]), C * kRows * (int)sizeof(Message));
  }
  cluster_arrive();  // waited for before the first store to another CTA's shared memory
  grid_dependency_wait();
  grid_dependents_launch();
  // The tables are read once, for every thread: what steers the barriers below
  // is the same throughout the CTA even if the caller changes them meanwhile.
  // Where not all CTAs fit the GPU at once, the clusters -- which start in the
  // order of their numbers -- take the requests with the most nodes first (T = 0
  // after others: they end without the race).  64 ragged chains: 39.2 us, 43.4
  // in the order given.
  if (p.rows < kRows && p.batch <= kThreads) {
    int o_t = 0, L_t = 0, key = -1;
    float temp_t = 1.f;
    if (tid < p.batch) {
      o_t = p.qo_indptr[tid];
      L_t = p.qo_indptr[tid + 1] - o_t;
      if (p.temperature) temp_t = p.temperature[tid];
      key = (2 * min(max(L_t, 0), 1 << 16) + (temp_t == 0.f ? 0 : 8)) * kThreads + (kThreads - 1 - tid);
    }
    sh.keys[tid] = key;
    __syncthreads();
    if (tid < p.batch) {
      int before = 0;
      for (int i = 0; i < p.batch; i += 4) {   // (behind the batch: -1)
        const int4 other = *reinterpret_cast<const int4*>(&sh.keys[i]);
        before += (other.x > key) + (other.y > key) + (other.z > key) + (other.w > key);
      }
      if (before == place) {
        sh.b = tid;
        sh.o = o_t;
        sh.L = L_t;
        sh.temp = temp_t;
      }
    }
  } else if (tid == 0) {
    const int o = p.qo_indptr[place];
    sh.b = place;
    sh.o = o;
    sh.L = p.qo_indptr[place + 1] - o;
    sh.temp = p.temperature ? p.temperature[place] : 1.f;
  }
  if (tid < kNodes) {
    sh.first[tid] = kNodes;
    sh.kids[tid] = 0;
  }
  __syncthreads();
  const int b = sh.b, o = sh.o, L = sh.L;
  const float temp = sh.temp;
  const bool table_ok = o >= 0 && L >= 0 && (int64_t)o + L <= p.total;
  const int V = p.vocab;
  const int c0 = (int)min((int64_t)V, (int64_t)rank * p.slice), c1 = (int)min((int64_t)V, (int64_t)c0 + p.slice);
  const float* noise = p.noise + (size_t)b * p.noise_stride;
  constexpr int LES = LB ? 2 : 4, QES = QT == 1 ? 2 : 4;
  const bool greedy = temp == 0.f;
  auto row_of = [&](int i) -> const void* {
    return static_cast<const uint8_t*>(p.logits) + (size_t)(o + i) * p.row_stride * LES;
  };
  auto qrow_of = [&](int i) -> const void* {
    return QT ? static_cast<const uint8_t*>(p.draft) + (size_t)(o + i) * p.draft_stride * QES : nullptr;
  };
  // this CTA's slice of node i's row, towards L2
  auto prefetch_row = [&](int i) {
    prefetch_l2(static_cast<const uint8_t*>(row_of(i)) + (size_t)c0 * LES, (int64_t)(c1 - c0) * LES);
  };
  // the noise (read last, but always) too: at once where SMs idle, else while
  // the first pass's exchange and decisions leave HBM idle -- asked for at the
  // start it would delay the rows (64 chains: 46.3 us, 44.5 behind them)
  const bool noise_first = p.rows == kRows;
  auto prefetch_noise = [&]() {
    if (!greedy) prefetch_l2(noise + c0, (int64_t)(c1 - c0) * 4);
  };
  // (by warps that have nothing of the tables to read)
  if (tid == kThreads - 32 && table_ok && L > 0) {
    prefetch_row(0);
    if (noise_first) prefetch_noise();
  }
  if (warp == kWarps - 2) {
    // log2(e) / T as a float pair: a rounded factor alone would tilt the whole
    // distribution by |logit difference| * 2^-25.  Rounded down, so that both
    // parts are positive and a logit of -inf stays -inf (log2(e) itself is
    // 1.4426950216 + 1.926e-8).
    const float hi = greedy ? 1.f : __fdiv_rd(1.4426950216293335f, temp);
    const float lo =
        greedy ? 1.f
               : fminf(fmaxf((fmaf(-hi, temp, 1.4426950216293335f) + 1.925963033500e-8f) / temp, 1e-45f), 3e38f);
    if (lane == 0) {
      sh.c_hi = hi;
      sh.c_lo = lo;
    }
  }
  int bad = 0;
  if (table_ok)
    for (int i = tid; i < L; i += kThreads) {
      const int par = p.parents[o + i];
      const bool wrong = i == 0 ? par >= 0 : (par < 0 || par >= i);
      bad |= wrong;
      if (L <= kNodes) {
        sh.par[i] = par;
        sh.tok[i] = p.tokens[o + i];
        sh.u[i] = p.uniforms[o + i];
        if (i > 0 && !wrong) {
          atomicMin(&sh.first[par], i);
          atomicAdd(&sh.kids[par], 1);
        }
      }
    }
  bad = __syncthreads_or(bad) || !table_ok || !(temp >= 0.f && temp < INFINITY);
  const float c_hi = sh.c_hi, c_lo = sh.c_lo;
  cluster_wait();

  // The exchange: lane k of the r-th warp sends its message of row r to CTA k,
  // and an mbarrier here counts the messages of all CTAs into sh.ex[phase][row]
  // [0 .. C): one way through the cluster's network, where a cluster barrier
  // behind plain stores takes two (a chain of 4 drafts: 7.5 us, 7.9 with it).  All kRows
  // messages are always sent, so every count is the same.  The two phases
  // alternate, so a CTA that runs ahead never writes what a slower one still
  // reads.  With them goes a tag of where the sender's walk stands.  Every CTA
  // computes the same walk from the same inputs; should they differ -- inputs
  // written while they are read -- all of them see it at the same exchange and
  // end there, before one waits for, or writes to, another that has left.
  int phase = 0;
  uint32_t parities = 0;
  bool late = false;
  // every thread, all lanes of a warp with the same words; false: the CTAs' walks differ
  auto exchange = [&](uint32_t tag, uint64_t a, uint32_t m) -> bool {
    phase ^= 1;
    if (warp < kRows && lane < C)
      cluster_store(smem_u32(&sh.ex[phase][warp][rank]), smem_u32(&sh.ex_bar[phase]), lane, a, (uint64_t)tag << 32 | m);
    bool here = false;
    for (uint32_t i = 0; i < kSpinLimit && !here; ++i)
      here = cluster_try_wait(smem_u32(&sh.ex_bar[phase]), (parities >> phase) & 1u);
    late = !__syncthreads_and(here);
    parities ^= 1u << phase;
    if (tid == 0) mbar_expect_tx(smem_u32(&sh.ex_bar[phase]), C * kRows * (int)sizeof(Message));   // its next use
    const uint32_t other = (uint32_t)(sh.ex[phase][0][lane < C ? lane : 0].b >> 32);
    return __all_sync(0xffffffffu, other == tag) && !late;
  };
  enum : uint32_t { kStats = 1u << 28, kResidual = 2u << 28, kBonus = 3u << 28, kEnd = 4u << 28, kNone = 5u << 28 };
  // no answer: the request's outputs say so
  auto give_up = [&](bool flag) {
    if (late) {   // nothing may arrive here after this CTA has ended: wait for the others to end too
      if (tid == 0 && p.status) atomicOr(p.status, VA_DEV_TIMEOUT);
      cluster_sync();
    }
    if (rank != 0) return;
    if (tid == 0) {
      p.accept_len[b] = 0;
      p.bonus[b] = -1;
      if (flag && p.status) atomicOr(p.status, VA_DEV_BAD_TABLE);
    }
    if (table_ok)
      for (int i = tid; i < L; i += kThreads) {
        p.path[o + i] = -1;
        if (p.logprobs) p.logprobs[o + i] = 0.f;
      }
  };
  if (bad || L == 0) {
    const bool same = exchange(kNone, 0, 0);
    give_up(bad || !same);
    return;
  }
  const uint64_t ch2 = f32x2(c_hi, c_hi), cl2 = f32x2(c_lo, c_lo);
  // 2^((x - m) log2(e) / T) of a pair: the difference first (exact for bf16
  // logits of like size), then the two-term product
  auto weight2 = [&](float x0, float x1, float m, float* w0, float* w1) {
    const uint64_t d = add_f32x2(f32x2(x0, x1), f32x2(-m, -m));
    const uint64_t y = fma_f32x2(d, ch2, fma_f32x2(d, cl2, 0ull));
    *w0 = ex2(f32x2_lo(y));
    *w1 = ex2(f32x2_hi(y));
  };
  // twice that, which is 2 at the maximum and below 2 elsewhere
  auto twice2 = [&](float x0, float x1, float m, float* w0, float* w1) {
    const uint64_t d = add_f32x2(f32x2(x0, x1), f32x2(-m, -m));
    const uint64_t y = fma_f32x2(d, ch2, fma_f32x2(d, cl2, f32x2(1.f, 1.f)));
    *w0 = ex2(f32x2_lo(y));
    *w1 = ex2(f32x2_hi(y));
  };
  auto weight = [&](float x, float m) {
    const float d = x - m;
    return ex2(fmaf(d, c_hi, d * c_lo));
  };

  const int32_t* par = L <= kNodes ? sh.par : p.parents + o;
  const int32_t* tok = L <= kNodes ? sh.tok : p.tokens + o;
  const float* uni = L <= kNodes ? sh.u : p.uniforms + o;
  int v = 0, k = 0;
  if (tid == 0 && rank == 0) p.path[o] = 0;
  for (;;) {
    // ---- the rows of this pass: the first child's always, those below it
    // while no node has a choice.  A chain of 4 drafts (32,016 tokens) took
    // 7.9 us with up to eight rows, 9.4 with four, 11.0 with two and 14.3 with one;
    // a wide tree 13.6 us with the first child's row and 16.8 without.
    // The host asks for eight rows where the whole batch fits the GPU, else for
    // four: 64 ragged chains took 39.6 us with four and 43.2 with eight, whose
    // rows past the accepted ones are read from HBM for nothing.
    int n = 1, mine = (warp & (kRows - 1)) == 0 ? v : -1;   // rows; the node that this warp decides about
    int n_kids = L;                                         // how many children it has at most
    if (L <= kNodes) {
      bool alone = true;
      int kids = sh.kids[v], at = sh.first[v];
      if (mine == v) n_kids = kids;
      for (; n < p.rows; ++n) {
        alone = alone && kids == 1;
        if (kids == 0 || (n > 1 && !alone)) break;
        if ((warp & (kRows - 1)) == n) mine = at;
        kids = sh.kids[at];
        at = sh.first[at];
        if ((warp & (kRows - 1)) == n) n_kids = kids;
      }
    }
    const int row_warps = kWarps / (n > 4 ? 8 : n > 2 ? 4 : n);   // warps of a row in the pass over them
    // slices that take more than one round of loads are asked for in one go,
    // by the warps that decide about no row
    if (warp >= kRows) {
      if (mine > 0 && lane == 0 && (int64_t)(c1 - c0) * LES > row_warps * 32 * 16 * kVectors) prefetch_row(mine);
      mine = -1;
    }

    // ---- its children, up to 32 at a time, one a lane: what they need is
    // asked for before the pass over the rows, so it arrives meanwhile
    RowState& rs = sh.row[warp & (kRows - 1)];
    const void* const row = row_of(max(mine, 0));
    const void* const qrow = qrow_of(max(mine, 0));
    int scan = mine + 1;   // the next node to look at
    uint32_t win = 0;      // lanes whose child has not been tried
    int kid = -1, ctok = -1;
    uint32_t cxb = 0, cqb = 0;                  // token's logit and draft probability as loaded,
    bool has = false;                           // if it is a token and nothing of it was rejected,
    float cx = -INFINITY, cq = 0.f, cu = 0.f;   // and as numbers; the child's number
    auto load_children = [&]() {
      int cnt = 0;
      if (n_kids == 1 && scan == mine + 1 && L <= kNodes) {   // a chain's only child
        if (lane == 0) rs.kid[0] = sh.first[mine];
        cnt = 1;
        scan = L;
      }
      if (n_kids == 0) scan = L;
      if (L <= kNodes && n_kids <= 32 && scan < L) {   // the whole tree at once
        bool is[kNodes / 32];
        uint32_t who[kNodes / 32];
#pragma unroll
        for (int c = 0; c < kNodes / 32; ++c) {
          const int i = 32 * c + lane;
          is[c] = i > mine && i < L && sh.par[i] == mine;
          who[c] = __ballot_sync(0xffffffffu, is[c]);
        }
#pragma unroll
        for (int c = 0; c < kNodes / 32; ++c) {
          if (is[c]) rs.kid[cnt + __popc(who[c] & ((1u << lane) - 1u))] = 32 * c + lane;
          cnt += __popc(who[c]);
        }
        scan = L;
      }
      while (scan < L && cnt < 32) {
        const int i = scan + lane;
        const bool is = i < L && par[i] == mine;
        const uint32_t m = __ballot_sync(0xffffffffu, is);
        const int pos = cnt + __popc(m & ((1u << lane) - 1u));
        if (is && pos < 32) rs.kid[pos] = i;
        const uint32_t full = __ballot_sync(0xffffffffu, is && pos == 31);
        cnt = min(32, cnt + __popc(m));
        scan += full ? __ffs(full) : 32;   // go on behind the 32nd
      }
      __syncwarp();
      win = cnt < 32 ? (1u << cnt) - 1u : 0xffffffffu;
      kid = ctok = -1;
      cu = 0.f;
      if (lane < cnt) {
        kid = rs.kid[lane];
        ctok = tok[kid];
        cu = uni[kid];
      }
      has = ctok >= 0 && ctok < V;
      cxb = load_bits<LB>(row, has ? ctok : 0);   // (not waited for here: see child_values)
      if (QT) cqb = load_bits<QT == 1>(qrow, has ? ctok : 0);
      if (!QT && cnt > 0) {
        // q one-hot: an earlier sibling's equal token was rejected before
        // this one, so nothing of it is left
        bool dup = (__match_any_sync(0xffffffffu, ctok) & ((1u << lane) - 1u)) != 0;
        const int n0 = rs.n_child, at = n0 + lane;
        for (int j = 0; j < min(n0, kChildList); ++j) dup |= rs.child_tok[j] == ctok;
        if (n0 > kChildList)
          for (int j = mine + 1; j < kid; ++j) dup |= par[j] == mine && tok[j] == ctok;
        if (dup) has = false;
        if (lane < cnt) {
          if (at < kChildList) rs.child_tok[at] = ctok;
          atomicOr(&rs.marks[(ctok >> 8) & (kMarks - 1)], 1u << ((ctok >> 3) & 31));
        }
        __syncwarp();
        if (lane == 0) rs.n_child = n0 + cnt;
      }
      __syncwarp();
    };
    auto child_values = [&]() {
      cx = has ? bits_value<LB>(cxb) : -INFINITY;
      cq = QT && has ? bits_value<QT == 1>(cqb) : 0.f;
    };
    if (mine >= 0) {
      rs.marks[lane] = 0;
      if (lane == 0) rs.n_child = 0;
      __syncwarp();
      load_children();
    }

    // ---- each row's maximum and sum over the slice (T = 0: its first argmax).
    // The warps are shared out among the rows, so that every row's loads are in
    // flight at once and each warp reduces once.
    const int r_mine = warp / row_warps, w_mine = warp - r_mine * row_warps;
    if (r_mine < n) {
      int i_row = v;
      for (int j = 0; j < r_mine; ++j) i_row = sh.first[i_row];
      const void* x_row = row_of(i_row);
      const int t0 = w_mine * 32 + lane, step = row_warps * 32;
      // 16-byte loads over the aligned middle of the slice, single elements at the ends
      constexpr int EPV = 16 / LES;
      const uintptr_t a0 = reinterpret_cast<uintptr_t>(x_row) + (uintptr_t)c0 * LES;
      const int head = min(c1 - c0, (int)(((16 - (a0 & 15)) & 15) / LES));
      const int nvec = (c1 - c0 - head) / EPV, v0 = c0 + head, v1 = v0 + nvec * EPV;
      const uint4* vp = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x_row) + (size_t)v0 * LES);
      const int n_end = head + (c1 - v1);
      auto end_at = [&](int i) { return i < head ? c0 + i : v1 + (i - head); };
      // Running maximum and sum, eight vectors at a time (T = 0: the maximum
      // and the eight vectors it was first met in).  Weights of 1, the maximum's
      // own, are counted apart: a small weight added to them would lose its
      // digits, which are all there is of log p where the model is sure (log p
      // near -1e-6 was off by a tenth of itself, now by 3e-7; it costs 2.0 of
      // 39.9 us of 64 chains, 0.3 of 7.7 us of a chain of 4 drafts).
      float m = -INFINITY, s = 0.f, ones = 0.f;
      int i_max = 0;
      constexpr int NV = kVectors;
      for (int i0 = t0; i0 < nvec; i0 += NV * step) {
        uint4 w[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int i = i0 + j * step;
          const uint32_t ninf = LB ? 0xff80ff80u : 0xff800000u;
          w[j] = i < nvec ? __ldg(vp + i) : make_uint4(ninf, ninf, ninf, ninf);
        }
        float mx;
        if constexpr (LB) {   // the maximum in bf16 pairs
          uint32_t v2 = w[0].x;
#pragma unroll
          for (int j = 0; j < NV; ++j)
            v2 = max_bf16x2(max_bf16x2(v2, w[j].x), max_bf16x2(w[j].y, max_bf16x2(w[j].z, w[j].w)));
          mx = fmaxf(__uint_as_float(v2 << 16), __uint_as_float(v2 & 0xffff0000u));
        } else {
          mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < NV; ++j)
            mx = fmaxf(fmaxf(mx, fmaxf(__uint_as_float(w[j].x), __uint_as_float(w[j].y))),
                       fmaxf(__uint_as_float(w[j].z), __uint_as_float(w[j].w)));
        }
        if (mx > m) {
          s = m == -INFINITY ? 0.f : (ones + s) * weight(m, mx);
          ones = 0.f;
          m = mx;
          i_max = i0;
        }
        if (greedy || m == -INFINITY) continue;
        float s0 = 0.f, s1 = 0.f;
        uint32_t at_max = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (i0 + j * step >= nvec) break;
          const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
          for (int q = 0; q < (LB ? 4 : 2); ++q) {
            float w0, w1;
            if (LB) twice2(__uint_as_float(u[q] << 16), __uint_as_float(u[q] & 0xffff0000u), m, &w0, &w1);
            else twice2(__uint_as_float(u[2 * q]), __uint_as_float(u[2 * q + 1]), m, &w0, &w1);
            // of numbers up to 2, 2 alone has bit 30, and no other bit
            at_max += __float_as_uint(w0) >> 30;
            at_max += __float_as_uint(w1) >> 30;
            s0 += __uint_as_float(__float_as_uint(w0) & 0xbfffffffu);
            s1 += __uint_as_float(__float_as_uint(w1) & 0xbfffffffu);
          }
        }
        ones += (float)at_max;
        s += 0.5f * (s0 + s1);
      }
      if (greedy) {
        // the lanes that hold the warp's maximum look it up where they met it
        // (10.3 us of a 4-row pass over 128,256 tokens came down to 3.9
        // against a key of value and index kept for every entry)
        uint64_t best = 0;
        for (int i = t0; i < n_end; i += step) {
          const float x = load_elem<LB>(x_row, end_at(i));
          if (x >= -INFINITY) best = max64(best, logit_key(x + 0.f, (uint32_t)end_at(i)));
        }
        const float wm = warp_max(m);
        if (m > -INFINITY && m == wm) {
          int at_max = -1;
#pragma unroll
          for (int j = NV - 1; j >= 0; --j) {
            const int i = i_max + j * step;
            if (i >= nvec) continue;
            const uint4 w = __ldg(vp + i);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = EPV - 1; q >= 0; --q) {
              const float x = !LB     ? __uint_as_float(u[q % 4])
                              : q & 1 ? __uint_as_float(u[q / 2] & 0xffff0000u)
                                      : __uint_as_float(u[q / 2] << 16);
              if (x == m) at_max = v0 + i * EPV + q;
            }
          }
          if (at_max >= 0) best = max64(best, logit_key(m + 0.f, (uint32_t)at_max));
        }
        best = warp_max64(best);
        if (lane == 0) sh.part[r_mine][w_mine] = best;
      } else {
        for (int i = t0; i < n_end; i += step) {
          const float x = load_elem<LB>(x_row, end_at(i));
          if (x > m) {
            s = m == -INFINITY ? 0.f : (ones + s) * weight(m, x);
            ones = 0.f;
            m = x;
          }
          if (m > -INFINITY) {
            const float w = weight(x, m);
            if (w >= 1.f) ones += 1.f;
            else s += w;
          }
        }
        // thread -> warp -> CTA -> cluster: each part against its own maximum,
        // joined against the common one, whose own weight -- in the first part
        // that has it -- is left out
        const float wm = warp_max(m);
        const uint32_t tops = __ballot_sync(0xffffffffu, m == wm);
        const float tail = warp_add(m == -INFINITY             ? 0.f
                                    : lane == __ffs(tops) - 1 ? (ones - 1.f) + s
                                                               : (ones + s) * weight(m, wm));
        if (lane == 0) sh.part[r_mine][w_mine] = (uint64_t)__float_as_uint(tail) << 32 | __float_as_uint(wm);
      }
    }
    __syncthreads();
    if (!noise_first && v == 0 && tid == kThreads - 1) prefetch_noise();
    // the lanes' maxima and tails, joined in every lane
    auto join = [&](float pm, float pt, float* mo) -> float {
      const float jm = warp_max(pm);
      const uint32_t tops = __ballot_sync(0xffffffffu, pm == jm);
      *mo = jm;
      return warp_add(pm == -INFINITY ? 0.f : lane == __ffs(tops) - 1 ? pt : (1.f + pt) * weight(pm, jm));
    };
    float m = -INFINITY, tail = 0.f;
    int am = -1;
    uint64_t mine_a = 0;
    if (mine >= 0) {
      const bool in = lane < row_warps;
      if (greedy) {
        mine_a = warp_max64(in ? sh.part[warp][lane] : 0);
      } else {
        const uint64_t part = in ? sh.part[warp][lane] : (uint64_t)0xff800000u;   // (no part: -inf)
        mine_a = __float_as_uint(join(__uint_as_float((uint32_t)part), __uint_as_float((uint32_t)(part >> 32)), &m));
      }
    }
    if (!exchange(kStats | ((uint32_t)v & 0xffffffu) << 4 | (uint32_t)n, mine_a, __float_as_uint(m))) {
      give_up(true);
      return;
    }

    // ---- each row's warp tries its children in index order.  The row's warp
    // of every CTA comes to the same decisions: the same numbers, read and
    // joined in the same order.
    bool dead = false, pending = false;   // pending (QT): a child was rejected and its B not yet summed
    float cw = 0.f, sf = 0.f;             // weight of the child's token: sum times its probability
    double A = 0.0, B = 1.0;
    float Af = 0.f, Bf = 1.f;             // (their fp32 values: conversions take the fp64 pipe)
    auto child_w = [&]() { return greedy ? (ctok == am && cx > -INFINITY ? 1.f : 0.f) : weight(cx, m); };
    // u q B < p - A q, times the sum, in fp64: where fp32 is too close to tell.
    // (The token's weight anew; sum, A and B as they are.)
    auto sum64 = [&]() { return 1.0 + (double)tail; };
    auto precisely = [&](float x, float q, float u, double b) {
      const double w = exp(((double)x - (double)m) / (double)sh.temp);
      const double sum = sum64();
      return (double)u * b * (double)q * sum < w - (QT ? A * (double)q * sum : 0.0);
    };
    auto decide = [&]() {
      int next = -1, more = 0;
      float nx = 0.f;
      while (!dead) {
        if (win == 0) {
          load_children();
          if (win == 0) break;
          child_values();
          cw = child_w();
        }
        if (pending) {
          more = 1;
          break;
        }
        if constexpr (QT == 0) {
          // every lane its own child: B is what the children before it leave
          float before = cw;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += y;
          }
          const float all = __shfl_sync(0xffffffffu, before, 31);
          before -= cw;
          // (rounding may put the weights before this child above all there is:
          // nothing is left then, and not less)
          const float lhs = greedy ? 0.f : cu * fmaxf(Bf * sf - before, 0.f);
          const bool near = !greedy && fabsf(cw - lhs) <= 4e-6f * (cw + sf) && cx > -INFINITY;
          const bool ok = cw > 0.f && lhs < cw;   // a weight of 0 is never accepted
          uint32_t may = __ballot_sync(0xffffffffu, (ok || near) && ((win >> lane) & 1u));
          const uint32_t close = __ballot_sync(0xffffffffu, near);
          while (may) {
            const int j = __ffs(may) - 1;
            const float xj = __shfl_sync(0xffffffffu, cx, j), uj = __shfl_sync(0xffffffffu, cu, j);
            bool yes = true;
            if ((close >> j) & 1u) {
              double b = B;
              for (int i = 0; i < j; ++i) b -= (double)__shfl_sync(0xffffffffu, cw, i) / sum64();
              yes = precisely(xj, 1.f, uj, fmax(b, 0.0));
            }
            if (yes) {
              next = __shfl_sync(0xffffffffu, kid, j);
              nx = xj;
              break;
            }
            may &= may - 1;
          }
          win = 0;
          if (next >= 0) break;
          if (!greedy && scan < L) {
            B = fmax(B - (double)(all / sf), 0.0);
            Bf = (float)B;
          }
        } else {
          const int j = __ffs(win) - 1;
          win &= win - 1;
          const float wj = __shfl_sync(0xffffffffu, cw, j), xj = __shfl_sync(0xffffffffu, cx, j);
          const float qj = __shfl_sync(0xffffffffu, cq, j), uj = __shfl_sync(0xffffffffu, cu, j);
          bool ok;
          if (greedy) {
            ok = wj > 0.f;
          } else {
            const float lhs = uj * Bf * qj * sf, aq = Af * qj * sf;
            ok = lhs < wj - aq;
            if (fabsf(wj - aq - lhs) <= 4e-6f * (wj + aq + lhs) && xj > -INFINITY) ok = precisely(xj, qj, uj, B);
          }
          if (ok) {
            next = __shfl_sync(0xffffffffu, kid, j);
            nx = xj;
            break;
          }
          if (greedy) continue;
          A += B;
          Af = (float)A;
          pending = true;
        }
      }
      pending = false;
      if (lane == 0) {
        sh.next[warp] = next;
        sh.more[warp] = more;
        rs.as = Af * sf;
        rs.x = nx;
      }
    };
    if (mine >= 0) {
      if (greedy) {
        const uint64_t key = warp_max64(lane < C ? sh.ex[phase][warp][lane].a : 0);
        dead = key <= logit_key(-INFINITY, 0);
        am = dead ? 0 : (int)(0xffffffffu - (uint32_t)key);
      } else {
        const Message in = sh.ex[phase][warp][lane < C ? lane : 0];
        tail = join(lane < C ? __uint_as_float((uint32_t)in.b) : -INFINITY, __uint_as_float((uint32_t)in.a), &m);
        dead = m == -INFINITY;
        sf = 1.f + tail;
      }
      child_values();
      if (!dead) cw = child_w();
      if (lane == 0) {
        sh.node[warp] = mine;
        rs.m = m;
        rs.tail = tail;
        rs.sf = sf;
        rs.am = am;
        rs.dead = dead;
      }
      decide();
    }
    __syncthreads();

    // ---- follow the decisions along the rows of the pass: a row whose accepted
    // child is the next row's node leads on to it, and all such are taken at once
    auto emit = [&](int r0, int count) {   // rows r0 .. accept their children: nodes k + 1 ..
      if (rank == 0 && tid < count) {
        const RowState& e = sh.row[r0 + tid];
        const int i = k + tid;
        p.path[o + i + 1] = sh.next[r0 + tid];
        if (i < kNodes) {
          sh.lx[i] = e.x;
          sh.lm[i] = e.m;
          sh.lt[i] = e.tail;
        } else if (p.logprobs) {
          p.logprobs[o + i] = greedy ? 0.f : log_prob(e.x, e.m, c_hi, c_lo, e.tail);
        }
      }
      k += count;
    };
    int r = 0, at, to;
    for (;;) {
      const int slot = lane & (kRows - 1);
      const int r_node = sh.node[slot], r_next = sh.next[slot], r_more = QT ? sh.more[slot] : 0;
      const int after = __shfl_down_sync(0xffffffffu, r_node, 1);
      const uint32_t leads = __ballot_sync(0xffffffffu, lane + 1 < n && !r_more && r_next == after);
      const int run = __ffs(~(leads >> r)) - 1;
      if (run) emit(r, run);
      r += run;
      at = __shfl_sync(0xffffffffu, r_node, r);
      to = __shfl_sync(0xffffffffu, r_next, r);
      if (!QT || !__shfl_sync(0xffffffffu, r_more, r)) break;
      // B = sum_x (p(x) - A q(x))+ of this row, in units of 2^-50
      const void *x_row = row_of(at), *q_row = qrow_of(at);
      const float rm = sh.row[r].m, inv = 1.f / sh.row[r].sf, as = sh.row[r].as;
      float t = 0.f;
      if (p.vec) {
#pragma unroll 2
        for (int i = c0 + 8 * tid; i < c1; i += 8 * kThreads) {
          float x[8], q[8];
          load8<LB>(x_row, i, x);
          load8<QT == 1>(q_row, i, q);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            float w0, w1;
            weight2(x[e], x[e + 1], rm, &w0, &w1);
            t += fmaxf(fmaf(-as, q[e], w0), 0.f) + fmaxf(fmaf(-as, q[e + 1], w1), 0.f);
          }
        }
      } else {
#pragma unroll 4
        for (int i = c0 + tid; i < c1; i += kThreads)
          t += fmaxf(fmaf(-as, load_elem<QT == 1>(q_row, i), weight(load_elem<LB>(x_row, i), rm)), 0.f);
      }
      uint64_t f = warp_add64(__float2ull_rn(t * inv * 0x1p50f));
      if (lane == 0) sh.part[0][warp] = f;
      __syncthreads();
      if (warp == 0) f = warp_add64(lane < kWarps ? sh.part[0][lane] : 0);
      if (!exchange(kResidual | ((uint32_t)at & 0xffffffu) << 4 | (uint32_t)r, f, 0)) {
        give_up(true);
        return;
      }
      if (warp == r) {
        f = warp_add64(lane < C ? sh.ex[phase][0][lane].a : 0);
        B = (double)f * 0x1p-50;
        Bf = (float)B;
        decide();
      }
      __syncthreads();
    }
    if (to >= 0) {
      emit(r, 1);
      v = to;
      continue;
    }

    // ---- no child accepted: the bonus token
    const RowState& last = sh.row[r];
    const void *x_row = row_of(at), *q_row = qrow_of(at);
    int bonus = -1;
    // its children's distribution counts where one of them was rejected
    const bool use_q = QT && last.as > 0.f;
    const int groups = (c1 - c0 + 8 * kThreads - 1) / (8 * kThreads);
    const bool prune = use_q && p.vec && groups >= 4 && groups <= kGroups;
    // all of its slice asked for at once: the loads below run behind it
    if (use_q && !prune && tid == 0 && !last.dead && !greedy)
      prefetch_l2(static_cast<const uint8_t*>(q_row) + (size_t)c0 * QES, (int64_t)(c1 - c0) * QES);
    if (last.dead || greedy) {
      if (!exchange(kEnd | ((uint32_t)at & 0xffffffu) << 4, 0, 0)) {
        give_up(true);
        return;
      }
      if (!last.dead) bonus = last.am;
    } else {
      const float rm = last.m, as = last.as;
      const int n_child = QT ? 0 : last.n_child;
      bool plain = QT ? !use_q : n_child == 0;   // draw from p_v itself: nothing rejected, or nothing left of the residual
      for (;;) {
        // the best of this thread's entries so far: w / e of the largest
        float best_w = 0.f, best_e = 1.f;
        int best_i = -1;
        // which of the entries i .. i + 7 (i a multiple of 8) are rejected tokens
        auto rejected8 = [&](int i) -> uint32_t {
          if (QT || plain || !((last.marks[(i >> 8) & (kMarks - 1)] >> ((i >> 3) & 31)) & 1u)) return 0u;
          uint32_t hit = 0;
          for (int j = 0; j < min(n_child, kChildList); ++j) {
            const uint32_t d = (uint32_t)(last.child_tok[j] - i);
            if (d < 8) hit |= 1u << d;
          }
          if (n_child > kChildList)
            for (int j = at + 1; j < L; ++j)
              if (par[j] == at && (uint32_t)(tok[j] - i) < 8u) hit |= 1u << (tok[j] - i);
          return hit;
        };
        // w / e compared by cross products (each within 2^-24, as the weights
        // are): no division or reciprocal an entry.  A thread's entries come in
        // rising order: an equal one does not replace.
        auto take = [&](float w, float q, float e, int i) {
          if (QT) w = fmaf(-as, q, w);
          const bool better = w * best_e > best_w * e;
          best_w = better ? w : best_w;
          best_e = better ? e : best_e;
          best_i = better ? i : best_i;
        };
        // every entry from i = c0 + 8 tid on
        auto race = [&](auto with_q) {
          constexpr bool Q = QT && decltype(with_q)::value;
          if (p.vec) {
#pragma unroll 2
            for (int i = c0 + 8 * tid; i < c1; i += 8 * kThreads) {
              float x[8], q[8], e[8];
              load8<LB>(x_row, i, x);
              if (Q) load8<QT == 1>(q_row, i, q);
              load8<false>(noise, i, e);
              const uint32_t hit = rejected8(i);
              if (!QT && hit) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = (hit >> j) & 1u ? -INFINITY : x[j];
              }
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                float w0, w1;
                weight2(x[j], x[j + 1], rm, &w0, &w1);
                take(w0, Q ? q[j] : 0.f, e[j], i + j);
                take(w1, Q ? q[j + 1] : 0.f, e[j + 1], i + j + 1);
              }
            }
          } else {
#pragma unroll 4
            for (int i = c0 + tid; i < c1; i += kThreads) {
              const float x = (rejected8(i & ~7) >> (i & 7)) & 1u ? -INFINITY : load_elem<LB>(x_row, i);
              take(weight(x, rm), Q ? load_elem<QT == 1>(q_row, i) : 0.f, __ldg(noise + i), i);
            }
          }
        };
        if constexpr (QT != 0) {
          if (plain) {
            race(std::false_type());
          } else if (prune) {
            // p / e bounds an entry's key from above, and only a handful in a
            // vocabulary lie above the best key of all: bounds of groups of
            // eight first, then a key to beat from the best group of each
            // warp, then the groups whose bounds reach it.  q is read for
            // those alone (64 chains: 25 MB less, 37.8 us, 39.3 with all of
            // q); a slice of less than four groups a thread is over sooner in
            // one go.
            auto exact = [&](int i) {
              float x[8], q[8], e[8];
              load8<LB>(x_row, i, x);
              load8<QT == 1>(q_row, i, q);
              load8<false>(noise, i, e);
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                float w0, w1;
                weight2(x[j], x[j + 1], rm, &w0, &w1);
                take(w0, q[j], e[j], i + j);
                take(w1, q[j + 1], e[j + 1], i + j + 1);
              }
            };
            const int i_first = c0 + 8 * tid;
            float top = 0.f;
            int top_g = 0;
#pragma unroll 4
            for (int g = 0; g < groups; ++g) {
              const int i = i_first + g * 8 * kThreads;
              float x[8], e[8], gw = 0.f, ge = 1.f;
              load8<LB>(x_row, min(i, c1 - 8), x);
              load8<false>(noise, min(i, c1 - 8), e);
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                float w[2];
                weight2(x[j], x[j + 1], rm, &w[0], &w[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const bool better = w[h] * ge > gw * e[j + h];
                  gw = better ? w[h] : gw;
                  ge = better ? e[j + h] : ge;
                }
              }
              // (cross products tell within 2^-23, the quotient within 2^-22)
              float bound = ge >= 1e-37f ? __fdividef(gw, fminf(ge, 1e37f)) * 1.000001f : gw > 0.f ? INFINITY : 0.f;
              if (i >= c1) bound = 0.f;
              bounds[g][tid] = bound;
              if (bound > top) {
                top = bound;
                top_g = g;
              }
            }
            const float warp_top = warp_max(top);
            const uint32_t owners = __ballot_sync(0xffffffffu, top == warp_top && top > 0.f);
            if (owners && lane == __ffs(owners) - 1) exact(i_first + top_g * 8 * kThreads);
            const float beat_warp = warp_max(best_i >= 0 ? __fdiv_rn(best_w, best_e) : 0.f);
            if (lane == 0) sh.beat[warp] = beat_warp;
            __syncthreads();
            const float beat = warp_max(lane < kWarps ? sh.beat[lane] : 0.f);
            best_w = 0.f;
            best_e = 1.f;
            best_i = -1;
            for (int g = 0; g < groups; ++g)
              if (bounds[g][tid] > 0.f && bounds[g][tid] >= beat) exact(i_first + g * 8 * kThreads);
          } else {
            race(std::true_type());
          }
        } else {
          race(std::false_type());
        }
        uint64_t key = warp_max64(best_i >= 0 ? race_key(__fdiv_rn(best_w, best_e), (uint32_t)best_i) : 0);
        if (lane == 0) sh.part[0][warp] = key;
        __syncthreads();
        if (warp == 0) key = warp_max64(lane < kWarps ? sh.part[0][lane] : 0);
        if (!exchange(kBonus | ((uint32_t)at & 0xffffffu) << 4 | (plain ? 1u : 0u), key, 0)) {
          give_up(true);
          return;
        }
        key = warp_max64(lane < C ? sh.ex[phase][0][lane].a : 0);
        if (key != 0) {
          bonus = (int)(0xffffffffu - (uint32_t)key);
          break;
        }
        if (plain) break;
        plain = true;
      }
    }
    if (rank == 0) {
      if (tid == 0) {
        p.accept_len[b] = k + 1;
        p.bonus[b] = bonus;
      }
      if (p.logprobs && warp == 0) {
        // every emitted token's, a lane each
        __syncwarp();
        for (int i = lane; i <= k; i += 32) {
          if (i < k && i >= kNodes) continue;   // (written on the way)
          const bool end = i == k;
          const float x = !end ? sh.lx[i] : bonus >= 0 ? load_elem<LB>(x_row, bonus) : 0.f;
          const float lp = greedy ? 0.f : log_prob(x, end ? last.m : sh.lm[i], c_hi, c_lo, end ? last.tail : sh.lt[i]);
          p.logprobs[o + i] = end && bonus < 0 ? 0.f : lp;
        }
      }
      for (int i = k + 1 + tid; i < L; i += kThreads) {
        p.path[o + i] = -1;
        if (p.logprobs) p.logprobs[o + i] = 0.f;
      }
    }
    return;
  }
}

}  // namespace

cudaError_t launch_accept_sample(const SampleParams& p, bool logits_bf16, int draft, cudaStream_t stream) {
  const void* kern;
  if (logits_bf16)
    kern = draft == 0   ? reinterpret_cast<const void*>(accept_sample_kernel<true, 0>)
           : draft == 1 ? reinterpret_cast<const void*>(accept_sample_kernel<true, 1>)
                        : reinterpret_cast<const void*>(accept_sample_kernel<true, 2>);
  else
    kern = draft == 0   ? reinterpret_cast<const void*>(accept_sample_kernel<false, 0>)
           : draft == 1 ? reinterpret_cast<const void*>(accept_sample_kernel<false, 1>)
                        : reinterpret_cast<const void*>(accept_sample_kernel<false, 2>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.batch * (unsigned)p.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {const_cast<SampleParams*>(&p)};
  return cudaLaunchKernelExC(&cfg, kern, args);
}

}  // namespace va
