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
// the vocabulary, so a step is one pass over the node's row and one exchange
// through distributed shared memory.  Rows of nodes that are not accepted are
// never read: a 64-node tree whose path is two nodes long reads two rows.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/verify_attn.h"
#include "va_device.cuh"
#include "va_kernels.h"

namespace va {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kChildList = 64;  // children's tokens kept in shared memory (further ones are searched)

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
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// Store 8 bytes at shared address `addr` (of this CTA) in the shared memory
// of CTA `cta` of the cluster.
__device__ __forceinline__ void cluster_store(uint32_t addr, uint32_t cta, uint64_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(cta));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

template <bool BF16>
__device__ __forceinline__ float load_elem(const void* row, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(row) + i) << 16);
  else
    return __ldg(static_cast<const float*>(row) + i);
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

struct Shared {
  uint64_t warp_a[kWarps], warp_b[kWarps];
  uint64_t ex_a[2][kMaxCluster], ex_b[2][kMaxCluster];  // the cluster's exchange, two phases
  int child_tok[kChildList];
  int n_child;
  int next, more;    // the accepted child (or -1); a residual's sum is wanted
  double a;          // A after the children tried so far
};

// LB: logits bf16 (else fp32).  QT: draft distributions: 0 none, 1 bf16, 2 fp32.
template <bool LB, int QT>
__global__ void __launch_bounds__(kThreads, 2) accept_sample_kernel(const SampleParams p) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = p.cluster;
  const int rank = (int)cluster_rank(), b = blockIdx.x / C;
  grid_dependency_wait();
  grid_dependents_launch();
  const int o = p.qo_indptr[b];
  const int L = p.qo_indptr[b + 1] - o;
  const float temp = p.temperature ? p.temperature[b] : 1.f;
  const bool table_ok = o >= 0 && L >= 0 && (int64_t)o + L <= p.total;
  int bad = 0;
  if (table_ok)
    for (int i = tid; i < L; i += kThreads) {
      const int par = p.parents[o + i];
      bad |= i == 0 ? par >= 0 : (par < 0 || par >= i);
    }
  bad = __syncthreads_or(bad) || !table_ok || !(temp >= 0.f && temp < INFINITY);
  if (bad || L == 0) {  // the same in every CTA of the cluster
    if (rank == 0) {
      if (tid == 0) {
        p.accept_len[b] = 0;
        p.bonus[b] = -1;
        if (bad && p.status) atomicOr(p.status, VA_DEV_BAD_TABLE);
      }
      if (table_ok)
        for (int i = tid; i < L; i += kThreads) {
          p.path[o + i] = -1;
          if (p.logprobs) p.logprobs[o + i] = 0.f;
        }
    }
    return;
  }

  cluster_sync();  // every CTA of the cluster runs before its shared memory is written

  const int V = p.vocab;
  const int c0 = (int)min((int64_t)V, (int64_t)rank * p.slice), c1 = (int)min((int64_t)V, (int64_t)c0 + p.slice);
  const float* noise = p.noise + (size_t)b * p.noise_stride;
  constexpr int LES = LB ? 2 : 4, QES = QT == 1 ? 2 : 4;
  const bool greedy = temp == 0.f;
  // log2(e) / T as a float pair: a rounded factor alone would tilt the whole
  // distribution by |logit difference| * 2^-25
  // (both parts > 0, so that -inf logits stay -inf)
  const double cd = greedy ? 1.0 : fmin(1.4426950408889634 / (double)temp, 3e38);
  const float c_hi = __double2float_rd(cd), c_lo = fmaxf((float)(cd - (double)c_hi), 1.1754944e-38f);
  const uint64_t ch2 = f32x2(c_hi, c_hi), cl2 = f32x2(c_lo, c_lo);
  // 2^((x - m) log2(e) / T) of a pair: the difference first (exact for bf16
  // logits of like size), then the two-term product
  auto weight2 = [&](float x0, float x1, float m, float* w0, float* w1) {
    const uint64_t d = add_f32x2(f32x2(x0, x1), f32x2(-m, -m));
    const uint64_t y = fma_f32x2(d, ch2, fma_f32x2(d, cl2, 0ull));
    *w0 = ex2(f32x2_lo(y));
    *w1 = ex2(f32x2_hi(y));
  };
  auto weight = [&](float x, float m) {
    const float d = x - m;
    return ex2(fmaf(d, c_hi, d * c_lo));
  };

  // Exchange one pair of words with the cluster: every CTA gets all of them
  // in sh.ex_a / ex_b [phase][0 .. C).  The two phases alternate, so a CTA that
  // runs ahead never writes what a slower one still reads.
  int phase = 0;
  auto exchange = [&](uint64_t a, uint64_t v) {  // called by every thread, values of thread 0
    phase ^= 1;
    if (tid == 0)
      for (int k = 0; k < C; ++k) {
        cluster_store(smem_u32(&sh.ex_a[phase][rank]), k, a);
        cluster_store(smem_u32(&sh.ex_b[phase][rank]), k, v);
      }
    __syncwarp();
    cluster_sync();
  };
  // Cluster-wide maximum of a key / sum of a double; the result in every thread.
  auto cluster_max = [&](uint64_t key) -> uint64_t {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) key = max64(key, __shfl_xor_sync(0xffffffffu, key, s));
    if (lane == 0) sh.warp_a[warp] = key;
    __syncthreads();
    if (tid == 0)
      for (int w = 1; w < kWarps; ++w) key = max64(key, sh.warp_a[w]);
    exchange(key, 0);
    key = sh.ex_a[phase][0];
    for (int k = 1; k < C; ++k) key = max64(key, sh.ex_a[phase][k]);
    return key;
  };
  auto cluster_sum = [&](float v) -> double {
    double s = v;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) sh.warp_a[warp] = __double_as_longlong(s);
    __syncthreads();
    if (tid == 0)
      for (int w = 1; w < kWarps; ++w) s += __longlong_as_double(sh.warp_a[w]);
    exchange(__double_as_longlong(s), 0);
    s = __longlong_as_double(sh.ex_a[phase][0]);
    for (int k = 1; k < C; ++k) s += __longlong_as_double(sh.ex_a[phase][k]);
    return s;
  };

  int v = 0, k = 0;
  for (;;) {
    const void* row = static_cast<const uint8_t*>(p.logits) + (size_t)(o + v) * p.row_stride * LES;
    const void* qrow = QT ? static_cast<const uint8_t*>(p.draft) + (size_t)(o + v) * p.draft_stride * QES : nullptr;
    if (tid == 0 && rank == 0) p.path[o + k] = v;

    // ---- the row's maximum and sum (T = 0: its first argmax)
    float m = -INFINITY;
    double sum = 0.0;
    int am = -1;
    {
      // 16-byte loads over the aligned middle of the slice, single elements at the ends
      constexpr int EPV = 16 / LES;
      const uintptr_t a0 = reinterpret_cast<uintptr_t>(row) + (uintptr_t)c0 * LES;
      const int head = min(c1 - c0, (int)(((16 - (a0 & 15)) & 15) / LES));
      const int nvec = (c1 - c0 - head) / EPV, v0 = c0 + head, v1 = v0 + nvec * EPV;
      const uint4* vp = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (size_t)v0 * LES);
      const int n_end = head + (c1 - v1);
      auto end_at = [&](int i) { return i < head ? c0 + i : v1 + (i - head); };
      if (greedy) {
        uint64_t best = 0;
        for (int i = tid; i < n_end; i += kThreads)
          best = max64(best, logit_key(load_elem<LB>(row, end_at(i)), (uint32_t)end_at(i)));
#pragma unroll 4
        for (int i = tid; i < nvec; i += kThreads) {
          const uint4 w = __ldg(vp + i);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
          const uint32_t e = (uint32_t)(v0 + i * EPV);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (LB) {
              best = max64(best, logit_key(__uint_as_float(u[q] << 16), e + 2 * q));
              best = max64(best, logit_key(__uint_as_float(u[q] & 0xffff0000u), e + 2 * q + 1));
            } else {
              best = max64(best, logit_key(__uint_as_float(u[q]), e + q));
            }
          }
        }
        am = (int)(0xffffffffu - (uint32_t)cluster_max(best));
      } else {
        // running maximum and sum, four vectors at a time
        float s = 0.f;
        constexpr int NV = 4;
        for (int i0 = tid; i0 < nvec; i0 += NV * kThreads) {
          uint4 w[NV];
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int i = i0 + j * kThreads;
            const uint32_t ninf = LB ? 0xff80ff80u : 0xff800000u;
            w[j] = i < nvec ? __ldg(vp + i) : make_uint4(ninf, ninf, ninf, ninf);
          }
          float x[NV][EPV];
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (LB) {
                x[j][2 * q] = __uint_as_float(u[q] << 16);
                x[j][2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
                mx = fmaxf(mx, fmaxf(x[j][2 * q], x[j][2 * q + 1]));
              } else {
                x[j][q] = __uint_as_float(u[q]);
                mx = fmaxf(mx, x[j][q]);
              }
            }
          }
          if (mx > m) {
            s = m == -INFINITY ? 0.f : s * weight(m, mx);
            m = mx;
          }
          if (m == -INFINITY) continue;
          float t0 = 0.f, t1 = 0.f;
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int q = 0; q < EPV; q += 2) {
              float w0, w1;
              weight2(x[j][q], x[j][q + 1], m, &w0, &w1);
              t0 += w0;
              t1 += w1;
            }
          s += t0 + t1;
        }
        for (int i = tid; i < n_end; i += kThreads) {
          const float x = load_elem<LB>(row, end_at(i));
          if (x > m) {
            s = m == -INFINITY ? 0.f : s * weight(m, x);
            m = x;
          }
          if (m > -INFINITY) s += weight(x, m);
        }
        // thread -> warp -> CTA -> cluster: the maximum first, then the sums
        // against it in double
        float wm = m;
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, j));
        double ws = m == -INFINITY ? 0.0 : (double)(s * weight(m, wm));
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, j);
        if (lane == 0) {
          sh.warp_a[warp] = __float_as_uint(wm);
          sh.warp_b[warp] = __double_as_longlong(ws);
        }
        __syncthreads();
        // the sums of parts against their common maximum, in part order
        auto join = [&](const uint64_t* pm, const uint64_t* ps, int n, float* mo) -> double {
          float mm = -INFINITY;
          for (int j = 0; j < n; ++j) mm = fmaxf(mm, __uint_as_float((uint32_t)pm[j]));
          double t = 0.0;
          for (int j = 0; j < n; ++j) {
            const float pj = __uint_as_float((uint32_t)pm[j]);
            if (pj > -INFINITY) t += __longlong_as_double(ps[j]) * (double)weight(pj, mm);
          }
          *mo = mm;
          return t;
        };
        float cm = -INFINITY;
        double cs = 0.0;
        if (tid == 0) cs = join(sh.warp_a, sh.warp_b, kWarps, &cm);
        exchange(__float_as_uint(cm), __double_as_longlong(cs));
        sum = join(sh.ex_a[phase], sh.ex_b[phase], C, &m);
      }
    }
    const bool dead = greedy ? !(load_elem<LB>(row, am) > -INFINITY) : !(sum > 0.0);

    // ---- the children in index order.  Warp 0 of every CTA comes to the
    // same decisions: the same numbers, read and reduced in the same order.
    double A = 0.0, B = 1.0;
    int base = v + 1 - 32;
    uint32_t win = 0;       // children in the window base .. base + 31 not yet tried
    bool pending = false;   // QT: a child was rejected and its B not yet summed
    double cp = 0.0, cq = 0.0, cu = 0.0;
    int ctok = -1;
    if (tid == 0) sh.n_child = 0;
    // the next window that holds a child of v: each lane its child's token,
    // number and probabilities
    auto load_window = [&]() -> bool {
      for (base += 32; base < L; base += 32) {
        const int i = base + lane;
        const bool is = i < L && p.parents[o + i] == v;
        win = __ballot_sync(0xffffffffu, is);
        if (win) {
          cp = cq = cu = 0.0;
          ctok = -1;
          if (is) {
            ctok = p.tokens[o + i];
            cu = p.uniforms[o + i];
            if (ctok >= 0 && ctok < V) {
              if (greedy) cp = ctok == am ? 1.0 : 0.0;
              else cp = exp(((double)load_elem<LB>(row, ctok) - (double)m) / (double)temp) / sum;
              if (QT) cq = load_elem<QT == 1>(qrow, ctok);
            }
          }
          if (!QT) {
            // q one-hot: an earlier sibling's equal token was rejected before
            // this one, so nothing of it is left
            bool dup = false;
            for (int j = 0; j < 32; ++j) {
              const int tj = __shfl_sync(0xffffffffu, ctok, j);
              dup |= j < lane && ((win >> j) & 1u) && tj == ctok;
            }
            for (int j = v + 1; j < base; ++j) dup |= p.parents[o + j] == v && p.tokens[o + j] == ctok;
            if (dup) cp = 0.0;
            const int n0 = sh.n_child, at = n0 + __popc(win & ((1u << lane) - 1u));
            if (is && at < kChildList) sh.child_tok[at] = ctok;
            __syncwarp();
            if (lane == 0) sh.n_child = n0 + __popc(win);
            __syncwarp();
          }
          return true;
        }
      }
      return false;
    };
    int to = -1;
    for (;;) {
      __syncthreads();
      if (warp == 0) {
        int next = -1, more = 0;
        while (!dead) {
          if (win == 0 && !load_window()) break;
          if (pending) {
            more = 1;
            break;
          }
          const int j = __ffs(win) - 1;
          win &= win - 1;
          const double pj = __shfl_sync(0xffffffffu, cp, j), qj = __shfl_sync(0xffffffffu, cq, j),
                       uj = __shfl_sync(0xffffffffu, cu, j);
          const bool ok = greedy ? pj > 0.0 : QT ? uj * B * qj < pj - A * qj : uj * B < pj;
          if (ok) {
            next = base + j;
            break;
          }
          if (greedy) continue;
          if (QT) {
            A += B;
            pending = true;
          } else {
            B -= pj;
          }
        }
        pending = false;
        if (lane == 0) {
          sh.next = next;
          sh.more = more;
          sh.a = A;
        }
      }
      __syncthreads();
      to = sh.next;
      A = sh.a;
      if (!QT || !sh.more) break;
      // B = sum_x (p(x) - A q(x))+
      const float inv = (float)(1.0 / sum), af = (float)A;
      float t = 0.f;
      if (p.vec) {
#pragma unroll 2
        for (int i = c0 + 8 * tid; i < c1; i += 8 * kThreads) {
          float x[8], q[8];
          load8<LB>(row, i, x);
          load8<QT == 1>(qrow, i, q);
#pragma unroll
          for (int e = 0; e < 8; ++e) t += fmaxf(fmaf(-af, q[e], weight(x[e], m) * inv), 0.f);
        }
      } else {
#pragma unroll 4
        for (int i = c0 + tid; i < c1; i += kThreads)
          t += fmaxf(fmaf(-af, load_elem<QT == 1>(qrow, i), weight(load_elem<LB>(row, i), m) * inv), 0.f);
      }
      B = cluster_sum(t);
    }
    if (to >= 0) {
      if (tid == 0 && rank == 0 && p.logprobs) {
        double lp = 0.0;
        if (!greedy)
          lp = ((double)load_elem<LB>(row, p.tokens[o + to]) - (double)m) / (double)temp - log(sum);
        p.logprobs[o + k] = (float)lp;
      }
      v = to;
      ++k;
      continue;
    }

    // ---- no child accepted: the bonus token
    int bonus = -1;
    if (!dead && greedy) {
      bonus = am;
    } else if (!dead) {
      const float inv = (float)(1.0 / sum);
      float af = (float)A;
      const int n_child = QT ? 0 : sh.n_child;
      bool plain = false;   // draw from p_v itself: nothing is left of the residual
      for (;;) {
        uint64_t best = 0;
        auto rejected = [&](int x) {
          for (int j = 0; j < min(n_child, kChildList); ++j)
            if (sh.child_tok[j] == x) return true;
          if (n_child > kChildList)
            for (int j = v + 1; j < L; ++j)
              if (p.parents[o + j] == v && p.tokens[o + j] == x) return true;
          return false;
        };
        auto take = [&](float x, float q, float e, int i) {
          float w = weight(x, m) * inv;
          if (QT && !plain) w = fmaf(-af, q, w);
          if (!(w > 0.f)) return;
          const uint64_t key = race_key(__fdiv_rn(w, e), (uint32_t)i);
          // a rejected token is looked for only when it would win
          if (key > best && (QT || plain || !rejected(i))) best = key;
        };
        if (p.vec) {
#pragma unroll 2
          for (int i = c0 + 8 * tid; i < c1; i += 8 * kThreads) {
            float x[8], q[8], e[8];
            load8<LB>(row, i, x);
            if (QT) load8<QT == 1>(qrow, i, q);
            load8<false>(noise, i, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) take(x[j], QT ? q[j] : 0.f, e[j], i + j);
          }
        } else {
#pragma unroll 4
          for (int i = c0 + tid; i < c1; i += kThreads)
            take(load_elem<LB>(row, i), QT ? load_elem<QT == 1>(qrow, i) : 0.f, __ldg(noise + i), i);
        }
        best = cluster_max(best);
        if (best != 0) {
          bonus = (int)(0xffffffffu - (uint32_t)best);
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
        if (p.logprobs) {
          double lp = 0.0;
          if (!greedy && bonus >= 0)
            lp = ((double)load_elem<LB>(row, bonus) - (double)m) / (double)temp - log(sum);
          p.logprobs[o + k] = (float)lp;
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
