// Norm, rotation and append of a step's new tokens in one pass over the rows
// of the projection: every head of q and k is divided by its root mean square
// and multiplied by a weight, rotated by RoPE at the token's position, and
// rounded once -- q to bf16 rows, k (and v, as it is) into the token's page
// slot, as bf16 or as e4m3(x / scale).
//
//   x' = x / sqrt(mean(x^2) + eps) * (w + offset)
//   (a, b) -> (a cos - b sin, a sin + b cos),  angle = position * frequency
//
// The work reads and writes every row once and computes about ten operations
// an element: HBM bounds it on prompts, the chain of dependent loads (request,
// tables, page id) on single tokens.  A row is held by head_dim / 8 neighbouring
// lanes, 16 bytes each, so a lane has the same columns of all rows and keeps
// for them, weight and rotation in one,
//   y = (x A + x' B) / rms,  A = w cos, B = -+ w' sin,  x' and w' the pair's other
// -- of which the raw 16 bytes come from the other lane by four shuffles.  In
// columns that do not turn x' may not come in by B = 0, which makes NaN of an
// infinity: there x' is x itself and A = B = w / 2 (exact without weights); with
// pairs of neighbours x' is masked to 0.
//
// A CTA takes a run of tokens, one each where they are few.  It finds the slots
// of eight tokens (a warp a token) and their angles at a time.  With one token
// the loads of its rows are started first, into registers, and the slot is
// found while they are under way.  With more, one thread brings the tokens' rows
// into shared memory by bulk copies, a token ahead of the one in work: rows
// loaded into registers one token ahead kept too little under way (10,240 tokens
// of 64 + 16 heads: 38 % of the DRAM's cycles, warps waiting for loads half of
// their time).  On one GB300 these 10,240 tokens take 83.5 us (5.0 TB/s; 90 into
// an fp8 cache), 334 tokens in 64 chains into an fp8 cache 8.6 us, one token (32
// + 16 heads) 3.2 us.
//
// Angles: the frequency is kept in turns as a 64-bit binary fraction, so
// position * frequency modulo one turn is one integer product, which adds
// position * 2^-64 turns to what the frequency's double has lost (below 2^-53 of
// a turn); its top 32 bits, rounded to fp32 (1e-7 of a radian), go through
// sincospi.  (A float product is off by position * 2^-24 of a radian.)
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/verify_attn.h"
#include "va_budget.h"
#include "va_device.cuh"
#include "va_kernels.h"
#include "va_tc.cuh"

namespace va {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;      // rows of q that a thread has in flight
constexpr int kTokens = 8;    // tokens whose slots and angles are found at a time
// CTAs that an SM holds and tokens whose rows each holds in shared memory: four
// of two tokens took a prompt's rows in 83.5 us, three of three in 89.2
constexpr int kResident = 4, kStages = 2;
constexpr int kMaxStages = 45 * 1024;
constexpr int kDrain = 1024;  // tries for a copy under way when the CTA gives up
// How a CTA gets its rows: one token's into registers, all that it likes while
// there is a CTA an SM at most (1 to 8 tokens of 64 + 16 heads 3.7 us, 4.4 with
// the registers of the next), or so that three CTAs share an SM, which spills
// (334 tokens 8.4 us, 9.3 with two and no spill); a run of tokens' through shared
// memory.
enum { kFew, kDirect, kStaged };

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(u[k] << 16);
    x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// e4m3 codes of x / scale: the correctly rounded quotient, to nearest even, saturated
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(x[e], scale);
  return make_uint2(e4m3x4_rn_satfinite(y[0], y[1], y[2], y[3]), e4m3x4_rn_satfinite(y[4], y[5], y[6], y[7]));
}

// `bytes` (a multiple of 16) from global to shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Weight and rotation of a lane's eight columns, as pairs of neighbours.
struct Coef {
  uint64_t a[4], b[4];
};
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// y = (x A + x' B) / rms of this lane's columns; all lanes of the warp call.
// (keep: all bits, or none where pairs of neighbours do not turn)
template <int D, bool PAIRS>
__device__ __forceinline__ void head(uint4 raw, const Coef& c, bool norm, bool rot, uint32_t keep, int partner, float eps, float (&y)[8]) {
  constexpr int LANES = D / 8;
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
  uint64_t x[4], v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = f32x2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = mul_f32x2(x[k], c.a[k]);
  if (rot) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (PAIRS) {
        v[k] = fma_f32x2(f32x2(__uint_as_float(u[k] & 0xffff0000u & keep), __uint_as_float((u[k] << 16) & keep)), c.b[k], v[k]);
      } else {
        const uint32_t o = __shfl_sync(0xffffffffu, u[k], partner, LANES);
        v[k] = fma_f32x2(f32x2(__uint_as_float(o << 16), __uint_as_float(o & 0xffff0000u)), c.b[k], v[k]);
      }
    }
  }
  if (norm) {
    uint64_t q = mul_f32x2(x[0], x[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) q = fma_f32x2(x[k], x[k], q);
    float ss = f32x2_lo(q) + f32x2_hi(q);
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float inv = rsqrtf(ss * (1.f / D) + eps);
    const uint64_t i2 = f32x2(inv, inv);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = mul_f32x2(v[k], i2);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    y[2 * k] = f32x2_lo(v[k]);
    y[2 * k + 1] = f32x2_hi(v[k]);
  }
}

template <int D, bool PAIRS, int MODE>
__global__ void __launch_bounds__(kThreads, MODE == kStaged ? kResident : MODE == kDirect ? 3 : 1) paged_qkv_append_kernel(const QkvParams p) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  constexpr bool STAGED = MODE == kStaged;
  __shared__ __align__(16) float cs[kTokens][D], sn[kTokens][D];   // by column: cos, -+ sin
  __shared__ __align__(16) float wt[2][D];
  __shared__ long long first_row[kTokens];   // cache row of the token's KV head 0, or -1
  extern __shared__ __align__(128) uint8_t stages[];   // STAGED: kStages x (q, k, v rows of a token)
  __shared__ __align__(8) uint64_t full[kStages];
  __shared__ int abort_shared;
  const int tid = threadIdx.x, lane = tid % LANES, grp = tid / LANES, warp = tid >> 5, wl = tid & 31;
  const long long i0 = (long long)blockIdx.x * p.per_cta, i1 = min(i0 + p.per_cta, (long long)p.total_new);
  grid_dependency_wait();
  grid_dependents_launch();
  const __nv_bfloat16* const q = static_cast<const __nv_bfloat16*>(p.q) + lane * 8;
  const __nv_bfloat16* const k = static_cast<const __nv_bfloat16*>(p.k) + lane * 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int v_lanes = p.head_dim_v / 8, v_total = p.h_kv * v_lanes;
  // STAGED: the token's rows in shared memory
  const uint32_t q_bytes = p.h_q * D * 2, k_bytes = p.h_kv * D * 2, v_bytes = v_total * 16;
  const uint32_t stage_bytes = q_bytes + k_bytes + v_bytes;
  auto bring = [&](long long i, int stage) {
    const uint32_t at = smem_u32(stages) + stage * stage_bytes, bar = smem_u32(full + stage);
    mbar_expect_tx(bar, stage_bytes);
    bulk_load(at, static_cast<const __nv_bfloat16*>(p.q) + i * p.q_stride, q_bytes, bar);
    bulk_load(at + q_bytes, static_cast<const __nv_bfloat16*>(p.k) + i * p.k_stride, k_bytes, bar);
    bulk_load(at + q_bytes + k_bytes, static_cast<const __nv_bfloat16*>(p.v) + i * p.v_stride, v_bytes, bar);
  };
  uint4 x[STAGED ? 1 : kRows], kx = zero, vx = zero;
  if constexpr (STAGED) {
    if (tid == 0) {
      for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(full + s), 1);
      abort_shared = 0;
      mbar_fence_init();
      for (int s = 0; s < kStages && i0 + s < i1; ++s) bring(i0 + s, s);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      x[j] = grp + j * GROUPS < p.h_q ? *reinterpret_cast<const uint4*>(q + i0 * p.q_stride + (grp + j * GROUPS) * D) : zero;
    if (grp < p.h_kv) kx = *reinterpret_cast<const uint4*>(k + i0 * p.k_stride + grp * D);
    if (tid < v_total) vx = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v) + i0 * p.v_stride)[tid];
  }
  int stage = 0, round = 0;
  if (tid >= kThreads - D) {
    const int e = tid - (kThreads - D);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const void* const w = t == 0 ? p.q_weight : p.k_weight;
      wt[t][e] = !w ? 1.f : (p.weight_f32 ? static_cast<const float*>(w)[e]
                                          : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[e])) + p.weight_offset;
    }
  }
  const int e0 = lane * 8, half = p.rot / 2;
  const bool rot = p.rot > 0, q_norm = p.q_weight != nullptr, k_norm = p.k_weight != nullptr;
  const uint32_t keep = !PAIRS || e0 < p.rot ? 0xffffffffu : 0u;
  const int partner = e0 >= p.rot ? lane : e0 < half ? lane + half / 8 : lane - half / 8;
  const long long step = p.nhd ? 1 : p.page_size;

  for (long long g0 = i0; g0 < i1; g0 += kTokens) {
    const int tokens = (int)min((long long)kTokens, i1 - g0);
    if (g0 > i0) __syncthreads();
    // A warp a token: its request -- as many end at or before it -- and its slot.
    // The tables of 128 requests are read at once, before it is known whose
    // they are: one round to memory instead of two.
    if (warp < tokens) {
      const long long i = g0 + warp;
      int b = 0, tab[5] = {0, 0, 0, 0, 0};
      for (int b0 = 0; b0 < p.batch; b0 += 128) {
        int v[4][5], in = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int at = min(b0 + c * 32 + wl, p.batch - 1);
          v[c][0] = p.append_indptr[at];
          v[c][1] = p.append_indptr[at + 1];
          v[c][2] = p.kv_indptr[at];
          v[c][3] = p.kv_indptr[at + 1];
          v[c][4] = p.last_page_len[at];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          in += __popc(__ballot_sync(0xffffffffu, b0 + c * 32 + wl < p.batch && v[c][1] <= i));
        b += in;
        if (in < 128) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int m = 0; m < 5; ++m) {
              const int x = __shfl_sync(0xffffffffu, v[c][m], in & 31);
              if (c == in >> 5) tab[m] = x;
            }
          break;
        }
      }
      if (wl == 0) {
        long long row = -1;   // (behind the last request: padding)
        if (b < p.batch) {
          const int a0 = tab[0], n = tab[1] - a0, pg0 = tab[2], npg = tab[3] - pg0, lpl = tab[4];
          const long long pos = (npg > 0 ? (long long)(npg - 1) * p.page_size + lpl : 0) - n + (i - a0);
          const bool ok = i >= a0 && i - a0 < n && pg0 >= 0 && npg > 0 && lpl >= 1 && lpl <= p.page_size && pos >= 0;
          const int page = ok ? p.kv_indices[pg0 + (int)(pos >> p.log2_page)] : -1;
          const long long slot = pos & (p.page_size - 1);
          if (ok && (unsigned)page < (unsigned)p.num_pages)
            row = p.nhd ? ((long long)page * p.page_size + slot) * p.h_kv : (long long)page * p.h_kv * p.page_size + slot;
          else if (p.status)
            atomicOr(p.status, ok ? VA_DEV_BAD_PAGE : VA_DEV_BAD_APPEND);
        }
        first_row[warp] = row;
      }
    }
    // the tokens' angles, a pair of columns a thread
    for (int c = tid; c < tokens * (D / 2); c += kThreads) {
      const int t = c / (D / 2), j = c % (D / 2);
      const bool turns = j < half;
      const int lo = PAIRS ? 2 * j : turns ? j : half + j, hi = PAIRS ? 2 * j + 1 : turns ? half + j : j + D / 2;
      float co = PAIRS || !rot ? 1.f : 0.5f, si = PAIRS ? -0.f : 0.5f;   // (-0: x A = -0 stays)
      if (turns) {
        const uint64_t a = (uint64_t)(int64_t)p.positions[g0 + t] * p.turn[j];
        sincospif((float)(int32_t)(uint32_t)(a >> 32) * 0x1p-31f, &si, &co);
      }
      cs[t][lo] = cs[t][hi] = co;
      sn[t][lo] = turns ? -si : si;
      sn[t][hi] = si;
    }
    __syncthreads();
    for (int t = 0; t < tokens; ++t) {
      const long long i = g0 + t, row0 = first_row[t];
      const bool live = row0 >= 0;
      const uint8_t* const at = stages + stage * stage_bytes;
      bool ok = true;
      if constexpr (STAGED) ok = mbar_wait(smem_u32(full + stage), round & 1, &abort_shared);
      Coef co;
      auto coef = [&](const float* w) {
        const float4* const c4 = reinterpret_cast<const float4*>(cs[t] + e0);
        const float4* const s4 = reinterpret_cast<const float4*>(sn[t] + e0);
        const float4* const w4 = reinterpret_cast<const float4*>(w + e0);
        const float4* const o4 = reinterpret_cast<const float4*>(w + (PAIRS ? lane : partner) * 8);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float4 c = c4[m], s = s4[m], a = w4[m];
          float4 o = o4[m];
          if constexpr (PAIRS) o = make_float4(o.y, o.x, o.w, o.z);
          co.a[2 * m] = f32x2(a.x * c.x, a.y * c.y);
          co.a[2 * m + 1] = f32x2(a.z * c.z, a.w * c.w);
          co.b[2 * m] = f32x2(o.x * s.x, o.y * s.y);
          co.b[2 * m + 1] = f32x2(o.z * s.z, o.w * s.w);
        }
      };
      coef(wt[0]);
      uint4* const qd = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + i * ((long long)p.h_q * D)) + lane;
      float y[8];
#pragma unroll 1
      for (int r0 = 0; r0 < p.h_q; r0 += kRows * GROUPS) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const int r = r0 + grp + j * GROUPS;
          if (r0 + j * GROUPS >= p.h_q) break;  // (the same for all lanes)
          uint4 raw = zero;
          if constexpr (STAGED) {
            if (r < p.h_q) raw = *reinterpret_cast<const uint4*>(at + (r * LANES + lane) * 16);
          } else {
            raw = x[j];
            // the next batch of the token
            const int rn = r + kRows * GROUPS;
            if (rn < p.h_q) x[j] = *reinterpret_cast<const uint4*>(q + i * p.q_stride + (size_t)rn * D);
          }
          head<D, PAIRS>(raw, co, q_norm, rot, keep, partner, p.eps, y);
          if (live && ok && r < p.h_q) qd[(size_t)r * LANES] = pack8(y);
        }
      }
      coef(wt[1]);
#pragma unroll 1
      for (int r0 = 0; r0 < p.h_kv; r0 += GROUPS) {
        const int r = r0 + grp;
        uint4 raw = zero;
        if (r < p.h_kv) {
          if constexpr (STAGED) raw = *reinterpret_cast<const uint4*>(at + q_bytes + (r * LANES + lane) * 16);
          else raw = r0 == 0 ? kx : *reinterpret_cast<const uint4*>(k + i * p.k_stride + (size_t)r * D);
        }
        head<D, PAIRS>(raw, co, k_norm, rot, keep, partner, p.eps, y);
        if (live && ok && r < p.h_kv) {
          const long long row = row0 + r * step;
          if (p.quant)
            reinterpret_cast<uint2*>(p.k_cache)[row * LANES + lane] = codes8(y, p.k_scale);
          else
            reinterpret_cast<uint4*>(p.k_cache)[row * LANES + lane] = pack8(y);
        }
      }
#pragma unroll 1
      for (int c = tid; c < v_total; c += kThreads) {
        uint4 v;
        if constexpr (STAGED) v = *reinterpret_cast<const uint4*>(at + q_bytes + k_bytes + c * 16);
        else v = c == tid ? vx : reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v) + i * p.v_stride)[c];
        if (live && ok) {
          const int h = c / v_lanes;
          const long long to = (row0 + h * step) * v_lanes + (c - h * v_lanes);
          if (p.quant) {
            unpack8(v, y);
            reinterpret_cast<uint2*>(p.v_cache)[to] = codes8(y, p.v_scale);
          } else {
            reinterpret_cast<uint4*>(p.v_cache)[to] = v;
          }
        }
      }
      if constexpr (STAGED) {
        // all have read the token's rows: its place is another's
        if (!__syncthreads_and(ok)) {
          if (tid == 0) {
            // nothing may still be on its way into the CTA's shared memory
            for (int s = 0; s < kStages && i + s < i1; ++s) {
              const int at_stage = (stage + s) % kStages, at_round = round + (stage + s) / kStages;
              for (int n = 0; n < kDrain && !mbar_try_wait(smem_u32(full + at_stage), at_round & 1); ++n) {}
            }
            if (p.status) atomicOr(p.status, VA_DEV_TIMEOUT);
          }
          return;
        }
        if (tid == 0 && i + kStages < i1) bring(i + kStages, stage);
        if (++stage == kStages) {
          stage = 0;
          ++round;
        }
      }
    }
  }
}

template <int D, bool PAIRS>
cudaError_t launch(const QkvParams& p, size_t stages, int num_sms, cudaStream_t stream) {
  void* args[] = {const_cast<QkvParams*>(&p)};
  const dim3 grid((unsigned)((p.total_new + p.per_cta - 1) / p.per_cta));
  const void* k = p.total_new <= num_sms ? reinterpret_cast<const void*>(paged_qkv_append_kernel<D, PAIRS, kFew>)
                                         : reinterpret_cast<const void*>(paged_qkv_append_kernel<D, PAIRS, kDirect>);
  if (stages) {
    k = reinterpret_cast<const void*>(paged_qkv_append_kernel<D, PAIRS, kStaged>);
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStages);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(k, grid, dim3(kThreads), stages, stream, args, /*pdl=*/true);
}

}  // namespace

cudaError_t launch_qkv_append(const QkvParams& params, int head_dim, int num_sms, cudaStream_t stream) {
  // One wave of CTAs, each with a run of tokens whose rows are brought into
  // shared memory; a token each where all are resident that way, or where a
  // token's rows leave no room for that many CTAs on an SM (more than 22.5 KB:
  // 10,240 tokens of 72 + 16 heads of 128 take 91 us, of 80 + 16 146 us).
  QkvParams p = params;
  const size_t token = ((size_t)(p.h_q + p.h_kv) * head_dim + (size_t)p.h_kv * p.head_dim_v) * 2;
  const long long most = (long long)num_sms * kResident;
  size_t stages = kStages * token;
  p.per_cta = (int)((p.total_new + most - 1) / most);
  if (p.per_cta <= 1 || stages > (size_t)kMaxStages) {
    p.per_cta = 1;
    stages = 0;
  }
  if (head_dim == 64) return p.interleaved ? launch<64, true>(p, stages, num_sms, stream) : launch<64, false>(p, stages, num_sms, stream);
  return p.interleaved ? launch<128, true>(p, stages, num_sms, stream) : launch<128, false>(p, stages, num_sms, stream);
}

}  // namespace va
