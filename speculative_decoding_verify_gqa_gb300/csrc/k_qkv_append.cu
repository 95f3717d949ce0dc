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
// tables, page id) on single tokens.  So a CTA takes one token: it starts the
// loads of all its rows first, finds the token's slot and its angles while
// they are under way, and every head uses the same angles.  A row is held by
// head_dim / 8 neighbouring lanes, 16 bytes each.
//
// Angles: the frequency is kept in turns as a 64-bit binary fraction, so
// position * frequency modulo one turn is one integer product, exact for any
// position to 2^-64 of the position; its top 32 bits go through sincospi.  (A
// float product is off by position * 2^-24 of a radian.)
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/verify_attn.h"
#include "va_device.cuh"
#include "va_kernels.h"

namespace va {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 5;  // rows of q and k that a thread has in flight

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

template <int D>
__global__ void __launch_bounds__(kThreads) paged_qkv_append_kernel(const QkvParams p) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  __shared__ __align__(16) float cs[64], sn[64], wt[2][D];
  const int tid = threadIdx.x, lane = tid % LANES, grp = tid / LANES;
  const long long i = blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  // the first rows of this thread's lane group, and its row of v
  const int nqk = p.h_q + p.h_kv;
  const uint4* const qs = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + i * p.q_stride) + lane;
  const uint4* const ks = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k) + i * p.k_stride) + lane;
  const uint4* const vs = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v) + i * p.v_stride);
  const int v_lanes = p.head_dim_v / 8, v_total = p.h_kv * v_lanes;
  uint4 x[kRows], vx = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int r = grp + j * GROUPS;
    x[j] = r < p.h_q ? qs[(size_t)r * LANES] : r < nqk ? ks[(size_t)(r - p.h_q) * LANES] : make_uint4(0, 0, 0, 0);
  }
  if (tid < v_total) vx = vs[tid];
  // angles and weights for all heads
  if (tid < p.rot / 2) {
    const uint64_t turns = (uint64_t)(int64_t)p.positions[i] * p.turn[tid];
    sincospif((float)(int32_t)(uint32_t)(turns >> 32) * 0x1p-31f, &sn[tid], &cs[tid]);
  }
  if (p.q_weight && tid < D)
    wt[0][tid] = (p.weight_f32 ? static_cast<const float*>(p.q_weight)[tid]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(p.q_weight)[tid])) + p.weight_offset;
  if (p.k_weight && tid >= kThreads - D) {
    const int e = tid - (kThreads - D);
    wt[1][e] = (p.weight_f32 ? static_cast<const float*>(p.k_weight)[e]
                             : __bfloat162float(static_cast<const __nv_bfloat16*>(p.k_weight)[e])) + p.weight_offset;
  }
  // the token's request: as many requests end at or before it
  int b = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads)
    b += __syncthreads_count(b0 + tid < p.batch && p.append_indptr[b0 + tid + 1] <= i);
  if (b >= p.batch) return;  // behind the last request: padding
  const int a0 = p.append_indptr[b], n = p.append_indptr[b + 1] - a0;
  const int pg0 = p.kv_indptr[b], npg = p.kv_indptr[b + 1] - pg0, lpl = p.last_page_len[b];
  const long long pos = (npg > 0 ? (long long)(npg - 1) * p.page_size + lpl : 0) - n + (i - a0);
  const bool pos_ok = i >= a0 && i - a0 < n && pg0 >= 0 && npg > 0 && lpl >= 1 && lpl <= p.page_size && pos >= 0;
  const int page = pos_ok ? p.kv_indices[pg0 + (int)(pos >> p.log2_page)] : -1;
  if (!pos_ok || (unsigned)page >= (unsigned)p.num_pages) {
    if (tid == 0 && p.status) atomicOr(p.status, pos_ok ? VA_DEV_BAD_PAGE : VA_DEV_BAD_APPEND);
    return;
  }
  // cache row of KV head h: row0 + h * step
  const long long slot = pos & (p.page_size - 1);
  const long long row0 = p.nhd ? ((long long)page * p.page_size + slot) * p.h_kv
                               : (long long)page * p.h_kv * p.page_size + slot;
  const long long step = p.nhd ? 1 : p.page_size;
  uint4* const qd = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + i * ((long long)p.h_q * D)) + lane;

  const int e0 = lane * 8, half = p.rot / 2;
  const bool turned = e0 < p.rot, low = e0 < half;
  const int partner = low ? lane + half / 8 : lane - half / 8;
  for (int r0 = 0; r0 < nqk; r0 += kRows * GROUPS) {
    if (r0 > 0) {
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int r = r0 + grp + j * GROUPS;
        x[j] = r < p.h_q ? qs[(size_t)r * LANES] : r < nqk ? ks[(size_t)(r - p.h_q) * LANES] : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = r0 + grp + j * GROUPS;
      if (r0 + j * GROUPS >= nqk) break;  // (the same for all lanes)
      const bool is_q = r < p.h_q;
      float y[8];
      unpack8(x[j], y);
      // (a warp's rows may be of both kinds: the shuffles stay outside the branches)
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
      for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
        const float* w = wt[is_q ? 0 : 1] + e0;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv * w[e];
      }
      if (p.rot > 0) {
        if (p.interleaved) {
          if (turned) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float c = cs[(e0 + e) / 2], s = sn[(e0 + e) / 2], a = y[e], z = y[e + 1];
              y[e] = a * c - z * s;
              y[e + 1] = a * s + z * c;
            }
          }
        } else {
          const int j0 = turned ? (low ? e0 : e0 - half) : 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float z = __shfl_sync(0xffffffffu, y[e], partner, LANES);
            const float c = cs[j0 + e], s = sn[j0 + e];
            if (turned) y[e] = low ? y[e] * c - z * s : y[e] * c + z * s;
          }
        }
      }
      if (is_q) {
        qd[(size_t)r * LANES] = pack8(y);
      } else if (r < nqk) {
        const long long row = row0 + (r - p.h_q) * step;
        if (p.quant)
          reinterpret_cast<uint2*>(p.k_cache)[row * LANES + lane] = codes8(y, p.k_scale);
        else
          reinterpret_cast<uint4*>(p.k_cache)[row * LANES + lane] = pack8(y);
      }
    }
  }
  for (int c = tid; c < v_total; c += kThreads) {
    if (c != tid) vx = vs[c];
    const int h = c / v_lanes;
    const long long at = (row0 + h * step) * v_lanes + (c - h * v_lanes);
    if (p.quant) {
      float y[8];
      unpack8(vx, y);
      reinterpret_cast<uint2*>(p.v_cache)[at] = codes8(y, p.v_scale);
    } else {
      reinterpret_cast<uint4*>(p.v_cache)[at] = vx;
    }
  }
}

}  // namespace

cudaError_t launch_qkv_append(const QkvParams& p, int head_dim, cudaStream_t stream) {
  void* args[] = {const_cast<QkvParams*>(&p)};
  const void* k = head_dim == 64 ? reinterpret_cast<const void*>(paged_qkv_append_kernel<64>)
                                 : reinterpret_cast<const void*>(paged_qkv_append_kernel<128>);
  return launch_kernel(k, dim3((unsigned)p.total_new), dim3(kThreads), 0, stream, args, /*pdl=*/true);
}

}  // namespace va
