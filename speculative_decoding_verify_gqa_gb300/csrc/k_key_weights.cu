// Attention weight that each cached key receives from a step's queries: for
// key j of request b and KV head h,
//
//   w[j] = base + sum over queries t that see j, heads g of h: exp(s_tgj - lse_tg)
//
// with s = q . k * sm_scale * k_scale, lse the attention's own log-sum-exp, and
// base = decay * w[j] for the keys of the prefix, 0 for the step's own.  With
// an accepted path only its queries and keys count: query k is node path[k],
// key prefix + k is read from slot prefix + path[k] and weighed in slot
// prefix + k, where compaction moves it.
//
// One thread per key: its row of K in registers, the queries broadcast from
// shared memory, so the sum over the queries never crosses threads and its
// order is fixed.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/verify_attn.h"
#include "va_device.cuh"
#include "va_kernels.h"

namespace va {
namespace {

constexpr int kTile = 128;   // keys of a CTA
constexpr int kQRows = 16;   // query rows in shared memory

struct Request {
  int o, L, n, pg0, npg;  // first query row, query tokens, those counted, page table
  int pre, keys;          // prefix length, keys weighed (0: nothing to do)
  bool bad;
};

__device__ __forceinline__ Request load_request(const KeyWeightParams& p, int b) {
  Request r;
  r.o = p.qo_indptr[b];
  r.L = p.qo_indptr[b + 1] - r.o;
  r.pg0 = p.kv_indptr[b];
  r.npg = p.kv_indptr[b + 1] - r.pg0;
  const int lpl = r.npg > 0 ? p.last_page_len[b] : 1;
  r.n = p.accept_len ? p.accept_len[b] : r.L;
  const long long len = r.npg > 0 ? (long long)(r.npg - 1) * p.page_size + lpl : 0, pre = len - r.L;
  r.bad = r.o < 0 || r.L < 0 || (long long)r.o + r.L > p.total_qo || r.npg < 0 || r.pg0 < 0 || lpl < 1 ||
          lpl > p.page_size || pre < 0 || len > 0x7fffffffLL || r.n < 0 || r.n > r.L;
  r.pre = r.bad ? 0 : (int)pre;
  r.keys = r.bad ? 0 : r.pre + r.n;
  return r;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kTile) verify_attn_key_weights_kernel(const KeyWeightParams p) {
  __shared__ __align__(16) float qs[kQRows][D];
  __shared__ float l2[kQRows];
  const int tid = threadIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  long long unit = 0;  // of (request, head, tile)
  for (int b = 0; b < p.batch; ++b) {
    const Request rq = load_request(p, b);
    int bad = rq.bad;
    if (!bad && p.accept_len)
      for (int k = tid; k < rq.n; k += kTile) {
        const int node = p.path[rq.o + k];
        bad |= node >= rq.L || node < k || (k > 0 && p.path[rq.o + k - 1] >= node);
      }
    bad = __syncthreads_or(bad);
    if (bad) {
      if (blockIdx.x == 0 && tid == 0 && p.status) atomicOr(p.status, VA_DEV_BAD_TABLE);
      continue;
    }
    const int tiles = (rq.keys + kTile - 1) / kTile;
    const long long units = (long long)tiles * p.h_kv;
    long long u = (long long)blockIdx.x - unit % gridDim.x;
    if (u < 0) u += gridDim.x;
    unit += units;
    for (; u < units; u += gridDim.x) {
      const int h = (int)(u / tiles), j = (int)(u % tiles) * kTile + tid;
      const bool live = j < rq.keys;
      const int at = live ? (j < rq.pre || !p.accept_len ? j : rq.pre + min(max(p.path[rq.o + j - rq.pre], 0), rq.L - 1)) : 0;
      auto row_of = [&](int pos) -> long long {
        const unsigned page = (unsigned)p.kv_indices[rq.pg0 + (pos >> p.log2_page)];
        if (page >= (unsigned)p.num_pages) return -1;
        const long long slot = pos & (p.page_size - 1);
        return p.nhd ? ((long long)page * p.page_size + slot) * p.h_kv + h
                     : ((long long)page * p.h_kv + h) * p.page_size + slot;
      };
      const long long src = live ? row_of(at) : -1, dst = live ? row_of(j) : -1;
      if (live && (src < 0 || dst < 0) && p.status) atomicOr(p.status, VA_DEV_BAD_PAGE);
      const bool ok = src >= 0 && dst >= 0;
      uint32_t k[D / 2];  // bf16 pairs
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        if constexpr (FP8) {
          const uint2 x = ok ? static_cast<const uint2*>(p.k_cache)[src * (D / 8) + c] : make_uint2(0, 0);
          k[4 * c] = e4m3x2_to_bf16x2((uint16_t)x.x);
          k[4 * c + 1] = e4m3x2_to_bf16x2((uint16_t)(x.x >> 16));
          k[4 * c + 2] = e4m3x2_to_bf16x2((uint16_t)x.y);
          k[4 * c + 3] = e4m3x2_to_bf16x2((uint16_t)(x.y >> 16));
        } else {
          const uint4 x = ok ? static_cast<const uint4*>(p.k_cache)[src * (D / 8) + c] : make_uint4(0, 0, 0, 0);
          k[4 * c] = x.x;
          k[4 * c + 1] = x.y;
          k[4 * c + 2] = x.z;
          k[4 * c + 3] = x.w;
        }
      }
      const int draft = j - rq.pre, len = rq.pre + rq.L;
      float sum = 0.f;
      for (int r0 = 0; r0 < rq.n * p.group; r0 += kQRows) {
        const int m = min(kQRows, rq.n * p.group - r0);
        __syncthreads();
        for (int i = tid; i < m * (D / 8); i += kTile) {
          const int r = i / (D / 8), c = i % (D / 8), t = (r0 + r) / p.group, g = (r0 + r) % p.group;
          const int row = rq.o + (p.accept_len ? min(max(p.path[rq.o + t], 0), rq.L - 1) : t);
          const uint4 x = reinterpret_cast<const uint4*>(p.q)[((long long)row * p.h_q + h * p.group + g) * (D / 8) + c];
          const uint32_t u4[4] = {x.x, x.y, x.z, x.w};
          for (int e = 0; e < 4; ++e) {
            qs[r][8 * c + 2 * e] = __uint_as_float(u4[e] << 16);
            qs[r][8 * c + 2 * e + 1] = __uint_as_float(u4[e] & 0xffff0000u);
          }
          if (c == 0) {
            const float lse = p.lse[(long long)row * p.h_q + h * p.group + g];
            l2[r] = lse == -INFINITY ? INFINITY : lse * kLog2e;  // a row that saw nothing counts nothing
          }
        }
        __syncthreads();
        for (int r = 0; r < m; ++r) {
          const int t = (r0 + r) / p.group;
          bool vis = draft <= t;
          if (p.mask) {
            vis = draft < 0;
            if (p.mask_full || (draft >= 0 && ok)) {
              const long long bit = p.mask_indptr[b] + (p.mask_full ? (long long)t * len + min(j, len - 1)
                                                                    : (long long)t * rq.L + draft);
              vis = (p.mask[bit >> 3] >> (bit & 7)) & 1;
            }
          }
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < D / 2; ++e) {
            s = fmaf(qs[r][2 * e], __uint_as_float(k[e] << 16), s);
            s = fmaf(qs[r][2 * e + 1], __uint_as_float(k[e] & 0xffff0000u), s);
          }
          if (vis) sum += ex2(fmaf(s, p.scale_log2, -l2[r]));
        }
      }
      if (ok) {
        float* const w = p.key_weights + dst;
        *w = j < rq.pre && p.decay != 0.f ? fmaf(p.decay, *w, sum) : sum;
      }
    }
  }
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightParams& p, int head_dim, bool kv_fp8, int num_sms, cudaStream_t stream) {
  void* args[] = {const_cast<KeyWeightParams*>(&p)};
  const void* k = head_dim == 64 ? (kv_fp8 ? reinterpret_cast<const void*>(verify_attn_key_weights_kernel<64, true>)
                                           : reinterpret_cast<const void*>(verify_attn_key_weights_kernel<64, false>))
                                 : (kv_fp8 ? reinterpret_cast<const void*>(verify_attn_key_weights_kernel<128, true>)
                                           : reinterpret_cast<const void*>(verify_attn_key_weights_kernel<128, false>));
  return launch_kernel(k, dim3((unsigned)num_sms * 4), dim3(kTile), 0, stream, args, /*pdl=*/true);
}

}  // namespace va
