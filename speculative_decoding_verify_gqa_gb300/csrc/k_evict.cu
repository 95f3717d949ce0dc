// Eviction from the paged cache by the attention weight that each key has
// received: of request b's kv_len keys, each layer and KV head keeps keep_len
// -- the first `sinks`, the last `recent`, and of those between the largest
// weights, the lower position among equals -- and moves them to the front in
// their order, with their weights.
//
// A unit (layer, request, KV head) belongs to one cluster of CTAs.  Each CTA
// finds the unit's survivors for itself: the weight that the last of them has
// by three passes of an 11-bit radix select over order-preserving integers,
// then one bit a key and the count of bits before each word in shared memory.
// Then the CTAs share the columns: CTA c moves its 16-byte column chunks of
// every surviving row, and CTA 0 the weights.
//
// In place: the row of rank k goes to position k and comes from a position >=
// k.  A batch of rows is read, the CTA meets, and the batch is written: what
// it overwrites has a rank no higher than its position, so it has been read.
// Columns are independent, so only the CTA's own threads have to meet; the
// cluster meets once, before CTA 0 overwrites weights that others still rank.
//
// Bound by the rows' copy (HBM) where many units move, and by the select's
// chain of passes where few do.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/verify_attn.h"
#include "va_device.cuh"
#include "va_kernels.h"

namespace va {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kDigit = 11, kBins = 1 << kDigit;
constexpr int kBatch = 8;    // rows' chunks in flight per thread
constexpr int kResolve = 256;  // ranks resolved at a time

// Weights as integers in their order: -0 counts as 0, NaN above everything.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}

// exclusive sum over the threads of the CTA; *total receives the whole sum
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int x = warp_sums[w];
    before += w < warp ? x : 0;
    all += x;
  }
  *total = all;
  return before + s - v;
}

__global__ void __launch_bounds__(kThreads) paged_kv_evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t dyn[];
  uint32_t* const bits = dyn;                                   // one bit a key: kept
  int* const before = reinterpret_cast<int*>(dyn + p.words);    // kept keys before each word
  __shared__ int hist[kBins];
  __shared__ long long src_row[kResolve], dst_row[kResolve];
  __shared__ int warp_sums[kWarps], geo[4], pick[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % p.cluster;
  const long long unit = blockIdx.x / p.cluster;
  const int head = (int)(unit % p.h_kv);
  const int b = (int)(unit / p.h_kv % p.batch), layer = (int)(unit / p.h_kv / p.batch);
  grid_dependency_wait();
  grid_dependents_launch();
  if (tid < 3) pick[tid] = 0;
  if (tid < 4) {
    const int32_t* const src[4] = {p.kv_indptr + b, p.kv_indptr + b + 1, p.last_page_len + b, p.keep_len + b};
    geo[tid] = *src[tid];
  }
  __syncthreads();
  const int pg0 = geo[0], npg = geo[1] - pg0, lpl = npg > 0 ? geo[2] : 1;
  const long long len = npg > 0 ? (long long)(npg - 1) * p.page_size + lpl : 0;
  const bool table_ok = npg >= 0 && pg0 >= 0 && lpl >= 1 && lpl <= p.page_size && geo[3] >= 0 && len <= p.max_kv_len;
  const bool first = layer == 0 && head == 0 && rank == 0 && tid == 0;
  if (!table_ok) {
    if (first && p.kv_len_out) p.kv_len_out[b] = len >= 0 && len <= 0x7fffffffLL && npg >= 0 ? (int)len : 0;
    if (first && p.status) atomicOr(p.status, VA_DEV_BAD_TABLE);
    return;
  }
  const int n = (int)len, keep = min(geo[3], n);
  int bad = 0;
  if (keep < n)
    for (int j = tid; j < npg; j += kThreads) bad |= (unsigned)p.kv_indices[pg0 + j] >= (unsigned)p.num_pages;
  bad = __syncthreads_or(bad);
  if (first) {
    if (p.kv_len_out) p.kv_len_out[b] = bad ? n : keep;
    if (bad && p.status) atomicOr(p.status, VA_DEV_BAD_PAGE);
  }
  if (bad || keep == n) return;

  const long long slot_rows = p.nhd ? p.h_kv : 1, page_rows = (long long)p.h_kv * p.page_size;
  const long long layer_row = (long long)layer * p.num_pages * page_rows + (p.nhd ? head : (long long)head * p.page_size);
  float* const w = p.key_weights;
  // row of position j of this layer and head; a page id that has changed since the check reads page 0
  auto row_of = [&](int j) {
    const unsigned page = (unsigned)p.kv_indices[pg0 + (j >> p.log2_page)];
    return layer_row + (page < (unsigned)p.num_pages ? page : 0u) * page_rows + (j & (p.page_size - 1)) * slot_rows;
  };

  // the middle [lo, hi) competes for `rest` places
  const int lo = min(p.sinks, keep), hi = n - min(p.recent, keep - lo), rest = keep - lo - (n - hi);
  uint32_t edge = 0xffffffffu;  // the last survivor's weight, and how many of the keys with just that weight survive
  int ties = 0;
  if (rest > 0) {
    uint32_t fixed = 0;
    int want = rest;  // rank, from above, of the last survivor among the keys that share the digits found so far
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, nb = pass == 2 ? 1024 : kBins;
      for (int k = tid; k < nb; k += kThreads) hist[k] = 0;
      __syncthreads();
      const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
      for (int j = lo + tid; j < hi; j += kThreads) {
        const uint32_t u = order_of(w[row_of(j)]);
        if ((u & above) == fixed) atomicAdd(&hist[(u >> shift) & (nb - 1)], 1);
      }
      __syncthreads();
      // bins from above: thread t holds bins nb - 1 - t * per ...
      const int per = nb / kThreads;
      int sum = 0;
      for (int k = 0; k < per; ++k) sum += hist[nb - 1 - tid * per - k];
      int all;
      int run = block_scan(sum, warp_sums, &all);
      if (run < want && run + sum >= want) {
        for (int k = 0; k < per; ++k) {
          const int bin = nb - 1 - tid * per - k, c = hist[bin];
          if (run + c >= want) {
            pick[0] = bin;
            pick[1] = want - run;
            break;
          }
          run += c;
        }
      }
      __syncthreads();
      fixed |= (uint32_t)pick[0] << shift;
      want = pick[1];
      __syncthreads();
    }
    edge = fixed;
    ties = want;
  }

  // one bit a key, in order: a warp takes a run of words; equals are counted first
  const int words = (n + 31) >> 5, per = (words + kWarps - 1) / kWarps;
  const int w0 = min(warp * per, words), w1 = min(w0 + per, words);
  int equal = 0;
  for (int k = w0; k < w1; ++k) {
    const int j = k * 32 + lane;
    const uint32_t u = j >= lo && j < hi && rest > 0 ? order_of(w[row_of(j)]) : 0u;
    const bool more = j < lo || (j >= hi && j < n) || (j >= lo && j < hi && rest > 0 && u > edge);
    const bool same = j >= lo && j < hi && rest > 0 && u == edge;
    const uint32_t mm = __ballot_sync(0xffffffffu, more), ms = __ballot_sync(0xffffffffu, same);
    if (lane == 0) {
      bits[k] = mm;
      before[k] = (int)ms;  // (until the equals are counted)
    }
    equal += __popc(ms);
  }
  int all;
  int eq_run = block_scan(lane == 0 ? equal : 0, warp_sums, &all);
  eq_run = __shfl_sync(0xffffffffu, eq_run, 0);
  int kept = 0;
  for (int k0 = w0; k0 < w1; k0 += 32) {
    // lane: one word; the equals before it in this warp's run
    const int k = k0 + lane;
    uint32_t ms = k < w1 ? (uint32_t)before[k] : 0u;
    const int c = __popc(ms);
    int s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += t;
    }
    int room = ties - (eq_run + s - c);  // equals of this word that still survive
    eq_run += __shfl_sync(0xffffffffu, s, 31);
    if (room < c) {
      uint32_t some = 0;
      for (; room > 0; --room) {
        const uint32_t one = ms & (0u - ms);
        some |= one;
        ms ^= one;
      }
      ms = some;
    }
    if (k < w1) {
      bits[k] |= ms;
      kept += __popc(bits[k]);
    }
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) kept += __shfl_xor_sync(0xffffffffu, kept, m);
  int run = block_scan(lane == 0 ? kept : 0, warp_sums, &all);
  run = __shfl_sync(0xffffffffu, run, 0);
  if (tid == 0) pick[2] = n;
  __syncthreads();
  for (int k0 = w0; k0 < w1; k0 += 32) {
    const int k = k0 + lane;
    const uint32_t m = k < w1 ? bits[k] : 0u;
    int s = __popc(m);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += t;
    }
    if (k < w1) {
      before[k] = run + s - __popc(m);
      if (m != 0xffffffffu) atomicMin(&pick[2], k * 32 + __ffs(~m) - 1);  // the first key that goes
    }
    run += __shfl_sync(0xffffffffu, s, 31);
  }
  if (p.cluster > 1) cluster_sync();
  __syncthreads();

  // ranks before the first gap stay where they are
  const int chunks = p.k_chunks + p.v_chunks;
  const int c0 = (int)((long long)chunks * rank / p.cluster), nc = (int)((long long)chunks * (rank + 1) / p.cluster) - c0;
  for (int k0 = min(pick[2], keep); k0 < keep; k0 += kResolve) {
    const int m = min(kResolve, keep - k0);
    __syncthreads();
    if (tid < m) {
      const int k = k0 + tid;
      int a = 0, z = words;  // the last word with before[word] <= k
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (before[mid] <= k) a = mid; else z = mid;
      }
      uint32_t x = bits[a];
      for (int t = k - before[a]; t > 0; --t) x &= x - 1;
      src_row[tid] = row_of(min(a * 32 + (x ? __ffs(x) - 1 : 0), n - 1));
      dst_row[tid] = row_of(k);
    }
    __syncthreads();
    const int total = m * nc;
    for (int i0 = 0; i0 < total; i0 += kThreads * kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * kThreads + tid;
        if (i < total) {
          const int r = i / nc, c = c0 + i - r * nc;
          v[j] = c < p.k_chunks ? static_cast<const uint4*>(p.k_cache)[src_row[r] * p.k_chunks + c]
                                : static_cast<const uint4*>(p.v_cache)[src_row[r] * p.v_chunks + c - p.k_chunks];
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * kThreads + tid;
        if (i < total) {
          const int r = i / nc, c = c0 + i - r * nc;
          if (c < p.k_chunks) static_cast<uint4*>(p.k_cache)[dst_row[r] * p.k_chunks + c] = v[j];
          else static_cast<uint4*>(p.v_cache)[dst_row[r] * p.v_chunks + c - p.k_chunks] = v[j];
        }
      }
    }
    if (rank == 0) {
      float v = 0.f;
      if (tid < m) v = w[src_row[tid]];
      __syncthreads();
      if (tid < m) w[dst_row[tid]] = v;
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  const long long units = (long long)p.layers * p.batch * p.h_kv;
  const size_t smem = (size_t)p.words * 8;
  const void* k = reinterpret_cast<const void*>(paged_kv_evict_kernel);
  // (the same value for every call: calls of several threads set it side by side)
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictMaxKeys / 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)p.cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {const_cast<EvictParams*>(&p)};
  return cudaLaunchKernelExC(&cfg, k, args);
}

}  // namespace va
