// Eviction from the paged cache by the attention weight that each key has
// received: of request b's kv_len keys, each layer and KV head keeps keep_len
// -- the first `sinks`, the last `recent`, and of those between the largest
// weights, the lower position among equals -- and moves them to the front in
// their order, with their weights.
//
// A unit (layer, request, KV head) belongs to one cluster of CTAs, one where
// there are units enough.  Each CTA holds a slice of the unit's weights as the
// order-preserving integers in shared memory, whole or, where they are too many,
// their upper halves (two CTAs then hold 131,072 keys; with four bytes a key it
// took eight, which did not fit the GPU at a time); where those are too many,
// too, every pass reads the cache.  The weight of the last survivor is found by
// a radix select from the top, by digits of 11, 5, 11 and 5 bits: the CTAs count
// their slices, and each adds up all counts by reading the others' shared
// memory.  Lower halves that are not held are read from the cache again, for the
// few keys that share the upper one.  It ends as soon as all keys that share the
// digits found survive.  (Up to 16,384 keys every CTA holds all weights and counts for itself:
// a meeting of the cluster costs about a microsecond, and a select has up to
// six.)  Then each CTA marks its slice, one bit a key, and every CTA gathers
// all bits and counts them by words, so that the k-th survivor is found by a
// search over the words.
//
// The move is shared by columns: a CTA moves its 16-byte chunks of every
// surviving row, CTA 0 the weights too.  In place: the row of rank k goes to
// position k and comes from a position >= k.  A batch of rows is read, the
// CTA meets, and the batch is written: what it overwrites has a rank no higher
// than its position, so it has been read.  Columns are independent, so only the
// CTA's own threads have to meet.
//
// Bound by the rows' copy (HBM) where rows move, and by the chain of loads and
// meetings of the select where they are few.  On one GB300, every row moving:
// half of up to 8,192 keys of 8 requests, 16 layers, 8 heads of 128 bf16 in 457
// us (6.4 TB/s); a quarter of 131,072 fp8 keys of 2 requests, 4 layers, NHD, in
// 297 us (3.8 TB/s); one request of 4,113 keys, one layer, in 17 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/verify_attn.h"
#include "va_budget.h"
#include "va_device.cuh"
#include "va_kernels.h"

namespace va {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1 << 11;
constexpr int kRanks = 1024;  // most rows of a batch
// Rows' chunks in flight per thread.  One CTA an SM with sixteen of them took the
// copies of 16 layers 458 us and of 131,072 keys 298 us, two CTAs with
// eight, whose loop then spills, in 505 and 411.
constexpr int kBatch = 16;
constexpr int kAhead = 8;   // weights in flight per thread

// Weights as integers in their order: -0 counts as 0, NaN above everything.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}
// shared memory of CTA `rank` of the cluster, at this CTA's address
__device__ __forceinline__ uint32_t remote(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ int4 ld_remote4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// position of the t-th set bit of x (t < popc(x))
__device__ __forceinline__ int nth_bit(uint32_t x, int t) {
  int pos = 0;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const int c = __popc(x & ((1u << w) - 1u));
    if (t >= c) {
      t -= c;
      x >>= w;
      pos += w;
    }
  }
  return pos;
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

__global__ void __launch_bounds__(kThreads, 1) paged_kv_evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t dyn[];
  uint32_t* const bits = dyn;                                  // one bit a key: it survives
  int* const before = reinterpret_cast<int*>(dyn + p.words);   // survivors before each word
  uint32_t* const slice32 = dyn + 2 * p.words;                   // this CTA's weights,
  uint16_t* const slice = reinterpret_cast<uint16_t*>(slice32);  // or their upper halves
  // the counts; later the rows of three batches, from and to
  __shared__ __align__(16) int hist[3][kBins];
  static_assert(2 * kRanks <= kBins, "a batch's rows");
  __shared__ int warp_sums[kWarps], geo[5], pick[3], count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.cluster, rank = blockIdx.x % C;
  const long long unit = blockIdx.x / C;
  const int head = (int)(unit % p.h_kv);
  const int b = (int)(unit / p.h_kv % p.batch), layer = (int)(unit / p.h_kv / p.batch);
  grid_dependency_wait();
  grid_dependents_launch();
  if (tid < 4) {
    const int32_t* const src[4] = {p.kv_indptr + b, p.kv_indptr + b + 1, p.last_page_len + b, p.keep_len + b};
    geo[tid] = *src[tid];
  }
  if (tid < 3) pick[tid] = 0;
  for (int k = tid; k < 2 * kBins; k += kThreads) hist[0][k] = 0;
  __syncthreads();
  const int pg0 = geo[0], npg = geo[1] - pg0, lpl = npg > 0 ? geo[2] : 1;
  const long long len = npg > 0 ? (long long)(npg - 1) * p.page_size + lpl : 0;
  const bool table_ok = npg >= 0 && pg0 >= 0 && lpl >= 1 && lpl <= p.page_size && geo[3] >= 0 && len <= p.max_kv_len;
  const bool first = layer == 0 && head == 0 && rank == 0 && tid == 0;
  const int n = table_ok ? (int)len : 0, keep = min(geo[3], n);
  int bad = 0;
  if (keep < n)
    for (int j = rank * kThreads + tid; j < npg; j += C * kThreads) bad |= (unsigned)p.kv_indices[pg0 + j] >= (unsigned)p.num_pages;
  bad = __syncthreads_or(bad);
  if (C > 1) {
    // The CTAs go on or leave together: each has checked its share of the pages,
    // and all have read the same tables (inputs that are written during the call
    // end it here).
    if (tid == 0) geo[4] = bad;
    cluster_sync();
    int odd = 0;
    if (tid < 5 * C) {
      const int v = (int)ld_remote(remote(smem_u32(geo + tid % 5), tid / 5));
      odd = tid % 5 == 4 ? v : (v != geo[tid % 5]) << 1;
    }
    const int any_bad = __syncthreads_or(odd & 1), differ = __syncthreads_or(odd & 2);
    bad = any_bad;
    if (bad || differ || !table_ok || keep == n) cluster_sync();   // nobody leaves while others read
    if (differ) {
      if (rank == 0 && tid == 0 && p.status) atomicOr(p.status, VA_DEV_BAD_TABLE);
      return;
    }
  }
  if (first) {
    if (p.kv_len_out) p.kv_len_out[b] = table_ok ? (bad ? n : keep) : len >= 0 && len <= 0x7fffffffLL && npg >= 0 ? (int)len : 0;
    if ((bad || !table_ok) && p.status) atomicOr(p.status, table_ok ? VA_DEV_BAD_PAGE : VA_DEV_BAD_TABLE);
  }
  if (!table_ok || bad || keep == n) return;

  // Rows count from the layer's first row of this head (32 bits hold them: a
  // row of K, V and its weight takes 132 bytes at least); a page id that has
  // changed since the check reads page 0.
  const uint32_t slot_rows = p.nhd ? p.h_kv : 1, page_rows = (uint32_t)p.h_kv * p.page_size;
  const long long layer_row = (long long)layer * p.num_pages * page_rows + (p.nhd ? head : (long long)head * p.page_size);
  float* const w = p.key_weights + layer_row;
  auto row_at = [&](int page, int j) -> uint32_t {
    return ((unsigned)page < (unsigned)p.num_pages ? (uint32_t)page : 0u) * page_rows + (uint32_t)(j & (p.page_size - 1)) * slot_rows;
  };
  auto row_of = [&](int j) { return row_at(p.kv_indices[pg0 + (j >> p.log2_page)], j); };

  // the middle [lo, hi) competes for `rest` places; this CTA looks after [s0, s1)
  const int lo = min(p.sinks, keep), hi = n - min(p.recent, keep - lo), rest = keep - lo - (n - hi);
  const bool alone = n <= kEvictAlone || C == 1;
  const int S = alone ? 1 : C, srank = alone ? 0 : rank;
  const int per = evict_slice(n, C), s0 = min(srank * per, n), s1 = min(s0 + per, n);
  const int m0 = max(s0, lo), m1 = min(s1, hi);
  // held whole, by upper halves, or (neither) read from the cache again by every pass
  const int how = evict_held(per, p.slice_cap);
  const bool whole = how == kEvictWhole, held = how == kEvictHalves;
  // the weight of key j as far as `mask` tells: the lower half is only looked at where the upper one is `fixed`'s
  auto weight_at = [&](int j, uint32_t fixed, uint32_t mask) -> uint32_t {
    if (whole) return slice32[j - s0];
    if (held) {
      const uint32_t u = (uint32_t)slice[j - s0] << 16;
      if ((mask & 0xffffu) == 0 || ((u ^ fixed) >> 16) != 0) return u;
    }
    return order_of(w[row_of(j)]);
  };

  // how the last survivor is told from the others: u & mask > fixed survives, `ties` of those with u & mask == fixed too
  uint32_t fixed = 0, mask = 0;
  int want = rest, same_all = 0;
  if (rest > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 16 : pass == 2 ? 5 : 0, nb = pass & 1 ? 32 : kBins;
      int* const h = hist[pass & 1];
      if (pass >= 2) {   // (the counts of two passes before have been read by all: they met in the last one)
        for (int k = tid; k < nb; k += kThreads) h[k] = 0;
        __syncthreads();
      }
      if (pass == 0) {
        for (int j0 = m0 + tid; j0 < m1; j0 += kThreads * kAhead) {
          int page[kAhead];
          float x[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) page[i] = p.kv_indices[pg0 + (min(j0 + i * kThreads, m1 - 1) >> p.log2_page)];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) x[i] = w[row_at(page[i], min(j0 + i * kThreads, m1 - 1))];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int j = j0 + i * kThreads;
            if (j < m1) {
              const uint32_t u = order_of(x[i]);
              if (whole) slice32[j - s0] = u;
              else if (held) slice[j - s0] = (uint16_t)(u >> 16);
              atomicAdd(&h[u >> 21], 1);
            }
          }
        }
      } else {
        auto add = [&](int j) {
          const uint32_t u = weight_at(j, fixed, pass == 1 ? 0xffff0000u : 0xffffffffu);
          if ((u & mask) == fixed) atomicAdd(&h[(u >> shift) & (nb - 1)], 1);
        };
        if (whole) {
#pragma unroll 4
          for (int j = m0 + tid; j < m1; j += kThreads) {
            const uint32_t u = slice32[j - s0];
            if ((u & mask) == fixed) atomicAdd(&h[(u >> shift) & (nb - 1)], 1);
          }
        } else if (held) {
          // eight upper halves at a time; few of them share the digits found
          const uint32_t want16 = fixed >> 16, mask16 = mask >> 16;
          for (int g = (m0 - s0) / 8 + tid; g * 8 < m1 - s0; g += kThreads) {
            const uint4 v = reinterpret_cast<const uint4*>(slice)[g];
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int j = s0 + g * 8 + e;
              if (((u[e / 2] >> (16 * (e & 1))) & mask16) == want16 && j >= m0 && j < m1) add(j);
            }
          }
        } else {
          for (int j = m0 + tid; j < m1; j += kThreads) add(j);
        }
      }
      if (S > 1) cluster_sync();
      __syncthreads();
      // bins from above: thread t holds four, nb - 1 - 4 t ..
      constexpr int kMost = kBins / kThreads;
      static_assert(kMost == 4, "bins of a thread");
      int c[kMost] = {0, 0, 0, 0};
      if (tid * kMost < nb) {
        const int4* const at = reinterpret_cast<const int4*>(h + nb - kMost - tid * kMost);
        int4 v = *at;
        if (S > 1) {
          const uint32_t a = smem_u32(at);
          int4 o[8];   // (all others' counts under way together)
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < S && r != rank) o[r] = ld_remote4(remote(a, r));
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < S && r != rank) v = make_int4(v.x + o[r].x, v.y + o[r].y, v.z + o[r].z, v.w + o[r].w);
        }
        c[0] = v.w;
        c[1] = v.z;
        c[2] = v.y;
        c[3] = v.x;
      }
      const int sum = c[0] + c[1] + c[2] + c[3];
      int all;
      int run = block_scan(sum, warp_sums, &all);
      if (run < want && run + sum >= want) {
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
          if (run < want && run + c[k] >= want) {
            pick[0] = nb - 1 - tid * kMost - k;
            pick[1] = want - run;
            pick[2] = c[k];
          }
          run += c[k];
        }
      }
      __syncthreads();
      fixed |= (uint32_t)pick[0] << shift;
      mask = 0xffffffffu << shift;
      want = pick[1];
      same_all = want == pick[2];   // all that share the digits survive
      if (same_all) break;
      __syncthreads();
    }
  }
  const int ties = want;

  // the slice's bits, in order: a warp takes a run of words
  const int words = (n + 31) >> 5, v0 = s0 >> 5, nv = s1 > s0 ? (s1 + 31) / 32 - v0 : 0;
  const int per_warp = (nv + kWarps - 1) / kWarps;
  const int w0 = v0 + min(warp * per_warp, nv), w1 = v0 + min((warp + 1) * per_warp, nv);
  if (held) {
    // a word a thread: compared by upper halves, the few equal ones with a lower digit by the weight itself
    const uint32_t want16 = fixed >> 16, mask16 = mask >> 16;
    const bool lower = (mask & 0xffffu) != 0;
    for (int k = v0 + tid; k < v0 + nv; k += kThreads) {
      const int j0 = k * 32;
      auto below = [&](int j) { return j <= j0 ? 0u : j >= j0 + 32 ? 0xffffffffu : (1u << (j - j0)) - 1u; };
      const uint32_t mid = rest > 0 ? below(hi) & ~below(lo) : 0u;   // keys that compete
      uint32_t gt = 0, eq = 0;
      if (mid) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 v = reinterpret_cast<const uint4*>(slice + (j0 - s0))[q];
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t x = (u[e / 2] >> (16 * (e & 1))) & mask16;
            gt |= (x > want16 ? 1u : 0u) << (q * 8 + e);
            eq |= (x == want16 ? 1u : 0u) << (q * 8 + e);
          }
        }
        gt &= mid;
        eq &= mid;
        if (lower)
          for (uint32_t left = eq; left; left &= left - 1) {
            const uint32_t one = left & (0u - left), u = order_of(w[row_of(j0 + __ffs(left) - 1)]) & mask;
            if (u > fixed) gt |= one;
            if (u != fixed) eq &= ~one;
          }
      }
      const uint32_t mm = gt | (below(n) & (below(lo) | ~below(hi)));
      bits[k] = same_all ? mm | eq : mm;
      before[k] = (int)eq;   // (until the equals are counted)
    }
  } else {
#pragma unroll 2
    for (int k = w0; k < w1; ++k) {
      const int j = k * 32 + lane;
      const bool mid = j >= lo && j < hi && rest > 0;
      const uint32_t u = mid ? (whole ? slice32[j - s0] : order_of(w[row_of(j)])) & mask : 0u;
      const bool more = j < lo || (j >= hi && j < n) || (mid && u > fixed), same = mid && u == fixed;
      const uint32_t mm = __ballot_sync(0xffffffffu, more), ms = __ballot_sync(0xffffffffu, same);
      if (lane == 0) {
        bits[k] = same_all ? mm | ms : mm;
        before[k] = (int)ms;
      }
    }
  }
  __syncthreads();
  int all;
  if (rest > 0 && !same_all) {
    // some of the equals go: those behind the first `ties` of all slices
    int equal = 0;
    for (int k = w0 + lane; k < w1; k += 32) equal += __popc((uint32_t)before[k]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) equal += __shfl_xor_sync(0xffffffffu, equal, m);
    int run = block_scan(lane == 0 ? equal : 0, warp_sums, &all);
    run = __shfl_sync(0xffffffffu, run, 0);
    if (S > 1) {
      if (tid == 0) count = all;
      cluster_sync();
      for (int r = 0; r < rank; ++r) run += (int)ld_remote(remote(smem_u32(&count), r));
    }
    for (int k0 = w0; k0 < w1; k0 += 32) {
      const int k = k0 + lane;   // lane: one word
      uint32_t ms = k < w1 ? (uint32_t)before[k] : 0u;
      const int c = __popc(ms);
      int s = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
      }
      int room = ties - (run + s - c);   // of this word's equals
      run += __shfl_sync(0xffffffffu, s, 31);
      if (room < c) {
        uint32_t some = 0;
        for (; room > 0; --room) {
          const uint32_t one = ms & (0u - ms);
          some |= one;
          ms ^= one;
        }
        ms = some;
      }
      if (k < w1) bits[k] |= ms;
    }
  }
  __syncthreads();
  if (S > 1) {
    // gather: words of CTA r's slice from its shared memory
    cluster_sync();
    const int words_per = per >> 5;
    for (int k = tid; k < words; k += kThreads)
      if (k < v0 || k >= v0 + nv) bits[k] = ld_remote(remote(smem_u32(bits + k), k / words_per));
    if (tid == 0) pick[2] = n;
    cluster_sync();   // nobody leaves, or moves weights, while others read
  } else {
    if (tid == 0) pick[2] = n;
    if (C > 1) cluster_sync();   // CTA 0 moves weights when all have read them
  }
  __syncthreads();
  {
    const int each = (words + kThreads - 1) / kThreads, k0 = min(tid * each, words), k1 = min(k0 + each, words);
    int sum = 0;
    for (int k = k0; k < k1; ++k) sum += __popc(bits[k]);
    int run = block_scan(sum, warp_sums, &all);
    for (int k = k0; k < k1; ++k) {
      const uint32_t m = bits[k];
      before[k] = run;
      run += __popc(m);
      if (m != 0xffffffffu) {   // the first key that goes
        atomicMin(&pick[2], k * 32 + __ffs(~m) - 1);
        for (++k; k < k1; ++k) {
          before[k] = run;
          run += __popc(bits[k]);
        }
      }
    }
  }
  __syncthreads();

  // ranks before the first gap stay where they are
  const int chunks = p.k_chunks + p.v_chunks;
  const int c0 = chunks * rank / C, nc = chunks * (rank + 1) / C - c0;
  const int par = kThreads / nc, my_r = tid / nc, my_c = c0 + tid - my_r * nc;   // this thread's first row, and its column
  const bool in_k = my_c < p.k_chunks;
  const int stride = in_k ? p.k_chunks : p.v_chunks;
  uint4* const col = (in_k ? static_cast<uint4*>(p.k_cache) + my_c : static_cast<uint4*>(p.v_cache) + (my_c - p.k_chunks)) +
                     layer_row * stride;
  // The rows of ranks k0 .. k0 + kRanks - 1: the last word with before[word] <=
  // k, its bit, the pages.  A list is made while rows of the one before are
  // under way: its positions and page loads before their loads, its rows behind.
  const int rows = min(par * kBatch, kRanks), top = 1 << (31 - __clz(words));
  constexpr int kEach = kRanks / kThreads;
  int pos[kEach], page[kEach], page_to[kEach];
  auto find = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) pos[i] = 0;
#pragma unroll 1
    for (int half = top; half > 0; half >>= 1) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int mid = pos[i] + half;
        if (mid < words && before[mid] <= k0 + tid + i * kThreads) pos[i] = mid;
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = min(k0 + tid + i * kThreads, keep - 1);
      pos[i] = min(pos[i] * 32 + nth_bit(bits[pos[i]], k - before[pos[i]]), n - 1);
      page[i] = p.kv_indices[pg0 + (pos[i] >> p.log2_page)];
      page_to[i] = p.kv_indices[pg0 + (k >> p.log2_page)];
    }
  };
  auto put = [&](int k0, uint32_t* list) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int r = tid + i * kThreads;
      list[r] = row_at(page[i], pos[i]);
      list[kRanks + r] = row_at(page_to[i], k0 + r);
    }
  };
  int k0 = min(pick[2], keep);
  __syncthreads();
  int next = 0;   // list that is made next
  uint32_t* list = reinterpret_cast<uint32_t*>(hist[0]);
  if (k0 < keep) {
    find(k0);
    put(k0, list);
  }
  __syncthreads();
  for (; k0 < keep; k0 += kRanks) {
    next = next == 2 ? 0 : next + 1;
    uint32_t* const list_next = reinterpret_cast<uint32_t*>(hist[next]);
    const int m = min(kRanks, keep - k0);
    const bool more = k0 + kRanks < keep;
    if (more) find(k0 + kRanks);
    for (int r0 = 0; r0 < m; r0 += rows) {
      uint4 v[kBatch];
      float x[kEach];
      const int end = min(m, r0 + rows);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + my_r + i * par;
        if (r < end && my_r < par) v[i] = col[(size_t)list[r] * stride];
      }
      if (rank == 0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int r = r0 + tid + i * kThreads;
          if (r < end) x[i] = w[list[r]];
        }
      }
      if (r0 == 0 && more) put(k0 + kRanks, list_next);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + my_r + i * par;
        if (r < end && my_r < par) col[(size_t)list[kRanks + r] * stride] = v[i];
      }
      if (rank == 0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int r = r0 + tid + i * kThreads;
          if (r < end) w[list[kRanks + r]] = x[i];
        }
      }
    }
    list = list_next;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  const long long units = (long long)p.layers * p.batch * p.h_kv;
  const size_t smem = evict_smem(p.words, p.slice_cap);
  const void* k = reinterpret_cast<const void*>(paged_kv_evict_kernel);
  // (the same value for every call: calls of several threads set it side by side)
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictMaxSmem);
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
