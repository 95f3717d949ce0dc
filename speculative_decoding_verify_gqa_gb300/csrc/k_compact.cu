// Compaction of accepted drafts in the paged cache: after a tree step the
// accepted nodes path[0] < path[1] < ... of request b sit at positions
// prefix + path[k]; the next step expects them at prefix + k.  For every
// layer, KV head and cache, row prefix + k is overwritten with row
// prefix + path[k], front to back.
//
// path[k] >= k and path ascends, so a row written (k) lies at or before every
// row still to be read (path[j] > path[k] >= k for j > k): in place and in
// order is safe, and so is reading a batch of rows before writing them.  A
// thread owns one 16-byte column chunk of all rows of one (layer, cache,
// head), so no two threads touch the same bytes and nothing waits.  The work
// is a copy of a few rows: bound by the chain of dependent reads (tables,
// path, page ids, rows), so a CTA resolves its request's rows once in shared
// memory and then keeps a few row loads in flight per thread.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/verify_attn.h"
#include "va_device.cuh"
#include "va_kernels.h"

namespace va {
namespace {

constexpr int kRows = 128;  // path entries resolved at a time
constexpr int kCtas = 4;    // CTAs an SM holds
constexpr int kBatch = 4;   // rows in flight per thread

__global__ void __launch_bounds__(256, kCtas) paged_kv_compact_kernel(const CompactParams p) {
  __shared__ long long src_row[kRows], dst_row[kRows];  // cache row (of head 0), or -1: nothing to do
  __shared__ int geo[6];
  const int b = blockIdx.y, tid = threadIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  // (read once for the CTA: the barriers below go by them)
  if (tid < 6) {
    const int32_t* const src[6] = {p.qo_indptr + b, p.qo_indptr + b + 1, p.kv_indptr + b, p.kv_indptr + b + 1,
                                   p.last_page_len + b, p.accept_len + b};
    geo[tid] = *src[tid];
  }
  __syncthreads();
  const int o = geo[0], L = geo[1] - o, pg0 = geo[2], npg = geo[3] - pg0;
  const int lpl = npg > 0 ? geo[4] : 1, n = geo[5];
  const long long kv_len = npg > 0 ? (long long)(npg - 1) * p.page_size + lpl : 0;
  const long long pre = kv_len - L;
  const bool table_ok = o >= 0 && L >= 0 && (long long)o + L <= p.total_qo && npg >= 0 && pg0 >= 0 && lpl >= 1 &&
                        lpl <= p.page_size && pre >= 0 && kv_len <= 0x7fffffffLL;
  // the whole path is checked before a row moves
  int bad = !table_ok || n < 0 || n > L;
  if (!bad)
    for (int k = tid; k < n; k += blockDim.x) {
      const int node = p.path[o + k];
      bad |= node >= L || node < k || (k > 0 && p.path[o + k - 1] >= node);
    }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0) {
    if (p.kv_len_out) p.kv_len_out[b] = bad ? (table_ok ? (int)kv_len : 0) : (int)(pre + n);
    if (bad && p.status) atomicOr(p.status, VA_DEV_BAD_TABLE);
  }
  if (bad) return;

  const int per_layer = p.h_kv * (p.k_chunks + p.v_chunks), total = p.layers * per_layer;
  // rows of one page and layer: HND [head][slot], NHD [slot][head]
  const size_t layer_rows = (size_t)p.num_pages * p.h_kv * p.page_size;
  int bad_page = 0;
  for (int k0 = 0; k0 < n; k0 += kRows) {
    const int m = min(kRows, n - k0);
    __syncthreads();
    for (int k = tid; k < m; k += blockDim.x) {
      const int node = p.path[o + k0 + k];
      const long long s = pre + node, d = pre + k0 + k;
      src_row[k] = -1;
      if (s == d || node < 0 || node >= L) continue;   // (checked above, should the path change meanwhile)
      const int ps = p.kv_indices[pg0 + (int)(s >> p.log2_page)], pd = p.kv_indices[pg0 + (int)(d >> p.log2_page)];
      if ((unsigned)ps >= (unsigned)p.num_pages || (unsigned)pd >= (unsigned)p.num_pages) {
        bad_page = 1;
        continue;
      }
      const long long slot_rows = p.nhd ? p.h_kv : 1, page_rows = (long long)p.h_kv * p.page_size;
      dst_row[k] = pd * page_rows + (d & (p.page_size - 1)) * slot_rows;
      src_row[k] = ps * page_rows + (s & (p.page_size - 1)) * slot_rows;
    }
    __syncthreads();
    // this thread's (layer, cache, head, chunk)s: layers outermost
    for (int idx = blockIdx.x * blockDim.x + tid; idx < total; idx += gridDim.x * blockDim.x) {
      const int layer = idx / per_layer, rem = idx - layer * per_layer;
      const bool is_v = rem >= p.h_kv * p.k_chunks;
      const int r2 = is_v ? rem - p.h_kv * p.k_chunks : rem, nch = is_v ? p.v_chunks : p.k_chunks;
      const int head = r2 / nch, ch = r2 - head * nch;
      uint4* base = static_cast<uint4*>(is_v ? p.v_cache : p.k_cache) +
                    ((size_t)layer * layer_rows + (p.nhd ? (size_t)head : (size_t)head * p.page_size)) * nch + ch;
      for (int k = 0; k < m; k += kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (k + j < m && src_row[k + j] >= 0) w[j] = base[src_row[k + j] * nch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (k + j < m && src_row[k + j] >= 0) base[dst_row[k + j] * nch] = w[j];
      }
    }
  }
  if (bad_page && blockIdx.x == 0 && p.status) atomicOr(p.status, VA_DEV_BAD_PAGE);
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  if (p.batch > 65535) return cudaErrorInvalidValue;
  // At most the CTAs that are resident together (kCtas on each SM): every CTA
  // of a request walks the same tables first, and a second wave would do so
  // after the first.
  const long long threads = (long long)p.layers * p.h_kv * (p.k_chunks + p.v_chunks);
  const long long most = std::max(1, kCtas * p.num_sms / p.batch);
  const long long blocks = std::min<long long>((threads + 255) / 256, most);
  void* args[] = {const_cast<CompactParams*>(&p)};
  return launch_kernel(reinterpret_cast<const void*>(paged_kv_compact_kernel),
                       dim3((unsigned)blocks, (unsigned)p.batch), dim3(256), 0, stream, args, /*pdl=*/true);
}

}  // namespace va
