// Kernel parameter blocks and launchers of the operators around a cache that is
// kept within a budget (internal to libverify_attn.so; every pointer is a
// device pointer unless it says otherwise).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace va {

// Norm, rotation and append of new queries, keys and values (see k_qkv_append.cu).
struct QkvParams {
  const void* q;              // bf16 rows of the projection: token i's heads at q + i * q_stride, ...
  const void* k;
  const void* v;
  const void* q_weight;       // nullable [head_dim]: the q heads are normalised
  const void* k_weight;
  const int32_t* append_indptr;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* last_page_len;
  const int32_t* positions;   // [total_new] when rot > 0
  void* q_out;                // [total_new, h_q, D] bf16
  void* k_cache;
  void* v_cache;
  int* status;                // nullable
  int64_t q_stride, k_stride, v_stride;  // elements, multiples of 8
  int64_t total_new;
  int batch, h_q, h_kv, page_size, log2_page, num_pages;
  int head_dim_v;
  int rot;                    // leading elements of a head that are rotated (a multiple of 16; 0: none)
  int interleaved;            // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
  int weight_f32;             // weights fp32 (else bf16)
  int quant;                  // e4m3 cache: stored = e4m3(x / scale)
  int nhd;
  float weight_offset, eps, k_scale, v_scale;
  int per_cta;                // tokens of a CTA (set by the launcher)
  uint64_t turn[64];          // frequency of pair i in turns per position, times 2^64
};
cudaError_t launch_qkv_append(const QkvParams& p, int head_dim, int num_sms, cudaStream_t stream);

// Attention weight received by each cached key (see k_key_weights.cu).
struct KeyWeightParams {
  const void* q;              // [total_qo, h_q, D] bf16
  const void* k_cache;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* last_page_len;
  const int32_t* qo_indptr;
  const uint8_t* mask;        // nullable: causal
  const int32_t* mask_indptr;
  const int32_t* accept_len;  // nullable: only the accepted path's queries and keys
  const int32_t* path;
  const float* lse;           // [total_qo, h_q]
  float* key_weights;         // one fp32 per cache row, in the cache's order of rows
  int* status;                // nullable
  int64_t total_qo;
  int batch, h_q, h_kv, group, page_size, log2_page, num_pages;
  int nhd, mask_full;
  float scale_log2;           // sm_scale * k_scale * log2(e)
  float decay;
  int box;                    // rows of a box of the K map (0: no map, rows are copied one by one)
};
// kmap: the K cache as [page][head][slot][element], boxes of `box` slots of one
// head: 64 bf16 columns with 128-byte swizzle, or whole e4m3 rows.
cudaError_t launch_key_weights(const KeyWeightParams& p, const CUtensorMap& kmap, int head_dim, bool kv_fp8,
                               int num_sms, cudaStream_t stream);

// Eviction of the keys with the least weight (see k_evict.cu).
constexpr int kEvictMaxKeys = 1 << 19;  // keys of a request: a bit and a count per word in shared memory
constexpr int kEvictAlone = 1 << 14;      // keys up to which every CTA ranks all of a unit's weights by itself
constexpr int kEvictMaxCluster = 8;
constexpr int kEvictStatic = 26 * 1024;   // static shared memory of a CTA, and what the system keeps of it
constexpr int kEvictMaxSmem = 227 * 1024 - kEvictStatic;
inline size_t evict_smem(int words, int slice) { return (size_t)words * 8 + (size_t)slice * 2; }
inline int evict_words(int64_t max_kv_len) { return (int)((max_kv_len + 63) / 64 * 2); }   // (what follows them starts on 16 bytes)

// CTAs per unit (layer, request, KV head), `units` of them: twice as many while
// all CTAs still run at a time, one an SM, and every one moves 64 bytes of a
// row of `chunks` 16-byte chunks -- or 32, where most of the GPU would stay idle.
inline int evict_cluster(int64_t units, int chunks, int num_sms) {
  int cluster = 1;
  for (int c = 2; c <= kEvictMaxCluster; c *= 2) {
    if (units * c > num_sms || chunks / c < (units * c * 2 <= num_sms ? 2 : 4)) break;
    cluster = c;
  }
  return cluster;
}
// Weights, two bytes each, that a CTA has room for: whole weights of up to 16,384
// keys; upper halves of as many as shared memory takes.  (Every CTA of a cluster
// ranks a request of up to 16,384 keys for itself.)
inline int evict_slice_cap(int64_t max_kv_len, int cluster) {
  const int64_t n = std::max(((max_kv_len + cluster - 1) / cluster + 31) / 32 * 32,
                             (std::min<int64_t>(max_kv_len, kEvictAlone) + 31) / 32 * 32);
  const int64_t room = ((int64_t)kEvictMaxSmem - (int64_t)evict_smem(evict_words(max_kv_len), 0)) / 64 * 32;
  return (int)std::min(n <= kEvictAlone ? 2 * n : n, room);
}
// Keys of a unit of n that each CTA of its cluster looks after, and how it holds
// their weights: whole, by upper halves, or not at all (every pass reads the cache).
__host__ __device__ inline int evict_slice(int n, int cluster) {
  const int ctas = n <= kEvictAlone ? 1 : cluster;
  return ((n + ctas - 1) / ctas + 31) & ~31;
}
enum { kEvictWhole, kEvictHalves, kEvictReread };
__host__ __device__ inline int evict_held(int slice, int slice_cap) {
  return slice <= slice_cap / 2 ? kEvictWhole : slice <= slice_cap ? kEvictHalves : kEvictReread;
}
struct EvictParams {
  float* key_weights;         // [layers, rows of a layer]
  const int32_t* keep_len;    // [batch]
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* last_page_len;
  void* k_cache;              // [layers, num_pages, ...]
  void* v_cache;
  int32_t* kv_len_out;        // nullable [batch]
  int* status;                // nullable
  int batch, layers, h_kv, page_size, log2_page, num_pages;
  int k_chunks, v_chunks;     // 16-byte chunks of a K / V row
  int nhd, sinks, recent;
  int max_kv_len, words;      // words: of 32 keys, that max_kv_len fills
  int cluster;                // CTAs per (layer, request, KV head)
  int slice_cap;              // weights that a CTA has room for
};
cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);

}  // namespace va
