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
// The product is taken transposed, S = K Q^T on the 5th-generation tensor cores
// (M = 128 keys, N = up to 128 query rows, accumulators in tensor memory): a
// key is a lane of tensor memory, so one thread holds a key and adds up its
// own weight -- the sum never crosses threads, needs no atomics, and its order
// is fixed.  K is read once and V not at all: HBM bounds the step of a serving
// batch, the tensor cores and the SFU's 2^x (one for each pair) a prompt's.
//
// On one GB300: 64 chains of up to 8 tokens behind up to 8,192 keys (64/8 heads,
// bf16) 106 us, 5.7 TB/s;
// 8 trees of 64 nodes behind 32,768 fp8 keys (32/8 heads) 191 us, 720 TFLOP/s;
// 10 prompts of 1,024 tokens (64/8 heads) 123 us, 697 TFLOP/s of visible pairs
// (345 us over an fp8 cache, where the loaders widen every chunk of q, too).
// The latter two wait for the warps that add: 32 rows take them some 500 cycles
// where the SFU needs 256 for the two of a scheduler, and a chunk's hand-offs --
// an mbarrier operation takes some 150 cycles -- come on top.  All roles share
// the instruction caches (87 % of requests hit), so the loops are kept short: the
// look at a mask out of line took the chains from 119 to 116 us, rows that all
// see the keys in a loop of their own the prompts from 131 to 124.
//
// A unit is one or two tiles of 128 keys of one (request, KV head).  One CTA per
// SM, its warps in roles that run through the same units:
//  * one warp walks the schedule: it posts a unit -- its geometry, its places in
//    all rings, the pages of its keys, which arrive by asynchronous copies -- in
//    a queue in shared memory, so that the others' loops stay short;
//  * 4 loader warps bring the tiles of K into the 128-byte-swizzled operand
//    layout: by TMA, a page or 32 slots of one a box, or for pages of fewer than
//    8 slots and tiles with keys of an accepted path row by row, in 16-byte
//    asynchronous copies; and the query rows of 128-row chunks by such copies.
//    e4m3 rows are widened to f16 between a raw buffer and the operand (exact),
//    and bf16 queries with them, as the attention kernels do;
//  * one thread issues tcgen05.mma: for each chunk of rows and tile of keys 4 or
//    8 steps of K = 16 into one of two buffers of the tile, and passes a chunk's
//    products on together;
//  * 4 warps per tile take 2^(s c - lse log2 e) of their lane's columns and add.
// Chunks of a (request, head) of up to 256 rows stay in shared memory from unit
// to unit.  Longer ones (prompts) are streamed, from the first chunk that sees
// the unit's keys on.
//
// Units are dealt in runs of neighbours where rows are few: they cost the same
// bytes, and the beginnings of heads are counted with them.  Where a request has more than 256 rows they are sorted by their number
// of chunks and dealt back and forth over the CTAs, the long ones first.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/verify_attn.h"
#include "va_budget.h"
#include "va_device.cuh"
#include "va_kernels.h"
#include "va_tc.cuh"

namespace va {
namespace {

constexpr int kTile = 128;    // keys of a tile, query rows of a chunk
constexpr int kEpiWarps = 8;  // 4 for each of the unit's tiles
constexpr int kLoadWarp = kEpiWarps, kMmaWarp = kLoadWarp + 4, kWalkWarp = kMmaWarp + 1, kThreads = 32 * (kWalkWarp + 1);
constexpr int kList = 512;    // units (of all heads) that are sorted
constexpr int kResident = 2;  // chunks that stay in shared memory
constexpr int kFlight = 3;    // e4m3: loads under way per loader thread
constexpr int kQueue = 6;     // units posted ahead
constexpr int kDrain = 1024;  // tries for a load under way when the CTA has given up

template <int D, bool FP8>
struct Cfg {
  static constexpr int OP = kTile * D * 2;         // one operand tile: [D / 64 halves][128 rows][128 bytes]
  static constexpr int RAW = FP8 ? kTile * D : 0;  // e4m3 rows as they are
  // Operand slots, the first for tiles of K and the rest for chunks of q: two
  // chunks stay where rows are few; where they are streamed they are what has
  // to come in, and a unit's own tiles are enough of K.
  static constexpr int SLOTS = FP8 ? 5 : 6;
  static constexpr int K_RUNS = SLOTS - kResident, K_SORTED = 2;
  static constexpr int OFF_RAW = SLOTS * OP, OFF_L2 = OFF_RAW + kFlight * RAW, OFF_LIST = OFF_L2 + (SLOTS - K_SORTED) * kTile * 4,
                       OFF_UNIT = OFF_LIST + kList * 8, OFF_PAGE = OFF_UNIT + kQueue * 128,
                       OFF_BAR = OFF_PAGE + kQueue * 2 * kTile * 4, SMEM = OFF_BAR + 512;
  static_assert(SMEM + 1024 <= 227 * 1024, "shared memory");
  static_assert(kList * 12 <= SLOTS * OP, "the unsorted list lies in the operand slots");
};

// Barriers: a slot full / free, products full / free, a unit posted / taken.
enum { B_FULL = 0, B_FREE = 6, B_SF = 12, B_SE = 14, B_UF = 16, B_UE = 22, B_RAW = 28, B_DONE = 31, B_COUNT = 32 };

// A place in a ring of n slots and the parity of its round.
struct Ring {
  int n, slot, round;
  __device__ explicit Ring(int n_, int slot_ = 0, int round_ = 0) : n(n_), slot(slot_), round(round_) {}
  __device__ void step() {
    if (++slot == n) {
      slot = 0;
      ++round;
    }
  }
};

struct Request {
  int o, L, n, pg0;  // first query row, query tokens, those counted, page table
  int pre, keys;     // prefix length, keys weighed (0: nothing to do)
  int rows, chunks;  // n * group query rows, in chunks
  bool bad;
};

__device__ __forceinline__ Request load_request(const KeyWeightParams& p, int b) {
  Request r;
  r.o = p.qo_indptr[b];
  r.L = p.qo_indptr[b + 1] - r.o;
  r.pg0 = p.kv_indptr[b];
  const int npg = p.kv_indptr[b + 1] - r.pg0;
  const int lpl = npg > 0 ? p.last_page_len[b] : 1;
  r.n = p.accept_len ? p.accept_len[b] : r.L;
  const long long len = npg > 0 ? (long long)(npg - 1) * p.page_size + lpl : 0, pre = len - r.L;
  r.bad = r.o < 0 || r.L < 0 || (long long)r.o + r.L > p.total_qo || npg < 0 || r.pg0 < 0 || lpl < 1 ||
          lpl > p.page_size || pre < 0 || len > 0x7fffffffLL - 2 * kTile || r.n < 0 || r.n > r.L ||
          (long long)r.n * p.group > 0x7fffffffLL - kTile;
  r.pre = r.bad ? 0 : (int)pre;
  r.keys = r.bad ? 0 : r.pre + r.n;
  r.rows = r.bad ? 0 : r.n * p.group;
  r.chunks = (r.rows + kTile - 1) / kTile;
  return r;
}

// What the roles share of the schedule.
struct Sched {
  unsigned tiles1, tiles2;            // tiles of 128 keys, units of 256, of all heads, counted as far as it matters
  int most_rows, entries;             // rows of the longest request, units of one head
  int kt;                             // tiles of a unit
  int sorted;                         // units are dealt from the sorted list
  int b0;                             // runs: first request, and units to skip there
  long long off, count;
};

// A unit as it is posted.
struct __align__(16) Unit {
  int nt;                  // tiles (0: no more units)
  int chunks, c0, c1;      // chunks of the request; the first that tile 0 / 1 takes part in
  int flags;               // kBad ..
  int rows, keys, pre;     // of the request, as in Request
  int key0, h, o, L;
  int n, mask_row;         // first bit of the request's mask
  int k_slot, k_round;     // ring places of tile 0 ...
  int k_slot1, k_round1;   // ... and 1,
  int q_slot, q_round;     // of chunk c0,
  int s0;                  // and number of the first products
  int pg0;                 // page table of the request
  int pad[10];
};
static_assert(sizeof(Unit) == 128, "Unit");
enum { kBad = 1, kFresh = 2, kLast = 4 };  // skipped; its chunks are loaded; its chunks' slots are given back

// The walk over the CTA's units; all lanes of the warp take the same steps.
struct Walk {
  const KeyWeightParams& p;
  const Sched& s;
  const int2* list;
  Request rq;
  long long at, left;
  int b, h, tile, tiles;
  int mask0;         // first bit of the request's mask
  bool fresh, last;  // first / last unit of this (request, head) in a row
  bool first;

  __device__ Walk(const KeyWeightParams& p_, const Sched& s_, const int2* l) : p(p_), s(s_), list(l), at(0), left(s_.count), b(-1), h(0), tile(0), tiles(0), mask0(0), first(true) {}

  __device__ void enter(int nb) {
    b = nb;
    mask0 = p.mask ? p.mask_indptr[b] : 0;
    const long long bits = p.mask ? (long long)p.mask_indptr[b + 1] - mask0 : 0;
    rq = load_request(p, b);
    // a mask is read where its offsets say: they span what the attention's plan takes, no other
    if (p.mask && (mask0 < 0 || bits != (long long)rq.L * (p.mask_full ? rq.keys : rq.L))) rq.bad = true;
    if (!rq.bad && p.accept_len) {
      bool bad = false;
      for (int k = threadIdx.x & 31; k < rq.n; k += 32) {
        const int node = p.path[rq.o + k];
        bad |= node >= rq.L || node < k || (k > 0 && p.path[rq.o + k - 1] >= node);
      }
      rq.bad = __any_sync(0xffffffffu, bad);
    }
    if (rq.bad) rq.rows = rq.chunks = 0;   // (its units are walked over)
    const int u = kTile * s.kt;
    tiles = (rq.keys + u - 1) / u;
  }
  __device__ bool next() {
    if (s.sorted) {
      const long long u = at * gridDim.x + ((at & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      ++at;
      if (u >= s.count) return false;
      const int2 e = list[u / p.h_kv];
      h = (int)(u % p.h_kv);
      if (e.x != b) enter(e.x);
      tile = e.y;
      fresh = last = true;
      return true;
    }
    if (left-- <= 0) return false;
    if (first) {
      first = false;
      enter(s.b0);
      if (tiles == 0) return false;   // (tables that change during the call)
      h = (int)(s.off / tiles);
      tile = (int)(s.off % tiles);
      fresh = true;
    } else {
      fresh = false;
      if (++tile == tiles) {
        tile = 0;
        fresh = true;
        if (++h == p.h_kv) {
          h = 0;
          do {
            if (b + 1 >= p.batch) return false;   // (the same)
            enter(b + 1);
          } while (tiles == 0);
        }
      }
    }
    last = tile == tiles - 1 || left == 0;
    return true;
  }
  __device__ int key0() const { return tile * kTile * s.kt; }
  __device__ int tiles_here() const { return min(s.kt, (rq.keys - key0() + kTile - 1) / kTile); }
  __device__ bool resident() const { return rq.chunks <= kResident; }
  // chunks before this one see none of the keys of the unit's tile t
  __device__ int chunk0(int t = 0) const {
    if (resident() || p.mask) return 0;
    return (int)min((long long)max(0, key0() + t * kTile - rq.pre) * p.group / kTile, (long long)rq.chunks);
  }
  // position that key j is read from
  __device__ int source(int j) const {
    return !p.accept_len || j < rq.pre ? j : rq.pre + min(max(p.path[rq.o + j - rq.pre], 0), rq.L - 1);
  }
};

// cache row of KV head h at position pos of a page, or -1 for a page outside the pool
__device__ __forceinline__ long long cache_row(const KeyWeightParams& p, int page, int pos, int h) {
  const long long slot = pos & (p.page_size - 1);
  const long long row = p.nhd ? ((long long)page * p.page_size + slot) * p.h_kv + h
                              : ((long long)page * p.h_kv + h) * p.page_size + slot;
  return (unsigned)page < (unsigned)p.num_pages ? row : -1;
}

__device__ __forceinline__ uint32_t op_addr(uint32_t base, int row, int chunk) {  // of a 16-byte chunk of an operand row
  return base + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// mbar_wait by a whole warp, with one answer
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}
// Wait for the tensor-memory loads under way; the registers pass through, so
// that nothing reads or moves them before.
__device__ __forceinline__ void tmem_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// f16 instruction descriptor: fp32 accumulator, both operands K-major
template <bool FP8>
__device__ __forceinline__ uint32_t idesc_n(int n) {
  return (1u << 4) | (FP8 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

// D[tmem] = A B^T, K = D, from shared-memory descriptors of the operands' first
// 16 columns: the next 16 lie 32 bytes on, the second 64 a half tile.
template <int D>
__device__ __forceinline__ void mma_tile(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
  constexpr int kHalf = kTile * 128 / 16;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n setp.ne.b32 p, %3, %3;\n"
      " add.s64 a1, %1, 2;\n add.s64 b1, %2, 2;\n add.s64 a2, %1, 4;\n add.s64 b2, %2, 4;\n"
      " add.s64 a3, %1, 6;\n add.s64 b3, %2, 6;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id)
      : "memory");
  if constexpr (D == 128)
    asm volatile(
        "{\n .reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n"
        " add.s64 a0, %1, %4;\n add.s64 b0, %2, %4;\n add.s64 a1, a0, 2;\n add.s64 b1, b0, 2;\n"
        " add.s64 a2, a0, 4;\n add.s64 b2, b0, 4;\n add.s64 a3, a0, 6;\n add.s64 b3, b0, 6;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %3, 1;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "n"(kHalf)
        : "memory");
}

// which of 32 query rows from `row` on see the key by the mask, bit row0 + token * width (out of line: rarely called)
__device__ __noinline__ uint32_t mask_bits(const uint8_t* mask, long long row0, int width, int row, int group, int n) {
  uint32_t on = 0;
  for (int tok = row / group, e = tok * group - row; e < 32 && tok < n; ++tok, e += group) {
    const long long bit = row0 + (long long)tok * width;
    if ((mask[bit >> 3] >> (bit & 7)) & 1) {   // rows e .. e + group - 1, those among the 32
      const int z = min(e + group, 32);
      on |= (z == 32 ? 0xffffffffu : (1u << z) - 1u) & (0xffffffffu << max(e, 0));
    }
  }
  return on;
}

// A warp's rows of a chunk of q that count nothing (`out`: this lane's own row)
// become 0: 2^(s c - lse log2 e) is 0 for lse = -inf where s is finite, and NaN
// where such a row holds NaN or infinity.  Behind the copies, which so need not
// wait for lse, and out of line: rarely called.
template <int QCH>
__device__ __noinline__ void leave_out(uint32_t base, int own, bool out) {
  cp_async_wait_all();
  __syncwarp();
  if (out)
#pragma unroll 1
    for (int ch = 0; ch < QCH; ++ch) sts128(op_addr(base, own, ch), make_uint4(0, 0, 0, 0));
  __syncwarp();
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    verify_attn_key_weights_kernel(const KeyWeightParams p, const __grid_constant__ CUtensorMap kmap) {
  using C = Cfg<D, FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Sched sched;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_shared;
  volatile int* const abort_flag = &abort_shared;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem), bars = sbase + C::OFF_BAR;
  auto bar = [&](int i) { return bars + 8 * i; };
  float* const l2s = reinterpret_cast<float*>(smem + C::OFF_L2);
  int2* const list = reinterpret_cast<int2*>(smem + C::OFF_LIST);

  if (tid == 0) {
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(bar(B_UF + i), 32 + 1);
      mbar_init(bar(B_UE + i), kEpiWarps + 4 + 1);
    }
    for (int i = 0; i < kFlight; ++i) mbar_init(bar(B_RAW + i), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_SF + i), 1);
      mbar_init(bar(B_SE + i), kEpiWarps);
    }
    mbar_init(bar(B_DONE), 1);
    abort_shared = 0;
    sched.tiles1 = sched.tiles2 = 0;
    sched.most_rows = sched.entries = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&tmem_slot), 512);
  grid_dependency_wait();
  grid_dependents_launch();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // ---- the schedule ----
  for (int b = tid; b < p.batch; b += kThreads) {
    const Request rq = load_request(p, b);
    if (rq.bad && blockIdx.x == 0 && p.status) atomicOr(p.status, VA_DEV_BAD_TABLE);
    if (rq.keys == 0) continue;
    const int one = (rq.keys + kTile - 1) / kTile, two = (one + 1) / 2;
    // (65,535 requests at most: 32 bits hold the sums)
    atomicAdd(&sched.tiles1, (unsigned)min((long long)one * p.h_kv, 65536ll));
    atomicAdd(&sched.tiles2, (unsigned)min((long long)two * p.h_kv, 65536ll));
    atomicMax(&sched.most_rows, rq.rows);
    atomicAdd(&sched.entries, min(two, kList + 1));
  }
  __syncthreads();
  const unsigned most = min(gridDim.x, 65535u);
  const int kt = sched.tiles1 <= most ? 1 : 2;
  const bool sorted = kt == 2 && sched.most_rows > kResident * kTile && sched.entries <= kList;
  if (sorted) {
    // rank = units with more chunks, or as many and listed before
    int* const cost = reinterpret_cast<int*>(smem);
    int2* const unit = reinterpret_cast<int2*>(smem + kList * 4);
    __syncthreads();
    if (tid == 0) sched.entries = 0;
    __syncthreads();
    for (int b = tid; b < p.batch; b += kThreads) {
      const Request rq = load_request(p, b);
      const int n = (rq.keys + 2 * kTile - 1) / (2 * kTile);
      if (n == 0) continue;
      const int first = atomicAdd(&sched.entries, n);
      for (int i = 0; i < n && first + i < kList; ++i) {
        const int skip = p.mask || rq.chunks <= kResident ? 0 : (int)((long long)max(0, i * 2 * kTile - rq.pre) * p.group / kTile);
        cost[first + i] = max(0, rq.chunks - skip);
        unit[first + i] = make_int2(b, i);
      }
    }
    __syncthreads();
    const int n = min(sched.entries, kList);
    for (int i = tid; i < n; i += kThreads) {
      const int c = cost[i];
      const int2 u = unit[i];
      int rank = 0;
      for (int k = 0; k < n; ++k) {
        // equals by request and tile: the atomics' order differs from CTA to CTA
        const int2 v = unit[k];
        rank += cost[k] > c || (cost[k] == c && (v.x < u.x || (v.x == u.x && v.y < u.y)));
      }
      list[rank] = u;
    }
  }
  if (warp == 0) {
    long long first = -1, end = 0;   // this CTA's units
    const unsigned all = kt == 1 ? sched.tiles1 : sched.tiles2;
    if (!sorted && all <= most) {
      // one at most
      const int at = blockIdx.x;
      end = at + 1;
      for (int b0 = 0, run = 0; b0 < p.batch && at < (int)all; b0 += 32) {
        int units = 0;
        if (b0 + lane < p.batch) units = (load_request(p, b0 + lane).keys + kTile * kt - 1) / (kTile * kt) * p.h_kv;
        int sum = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += t;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, run + sum > at);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            sched.b0 = b0 + lane;
            sched.off = at - (run + sum - units);
          }
          first = at;
          break;
        }
        run += __shfl_sync(0xffffffffu, sum, 31);
      }
    } else if (!sorted) {
      // units, and their cost by halves of a unit: two for a unit, and one for each chunk that is loaded when a
      // request's head begins (64 chains, 2 to 17 beginnings a CTA: 115 -> 106 us)
      long long total = 0, cost = 0;
      for (int b = lane; b < p.batch; b += 32) {
        const Request rq = load_request(p, b);
        const long long units = (rq.keys + 2 * kTile - 1) / (2 * kTile);
        total += units * p.h_kv;
        cost += (2 * units + (units ? min(rq.chunks, kResident) : 0)) * p.h_kv;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        cost += __shfl_xor_sync(0xffffffffu, cost, o);
      }
      // Runs of equal cost.  Unit i of a head lies at half `loads` + 2 i + 1 of its cost and belongs to the run that
      // this half lies in.
      const long long lo = cost * blockIdx.x / gridDim.x, hi = cost * (blockIdx.x + 1) / gridDim.x;
      long long run = 0, before = 0;   // cost and units before the 32 requests
      end = total;
      if (lo < hi)
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
          long long units = 0, each = 0, loads = 0;   // of a head; its cost
          if (b0 + lane < p.batch) {
            const Request rq = load_request(p, b0 + lane);
            units = (rq.keys + 2 * kTile - 1) / (2 * kTile);
            loads = units == 0 ? 0 : min(rq.chunks, kResident);
            each = 2 * units + loads;
          }
          long long sum = each * p.h_kv, tiles = units * p.h_kv;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, sum, o), v = __shfl_up_sync(0xffffffffu, tiles, o);
            if (lane >= o) {
              sum += t;
              tiles += v;
            }
          }
          // units before half x of the cost, of this lane's request
          auto units_before = [&](long long x) {
            const long long at = x - (run + sum - each * p.h_kv), h = at / each;
            return h * units + max(0ll, at - h * each - loads) / 2;
          };
          const uint32_t hit_lo = first < 0 ? __ballot_sync(0xffffffffu, run + sum > lo) : 0u;
          if (hit_lo) {
            const int from = __ffs(hit_lo) - 1;
            if (lane == from) {
              sched.b0 = b0 + lane;
              sched.off = units_before(lo);
              first = before + tiles - units * p.h_kv + sched.off;
            }
            first = __shfl_sync(0xffffffffu, first, from);
          }
          const uint32_t hit_hi = __ballot_sync(0xffffffffu, run + sum > hi);
          if (hit_hi) {
            const int from = __ffs(hit_hi) - 1;
            if (lane == from) end = before + tiles - units * p.h_kv + units_before(hi);
            end = __shfl_sync(0xffffffffu, end, from);
            break;
          }
          run += __shfl_sync(0xffffffffu, sum, 31);
          before += __shfl_sync(0xffffffffu, tiles, 31);
        }
    }
    if (lane == 0) {
      // Full: each loader warp's own arrival, for what it has stored (a chunk's
      // lse, widened rows) and behind the asynchronous ones of its copies.
      // A chunk's slot is free when its products are done and the sums' warps
      // have read its lse.
      for (int i = 0; i < C::SLOTS; ++i) {
        const bool k = i < (sorted ? C::K_SORTED : C::K_RUNS);
        mbar_init(bar(B_FULL + i), 4);
        mbar_init(bar(B_FREE + i), k ? 1 : 1 + kEpiWarps);
      }
      mbar_fence_init();
      sched.kt = kt;
      sched.sorted = sorted;
      sched.count = sorted ? (long long)min(sched.entries, kList) * p.h_kv : first < 0 ? 0 : end - first;
    }
  }
  __syncthreads();

  const int nk = sorted ? C::K_SORTED : C::K_RUNS, nq = C::SLOTS - nk;
  Unit* const units = reinterpret_cast<Unit*>(smem + C::OFF_UNIT);
  int* const unit_pages = reinterpret_cast<int*>(smem + C::OFF_PAGE);   // page of each key of a unit
  Ring ur(kQueue);   // this role's place in the queue
  bool live = true;

  if (warp == kWalkWarp) {
    // ---------------- the walk ----------------
    Walk w(p, sched, list);
    Ring kr(nk), qr(nq), hold(nq);
    int sn = 0;
    while (live) {
      const bool more = w.next();
      const Request& rq = w.rq;
      if (more && rq.bad && lane == 0 && p.status) atomicOr(p.status, VA_DEV_BAD_TABLE);
      if (ur.round > 0) live = warp_wait(bar(B_UE + ur.slot), (ur.round - 1) & 1, abort_flag);
      if (!live) break;
      const int key0 = more ? w.key0() : 0, nt = more ? w.tiles_here() : 0;
      if (more && !rq.bad) {
        // the pages of the unit's keys arrive by themselves: a load would take its turn behind all of the SM's copies
        const bool moved = p.accept_len && key0 + 2 * kTile > rq.pre;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= 4 * sched.kt) break;
          const int j = min(key0 + i * 32 + lane, rq.keys - 1), src = moved ? w.source(j) : j;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                           sbase + C::OFF_PAGE + (ur.slot * 2 * kTile + i * 32 + lane) * 4),
                       "l"(p.kv_indices + rq.pg0 + (src >> p.log2_page)));
        }
      }
      if (lane == 0) {
        Unit u;
        u.nt = nt;
        if (more) {
          u.chunks = rq.chunks;
          u.c0 = w.chunk0();
          u.c1 = nt == 2 ? w.chunk0(1) : rq.chunks;
          u.flags = (rq.bad ? kBad : 0) | (w.fresh || !w.resident() ? kFresh : 0) | (w.last || !w.resident() ? kLast : 0);
          u.rows = rq.rows;
          u.keys = rq.keys;
          u.pre = rq.pre;
          u.key0 = key0;
          u.h = w.h;
          u.o = rq.o;
          u.L = rq.L;
          u.pg0 = rq.pg0;
          u.n = rq.n;
          u.mask_row = w.mask0;
          if (rq.chunks > 0) {
            u.k_slot = kr.slot;
            u.k_round = kr.round;
            kr.step();
            u.k_slot1 = kr.slot;
            u.k_round1 = kr.round;
            if (nt == 2) kr.step();
            if (u.flags & kFresh) {
              hold = qr;
              for (int c = u.c0; c < rq.chunks; ++c) qr.step();
            }
            u.q_slot = hold.slot;
            u.q_round = hold.round;
            u.s0 = sn;
            sn += rq.chunks - u.c0;
          }
        }
        units[ur.slot] = u;
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(B_UF + ur.slot)) : "memory");
      if (lane == 0) mbar_arrive(bar(B_UF + ur.slot));
      ur.step();
      if (!more) break;
    }
    cp_async_wait_all();
  } else if (warp < kEpiWarps) {
    // ---------------- weights: one thread per key ----------------
    const int t = warp >> 2, slot = (warp & 3) * 32 + lane;
    const uint32_t cols = tmem + t * 256 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint64_t scale = f32x2(p.scale_log2, p.scale_log2);
    long long late = -1;
    float late_old = 0.f, late_sum = 0.f;
    while (live) {
      live = warp_wait(bar(B_UF + ur.slot), ur.round & 1, abort_flag);
      if (!live) break;
      const Unit u = units[ur.slot];
      int page = unit_pages[ur.slot * 2 * kTile + t * kTile + slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_UE + ur.slot));
      ur.step();
      if (u.nt == 0) break;
      if (u.flags & kBad) continue;
      const int j = u.key0 + t * kTile + slot;
      const bool mine = t < u.nt && j < u.keys;
      const int draft = j - u.pre, border = draft - lane;   // the warp's first key among the step's own
      long long dst = -1;
      float old = 0.f;
      if (mine) {
        bool ok = (unsigned)page < (unsigned)p.num_pages;
        // a key of the path is read from its node's slot and weighed in the one that it moves to
        if (p.accept_len && draft >= 0) page = p.kv_indices[u.pg0 + (j >> p.log2_page)];
        dst = cache_row(p, page, j, u.h);
        if (!ok) dst = -1;
        if (dst < 0 && p.status) atomicOr(p.status, VA_DEV_BAD_PAGE);
        if (dst >= 0 && draft < 0 && p.decay != 0.f) old = p.key_weights[dst];
      }
      float sum = 0.f;
      Ring qr(nq, u.q_slot, u.q_round);
      int product = u.s0;
      const int c_mine = t < u.nt ? (t == 0 ? u.c0 : u.c1) : u.chunks;
      for (int c = u.c0; c < u.chunks; ++c) {
        // the chunk's lse are there, and the products; a warp whose tile skips the chunk keeps in step
        const int qs = qr.slot, buf = product & 1;
        const uint32_t bq = bar(B_FULL + nk + qs), bs = bar(B_SF + buf);
        const uint32_t pq = qr.round & 1, ps = (product >> 1) & 1;
        // (both at once: each takes a few hundred cycles to answer)
        const bool hit_q = mbar_try_wait(bq, pq), hit_s = mbar_try_wait(bs, ps);
        if (!__all_sync(0xffffffffu, hit_q && hit_s)) {
          live = warp_wait(bq, pq, abort_flag);
          if (live) live = warp_wait(bs, ps, abort_flag);
        }
        qr.step();
        if (!live) break;
        ++product;
        if (c >= c_mine) {
          tc_fence_after();
          const int r0 = c * kTile, nr = min(kTile, u.rows - r0);
          // of the chunk's rows, those before `from` see none of the warp's keys, those from `vis` on all of them
          int from = 0, vis = 0;
          if (p.mask) {
            if (p.mask_full || border + 31 >= 0) vis = kTile;
          } else {
            from = min(max(max(border, -64) * p.group - r0, 0), kTile) & ~31;
            vis = max(max(border + 31, -64) * p.group - r0, 0);
          }
          const uint32_t at = cols + buf * kTile;
          const float* const l2 = l2s + qs * kTile;
          uint64_t acc0 = 0, acc1 = 0;
          // four logits: 2^(s c - lse log2 e)
          auto add4 = [&](const uint32_t* x, int k, bool o0, bool o1, bool o2, bool o3) {
            const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(l2 + k);
            const uint64_t a = fma_f32x2(f32x2(__uint_as_float(x[0]), __uint_as_float(x[1])), scale, l.x);
            const uint64_t b = fma_f32x2(f32x2(__uint_as_float(x[2]), __uint_as_float(x[3])), scale, l.y);
            acc0 = add_f32x2(acc0, f32x2(o0 ? ex2(f32x2_lo(a)) : 0.f, o1 ? ex2(f32x2_hi(a)) : 0.f));
            acc1 = add_f32x2(acc1, f32x2(o2 ? ex2(f32x2_lo(b)) : 0.f, o3 ? ex2(f32x2_hi(b)) : 0.f));
          };
          // 32 rows at a time: those that all see the warp's keys, then the others
          const int k0 = min(max(from, (vis + 31) & ~31), nr), k1 = max(k0, nr & ~31);
#pragma unroll 1
          for (int k = k0; k < k1; k += 32) {
            uint32_t x[32];
            tmem_ld32(at + k, x);
            tmem_wait32(x);
#pragma unroll
            for (int i = 0; i < 32; i += 4) add4(x + i, k + i, true, true, true, true);
          }
          for (int k = from == k0 ? k1 : from; k < nr; k = k + 32 == k0 ? k1 : k + 32) {
            // which of the 32 rows see the key: up to the chunk's end, from the causal border on, or by the mask
            uint32_t x[32];
            tmem_ld32(at + k, x);
            uint32_t on = 0xffffffffu;
            if (k < vis) {
              const int row = r0 + k;
              if (!p.mask || (!p.mask_full && draft < 0)) {
                const int lo = draft * p.group - row;
                on = lo >= 32 ? 0u : on << max(lo, 0);
              } else {
                on = 0;
                if (mine) {
                  const long long row0 = u.mask_row + (p.mask_full ? j : draft);
                  const int width = p.mask_full ? u.keys : u.L;
                  on = mask_bits(p.mask, row0, width, row, p.group, u.n);
                }
              }
            }
            if (nr - k < 32) on &= (1u << (nr - k)) - 1u;
            tmem_wait32(x);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              add4(x + i, k + i, on & (1u << i), on & (2u << i), on & (4u << i), on & (8u << i));
          }
          tc_fence_before();
          acc0 = add_f32x2(acc0, acc1);
          sum += f32x2_lo(acc0) + f32x2_hi(acc0);
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_SE + buf));
          if (u.flags & kLast) mbar_arrive(bar(B_FREE + nk + qs));   // the chunk's lse have been read
        }
      }
      // the store of the unit before, whose old weight has had this unit's time to arrive
      if (late >= 0) p.key_weights[late] = fmaf(p.decay, late_old, late_sum);
      late = live ? dst : -1;
      late_old = old;
      late_sum = sum;
    }
    if (late >= 0) p.key_weights[late] = fmaf(p.decay, late_old, late_sum);
    tc_fence_before();
  } else if (warp < kMmaWarp) {
    // ---------------- loads ----------------
    constexpr int KCH = (FP8 ? D : 2 * D) / 16, QCH = 2 * D / 16;  // 16-byte chunks of a row
    const int lw = warp - kLoadWarp, own = lw * 32 + lane;          // this thread's row of a chunk
    int p0 = 0, p1 = 0, p2 = 0, np = 0;  // e4m3: loads under way, the oldest first: 0: K, 8 and its slot: a chunk of q
    Ring rr(FP8 ? kFlight : nk);         // the next load's buffer: raw, or the tile's slot
    Ring rf(kFlight);                    // e4m3: the raw buffer that is widened next
    Ring kf(nk);                         // the K slot that is widened into next
    // e4m3: the oldest load has landed: widen it, and pass it on
    auto finish = [&]() {
      int slot = p0 & 7;
      const bool is_q = p0 & 8;
      p0 = p1;
      p1 = p2;
      --np;
      if (is_q) {
        cp_async_wait_all();
        const uint32_t base = sbase + slot * C::OP;
#pragma unroll
        for (int s = 0; s < QCH; ++s) {
          const uint32_t a = op_addr(base, lw * 32 + s * (32 / QCH) + lane / QCH, lane % QCH);
          uint4 v = lds128(a);
          v.x = bf16x2_to_f16x2(v.x);
          v.y = bf16x2_to_f16x2(v.y);
          v.z = bf16x2_to_f16x2(v.z);
          v.w = bf16x2_to_f16x2(v.w);
          sts128(a, v);
        }
      } else {
        slot = kf.slot;
        live = warp_wait(bar(B_RAW + rf.slot), rf.round & 1, abort_flag);
        if (!live) return;
        if (kf.round > 0 && !warp_wait(bar(B_FREE + slot), (kf.round - 1) & 1, abort_flag)) {
          live = false;
          return;
        }
        kf.step();
        const uint32_t raw = sbase + C::OFF_RAW + rf.slot * C::RAW, base = sbase + slot * C::OP;
        rf.step();
        uint4 raws[KCH];   // (all loads first)
#pragma unroll
        for (int s = 0; s < KCH; ++s)
          raws[s] = lds128(raw + (lw * 32 + s * (32 / KCH) + lane / KCH) * D + ((lane % KCH) << 4));
#pragma unroll
        for (int s = 0; s < KCH; ++s) {
          const int row = lw * 32 + s * (32 / KCH) + lane / KCH, ch = lane % KCH;
          const uint4 v = raws[s];
          sts128(op_addr(base, row, 2 * ch), make_uint4(e4m3x2_to_f16x2((uint16_t)v.x), e4m3x2_to_f16x2((uint16_t)(v.x >> 16)),
                                                        e4m3x2_to_f16x2((uint16_t)v.y), e4m3x2_to_f16x2((uint16_t)(v.y >> 16))));
          sts128(op_addr(base, row, 2 * ch + 1), make_uint4(e4m3x2_to_f16x2((uint16_t)v.z), e4m3x2_to_f16x2((uint16_t)(v.z >> 16)),
                                                            e4m3x2_to_f16x2((uint16_t)v.w), e4m3x2_to_f16x2((uint16_t)(v.w >> 16))));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_FULL + slot));
    };
    // e4m3: room for one more load under way
    auto room = [&]() {
      if constexpr (FP8)
        if (np == kFlight) finish();
    };
    // wait for a buffer to be free: what its readers may wait for is passed on meanwhile
    auto wait_free = [&](uint32_t b, uint32_t parity) {
      if constexpr (FP8)
        while (live && np > 0 && !__all_sync(0xffffffffu, mbar_try_wait(b, parity))) finish();
      if (live) live = warp_wait(b, parity, abort_flag);
    };
    // e4m3: one more load under way
    auto put = [&](int what) {
      if (np == 0) p0 = what;
      else if (np == 1) p1 = what;
      else p2 = what;
      ++np;
    };
    // the warp's arrival behind the asynchronous ones of its copies so far
    auto arrive_behind = [&](uint32_t b) {
      asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(b) : "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    const uint8_t* const kbase = static_cast<const uint8_t*>(p.k_cache) + (lane % KCH) * 16;
    const uint8_t* const qbase = static_cast<const uint8_t*>(p.q) + (lane % QCH) * 16;
    while (live) {
      // (posted units may be awaited for longer than the loads under way: pass those on first)
      wait_free(bar(B_UF + ur.slot), ur.round & 1);
      if (!live) break;
      const Unit u = units[ur.slot];
      const int done = ur.slot;
      ur.step();
      if (u.nt > 0 && u.chunks > 0) {
        for (int t = 0; t < u.nt && live; ++t) {
          room();
          if constexpr (!FP8)
            if (live && rr.round > 0) wait_free(bar(B_FREE + rr.slot), (rr.round - 1) & 1);
          if (!live) break;
          const uint32_t base = sbase + (FP8 ? C::OFF_RAW + rr.slot * C::RAW : rr.slot * C::OP);
          const uint32_t full = bar((FP8 ? B_RAW : B_FULL) + rr.slot);
          const int tile0 = u.key0 + t * kTile;
          const int* const pages = unit_pages + done * 2 * kTile + t * kTile + lw * 32;
          const bool moved = p.accept_len && tile0 + kTile > u.pre;
          if (p.box > 0 && !moved) {
            // whole pages, or 32 rows of one: lane i copies the box of rows i * box ..
            const int r = lane * p.box, j = tile0 + lw * 32 + r;
            const int page = lane * p.box < 32 && j < u.keys ? pages[r] : -1;
            const bool on = (unsigned)page < (unsigned)p.num_pages;   // (the others: whatever the buffer holds stays in its own lane)
            const int n = __popc(__ballot_sync(0xffffffffu, on));
            if (lane == 0) {
              if (n > 0) mbar_expect_tx(full, n * p.box * (FP8 ? D : 2 * D));
              else mbar_arrive(full);
            }
            __syncwarp();
            if (on) {
              const int at = j & (p.page_size - 1), row = lw * 32 + r;
              if constexpr (FP8) {
                tma_load_4d(base + row * D, &kmap, 0, at, u.h, page, full);
              } else {
                tma_load_4d(base + row * 128, &kmap, 0, at, u.h, page, full);
                if constexpr (D == 128) tma_load_4d(base + kTile * 128 + row * 128, &kmap, 64, at, u.h, page, full);
              }
            }
          } else {
#pragma unroll 4
            for (int s = 0; s < KCH; ++s) {
              const int i = s * (32 / KCH) + lane / KCH, r = lw * 32 + i, j = tile0 + r, ch = lane % KCH;
              if (j < u.keys) {
                const int src = moved && j >= u.pre ? u.pre + min(max(p.path[u.o + j - u.pre], 0), u.L - 1) : j;
                const long long k = cache_row(p, pages[i], src, u.h);
                if (k >= 0) cp_async_16(FP8 ? base + r * D + (ch << 4) : op_addr(base, r, ch), kbase + k * (KCH * 16), 16);
              }
            }
            arrive_behind(full);
          }
          if constexpr (FP8) put(0);
          rr.step();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_UE + done));
      if (u.nt == 0) break;
      if (!live || u.chunks == 0 || !(u.flags & kFresh)) continue;
      // row c of the chunks and its lse, one chunk ahead
      auto q_row = [&](int c) -> long long {
        const int r = c * kTile + own;
        if (r >= u.rows) return -1;
        const int tok = r / p.group, g = r - tok * p.group;
        const int node = p.accept_len ? min(max(p.path[u.o + tok], 0), u.L - 1) : tok;
        return (long long)(u.o + node) * p.h_q + u.h * p.group + g;
      };
      Ring qr(nq, u.q_slot, u.q_round);
      long long qrow = q_row(u.c0);
      float lse = qrow >= 0 ? p.lse[qrow] : -INFINITY;
      for (int c = u.c0; c < u.chunks && live; ++c) {
        const long long qnext = c + 1 < u.chunks ? q_row(c + 1) : -1;
        const float lnext = qnext >= 0 ? p.lse[qnext] : -INFINITY;
        room();
        if (live && qr.round > 0) wait_free(bar(B_FREE + nk + qr.slot), (qr.round - 1) & 1);
        if (!live) break;
        const uint32_t base = sbase + (nk + qr.slot) * C::OP;
#pragma unroll
        for (int s = 0; s < QCH; ++s) {
          const int from = s * (32 / QCH) + lane / QCH;
          const long long k = __shfl_sync(0xffffffffu, qrow, from);
          cp_async_16(op_addr(base, lw * 32 + from, lane % QCH), qbase + max(k, 0ll) * (QCH * 16), k >= 0 ? 16 : 0);
        }
        // rows past the end, and rows that saw nothing, count nothing
        l2s[qr.slot * kTile + own] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
        const bool out = qrow >= 0 && lse == -INFINITY;
        if (__any_sync(0xffffffffu, out)) leave_out<QCH>(base, own, out);
        if constexpr (FP8) put(8 | (nk + qr.slot));
        else arrive_behind(bar(B_FULL + nk + qr.slot));
        qr.step();
        qrow = qnext;
        lse = lnext;
      }
    }
    if constexpr (FP8)
      while (np > 0 && live) finish();
    cp_async_wait_all();
    if (!live)   // given up: nothing may still be on its way into the CTA's shared memory
      for (int i = 0; i < rr.n; ++i) {   // (every buffer's last load)
        const int round = i < rr.slot ? rr.round : rr.round - 1;
        for (int k = 0; k < kDrain && round >= 0 && !mbar_try_wait(bar((FP8 ? B_RAW : B_FULL) + i), round & 1); ++k) {}
      }
  } else if (lane == 0) {
    // ---------------- products: one thread ----------------
    const uint64_t desc0 = smem_desc_sw128(0, 16, 1024);
    bool issued = false;
    while (live) {
      live = mbar_wait(bar(B_UF + ur.slot), ur.round & 1, abort_flag);
      if (!live) break;
      const Unit& un = units[ur.slot];
      const int nt = un.nt, chunks = un.chunks, c0 = un.c0, c1 = un.c1, rows = un.rows;
      const bool last = un.flags & kLast;
      const int ks[2] = {un.k_slot, un.k_slot1}, kround[2] = {un.k_round, un.k_round1};
      int sn = un.s0;
      Ring qr(nq, un.q_slot, un.q_round);
      mbar_arrive(bar(B_UE + ur.slot));
      ur.step();
      if (nt == 0) break;
      for (int c = c0; live && c < chunks; ++c, ++sn) {
        const int qs = nk + qr.slot, buf = sn & 1;
        live = mbar_wait(bar(B_FULL + qs), qr.round & 1, abort_flag);
        qr.step();
        if (live && c == c0) live = mbar_wait(bar(B_FULL + ks[0]), kround[0] & 1, abort_flag);
        if (live && c == c1 && nt == 2) live = mbar_wait(bar(B_FULL + ks[1]), kround[1] & 1, abort_flag);
        if (live && sn >= 2) live = mbar_wait(bar(B_SE + buf), ((sn >> 1) - 1) & 1, abort_flag);
        if (!live) break;
        tc_fence_after();
        // what the copies and the loaders' stores left is there for the tensor cores: the fence stands here and not
        // with the loaders, where it would wait for all their copies under way
        fence_proxy_async();
        const uint32_t id = idesc_n<FP8>((min(kTile, rows - c * kTile) + 15) & ~15);
        const uint64_t qd = desc0 + (uint64_t)((sbase + qs * C::OP) >> 4);
        mma_tile<D>(tmem + buf * kTile, desc0 + (uint64_t)((sbase + ks[0] * C::OP) >> 4), qd, id);
        if (nt == 2 && c >= c1)
          mma_tile<D>(tmem + 256 + buf * kTile, desc0 + (uint64_t)((sbase + ks[1] * C::OP) >> 4), qd, id);
        umma_commit(bar(B_SF + buf));
        if (last) umma_commit(bar(B_FREE + qs));
        if (c == chunks - 1) {
          umma_commit(bar(B_FREE + ks[0]));
          if (nt == 2) umma_commit(bar(B_FREE + ks[1]));
        }
        issued = true;
      }
    }
    if (issued) {   // every commit has arrived before the CTA's shared memory goes away
      umma_commit(bar(B_DONE));
      mbar_wait(bar(B_DONE), 0, abort_flag);
    }
  }

  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && *abort_flag && p.status) atomicOr(p.status, VA_DEV_TIMEOUT);
}

template <int D, bool FP8>
cudaError_t launch(const KeyWeightParams& p, const CUtensorMap& kmap, int num_sms, cudaStream_t stream) {
  using C = Cfg<D, FP8>;
  const void* k = reinterpret_cast<const void*>(verify_attn_key_weights_kernel<D, FP8>);
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<KeyWeightParams*>(&p), const_cast<CUtensorMap*>(&kmap)};
  return launch_kernel(k, dim3((unsigned)num_sms), dim3(kThreads), C::SMEM, stream, args, /*pdl=*/true);
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightParams& p, const CUtensorMap& kmap, int head_dim, bool kv_fp8,
                               int num_sms, cudaStream_t stream) {
  if (head_dim == 64) return kv_fp8 ? launch<64, true>(p, kmap, num_sms, stream) : launch<64, false>(p, kmap, num_sms, stream);
  return kv_fp8 ? launch<128, true>(p, kmap, num_sms, stream) : launch<128, false>(p, kmap, num_sms, stream);
}

}  // namespace va
