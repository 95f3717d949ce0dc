// Host planner for batches that share a prefix (no CUDA calls).
//
// Consecutive requests of a group list the same leading pages.  Softmax
// attention splits over any partition of a row's keys and joins by LSE, so
// the keys of the shared pages become work items of the group: every query
// row of the group's requests -- they are consecutive rows of q -- against
// the shared keys, read once and multiplied in full row blocks, while each
// request keeps items for the keys of its own.  The split kernels run both in
// one launch; the merge joins a row's own partials with those of its group.
//
// A group's partials are laid out [KV head][split][row of the group], so the
// merge finds a row's without knowing how the rows were cut into blocks.
#include <algorithm>
#include <cstring>
#include <functional>
#include <map>
#include <utility>
#include <vector>

#include "../../include/verify_attn.h"
#include "va_internal.h"
#include "va_planner.h"

namespace va {

namespace {

// Rows row0 .. of request b (b < batch) or group b - batch, against keys [lo, hi).
struct SharedUnit {
  int32_t b, row0, nrows, lo, hi;
  int32_t group;   // group whose partials the rows are merged with, or -1
};

}  // namespace

// Groups of consecutive requests whose page lists start alike.  A request
// joins the group before it when that does not lower the pages saved,
// pages * (requests - 1).
int shared_groups(const int32_t* kv_indptr, const int32_t* kv_indices, const int32_t* qo_indptr,
                  const int32_t* last_page_len, int batch, int page_size, int min_pages,
                  int32_t* group_indptr, int32_t* shared_pages, int* num_groups) {
  if (!num_groups || !group_indptr || batch < 0 || page_size <= 0 || !kv_indptr || !qo_indptr ||
      (batch > 0 && (!last_page_len || !shared_pages)))
    return VA_ERR_INVALID_ARGUMENT;
  if (kv_indptr[0] < 0 || qo_indptr[0] < 0) return VA_ERR_INVALID_ARGUMENT;
  const int64_t least = std::max(1, min_pages);
  // whole pages of request b before its drafts
  std::vector<int64_t> whole((size_t)batch);
  for (int b = 0; b < batch; ++b) {
    const int64_t np = (int64_t)kv_indptr[b + 1] - kv_indptr[b], L = (int64_t)qo_indptr[b + 1] - qo_indptr[b];
    if (np < 0 || L < 0 || (np > 0 && (!kv_indices || last_page_len[b] < 1 || last_page_len[b] > page_size)))
      return VA_ERR_INVALID_ARGUMENT;
    const int64_t kv_len = np > 0 ? (np - 1) * page_size + last_page_len[b] : 0;
    if (kv_len < L) return VA_ERR_INVALID_ARGUMENT;
    whole[(size_t)b] = (kv_len - L) / page_size;
  }
  int n = 0;
  group_indptr[0] = 0;
  for (int b = 0; b < batch;) {
    int64_t s = whole[(size_t)b];
    int e = b + 1;
    for (; e < batch; ++e) {
      const int64_t most = std::min(s, whole[(size_t)e]);
      const int32_t *x = kv_indices + kv_indptr[b], *y = kv_indices + kv_indptr[e];
      int64_t k = 0;
      while (k < most && x[k] == y[k]) ++k;
      if (k < least || k * (e - b) < s * (e - b - 1)) break;
      s = k;
    }
    shared_pages[n] = e - b > 1 ? (int32_t)s : 0;
    group_indptr[++n] = e;
    b = e;
  }
  *num_groups = n;
  return VA_OK;
}

int plan_shared_bounds(int batch, int num_groups, int64_t total_qo, int num_qo_heads, int num_kv_heads,
                       int head_dim, int num_sms, size_t* plan_bytes, size_t* workspace_bytes) {
  if (!plan_bytes || !workspace_bytes || batch < 0 || num_groups < 0 || total_qo < 0 || num_sms <= 0 ||
      num_qo_heads <= 0 || num_kv_heads <= 0 || num_qo_heads % num_kv_heads || head_dim <= 0)
    return VA_ERR_INVALID_ARGUMENT;
  // Units of the requests and of the groups, each at least 64 rows but the
  // last of a request or group; a unit of cost w is cut into at most w / T + 1
  // items, T >= (sum of w) / target.
  const int64_t rows = (int64_t)num_qo_heads * total_qo;
  const int64_t units = ceil_div(rows, 64) + (int64_t)num_kv_heads * batch;
  const int64_t gunits = ceil_div(rows, 64) + (int64_t)num_kv_heads * num_groups;
  const int64_t target = (int64_t)kMaxTargetPerSm * num_sms;
  const int64_t items = target + units + gunits;
  // one partial of every row per part, and the further splits' blocks of <= 256 rows
  const int64_t part_rows = 2 * rows + 256 * target;
  *plan_bytes = sizeof(PlanHeader) + (size_t)(items + units + num_groups) * 32;
  size_t ws = kWsAlign + (size_t)(items + units + num_groups) * 32;
  ws = align_up(ws, kWsAlign) + (size_t)part_rows * 4;
  ws = align_up(ws, kWsAlign) + (size_t)part_rows * std::max(head_dim, kMaxHeadDimV) * 4;
  *workspace_bytes = align_up(ws, kWsAlign);
  return VA_OK;
}

int plan_shared_host(const int32_t* kv_indptr, const int32_t* qo_indptr, const int32_t* last_page_len,
                     const int32_t* mask_indptr, int batch, const int32_t* group_indptr,
                     const int32_t* shared_pages, int num_groups, int num_qo_heads, int num_kv_heads,
                     int head_dim, int page_size, int q_dtype, int kv_dtype, int has_mask, int num_sms,
                     const va_plan_options_t* opts, void* plan_h, size_t plan_bytes,
                     size_t* workspace_bytes) {
  if (!workspace_bytes || !plan_h || batch < 0 || num_groups < 0 || num_sms <= 0) return VA_ERR_INVALID_ARGUMENT;
  if (!kv_indptr || !qo_indptr || (batch > 0 && !last_page_len) || (has_mask && !mask_indptr) || !group_indptr ||
      (num_groups > 0 && !shared_pages))
    return VA_ERR_INVALID_ARGUMENT;
  int rc = check_common(num_qo_heads, num_kv_heads, head_dim, page_size, q_dtype, kv_dtype);
  if (rc) return rc;
  va_plan_options_t o;
  std::memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  if (o.max_splits < 0 || o.min_chunk < 0 || o.target_ctas < 0 || o.head_dim_v < 0) return VA_ERR_INVALID_ARGUMENT;
  if ((o.kv_layout != VA_LAYOUT_HND && o.kv_layout != VA_LAYOUT_NHD) || (o.rope != 0 && o.rope != 1) ||
      (o.q_fp8 != 0 && o.q_fp8 != 1) || o.draft_items < -1 || o.draft_items > 1 ||
      (o.mask_layout != VA_MASK_QLEN && o.mask_layout != VA_MASK_FULL))
    return VA_ERR_INVALID_ARGUMENT;
  if (o.kernel < VA_KERNEL_AUTO || o.kernel > VA_KERNEL_TC_256) return VA_ERR_INVALID_ARGUMENT;
  // a full-prefix mask may hide shared keys from single rows
  if (o.mask_layout == VA_MASK_FULL || o.draft_items == 1) return VA_ERR_UNSUPPORTED;
  const int dv = o.head_dim_v ? o.head_dim_v : head_dim;
  if (dv != 64 && dv != 128) return VA_ERR_UNSUPPORTED;
  if (o.q_fp8 && kv_dtype != VA_DTYPE_FP8_E4M3) return VA_ERR_UNSUPPORTED;
  // a work item names request b as b and group g as batch + g
  if ((int64_t)batch + num_groups > INT32_MAX) return VA_ERR_UNSUPPORTED;

  const int G = num_qo_heads / num_kv_heads;
  if (qo_indptr[0] < 0 || kv_indptr[0] < 0 || group_indptr[0] != 0 || group_indptr[num_groups] != batch)
    return VA_ERR_INVALID_ARGUMENT;
  std::vector<int64_t> prefix((size_t)batch), qlen((size_t)batch), pages((size_t)batch);
  for (int b = 0; b < batch; ++b) {
    const int64_t np = (int64_t)kv_indptr[b + 1] - kv_indptr[b], L = (int64_t)qo_indptr[b + 1] - qo_indptr[b];
    if (np < 0 || L < 0) return VA_ERR_INVALID_ARGUMENT;
    int64_t kv_len = 0;
    if (np > 0) {
      if (last_page_len[b] < 1 || last_page_len[b] > page_size) return VA_ERR_INVALID_ARGUMENT;
      kv_len = (np - 1) * page_size + last_page_len[b];
    }
    if (kv_len > INT32_MAX) return VA_ERR_UNSUPPORTED;
    if (kv_len < L) return VA_ERR_INVALID_ARGUMENT;
    if (has_mask && (mask_indptr[b] < 0 || (int64_t)mask_indptr[b + 1] - mask_indptr[b] != L * L))
      return VA_ERR_INVALID_ARGUMENT;
    prefix[(size_t)b] = kv_len - L;
    qlen[(size_t)b] = L;
    pages[(size_t)b] = np;
  }
  const bool tc_ok = head_dim == 128 && dv == head_dim && page_size % 16 == 0 && 128 % G == 0;
  if ((o.kernel == VA_KERNEL_TC_128 || o.kernel == VA_KERNEL_TC_256) && !tc_ok) return VA_ERR_UNSUPPORTED;
  if (o.q_fp8 && (!tc_ok || o.kernel == VA_KERNEL_MMA_64 || o.kernel == VA_KERNEL_MMA_128)) return VA_ERR_UNSUPPORTED;

  const int es = kv_dtype == VA_DTYPE_FP8_E4M3 ? 1 : 2;
  const int64_t key_bytes = (int64_t)(head_dim + dv) * es;
  // Groups worth a pass of their own: the K / V bytes that the requests after
  // the first do not read again outweigh the fp32 partials that the split
  // adds, written and read once each for both parts of every row.
  std::vector<GroupRec> groups((size_t)num_groups);
  std::vector<int32_t> group_of((size_t)batch, -1);
  int64_t max_rows = 0;
  for (int g = 0; g < num_groups; ++g) {
    const int r0 = group_indptr[g], r1 = group_indptr[g + 1];
    const int64_t S = (int64_t)shared_pages[g] * page_size;
    if (r1 < r0 || r1 > batch || shared_pages[g] < 0) return VA_ERR_INVALID_ARGUMENT;
    int64_t members = 0;
    for (int b = r0; b < r1; ++b) {
      if (pages[(size_t)b] < shared_pages[g] || (qlen[(size_t)b] > 0 && prefix[(size_t)b] < S))
        return VA_ERR_INVALID_ARGUMENT;
      members += qlen[(size_t)b] > 0;
      max_rows = std::max(max_rows, (int64_t)G * qlen[(size_t)b]);
    }
    GroupRec& gr = groups[(size_t)g];
    std::memset(&gr, 0, sizeof(gr));
    gr.r0 = r0;
    gr.r1 = r1;
    gr.pages = shared_pages[g];
    const int64_t L = r1 > r0 ? (int64_t)qo_indptr[r1] - qo_indptr[r0] : 0;
    if ((int64_t)G * L > INT32_MAX) return VA_ERR_UNSUPPORTED;
    const int64_t saved = (members - 1) * S * num_kv_heads * key_bytes;
    const int64_t added = 2 * 2 * L * num_qo_heads * 4LL * dv;
    if (members < 2 || S == 0 || saved <= added) continue;
    gr.rows = (int32_t)(G * L);
    for (int b = r0; b < r1; ++b) group_of[(size_t)b] = g;
    max_rows = std::max(max_rows, (int64_t)gr.rows);
  }
  // Units of work for a kernel, and how it would cut and pack them.
  std::vector<SharedUnit> units;
  int BM = 0, TK = 0;
  int64_t slots = 0, tile1 = 0, tile2 = 0, fixed = 0;
  const int64_t cap = (int64_t)kMaxTargetPerSm * num_sms;
  auto set_kernel = [&](int kernel) {
    BM = kernel_rows(kernel);
    TK = kernel_is_tc(kernel) ? kTcTileKeys : kTileKeys;
    slots = (int64_t)num_sms * (kernel_is_tc(kernel) ? 1 : kernel_ctas_per_sm(kernel));
    // Measured on one GB300, in units of 0.1 us: a key tile of the one-Q-tile
    // kernel 1.5 us (fp8 caches: 1.7), of the two-Q-tile kernel 2.3 us with two
    // (2.6) and 1.9 us with one in use (2.0), and what an item costs beside its
    // tiles (loads, pipeline fill, epilogue), 2 to 3.5 us.
    const bool fp8 = kv_dtype == VA_DTYPE_FP8_E4M3;
    tile1 = kernel == kKernelTc256 ? (fp8 ? 20 : 19) : (fp8 ? 17 : 15);
    tile2 = fp8 ? 26 : 23;
    fixed = kernel == kKernelTc256 ? 35 : 25;
    units.clear();
    auto add_units = [&](int32_t b, int64_t R, int64_t lo, int32_t group, auto&& end_of) {
      for (int64_t row0 = 0; row0 < R; row0 += BM) {
        const int32_t nrows = (int32_t)std::min<int64_t>(BM, R - row0);
        units.push_back({b, (int32_t)row0, nrows, (int32_t)lo, (int32_t)end_of(row0 + nrows - 1), group});
      }
    };
    for (int g = 0; g < num_groups; ++g) {
      const int64_t S = (int64_t)groups[(size_t)g].pages * page_size;
      if (groups[(size_t)g].rows > 0)
        add_units(batch + g, groups[(size_t)g].rows, 0, -1, [&](int64_t) { return S; });
    }
    for (int b = 0; b < batch; ++b) {
      const int32_t g = group_of[(size_t)b];
      const int64_t lo = g >= 0 ? (int64_t)groups[(size_t)g].pages * page_size : 0, pre = prefix[(size_t)b];
      const int64_t L = qlen[(size_t)b];
      // without a mask a row block's last visible key is that of its last token
      add_units(b, G * L, lo, g, [&](int64_t r) { return has_mask ? pre + L : pre + r / G + 1; });
    }
  };
  auto tiles_of = [&](const SharedUnit& u) { return ceil_div(u.hi - u.lo, TK); };
  // cost of a key tile; the row blocks of a group all as its first, so that they are cut alike
  auto tile_cost = [&](const SharedUnit& u) -> int64_t {
    const int32_t rows = u.b >= batch ? std::min(BM, groups[(size_t)(u.b - batch)].rows) : u.nrows;
    return rows > kTcRowsPerTile ? tile2 : tile1;
  };
  // chunk length of a unit, in keys, when items of cost T are aimed at
  const int64_t min_chunk = o.min_chunk;
  auto chunk_of = [&](const SharedUnit& u, int64_t T) -> int64_t {
    const int64_t t = tiles_of(u), min_tiles = std::max<int64_t>(1, min_chunk > 0 ? ceil_div(min_chunk, TK) : 2);
    int64_t n = std::min(ceil_div(t * tile_cost(u), T), std::max<int64_t>(1, t / min_tiles));
    if (o.max_splits > 0) n = std::min<int64_t>(n, o.max_splits);
    return ceil_div(t, std::max<int64_t>(1, n)) * TK;
  };
  auto splits_of = [&](const SharedUnit& u, int64_t cu) { return ceil_div(u.hi - u.lo, cu); };
  // The aimed-at item cost T and the finish it is estimated to give.
  auto choose = [&](bool tc, int64_t* T) -> int64_t {
    int64_t W = 0, key_tiles = 0;
    for (const SharedUnit& u : units) {
      W += tiles_of(u) * tile_cost(u) * num_kv_heads;
      key_tiles += tiles_of(u) * num_kv_heads;
    }
    // Few key tiles per SM: two thirds of the SMs, as in the planner without
    // groups (the set-up of more CTAs and a merge of more partials cost more).
    const bool latency = tc && key_tiles * TK * key_bytes <= 4LL * 64 * 1024 * num_sms;
    const int64_t cand_slots = latency ? std::max<int64_t>(1, 2 * (int64_t)num_sms / 3) : slots;
    int64_t best = -1;
    std::vector<std::pair<int64_t, int64_t>> load_of;
    // Candidates: items aimed at 3/4 to 4 waves of the slots, packed longest
    // first, plus the partials, written once and read once at about 6 TB/s
    // (without that term 3 groups of 8 17-node trees behind 16,384 fp8 keys
    // were cut into 480 items, 114.3 us; with it into 320, 107.7 us).  The
    // first within 1 % of the best is taken: fewer items.
    int64_t seen = -1;
    for (const int eighths : {6, 7, 8, 9, 10, 12, 14, 16, 20, 24, 32}) {
      int64_t target = std::min(eighths * cand_slots / 8, cap);
      if (o.target_ctas > 0) target = std::min<int64_t>(o.target_ctas, cap);
      const int64_t t = std::max<int64_t>(1, ceil_div(W, std::max<int64_t>(1, target)));
      load_of.clear();   // (cost, items)
      int64_t cuts = 0, part_rows = 0;
      for (const SharedUnit& u : units) {
        const int64_t cu = chunk_of(u, t), n = splits_of(u, cu);
        cuts += n;
        if (n > 1 || u.group >= 0 || u.b >= batch) part_rows += n * u.nrows * num_kv_heads;
        const int64_t last = tiles_of(u) - (n - 1) * (cu / TK);
        if (n > 1) load_of.push_back({fixed + cu / TK * tile_cost(u), (n - 1) * num_kv_heads});
        load_of.push_back({fixed + last * tile_cost(u), (int64_t)num_kv_heads});
      }
      if (cuts == seen) continue;   // the same cuts as the candidate before
      seen = cuts;
      std::sort(load_of.begin(), load_of.end(), std::greater<std::pair<int64_t, int64_t>>());
      std::map<int64_t, int64_t> levels;   // slot load -> slots
      levels[0] = cand_slots;
      for (const auto& x : load_of)
        for (int64_t left = x.second; left > 0;) {
          auto lo = levels.begin();
          const int64_t level = lo->first, take = std::min(left, lo->second);
          if ((lo->second -= take) == 0) levels.erase(lo);
          levels[level + x.first] += take;
          left -= take;
        }
      const int64_t finish = levels.rbegin()->first + part_rows * 8 * dv / 600000;
      if (best < 0 || finish * 100 < best * 99) {
        best = finish;
        *T = t;
      }
      if (o.target_ctas > 0) break;
    }
    return best;
  };
  int kernel = o.kernel;
  int64_t T = 1;
  if (kernel == VA_KERNEL_AUTO) {
    if (!tc_ok) {
      kernel = max_rows <= 64 ? kKernelMma64 : kKernelMma128;
    } else if (max_rows <= 128) {
      kernel = kKernelTc128;
    } else {
      // Two Q tiles a CTA do more per key tile, but items that fill only one
      // run slower there: the kernel with the earlier finish.
      int64_t t256 = 1;
      set_kernel(kKernelTc128);
      const int64_t f128 = choose(true, &T);
      set_kernel(kKernelTc256);
      const int64_t f256 = choose(true, &t256);
      kernel = f256 < f128 ? kKernelTc256 : kKernelTc128;
      if (kernel == kKernelTc256) T = t256;
    }
  }
  const bool chosen = T > 1;
  if (units.empty() || BM != kernel_rows(kernel) || !kernel_is_tc(kernel)) set_kernel(kernel);
  if (!chosen) choose(kernel_is_tc(kernel), &T);

  // The items and their partials.
  std::vector<PlanItem> items;
  std::vector<MergeItem> merges;
  int64_t part_rows = 0, max_nsplit = 0;
  for (const SharedUnit& u : units) {
    const int64_t cu = chunk_of(u, T);
    int64_t n = splits_of(u, cu);
    // a last chunk shorter than one key tile joins the one before it (the
    // tcgen05 kernels; see the planner without groups), but not a group's:
    // its row blocks are cut alike
    if (u.b < batch && kernel_is_tc(kernel) && n > 1 && u.hi - (u.lo + (n - 1) * cu) < TK) --n;
    GroupRec* gr = u.b >= batch ? &groups[(size_t)(u.b - batch)] : nullptr;
    const bool part = gr || u.group >= 0 || n > 1;
    if (gr && u.row0 == 0) {
      if (part_rows > INT32_MAX) return VA_ERR_UNSUPPORTED;
      gr->nsplit = (int32_t)n;
      gr->part_row0 = (int32_t)part_rows;
      part_rows += (int64_t)num_kv_heads * n * gr->rows;
    }
    for (int h = 0; h < num_kv_heads; ++h) {
      int64_t base = -1, stride = 0;
      if (gr) {
        base = gr->part_row0 + (int64_t)h * n * gr->rows + u.row0;
        stride = gr->rows;
      } else if (part) {
        if (part_rows > INT32_MAX) return VA_ERR_UNSUPPORTED;
        base = part_rows;
        stride = u.nrows;
        part_rows += n * u.nrows;
        merges.push_back({u.b, h, u.row0, u.nrows, (int32_t)base, (int32_t)n, u.group + 1, 0});
        max_nsplit = std::max(max_nsplit, n + (u.group >= 0 ? groups[(size_t)u.group].nsplit : 0));
      }
      for (int64_t s = 0; s < n; ++s) {
        const int64_t lo = u.lo + s * cu, hi = s == n - 1 ? u.hi : lo + cu;
        WorkItem w{u.b, h, u.row0, u.nrows, (int32_t)lo, (int32_t)hi, part ? (int32_t)(base + s * stride) : -1, -1};
        const int64_t cost = u.nrows > kTcRowsPerTile ? tile2 : tile1;
        items.push_back({w, fixed + ceil_div(hi - lo, TK) * cost});
      }
    }
  }
  if (part_rows > INT32_MAX) return VA_ERR_UNSUPPORTED;
  sort_items(items);
  const int64_t n_ctas = kernel_is_tc(kernel) && !items.empty() ? deal_chains(items, num_sms, TK, true) : 0;

  const size_t need = sizeof(PlanHeader) + (items.size() + merges.size() + groups.size()) * 32;
  if (plan_bytes < need) {
    *workspace_bytes = need;
    return VA_ERR_PLAN_BUFFER_TOO_SMALL;
  }
  int64_t merge_rows = 0;   // requests' row blocks are short next to the groups': the merge's grid
  for (const MergeItem& m : merges) merge_rows = std::max<int64_t>(merge_rows, m.nrows);
  PlanHeader hd;
  std::memset(&hd, 0, sizeof(hd));
  hd.magic = kPlanMagic;
  hd.version = kPlanVersion;
  hd.batch = batch;
  hd.h_q = num_qo_heads;
  hd.h_kv = num_kv_heads;
  hd.head_dim = head_dim;
  hd.head_dim_v = dv;
  hd.max_nsplit = max_nsplit;
  hd.page_size = page_size;
  hd.q_dtype = q_dtype;
  hd.kv_dtype = kv_dtype;
  hd.has_mask = has_mask ? 1 : 0;
  hd.group = G;
  hd.kernel = kernel;
  hd.block_rows = BM;
  hd.tile_keys = TK;
  hd.n_items = (int32_t)items.size();
  hd.n_merge = (int32_t)merges.size();
  hd.n_units = (int32_t)units.size();
  hd.num_sms = num_sms;
  hd.total_qo = batch > 0 ? qo_indptr[batch] : 0;
  hd.part_rows = part_rows;
  hd.chunk = T;
  hd.off_status = 0;
  hd.off_items = kWsAlign;
  hd.off_merge = hd.off_items + items.size() * sizeof(WorkItem);
  hd.off_part_lse =
      align_up(hd.off_merge + merges.size() * sizeof(MergeItem) + groups.size() * sizeof(GroupRec), kWsAlign);
  hd.off_part_out = align_up(hd.off_part_lse + (size_t)part_rows * 4, kWsAlign);
  hd.ws_bytes = align_up(hd.off_part_out + (size_t)part_rows * dv * 4, kWsAlign);
  hd.plan_bytes = need;
  hd.n_ctas = n_ctas;
  hd.flags = (o.kv_layout == VA_LAYOUT_NHD ? kPlanNhd : 0) | (o.rope ? kPlanRope : 0) | (o.q_fp8 ? kPlanF8Mma : 0) |
             (merge_rows << kPlanMergeRowsShift) | ((int64_t)num_groups << kPlanGroupShift);
  char* dst = static_cast<char*>(plan_h);
  std::memcpy(dst, &hd, sizeof(hd));
  dst += sizeof(hd);
  for (const PlanItem& x : items) {
    std::memcpy(dst, &x.it, sizeof(WorkItem));
    dst += sizeof(WorkItem);
  }
  if (!merges.empty()) std::memcpy(dst, merges.data(), merges.size() * sizeof(MergeItem));
  if (!groups.empty())
    std::memcpy(dst + merges.size() * sizeof(MergeItem), groups.data(), groups.size() * sizeof(GroupRec));
  *workspace_bytes = hd.ws_bytes;
  return VA_OK;
}

}  // namespace va
