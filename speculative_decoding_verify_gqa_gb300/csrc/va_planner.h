// What the planners (one plan per request, or with shared prefixes) have in
// common.  Host code, no CUDA calls.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <vector>

#include "../../include/verify_attn.h"
#include "va_internal.h"

namespace va {

constexpr int kMaxTargetPerSm = 4;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A work item with the weight it is sorted by.
struct PlanItem {
  WorkItem it;
  int64_t cost;
};

// Longest first; among equals by (b, h, kv_lo, row0), which identifies an
// item, so that row blocks reading the same keys sit next to each other.
void sort_items(std::vector<PlanItem>& items);

// The chains of the persistent tcgen05 variants: the sorted items dealt to at
// most num_sms chains, reordered and linked through next.  An item weighs its
// key tiles plus one, or (by_cost) its cost.  Returns the number of chains.
int64_t deal_chains(std::vector<PlanItem>& items, int num_sms, int TK, bool by_cost = false);

int check_common(int num_qo_heads, int num_kv_heads, int head_dim, int page_size, int q_dtype,
                 int kv_dtype);

}  // namespace va
