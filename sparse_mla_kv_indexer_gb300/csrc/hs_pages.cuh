// What hs_copy_pages keeps between its two launches, behind the pool's status word in one allocation.
#pragma once

#include "hs_internal.cuh"

namespace hs {

// int32 words: the status word; the number of the last call that marked pages, and how many of the running one's CTAs
// have read it; which of the call's copies of either kind are made; where each page of either kind went, and in the call
// of which number.
constexpr size_t PG_EPOCH = 2, PG_OK = 64, PG_MAP = PG_OK + 2 * HS_COPY_MAX_PAGES / 4;
inline size_t page_state_words(int num_pages, int num_idx_pages) { return PG_MAP + 2 * ((size_t)num_pages + num_idx_pages); }

__device__ __forceinline__ uint32_t* copy_epoch(const Dev& D) { return reinterpret_cast<uint32_t*>(D.status) + PG_EPOCH; }
__device__ __forceinline__ uint8_t* copy_made_flags(const Dev& D, bool kv) {
  return reinterpret_cast<uint8_t*>(D.status + PG_OK) + (kv ? 0 : HS_COPY_MAX_PAGES);
}
__device__ __forceinline__ int2* page_map(const Dev& D, bool kv) {
  return reinterpret_cast<int2*>(D.status + PG_MAP) + (kv ? 0 : D.num_pages);
}

}  // namespace hs
