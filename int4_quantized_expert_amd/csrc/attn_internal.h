// Declarations shared by the attention entry points (include/attention.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "device_common.h"

namespace moe {

int attn_bad(const char* fmt, long long x = 0, long long y = 0);   // MOE_EINVAL with the text
int check_attn(const attn_desc* d);
int check_attn_batch(int32_t B, int32_t N, const int32_t* cu, const int32_t* lens, const int32_t* table);

inline bool attn_overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && pa < pb + static_cast<uintptr_t>(nb) && pb < pa + static_cast<uintptr_t>(na);
}
inline bool attn_aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Where the tokens of a batch lie, as both kernels read it.
struct AttnBatch {
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  int B, N;
  int shift;            // log2 of page_size
  int max_pages;
  int64_t n_pages;
  int64_t page_elems;   // 2 n_kv page_size head_dim
  int64_t half_elems;   // n_kv page_size head_dim: from a page's keys to its values
};

inline AttnBatch attn_batch(const attn_desc* d, int32_t B, int32_t N, const int32_t* cu, const int32_t* lens,
                            const int32_t* table) {
  AttnBatch a;
  a.cu = cu;
  a.lens = lens;
  a.table = table;
  a.B = B;
  a.N = N;
  a.shift = __builtin_ctz(static_cast<unsigned>(d->page_size));
  a.max_pages = d->max_pages;
  a.n_pages = d->n_pages;
  a.half_elems = static_cast<int64_t>(d->n_kv_heads) * d->page_size * d->head_dim;
  a.page_elems = 2 * a.half_elems;
  return a;
}

}  // namespace moe
