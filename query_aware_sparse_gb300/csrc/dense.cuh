// Device helpers shared by the dense-layer operators: which keys a query row
// sees and what happens to a logit before the softmax.
#pragma once

#include "common.cuh"
#include "dense.h"

namespace quest {

// Visible keys lo <= j < hi of the row at position pos of a request of len
// tokens (hi <= lo: none). doc and prefix are 0 where the call has none.
struct Seen { int lo, hi; };
__device__ __forceinline__ Seen seen_keys(int pos, int len, int window, int doc, int prefix) {
  Seen s;
  s.hi = min(len, max(pos + 1, prefix));
  s.lo = max(0, doc);
  if (window > 0 && pos >= window) s.lo = max(s.lo, pos - window + 1);
  return s;
}

// A request's tokens that its page table holds.
__device__ __forceinline__ int held_tokens(int len, int table_pages, int page_size, unsigned* err) {
  if (len <= 0) return 0;
  if ((len - 1) / page_size >= table_pages) {
    report(err, QUEST_DEVERR_TABLE_RANGE);
    return max(0, table_pages) * page_size;
  }
  return len;
}

// cap tanh(x / cap): for |x| < cap the product of x and a polynomial in
// (x / cap)^2 (tanh(u) / u fitted at Chebyshev nodes for |u| < 1, 1.1e-7 of
// itself off at most, so small logits keep their relative accuracy), else
// tanhf. Which of the two a value takes goes by itself alone; a warp without a
// large one skips tanhf. Converged warps only.
__device__ __forceinline__ float capped(float x, float cap, float inv_cap) {
  const float u = x * inv_cap;
  const float w = u * u;
  float q = -0.00042374664917588234f;
  q = fmaf(q, w, 0.0025196773931384087f);
  q = fmaf(q, w, -0.008229382336139679f);
  q = fmaf(q, w, 0.021665599197149277f);
  q = fmaf(q, w, -0.05393609404563904f);
  q = fmaf(q, w, 0.13333140313625336f);
  q = fmaf(q, w, -0.3333333134651184f);
  float y = x * fmaf(q, w, 1.f);
  if (__any_sync(FULL, !(fabsf(u) < 1.f))) y = fabsf(u) < 1.f ? y : cap * tanhf(u);
  return y;
}

}  // namespace quest
