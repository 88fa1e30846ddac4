// thinkv_pages.cuh -- granting pages from a class pool.
//
// A pool hands out released pages first, the last released on top, then pages
// it never handed out.  The page_bump buffer (include/thinkv.h) holds, as
// int32: [0, 3) the pages ever handed out per class, [3, 6) the released pages
// per class, then one stack of released page ids per class (pool_pages[c]
// entries, class after class).
//
// A call that takes several pages numbers them in call order.  Its g-th page of
// class c (g counted from 0 over the call) has the virtual number
//   v = bump - released + g
// with bump and released the counters at the start of the call: v >= bump is
// the page id itself, v < bump stands for the stack entry bump - 1 - v.  So one
// base per run (virtual numbers may be negative) serves both sources, and with
// nothing released v is the page id, as if there were no stack.
#pragma once

#include <stdint.h>

#include "thinkv_internal.h"

namespace thinkv {

constexpr int kBumpHeader = 6;

__device__ inline const int32_t* released_stack(const CacheView& C, int c) {
  const int64_t before = c == 0 ? 0 : (c == 1 ? (int64_t)C.L.pool_pages[0]
                                              : (int64_t)C.L.pool_pages[0] + C.L.pool_pages[1]);
  return C.page_bump + kBumpHeader + before;
}

// The page with virtual number v of class c; bump: the class's count of pages
// ever handed out at the start of the call.
__device__ inline int granted_page(const CacheView& C, int c, int v, int bump) {
  return v >= bump ? v : released_stack(C, c)[bump - 1 - v];
}

// Whether class c's pool can give `total` pages.
__device__ inline bool pool_has(const CacheView& C, int c, int bump, int released, int64_t total) {
  return (int64_t)bump - released + total <= C.L.pool_pages[c];
}

// Counters after `total` pages of class c were granted.
__device__ inline void take_pages(const CacheView& C, int c, int bump, int released, int total) {
  const int from_stack = total < released ? total : released;
  C.page_bump[3 + c] = released - from_stack;
  C.page_bump[c] = bump + total - from_stack;
}

}  // namespace thinkv
