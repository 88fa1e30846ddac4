// thinkv_shared.h -- structures of shared-prefix decode (thinkv_shared.cu,
// thinkv_prefix.cu, and the split and combine kernels of thinkv_decode.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "thinkv_internal.h"

namespace thinkv {

constexpr int kTilePages = 8;                 // pages of a key tile (128 tokens)
constexpr int kBlockRows = 256;               // query rows of a prefix block, at most

// When the prefix kernel takes a run, in page-steps of the split kernel (live page
// x kv-head x sequence): it spares (count - 1) * pages * H of them and costs about
// kTileCost per unit (row block x key tile x kv-head).  Runs that spare more than
// they cost are taken where together they gain kWorthPageSteps, which pays for the
// launch, the start-up chain and the larger merge.  Measured, us a call, prefix kernel
// against split kernel alone, rows x 40 own tokens on one prefix:
//   32 q-heads, 8 kv-heads, d = 128   2 rows on 20,000 tokens 56 / 41, 4 rows 57 / 56,
//     8 rows 59 / 87; 8 rows on 2,048 tokens 41 / 27, 32 rows 47 / 50; on 65,536 tokens
//     2 rows 101 / 83, 3 rows 103 / 107: even at a gain of 18,000 to 31,000
//   8 q-heads, 8 kv-heads, d = 128    11,000 to 18,000 (8 rows on 8,192 tokens 43 / 54)
//   64 q-heads, 8 kv-heads, d = 64    28,000 to 40,000 (16 rows on 8,192 tokens 47 / 54)
//   8 q-heads, 1 kv-head, d = 128     40,000 to 80,000 (32 rows on 20,000 tokens 71 / 60,
//     on 65,536 tokens 77 / 138)
constexpr int64_t kTileCost = 10;
constexpr int64_t kWorthPageSteps = 24000;

// One run of neighbours with the same prefix whose prefix goes through the
// prefix kernel.
struct SharedRun {
  int32_t first, count;                       // members [first, first + count) of the call
  int32_t prefix, pages;                      // the prefix sequence and its live pages
};

// What the plan kernel leaves for the others (workspace).
struct SharedPlan {
  int4* item;          // [n] sequence (-1: decoded as empty), prefix read with its own pages (or
                       // -1), live pages of that prefix, run of the prefix kernel (or -1)
  int64_t* pref;       // [n + 1] pages the split kernel reads for the calls before i
  SharedRun* run;      // [n / 2] runs of the prefix kernel
  int64_t* rstart;     // [n / 2 + 1] their first unit (unit: kv-head, row block, key tile)
  int32_t* nruns;
  int32_t* start;      // [n + 1] scratch of the plan: first member of every run of neighbours
  int32_t* used;       // [n] scratch of the plan: a run of neighbours' number among `run`, or -1
};

// A run's rows: blocks of whole members, as equal as possible.
struct RunShape {
  int blocks, members;                        // row blocks, members of a block (the last may have fewer)
  int64_t tiles;                              // key tiles of the prefix
};
__host__ __device__ inline RunShape run_shape(int count, int pages, int Gq) {
  RunShape s;
  const int most = kBlockRows / Gq;
  s.blocks = (count + most - 1) / most;
  s.members = (count + s.blocks - 1) / s.blocks;
  s.tiles = (pages + kTilePages - 1) / kTilePages;
  return s;
}

// Partial rows of the prefix kernel: CTA c's piece of segment (run, kv-head,
// block) starts at row 2 * (rows of the segments before it) + c * kBlockRows.
// A block of more than 128 rows keeps one partial per row; a smaller one keeps
// two (even and odd key tiles), the second `rows` rows further on.
__host__ __device__ inline int64_t partial_row(const SharedRun& r, const RunShape& s, int Hkv, int Gq, int h,
                                               int b, int64_t cta) {
  return 2 * ((int64_t)r.first * Gq * Hkv + (int64_t)h * r.count * Gq + (int64_t)b * s.members * Gq) +
         cta * kBlockRows;
}

struct PrefixParams {
  const uint8_t* pool[3];
  int32_t phb[3];
  int32_t bits[3];     // + 256: float format
  const uint64_t* table;
  const uint64_t* live_list;
  int32_t max_blocks, Hkv, Hq, Gq;
  const uint16_t* q;
  float scale_log2;
  SharedPlan plan;
  float* o;            // [rows][D] unnormalised partial rows
  float2* ml;          // [rows] their (reference exponent, sum)
  int32_t* status;
};

// rows of the partials' arrays
inline int64_t partial_rows(const thinkv_layout& L, int32_t n, int grid) {
  return 2 * (int64_t)n * L.num_q_heads + (int64_t)grid * kBlockRows;
}

cudaError_t launch_shared_plan(const CacheView& C, int32_t n, const int32_t* seq, const int32_t* prefix,
                               bool inline_only, const SharedPlan& plan, cudaStream_t stream);
cudaError_t launch_prefix(const PrefixParams& p, int D, int G, int grid, cudaStream_t stream);

}  // namespace thinkv
