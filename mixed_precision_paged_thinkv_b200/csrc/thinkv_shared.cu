// thinkv_shared.cu -- shared-prefix decode: who reads which pages.
//
// A sequence's row attends over its prefix's live pages and its own.  Runs of
// neighbours with the same prefix can have the prefix read once for all their
// rows (thinkv_prefix.cu); every other page is read sequence by sequence by the
// split kernel of thinkv_decode.cu.  One CTA decides, since lengths and ids are
// known on the device only.
#include <stdint.h>

#include "thinkv_common.cuh"
#include "thinkv_internal.h"
#include "thinkv_shared.h"

namespace thinkv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Page-steps (live page x kv-head x sequence) that the split kernel has to be
// spared before the prefix kernel is worth its own latency.
constexpr int64_t kWorthPageSteps = 8192;

__device__ int64_t block_scan(int64_t v, int64_t* sh, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    sh[lane] = w;
  }
  __syncthreads();
  const int64_t before = warp ? sh[warp - 1] : 0;
  *total = sh[kWarps - 1];
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kThreads)
    shared_plan_kernel(CacheView C, int32_t n, const int32_t* __restrict__ seq,
                       const int32_t* __restrict__ prefix, bool inline_only, SharedPlan plan) {
  __shared__ int64_t sh[kWarps];
  const int tid = threadIdx.x, H = C.L.num_kv_heads, Gq = C.L.num_q_heads / H;
  pdl_launch_dependents();
  pdl_wait();
  auto row_prefix = [&](int i) {                 // the prefix row i really has (-1: none)
    const int s = seq[i], x = prefix[i];
    return s >= 0 && s < C.L.max_seqs && x >= 0 && x < C.L.max_seqs ? x : -1;
  };
  int64_t total, carry = 0;
  // ---- runs of neighbours with the same prefix ----
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    const bool start = i < n && (i == 0 || row_prefix(i) != row_prefix(i - 1));
    const int64_t k = carry + block_scan(start, sh, &total);
    if (start) plan.start[k] = i;
    carry += total;
  }
  const int nruns = (int)carry;
  if (tid == 0) plan.start[nruns] = n;
  __syncthreads();
  // ---- what the prefix kernel would spare the split kernel ----
  int64_t spared = 0;
  for (int base = 0; base < nruns; base += kThreads) {
    const int k = base + tid;
    int64_t v = 0;
    if (k < nruns) {
      const int first = plan.start[k], count = plan.start[k + 1] - first, x = row_prefix(first);
      if (!inline_only && x >= 0 && count >= 2) v = (int64_t)(count - 1) * C.num_live[x] * H;
    }
    block_scan(v, sh, &total);
    spared += total;
  }
  const bool use = spared >= kWorthPageSteps;
  int64_t nused = 0, units = 0;
  for (int base = 0; base < nruns; base += kThreads) {
    const int k = base + tid;
    bool mine = false;
    SharedRun r = {0, 0, -1, 0};
    RunShape s = {0, 0, 0};
    if (k < nruns) {
      r.first = plan.start[k];
      r.count = plan.start[k + 1] - r.first;
      r.prefix = row_prefix(r.first);
      r.pages = r.prefix >= 0 ? C.num_live[r.prefix] : 0;
      mine = use && r.count >= 2 && r.pages > 0;
      if (mine) s = run_shape(r.count, r.pages, Gq);
    }
    const int64_t e = nused + block_scan(mine, sh, &total);
    nused += total;
    const int64_t u = units + block_scan(mine ? H * (int64_t)s.blocks * s.tiles : 0, sh, &total);
    units += total;
    if (k < nruns) plan.used[k] = mine ? (int)e : -1;
    if (mine) {
      plan.run[e] = r;
      plan.rstart[e] = u;
    }
  }
  if (tid == 0) {
    plan.rstart[nused] = units;
    *plan.nruns = (int)nused;
  }
  __syncthreads();
  // ---- every sequence's own reading ----
  int64_t k0 = 0, pages = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    const bool start = i < n && (i == 0 || row_prefix(i) != row_prefix(i - 1));
    const int64_t before = block_scan(start, sh, &total);
    const int64_t k = k0 + before + start - 1;
    k0 += total;
    int4 item = make_int4(-1, -1, 0, -1);
    int64_t v = 0;
    if (i < n) {
      const int s = seq[i], x = prefix[i];
      if (s < 0 || s >= C.L.max_seqs || x < -1 || x >= C.L.max_seqs) {
        set_status(C.status, THINKV_ERR_INVALID);    // decoded as empty
      } else {
        item.x = s;
        v = C.num_live[s];
        if (x >= 0) {
          item.w = plan.used[k];
          if (item.w < 0) {
            item.y = x;
            item.z = C.num_live[x];
            v += item.z;
          }
        }
      }
    }
    const int64_t at = pages + block_scan(v, sh, &total);
    pages += total;
    if (i < n) {
      plan.item[i] = item;
      plan.pref[i] = at;
    }
  }
  if (tid == 0) plan.pref[n] = pages;
}

}  // namespace

cudaError_t launch_shared_plan(const CacheView& C, int32_t n, const int32_t* seq, const int32_t* prefix,
                               bool inline_only, const SharedPlan& plan, cudaStream_t stream) {
  return launch_pdl(shared_plan_kernel, dim3(1), dim3(kThreads), 0, stream, C, n, seq, prefix, inline_only,
                    plan);
}

}  // namespace thinkv
