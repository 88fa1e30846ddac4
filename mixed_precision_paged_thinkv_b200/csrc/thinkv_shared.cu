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

// Exclusive prefix of N values per thread over the block (sh: N * 33 words);
// tot: the block's sums.
template <int N>
__device__ void block_scan(int64_t (&v)[N], int64_t (&tot)[N], int64_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    x[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x[k], o);
      if (lane >= o) x[k] += y;
    }
    if (lane == 31) sh[k * 33 + warp] = x[k];
  }
  __syncthreads();
  if (warp < N) {                                // warp k scans the warps' sums of value k
    int64_t w = lane < warps ? sh[warp * 33 + lane] : 0;
    const int64_t own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < warps) sh[warp * 33 + lane] = w - own;
    if (lane == 31) sh[warp * 33 + 32] = w;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = sh[k * 33 + warp] + x[k] - v[k];
    tot[k] = sh[k * 33 + 32];
  }
  __syncthreads();
}

// One row as the plan sees it.
struct Row {
  int s, x;            // its sequence (-1: the row is empty) and prefix (-1: none)
};

__global__ void __launch_bounds__(kThreads)
    shared_plan_kernel(CacheView C, int32_t n, const int32_t* __restrict__ seq,
                       const int32_t* __restrict__ prefix, bool inline_only, SharedPlan plan) {
  __shared__ int64_t sh[3 * 33];
  const int tid = threadIdx.x, nt = blockDim.x, H = C.L.num_kv_heads, Gq = C.L.num_q_heads / H;
  const int max_seqs = C.L.max_seqs;
  pdl_launch_dependents();
  auto row = [&](int i) {
    Row r;
    r.s = seq[i];
    r.x = prefix[i];
    if (r.s < 0 || r.s >= max_seqs || r.x < -1 || r.x >= max_seqs) r.s = r.x = -1;
    return r;
  };
  // a call of one row per thread reads its inputs while the previous kernel ends
  Row mine = {-1, -1}, before = {-1, -1};
  const bool one_pass = n <= nt;
  if (tid < n) mine = row(tid);
  if (tid < n && tid > 0) before = row(tid - 1);
  pdl_wait();
  // live pages of the row's sequence and prefix, in flight over the first scan
  int own = 0, shared = 0;
  if (one_pass && tid < n) {
    if (mine.s >= 0) own = C.num_live[mine.s];
    if (mine.x >= 0) shared = C.num_live[mine.x];
  }
  // ---- runs of neighbours with the same prefix ----
  int64_t carry = 0, my_run = 0;
  for (int base = 0; base < n; base += nt) {
    const int i = base + tid;
    if (!one_pass && i < n) {
      mine = row(i);
      if (i > 0) before = row(i - 1);
    }
    const bool start = i < n && (i == 0 || mine.x != before.x);
    int64_t v[1] = {start}, tot[1];
    block_scan<1>(v, tot, sh);
    if (start) plan.start[carry + v[0]] = i;
    my_run = carry + v[0] + start - 1;           // (one pass: this row's run)
    carry += tot[0];
  }
  const int nruns = (int)carry;
  if (tid == 0) plan.start[nruns] = n;
  __syncthreads();
  // ---- the runs that the prefix kernel could take, and what that would gain ----
  int64_t gained = 0, nused = 0, units = 0;
  for (int base = 0; base < nruns; base += nt) {
    const int k = base + tid;
    int64_t v[3] = {0, 0, 0}, tot[3];
    SharedRun r = {0, 0, -1, 0};
    if (k < nruns) {
      r.first = plan.start[k];
      r.count = plan.start[k + 1] - r.first;
      r.prefix = row(r.first).x;
      r.pages = r.prefix >= 0 ? C.num_live[r.prefix] : 0;
      if (!inline_only && r.count >= 2 && r.pages > 0) {
        const RunShape s = run_shape(r.count, r.pages, Gq);
        const int64_t n_units = H * (int64_t)s.blocks * s.tiles;
        const int64_t gain = (int64_t)(r.count - 1) * r.pages * H - kTileCost * n_units;
        if (gain > 0) {
          v[0] = gain;
          v[1] = 1;
          v[2] = n_units;
        }
      }
    }
    const bool fit = v[1] != 0;
    block_scan<3>(v, tot, sh);
    if (k < nruns) plan.used[k] = fit ? (int)(nused + v[1]) : -1;
    if (fit) {
      plan.run[nused + v[1]] = r;
      plan.rstart[nused + v[1]] = units + v[2];
    }
    gained += tot[0];
    nused += tot[1];
    units += tot[2];
  }
  const bool use = gained >= kWorthPageSteps;
  if (tid == 0) {
    plan.rstart[use ? nused : 0] = use ? units : 0;
    *plan.nruns = use ? (int)nused : 0;
  }
  __syncthreads();
  // ---- every sequence's own reading ----
  int64_t k0 = 0, pages = 0;
  for (int base = 0; base < n; base += nt) {
    const int i = base + tid;
    if (!one_pass) {
      int64_t v[1] = {0}, tot[1];
      if (i < n) {
        mine = row(i);
        v[0] = i == 0 || mine.x != row(i - 1).x;
        own = mine.s >= 0 ? C.num_live[mine.s] : 0;
        shared = mine.x >= 0 ? C.num_live[mine.x] : 0;
      }
      const int64_t start = v[0];
      block_scan<1>(v, tot, sh);
      my_run = k0 + v[0] + start - 1;
      k0 += tot[0];
    }
    int4 item = make_int4(-1, -1, 0, -1);
    int64_t v[1] = {0}, tot[1];
    if (i < n) {
      if (mine.s < 0) {
        set_status(C.status, THINKV_ERR_INVALID);    // decoded as empty
      } else {
        item.x = mine.s;
        v[0] = own;
        if (mine.x >= 0) {
          item.w = use ? plan.used[my_run] : -1;
          if (item.w < 0) {
            item.y = mine.x;
            item.z = shared;
            v[0] += shared;
          }
        }
      }
    }
    block_scan<1>(v, tot, sh);
    if (i < n) {
      plan.item[i] = item;
      plan.pref[i] = pages + v[0];
    }
    pages += tot[0];
  }
  if (tid == 0) plan.pref[n] = pages;
}

}  // namespace

cudaError_t launch_shared_plan(const CacheView& C, int32_t n, const int32_t* seq, const int32_t* prefix,
                               bool inline_only, const SharedPlan& plan, cudaStream_t stream) {
  int threads = (n + 31) / 32 * 32;              // a row a thread where that is possible
  if (threads < 96) threads = 96;                // (a warp for each of a scan's three values)
  if (threads > kThreads) threads = kThreads;
  return launch_pdl(shared_plan_kernel, dim3(1), dim3(threads), 0, stream, C, n, seq, prefix, inline_only,
                    plan);
}

}  // namespace thinkv
