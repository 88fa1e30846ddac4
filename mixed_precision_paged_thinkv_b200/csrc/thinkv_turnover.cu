// thinkv_turnover.cu -- release and fork: the turnover of sequences in a batch.
//
// "ThinKV: Thought-Adaptive KV Cache Compression for Efficient Reasoning
// Models" keeps evicted slots inside their sequence (explainer, Methodologie,
// "Implementation Systeme: Pensee Continue (CT)") and says nothing of whole
// sequences that end or start from another one; these two calls add that.
//
//   release: the pages of each listed sequence go onto their class's stack of
//   released pages, the last page of the call first, so that later grants take
//   the call's pages in call order; the sequence becomes empty.
//   fork: dst[i] becomes a copy of src[i]: as many pages of each class, granted
//   in call order (released pages first, thinkv_pages.cuh), the same bytes,
//   slot positions, free stacks, FIFO windows, live list and counters.
//
// Two kernels per call.
//   plan: a CTA per listed sequence counts its pages per class, chunk by chunk
//   (32 table entries), and leaves each chunk's first rank within its class.
//   The CTA that arrives last checks the call (ids, distinctness, empty
//   destinations, pool space), scans the counts in call order and advances the
//   pools' counters; nothing has been changed before that point.
//   apply: a warp per chunk (release) or per chunk and kv-head (fork); the lane
//   holds one table entry, ballots give its rank and so its place on the stack
//   or its new page.
// Fork is bound by HBM writes.  A warp reads a page-head block once, into
// registers, and writes it to up to eight neighbouring copies of one source with
// streaming 16-byte stores; 64 copies of 20,000 tokens (1.1 GB written) take 232 us,
// 4.8 TB/s.  Reading once per copy took 331 us (reads from L2 and writes share the
// way to the SMs), bulk copies through shared memory 402 us for one copy each and
// the present time for eight at once, plain stores 5 % more; the number of
// copies together, of warps a chunk and of loads in flight change 3 % either way.
#include <stdint.h>

#include "thinkv_common.cuh"
#include "thinkv_internal.h"
#include "thinkv_pages.cuh"

namespace thinkv {

namespace {

constexpr int kChunk = 32;                     // table entries of a chunk (one per lane)
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBatch = 4;                  // chunks per warp and pass (loads in flight)
constexpr int kApplyWarps = 8;
constexpr int kForkCtas = 4;                   // CTAs of the copy per SM (32 warps)
constexpr int kCopyDepth = 4;                  // 16-byte loads a lane has in flight
constexpr int kParts = 8;                      // warps that share a chunk's blocks of one kv-head
constexpr int kCopies = 8;                     // neighbouring copies of one source made together

struct TurnoverWs {
  uint32_t* arrive;    // arrival counter of the plan kernel, zero between calls
  int32_t* head;       // [0] 1 once the call was accepted; [1 + c] pages of the call;
                       // [4 + c], [7 + c]: page_bump and released count before it
  int32_t* nb;         // [n] table entries of each listed (source) sequence
  int32_t* tot;        // [n][3] its pages per class
  int32_t* base;       // [n][3] pages of the sequences before it in the call
  int32_t* ubase;      // [n + 1] chunks before it (an empty sequence counts as one; a copy that
                       // leads no group counts as none)
  int32_t* crank;      // [n][chunks][3] a chunk's first rank within its sequence and class
  int64_t chunks;      // chunks of a full table
};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int64_t table_chunks(const thinkv_layout& L) { return (L.max_blocks_per_seq + kChunk - 1) / kChunk; }

TurnoverWs carve(const thinkv_layout& L, void* ws, int32_t n) {
  TurnoverWs w;
  uint8_t* p = static_cast<uint8_t*>(ws);
  w.arrive = reinterpret_cast<uint32_t*>(p);
  w.head = reinterpret_cast<int32_t*>(p + 128);
  p += 256;
  w.nb = reinterpret_cast<int32_t*>(p);
  p += round256((size_t)n * 4);
  w.tot = reinterpret_cast<int32_t*>(p);
  p += round256((size_t)n * 12);
  w.base = reinterpret_cast<int32_t*>(p);
  p += round256((size_t)n * 12);
  w.ubase = reinterpret_cast<int32_t*>(p);
  p += round256(((size_t)n + 1) * 4);
  w.crank = reinterpret_cast<int32_t*>(p);
  w.chunks = table_chunks(L);
  return w;
}

// Whether pair x of a fork leads a group: neighbours with one source, up to
// kCopies of them, are copied together.
__device__ inline bool leads_group(const int32_t* src, int x) {
  return x % kCopies == 0 || src[x] != src[x - 1];
}

// Exclusive prefix over the block of four values per thread; tot: block totals.
__device__ void block_scan4(int (&v)[4], int (&tot)[4], int (*sh)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = v[j];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x[j], o);
      if (lane >= o) x[j] += y;
    }
    if (lane == 31) sh[warp][j] = x[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int before = 0;
    tot[j] = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
      if (w < warp) before += sh[w][j];
      tot[j] += sh[w][j];
    }
    v[j] = before + x[j] - v[j];
  }
  __syncthreads();
}

// seq: the sequences whose tables are read (release: the released ones; fork:
// the sources); dst: the fork's destinations, null for a release.
__global__ void __launch_bounds__(kPlanThreads)
    turnover_plan_kernel(CacheView C, int32_t n, const int32_t* __restrict__ seq,
                         const int32_t* __restrict__ dst, TurnoverWs ws) {
  extern __shared__ uint32_t seen[];            // max_seqs bits
  __shared__ int sh[kPlanWarps][4];
  __shared__ int s_cnt[2][kPlanWarps * kPlanBatch][3];
  __shared__ int s_last, s_err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = blockIdx.x;
  const int max_seqs = C.L.max_seqs;
  pdl_launch_dependents();
  const int s = seq[i];
  pdl_wait();

  // ---- this sequence's pages per class, and each chunk's first ranks ----
  const int nb = (s >= 0 && s < max_seqs) ? C.num_blocks[s] : 0;
  const uint64_t* table = C.block_table + (int64_t)(nb ? s : 0) * C.L.max_blocks_per_seq;
  int32_t* crank = ws.crank + (int64_t)i * ws.chunks * 3;
  int run[3] = {0, 0, 0};
  uint64_t ent[kPlanBatch];
  constexpr int kPass = kPlanWarps * kPlanBatch;      // chunks of a pass
  auto load = [&](int chunk0) {
#pragma unroll
    for (int j = 0; j < kPlanBatch; ++j) {
      const int64_t e = (int64_t)(chunk0 + warp * kPlanBatch + j) * kChunk + lane;
      ent[j] = e < nb ? table[e] : ~0ull;
    }
  };
  load(0);
  int buf = 0;
  for (int chunk0 = 0; (int64_t)chunk0 * kChunk < nb; chunk0 += kPass, buf ^= 1) {
#pragma unroll
    for (int j = 0; j < kPlanBatch; ++j) {
      const int c = entry_class(ent[j]);
#pragma unroll
      for (int cc = 0; cc < 3; ++cc) {
        const int cnt = __popc(__ballot_sync(0xFFFFFFFFu, c == cc));
        if (lane == 0) s_cnt[buf][warp * kPlanBatch + j][cc] = cnt;
      }
    }
    load(chunk0 + kPass);                             // the next pass, in flight over the barrier
    __syncthreads();
    if (warp < 3) {                                   // warp cc scans class cc over the pass's chunks
      const int v = s_cnt[buf][lane][warp];
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      if ((int64_t)(chunk0 + lane) * kChunk < nb) crank[(int64_t)(chunk0 + lane) * 3 + warp] = run[0] + x - v;
      run[0] += __shfl_sync(0xFFFFFFFFu, x, 31);
    }
  }
  static_assert(kPass == 32, "a lane per chunk of a pass");
  if (warp < 3 && lane == 0) ws.tot[i * 3 + warp] = run[0];
  if (tid == 0) ws.nb[i] = nb;

  // ---- the last CTA to arrive checks and scans the call ----
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(ws.arrive, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  if (tid == 0) {
    *ws.arrive = 0u;
    s_err = *C.status != 0 ? -1 : 0;
  }
  for (int x = tid; x < (max_seqs + 31) / 32; x += kPlanThreads) seen[x] = 0;
  __syncthreads();
  const int32_t* own = dst ? dst : seq;               // the sequences that change
  for (int x = tid; x < n; x += kPlanThreads) {
    const int t = own[x];
    bool bad = t < 0 || t >= max_seqs || seq[x] < 0 || seq[x] >= max_seqs;
    if (!bad) bad = (atomicOr(&seen[t >> 5], 1u << (t & 31)) >> (t & 31)) & 1u;   // twice in the call
    if (!bad && dst) bad = C.num_blocks[t] != 0;      // a destination is empty
    if (bad && s_err == 0) s_err = THINKV_ERR_INVALID;
  }
  __syncthreads();
  if (dst)                                            // no destination is also a source
    for (int x = tid; x < n; x += kPlanThreads) {
      const int t = seq[x];
      if (t >= 0 && t < max_seqs && ((seen[t >> 5] >> (t & 31)) & 1u) && s_err == 0) s_err = THINKV_ERR_INVALID;
    }
  int carry[4] = {0, 0, 0, 0};
  for (int x0 = 0; x0 < n; x0 += kPlanThreads) {
    const int x = x0 + tid;
    int v[4] = {0, 0, 0, 0}, tot[4];
    if (x < n) {
#pragma unroll
      for (int c = 0; c < 3; ++c) v[c] = __ldcg(&ws.tot[x * 3 + c]);
      const int b = __ldcg(&ws.nb[x]);
      v[3] = b > 0 ? (b + kChunk - 1) / kChunk : 1;
      if (dst && !leads_group(seq, x)) v[3] = 0;
    }
    block_scan4(v, tot, sh);
    if (x < n) {
#pragma unroll
      for (int c = 0; c < 3; ++c) ws.base[x * 3 + c] = carry[c] + v[c];
      ws.ubase[x] = carry[3] + v[3];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) carry[j] += tot[j];
  }
  __syncthreads();
  if (tid == 0) {
    int err = s_err;
    if (err == 0 && dst)
      for (int c = 0; c < 3; ++c)
        if (!pool_has(C, c, C.page_bump[c], C.page_bump[3 + c], carry[c])) err = THINKV_ERR_OUT_OF_PAGES;
    ws.ubase[n] = carry[3];
    ws.head[0] = err == 0;
    if (err > 0) set_status(C.status, err);
    if (err == 0)
      for (int c = 0; c < 3; ++c) {
        const int bump = C.page_bump[c], released = C.page_bump[3 + c];
        ws.head[1 + c] = carry[c];
        ws.head[4 + c] = bump;
        ws.head[7 + c] = released;
        if (dst) take_pages(C, c, bump, released, carry[c]);
        else C.page_bump[3 + c] = released + carry[c];
      }
  }
}

// Rank within its class (from the call's start) of the table entry e_this
// lane holds in chunk k of listed sequence i.
__device__ inline int call_rank(const TurnoverWs& ws, int i, int k, int c, bool valid) {
  unsigned mine = 0;
#pragma unroll
  for (int cc = 0; cc < 3; ++cc) {
    const unsigned b = __ballot_sync(0xFFFFFFFFu, valid && c == cc);
    if (c == cc) mine = b;
  }
  unsigned below;
  asm("mov.u32 %0, %%lanemask_lt;" : "=r"(below));
  if (!valid) return 0;
  return ws.base[i * 3 + c] + ws.crank[((int64_t)i * ws.chunks + k) * 3 + c] + __popc(mine & below);
}

// Listed sequence of chunk u: the last i with ubase[i] <= u.
__device__ inline int sequence_of_chunk(const TurnoverWs& ws, int32_t n, int u) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ws.ubase[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kApplyWarps * 32)
    release_apply_kernel(CacheView C, int32_t n, const int32_t* __restrict__ seq, int32_t* nseg,
                         int32_t* settled, TurnoverWs ws) {
  pdl_launch_dependents();
  pdl_wait();
  if (ws.head[0] == 0) return;                        // the call was refused
  const int lane = threadIdx.x & 31;
  const int units = ws.ubase[n], nw = gridDim.x * kApplyWarps;
  for (int u = blockIdx.x * kApplyWarps + (threadIdx.x >> 5); u < units; u += nw) {
    const int i = sequence_of_chunk(ws, n, u), k = u - ws.ubase[i], s = seq[i];
    const int64_t row = (int64_t)s * C.L.max_blocks_per_seq;
    const int e = k * kChunk + lane;
    const bool valid = e < ws.nb[i];
    const uint64_t ent = valid ? C.block_table[row + e] : 0;
    const int c = entry_class(ent);
    const int page = (int)entry_page(ent);
    const int rank = call_rank(ws, i, k, c, valid);
    if (valid) {
      // the call's first page ends on top
      int32_t* stack = const_cast<int32_t*>(released_stack(C, c));
      stack[ws.head[7 + c] + ws.head[1 + c] - 1 - rank] = page;
      C.block_table[row + e] = 0;
      C.live_index[row + e] = -1;
    }
    const int cnt = min(kChunk, ws.nb[i] - k * kChunk);
    for (int j = 0; j < cnt; j += 2) {                // slot positions, two pages at a time
      const int from = j + (lane >> 4);
      const int pc = __shfl_sync(0xFFFFFFFFu, c, from & 31), pp = __shfl_sync(0xFFFFFFFFu, page, from & 31);
      if (from < cnt) C.slot_pos[pc][(int64_t)pp * kPage + (lane & 15)] = -1;
    }
    if (k == 0) {
      if (lane < 3) {
        C.free_top[s * 3 + lane] = 0;
        C.fifo_head[s * 3 + lane] = 0;
        C.fifo_tail[s * 3 + lane] = 0;
      }
      if (lane == 0) {
        C.num_blocks[s] = 0;
        C.live_count[s] = 0;
        C.num_live[s] = 0;
        if (nseg) {
          nseg[s] = 0;
          settled[s] = 0;
        }
      }
    }
  }
}

// The sequence's state that is not in pages: chunk k of K copies its share.
__device__ void fork_state(const CacheView& C, int s, int t, int k, int K, const int4* seg, int4* segw,
                           int32_t* nseg, int32_t* settled) {
  const int lane = threadIdx.x & 31;
  const int64_t cap = (int64_t)C.L.max_blocks_per_seq * kPage;
  const int first = k * 32 + lane, step = K * 32;
#pragma unroll 1
  for (int c = 0; c < 3; ++c) {
    const int64_t a = ((int64_t)s * 3 + c) * cap, b = ((int64_t)t * 3 + c) * cap;
    const int top = C.free_top[s * 3 + c];
#pragma unroll 4
    for (int x = first; x < top; x += step) C.free_slots[b + x] = C.free_slots[a + x];
    const int h = C.fifo_head[s * 3 + c], len = C.fifo_tail[s * 3 + c] - h;
    const int64_t h0 = h % cap;
#pragma unroll 4
    for (int x = first; x < len; x += step) {
      int64_t r = h0 + x;
      if (r >= cap) r -= cap;
      C.fifo[b + r] = C.fifo[a + r];
    }
  }
  if (seg)
    for (int x = first; x < nseg[s]; x += step) segw[(int64_t)t * cap + x] = seg[(int64_t)s * cap + x];
  if (k == 0) {
    if (lane < 3) {
      C.free_top[t * 3 + lane] = C.free_top[s * 3 + lane];
      C.fifo_head[t * 3 + lane] = C.fifo_head[s * 3 + lane];
      C.fifo_tail[t * 3 + lane] = C.fifo_tail[s * 3 + lane];
    }
    if (lane == 0) {
      C.num_blocks[t] = C.num_blocks[s];
      C.live_count[t] = C.live_count[s];
      C.num_live[t] = C.num_live[s];
      if (seg) {
        nseg[t] = nseg[s];
        settled[t] = settled[s];
      }
    }
  }
}

__global__ void __launch_bounds__(kApplyWarps * 32, kForkCtas)
    fork_apply_kernel(CacheView C, int32_t n, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, int4* seg, int32_t* nseg, int32_t* settled,
                      TurnoverWs ws) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  if (ws.head[0] == 0) return;                        // the call was refused
  const int H = C.L.num_kv_heads, warps = H * kParts;   // warps of a chunk
  const int64_t items = (int64_t)ws.ubase[n] * warps, nw = (int64_t)gridDim.x * kApplyWarps;
  for (int64_t it = (int64_t)blockIdx.x * kApplyWarps + warp; it < items; it += nw) {
    const int u = (int)(it / warps), hp = (int)(it - (int64_t)u * warps);
    const int h = hp / kParts, part = hp - h * kParts;
    const int i = sequence_of_chunk(ws, n, u), k = u - ws.ubase[i], s = src[i];
    const int64_t srow = (int64_t)s * C.L.max_blocks_per_seq;
    const int nb = ws.nb[i], e = k * kChunk + lane;
    int members = 1;                                  // copies of this source made here
    while (i + members < n && (i + members) % kCopies != 0 && src[i + members] == s) ++members;
    const bool valid = e < nb;
    const uint64_t ent = valid ? C.block_table[srow + e] : 0;
    const int c = entry_class(ent);
    const int64_t page = entry_page(ent);
    const int rank = call_rank(ws, i, k, c, valid) - (valid ? ws.base[i * 3 + c] : 0);   // in the source
    const int cnt = min(kChunk, nb - k * kChunk);
    const int64_t phb = page_head_bytes(C.L.head_dim, C.L.group_size, C.L.bits[c]);
    const uint64_t from_ptr = reinterpret_cast<uint64_t>(C.pool[c]) + (page * H + h) * phb;
    int to[kCopies];                                  // this entry's page in each copy
#pragma unroll
    for (int m = 0; m < kCopies; ++m) {
      to[m] = 0;
      if (valid && m < members)
        to[m] = granted_page(C, c, ws.head[4 + c] - ws.head[7 + c] + ws.base[(i + m) * 3 + c] + rank, ws.head[4 + c]);
    }
    for (int j = part; j < cnt; j += kParts) {        // this part's page-head blocks: read once
      const uint4* a = reinterpret_cast<const uint4*>(__shfl_sync(0xFFFFFFFFu, from_ptr, j));
      const int cj = __shfl_sync(0xFFFFFFFFu, c, j), quads = __shfl_sync(0xFFFFFFFFu, (int)(phb / 16), j);
      uint4* pool = reinterpret_cast<uint4*>(C.pool[cj]) + (int64_t)h * quads;
      for (int q = lane; q < quads + lane; q += 32 * kCopyDepth) {
        uint4 v[kCopyDepth];
#pragma unroll
        for (int x = 0; x < kCopyDepth; ++x)
          if (q + 32 * x < quads) v[x] = __ldcg(a + q + 32 * x);   // (not the read-only path: written by kernels before)
#pragma unroll
        for (int m = 0; m < kCopies; ++m) {
          if (m >= members) break;
          uint4* b = pool + (int64_t)__shfl_sync(0xFFFFFFFFu, to[m], j) * H * quads;
#pragma unroll
          for (int x = 0; x < kCopyDepth; ++x)
            if (q + 32 * x < quads) __stcs(b + q + 32 * x, v[x]);   // (streaming: 5 % faster)
        }
      }
    }
    // the bookkeeping of the chunk, three tasks a copy, spread over its warps
    for (int id = hp; id < 3 * members; id += warps) {
      const int m = id / 3, task = id - 3 * m, t = dst[i + m];
      const int64_t trow = (int64_t)t * C.L.max_blocks_per_seq;
      int mine = 0;
#pragma unroll
      for (int x = 0; x < kCopies; ++x) mine = x == m ? to[x] : mine;
      if (task == 0) {
        if (valid) {
          const int index = C.live_index[srow + e];
          C.block_table[trow + e] = make_entry((uint32_t)mine, c, entry_mask(ent));
          C.live_index[trow + e] = index;
          if (index >= 0) C.live_list[trow + index] = make_live_desc((uint32_t)mine, c, e);
        }
      } else if (task == 1) {                         // slot positions, two pages at a time
#pragma unroll 4
        for (int j = 0; j < kChunk; j += 2) {
          const int from = j + (lane >> 4);
          const int pc = __shfl_sync(0xFFFFFFFFu, c, from);
          const int64_t pa = __shfl_sync(0xFFFFFFFFu, page, from), pb = __shfl_sync(0xFFFFFFFFu, mine, from);
          if (from < cnt) {
            int32_t* pos = C.slot_pos[pc] + (lane & 15);
            pos[pb * kPage] = __ldcg(pos + pa * kPage);
          }
        }
      } else {
        fork_state(C, s, t, k, max(1, (nb + kChunk - 1) / kChunk), seg, seg, nseg, settled);
      }
    }
  }
}

cudaError_t launch_plan(const CacheView& C, int32_t n, const int32_t* seq, const int32_t* dst,
                        const TurnoverWs& ws, cudaStream_t stream) {
  const size_t seen = (size_t)((C.L.max_seqs + 31) / 32) * 4;
  return launch_pdl(turnover_plan_kernel, dim3(n), dim3(kPlanThreads), seen, stream, C, n, seq, dst, ws);
}

}  // namespace

size_t turnover_workspace_bytes(const thinkv_layout& L, int32_t n) {
  return 256 + round256((size_t)n * 4) + 2 * round256((size_t)n * 12) + round256(((size_t)n + 1) * 4) +
         round256((size_t)n * table_chunks(L) * 12);
}

cudaError_t launch_release(const CacheView& C, int32_t n, const int32_t* seq, int32_t* nseg,
                           int32_t* settled, void* workspace, int num_sms, cudaStream_t stream) {
  const TurnoverWs ws = carve(C.L, workspace, n);
  cudaError_t e = launch_plan(C, n, seq, nullptr, ws, stream);
  if (e != cudaSuccess) return e;
  int64_t grid = ((int64_t)n * ws.chunks + kApplyWarps - 1) / kApplyWarps;
  if (grid > (int64_t)num_sms * 8) grid = (int64_t)num_sms * 8;
  return launch_pdl(release_apply_kernel, dim3((unsigned)grid), dim3(kApplyWarps * 32), 0, stream, C, n, seq,
                    nseg, settled, ws);
}

cudaError_t launch_fork(const CacheView& C, int32_t n, const int32_t* src, const int32_t* dst, int4* seg,
                        int32_t* nseg, int32_t* settled, void* workspace, int num_sms,
                        cudaStream_t stream) {
  const TurnoverWs ws = carve(C.L, workspace, n);
  cudaError_t e = launch_plan(C, n, src, dst, ws, stream);
  if (e != cudaSuccess) return e;
  int64_t grid = ((int64_t)n * ws.chunks * C.L.num_kv_heads * kParts + kApplyWarps - 1) / kApplyWarps;
  if (grid > (int64_t)num_sms * kForkCtas) grid = (int64_t)num_sms * kForkCtas;
  return launch_pdl(fork_apply_kernel, dim3((unsigned)grid), dim3(kApplyWarps * 32), 0, stream, C, n, src, dst,
                    seg, nseg, settled, ws);
}

}  // namespace thinkv
