// thinkv_prefix.cu -- attention of many query rows over one sequence's pages:
// the shared part of shared-prefix decode.
//
// A run of count sequences with the same prefix has count * Gq query rows per
// kv-head that read the same keys, so the products are matrix products with up
// to 256 rows: work for tcgen05, where the per-sequence kernel
// (thinkv_decode.cu) is a stream of 16-token steps with 8 columns.
//
// Units of work are (run, kv-head, block of up to 256 rows, tile of 128 key
// slots = 8 live pages); every CTA of the grid (one per SM) takes an equal
// contiguous share of them and leaves one partial (reference exponent, sum,
// unnormalised row) per row and segment it touched, merged by merge_kernel
// (thinkv_decode.cu).  Inside a CTA the roles are
//   warp 17      loads page-head blocks into a byte ring (cp.async.bulk), a tile
//                at a time, descriptors and masks requested one and two batches ahead;
//   warps 8-15   page p of a tile belongs to warp 8 + p: codes and params
//                become fp16 keys and values, written as the K-major,
//                128-byte-swizzled operands of tcgen05.mma (values transposed:
//                the packed V codes pair two tokens of a channel);
//   warp 16      issues S = Q K^T and O += P V (accumulators and P in tensor
//                memory, P over its own scores);
//   warps 0-7    two softmax groups, a thread per row: P = 2^(s - reference) in
//                fp16, sums in fp32, one pass over the scores.  The groups
//                alternate, so that one's exponentials run under the other's products: a
//                block of more than 128 rows gives each group its own rows, a
//                smaller one even and odd key tiles.
// The reference exponent trails the running maximum, by whole numbers: P may
// grow to 2^15 before it is rescaled by a power of two, and starts at 2^7, so that
// the small weights of a long flat row keep fp16's normal precision.  A rescale
// is exact for the fp32 sums and accumulators; weights of the same tile that are
// already stored as fp16 lose what falls below 2^-24, about as if weighed under the
// new reference at once: 2^-24 each at most beside a largest weight of 2^6 or more.
//
// Rounding: keys, values and P enter the products as fp16, the widest type that
// the tensor cores take at full rate beside bf16 (each key or value is one fused
// multiply-add zero + scale * code, rounded once); everything summed is fp32.
//
// 512 rows x 65,536 keys x 8 kv-heads, d = 128, codes of 8, 4 and 2 bits (137
// GFLOP, 84 us at the measured bf16 rate): 183-205 us.  No unit is busy half the time (issue
// slots 55 %, products 38 %): what bounds it is each group's chain of scores ->
// weights -> products, about 5,300 cycles a tile of which 3,000 are softmax; leaving
// out the exponentials, the unpacking or the products alone takes off 10 to 20 %.
// Measured on the way: generic instead of shared-space pointers 259 us,
// operands of the products not warp-uniform (same step), straight-line page writers
// 350 us and masked softmax code unrolled 611 us (both the instruction cache), pages
// waited for one by one 403 us, half tiles with two score buffers per group slower (a
// product of 64 columns costs what one of 128 does), keys written a tile ahead of
// values no faster, spinning instead of suspended waits no faster.

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "thinkv_common.cuh"
#include "thinkv_internal.h"
#include "thinkv_shared.h"

namespace thinkv {

namespace {

constexpr int kTile = kTilePages * kPage;     // 128 key slots
constexpr int kDequantWarps = kTilePages;
constexpr int kWarpMma = 16, kWarpLoad = 17;
// Five warpgroups, so that registers can move between them (setmaxnreg): the
// launch's 640 x 96 become 152 for softmax, 56 for the dequantising warps and 64
// for the last group.
constexpr int kThreads = 20 * 32;
constexpr int kRegsSoftmax = 152, kRegsDequant = 56, kRegsLast = 64;
static_assert(256 * kRegsSoftmax + 256 * kRegsDequant + 128 * kRegsLast <= kThreads * 96, "register shares");
constexpr int kSlots = 4;                     // tiles of raw pages in flight
constexpr float kHeadroom = 7.f;              // P starts at 2^7 at a row's maximum
constexpr float kSlack = 8.f;                 // and grows by up to 2^8 before a rescale

template <int D>
struct Shape {
  static constexpr int kv_bytes = kTile * D * 2;            // one key or value tile
  static constexpr int q_bytes = 128 * D * 2;               // one query tile
  static constexpr int kv_bufs = D == 128 ? 3 : 6;
  static constexpr int ring = 65536;                        // raw bytes in flight
  // tensor memory: score tiles (two, or three where the accumulators leave room:
  // a group's next scores are then made while it still weighs the present ones),
  // then the groups' accumulators
  static constexpr int s_bufs = D == 128 ? 2 : 3;
  static constexpr int col_o = s_bufs * kTile;
  static_assert(col_o + 2 * D <= 512, "tensor memory columns");
  static constexpr int off_q = 0;
  static constexpr int off_kv = 2 * q_bytes;
  static constexpr int off_ring = off_kv + kv_bufs * kv_bytes;
  static constexpr int off_misc = off_ring + ring;
  static constexpr int smem = off_misc + 2048 + 1024;       // + alignment of the base
};

struct Misc {
  uint64_t raw_full[kSlots], raw_empty[kSlots];
  uint64_t kv_full[6], kv_empty[6];
  uint64_t s_full[3], p_full[3];              // of the score tiles
  uint64_t o_done[2][2];                      // [group][odd]: products, counted per group
  uint64_t q_full, drain;
  uint32_t slot_off[kSlots][kTilePages];      // where each page's block lies in the ring
  uint32_t slot_bits[kSlots][kTilePages];     // its class's bits | live mask << 16 (0: no page)
  alignas(16) uint16_t mask[4][kTilePages];   // live masks of the last four tiles
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(Misc) <= 2048, "misc area");

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
// K-major operand, 128-byte swizzle: rows of 128 bytes, 8-row groups 1024 apart
__device__ inline uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// fp16 x fp16 -> fp32, both operands K-major, M = 128
__host__ __device__ constexpr uint32_t instr_desc(int n) {
  return (1u << 4) | ((uint32_t)(n / 8) << 17) | ((uint32_t)(128 / 16) << 24);
}
__device__ inline void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ inline void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ inline void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ inline void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ inline void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ inline void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this thread's row
__device__ inline void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
// Waits for this thread's loads; r, the registers of one of them, are used after it.
__device__ inline void tc_wait_ld_of(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ inline void tc_wait_ld_of(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ inline void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ inline void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ inline void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ inline void mbar_arrive(uint64_t* bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for a phase, with a limit on the probes; false when they ran out or
// another role gave up.  (A probe with a time hint of its own is compiled to
// a loop of sleeps, which wakes late.)
__device__ __forceinline__ bool wait_role(Misc* m, uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t it = 0; it < kWaitLimit; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if (m->abort) return false;
  }
  m->abort = 1;
  return false;
}
// The same for a whole warp, which goes on or gives up together.
__device__ inline bool wait_warp(Misc* m, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, wait_role(m, bar, parity));
}

// ---------------------------------------------------------------------------
// one segment's share of this CTA: which rows, which key tiles
// ---------------------------------------------------------------------------
struct Piece {
  SharedRun run;
  int h, rows;                 // kv-head; query rows of the block
  int first_member;            // call index of the block's first sequence
  int64_t t0, t1;              // key tiles [t0, t1)
  int64_t row;                 // first partial row
  bool pair;                   // more than 128 rows: the groups take 128 rows each
};

__device__ inline Piece piece_at(const PrefixParams& p, int nruns, int64_t u, int64_t U1, int64_t cta) {
  int lo = 0, hi = nruns;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(&p.plan.rstart[mid]) <= u) lo = mid; else hi = mid;
  }
  Piece x;
  const int4 rr = __ldcg(reinterpret_cast<const int4*>(p.plan.run) + lo);
  x.run.first = rr.x; x.run.count = rr.y; x.run.prefix = rr.z; x.run.pages = rr.w;
  const RunShape s = run_shape(x.run.count, x.run.pages, p.Gq);
  const int64_t rel = u - __ldcg(&p.plan.rstart[lo]);
  const int seg = (int)(rel / s.tiles);
  x.t0 = rel - (int64_t)seg * s.tiles;
  x.t1 = min(s.tiles, x.t0 + (U1 - u));
  x.h = seg / s.blocks;
  const int b = seg - x.h * s.blocks;
  x.first_member = x.run.first + b * s.members;
  x.rows = min(s.members, x.run.count - b * s.members) * p.Gq;
  x.row = partial_row(x.run, s, p.Hkv, p.Gq, x.h, b, cta);
  x.pair = x.rows > 128;
  return x;
}

// ---------------------------------------------------------------------------
// codes -> fp16 operands
// ---------------------------------------------------------------------------
__device__ inline __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ inline uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

template <int B, int F>
__device__ constexpr float largest_code() {
  return F == 1 ? (B == 8 ? 448.f : B == 4 ? 6.f : 2.f) : (float)((1 << B) - 1);   // (ternary codes: 0..2)
}
// A finite scale whose largest value zero + scale * code would round past fp16's
// range (from 65504 + 16 on, which would become inf) is lowered to what fits.  A
// scale or zero that is infinite or not a number stays what it is, and so does
// the other scale of a pair.
template <int B, int F>
__device__ __forceinline__ __half2 fitting(__half2 s, __half2 z) {
  const __half2 top = __hfma2(s, __float2half2_rn(largest_code<B, F>()), z);
  if (!__hble2(top, __float2half2_rn(65504.f))) {
    const float2 sf = __half22float2(s), zf = __half22float2(z);
    auto fit = [](float sc, float ze) {
      const float t = fmaf(sc, largest_code<B, F>(), ze);
      return t >= 65520.f && t < INFINITY ? (65504.f - ze) * (1.f / largest_code<B, F>()) : sc;
    };
    s = __halves2half2(__float2half_rd(fit(sf.x, zf.x)), __float2half_rd(fit(sf.y, zf.y)));
  }
  return s;
}

// Codes k of both half-words of w as fp16 numbers (float formats: their values).
// A b-bit code at bit j of its half-word becomes 1024 + code * 2^j by setting the
// exponent, j below a byte; one operation takes it back to the code, exactly.
template <int B, int F>
__device__ inline __half2 code_pair(uint32_t w, int k) {
  if constexpr (F == 1 && B != 2) {
    return as_half2(unpack_float_pair<B>(w, k));
  } else if constexpr (B == 8) {
    return __hsub2(as_half2(unpack_pair<8>(w, k)), __float2half2_rn(1024.f));
  } else {
    const int j = (B * k) % 8;
    const uint32_t m = ((1u << B) - 1u) << j;
    const __half2 x = as_half2(((w >> (B * k / 8 * 8)) & (m | (m << 16))) | 0x64006400u);
    if (j == 0) return __hsub2(x, __float2half2_rn(1024.f));
    const float f = 1.f / (float)(1 << j);
    return __hfma2(x, __float2half2_rn(f), __float2half2_rn(-1024.f * f));
  }
}

// NW words of this lane's portion from byte o on.
template <int LB, int NW>
__device__ __forceinline__ void piece_words(const uint8_t* region, int o, uint32_t (&w)[NW]) {
  const uint8_t* at = region + lane_off(threadIdx.x & 31, o, LB);
  if constexpr (NW == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (NW == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}

// The page writers below stay loops over eight-pair bodies.  Eight warps run
// them for three classes next to the softmax and the products, and the
// instruction cache is what limits them: with straight-line bodies (a quarter
// fewer instructions) the kernel took 350 us instead of 280 on 512 rows x 65,536
// keys x 8 heads.

// Keys of one page-head: rows page * 16 + slot of the key tile.
template <int D, int G, int B, int F>
__device__ __forceinline__ void write_keys(const uint8_t* blk, uint8_t* tile, int page) {
  constexpr int NG = D / G, LANE_BYTES = D * B / 16;
  constexpr int PB = G * B / 32;                       // bytes of a piece (group, slot half)
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t* kpar = reinterpret_cast<const uint32_t*>(blk + 4 * D * B) + g;
  // a row's 16-byte chunks are exchanged with the row's number in its group of eight
  uint8_t* dst = tile + page * (kPage * 128) + g * 128;
  const int off = ((G == 64 ? 2 * t : t) ^ g) << 4;
#pragma unroll 1
  for (int y = 0; y < 2 * NG; ++y) {
    const int gr = y >> 1, r = y & 1;
    uint8_t* to = dst + (gr * G / 64) * (kTile * 128) + r * 1024;
    const int first = G == 64 ? off : off ^ ((gr & 1) << 6);
    if constexpr (B == 16) {
#pragma unroll
      for (int c = 0; c < G / 32; ++c) {
        uint32_t w[4];
        piece_words<LANE_BYTES, 4>(blk, y * PB + 16 * c, w);
        *reinterpret_cast<uint4*>(to + (first ^ (c << 4))) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      uint32_t w[PB >= 4 ? PB / 4 : 1];
      if constexpr (PB == 2) {                         // 4 + 4 codes: bytes -> half-words
        const uint32_t h16 = *reinterpret_cast<const uint16_t*>(blk + lane_off(lane, y * PB, LANE_BYTES));
        w[0] = __byte_perm(h16, 0u, 0x4140);
      } else {
        piece_words<LANE_BYTES, PB / 4>(blk, y * PB, w);
      }
      const __half2 sz = as_half2(kpar[gr * 16 + 8 * r]);
      const __half2 z = __high2half2(sz), s = fitting<B, F>(__low2half2(sz), z);
      constexpr int PAIRS = PB == 2 ? 4 : 16 / B;      // pairs of a word
#pragma unroll
      for (int c = 0; c < G / 32; ++c) {               // 16-byte chunks of the piece
        uint32_t v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int u = c * 4 + x;
          v[x] = as_bits(__hfma2(code_pair<B, F>(w[u / PAIRS], u % PAIRS), s, z));
        }
        *reinterpret_cast<uint4*>(to + (first ^ (c << 4))) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

// Values of one page-head, transposed: row = channel, tokens along the row.
template <int D, int G, int B, int F>
__device__ __forceinline__ void write_values(const uint8_t* blk, uint8_t* tile, int page, uint32_t mask) {
  constexpr int NG = D / G, LANE_BYTES = D * B / 16;
  constexpr int Q = B == 16 ? D / 8 : D * B / 128;     // words per token pair
  constexpr int PER = B == 16 ? 1 : 16 / B;            // codes per half-word
  constexpr int NW = B == 16 ? 4 : B / 2;              // words of a body: 64 channels (raw: 32)
  constexpr int NB = Q / NW;                           // bodies per token pair
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t* vpar = reinterpret_cast<const uint32_t*>(blk + 4 * D * B + 64 * NG) + 2 * t;
  uint8_t* at = tile + (page / 4) * (D * 128) + g * 128 + 4 * t;
  const int off = (((page % 4) * 2) ^ g) << 4;
  // a dead slot's weight is 0, but what its bytes decode to may not be finite:
  // its scale and zero become 0 (codes are finite), or the value (raw fp16, E4M3)
  constexpr bool by_value = B == 16 || (B == 8 && F == 1);
#pragma unroll 1
  for (int y = 0; y < 2 * NB; ++y) {
    const int P = y / NB, b = y % NB;
    const uint32_t tm = mask >> (2 * t + 8 * P);
    const uint32_t dm = ((tm & 1u) ? 0xFFFFu : 0u) | ((tm & 2u) ? 0xFFFF0000u : 0u);
    uint8_t* to = at + (off ^ (P << 4)) + b * (NW * PER * 1024);
    uint32_t w[NW];
    piece_words<LANE_BYTES, NW>(blk + 2 * D * B, (P * Q + b * NW) * 4, w);
    constexpr int GB = B == 16 ? 1 : 64 / G;           // groups of a body
    __half2 s[GB], z[GB];
    if constexpr (B < 16) {
#pragma unroll
      for (int gr = 0; gr < GB; ++gr) {
        const uint32_t* pp = vpar + (b * GB + gr) * 16 + 8 * P;
        const uint32_t p0 = pp[0], p1 = pp[1];
        z[gr] = as_half2(__byte_perm(p0, p1, 0x7632) & dm);
        s[gr] = fitting<B, F>(as_half2(__byte_perm(p0, p1, 0x5410) & dm), z[gr]);
      }
    }
#pragma unroll
    for (int x = 0; x < NW * PER; ++x) {               // channel 16 * (e / 2) + g + 8 * (e % 2), e from b on
      uint32_t v;
      if constexpr (B == 16) {
        v = w[x];
      } else {
        const int gr = x * 8 / G;
        v = as_bits(__hfma2(code_pair<B, F>(w[x / PER], x % PER), s[gr], z[gr]));
      }
      *reinterpret_cast<uint32_t*>(to + x * 1024) = by_value ? v & dm : v;
    }
  }
}

template <int D>
__device__ inline void zero_values(uint8_t* tile, int page) {
  const int lane = threadIdx.x & 31;
  uint8_t* base = tile + (page / 4) * (D * 128);
  for (int x = lane; x < 2 * D; x += 32) {
    const int ch = x >> 1, chunk = (page % 4) * 2 + (x & 1);
    *reinterpret_cast<uint4*>(base + ch * 128 + ((chunk ^ (ch & 7)) << 4)) = make_uint4(0, 0, 0, 0);
  }
}

template <int D, int G, bool KEYS>
__device__ inline void write_page(const uint8_t* blk, uint32_t bits, uint8_t* tile, int page, uint32_t mask) {
  auto go = [&](auto b, auto f) {
    if constexpr (KEYS) write_keys<D, G, b.value, f.value>(blk, tile, page);
    else write_values<D, G, b.value, f.value>(blk, tile, page, mask);
  };
  using std::integral_constant;
  switch (bits) {
    case 256 + 8: go(integral_constant<int, 8>{}, integral_constant<int, 1>{}); break;
    case 256 + 4: go(integral_constant<int, 4>{}, integral_constant<int, 1>{}); break;
    case 256 + 2: go(integral_constant<int, 2>{}, integral_constant<int, 1>{}); break;
    case 8: go(integral_constant<int, 8>{}, integral_constant<int, 0>{}); break;
    case 4: go(integral_constant<int, 4>{}, integral_constant<int, 0>{}); break;
    case 2: go(integral_constant<int, 2>{}, integral_constant<int, 0>{}); break;
    default: go(integral_constant<int, 16>{}, integral_constant<int, 0>{}); break;
  }
}

// Scores of two pages: -inf for dead slots, whatever their keys decoded to.
__device__ __forceinline__ void hide_dead(uint32_t (&s)[32], uint32_t live) {
#pragma unroll
  for (int e = 0; e < 32; ++e) s[e] = (live >> e) & 1u ? s[e] : 0xFF800000u;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 operations in one instruction (each rounded as the single one).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
#pragma unroll
  for (int e = 2; e < 30; e += 4) {
    a = max3(a, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
    b = max3(b, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
  }
  return fmaxf(max3(a, __uint_as_float(s[30]), __uint_as_float(s[31])), b);
}

// N * 32 columns of this thread's row, times f
template <int N>
__device__ __forceinline__ void scale_columns(uint32_t addr, float f) {
#pragma unroll 1
  for (int c = 0; c < N; ++c) {
    uint32_t o[32];
    tmem_ld32(addr + c * 32, o);
    tc_wait_ld_of(o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
    tmem_st32(addr + c * 32, o);
  }
}
// 32 weights (fp16, 16 columns) of this thread's row, times f, a power of two, in
// two steps: as one fp16 factor f would be 0 from 2^-25 on, where weights of up to
// 2^15 are not.
__device__ __forceinline__ void scale_weights(uint32_t addr, float f) {
  uint32_t w[16];
  tmem_ld16(addr, w);
  tc_wait_ld_of(w);
  const __half2 f1 = __float2half2_rn(fmaxf(f, 0x1p-14f)), f2 = __float2half2_rn(fminf(f * 0x1p14f, 1.f));
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = as_bits(__hmul2(__hmul2(as_half2(w[e]), f1), f2));
  tmem_st16(addr, w);
}

// P of 32 scores, 2^(s * scale - ref) in fp16, to 16 columns from `to` on; the
// fp32 weights go into the running sums.
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], float scale, float ref, float2 (&add)[2],
                                          uint32_t to) {
  uint32_t pk[16];
  const float2 k2 = make_float2(scale, scale), r2 = make_float2(-ref, -ref);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float2 y = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), k2, r2);
    y.x = exp2_approx(y.x);
    y.y = exp2_approx(y.y);
    add[(e >> 1) & 1] = add2(add[(e >> 1) & 1], y);
    pk[e / 2] = pack_half2_rn(y.x, y.y);
  }
  tmem_st16(to, pk);
}

// 1 in one lane of the (converged) warp, 0 in the others
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t lead;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(lead));
  return lead;
}

template <int N>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(PrefixParams p) {
  using S = Shape<D>;
  extern __shared__ uint8_t raw_smem[];
  // (an offset from the array, not a rounded address: a pointer made from an integer
  // would be a generic one, and every access slower)
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  Misc* m = reinterpret_cast<Misc*>(smem + S::off_misc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();                                   // the plan
  pdl_launch_dependents();
  const int nruns = __ldcg(p.plan.nruns);
  const int64_t U = __ldcg(&p.plan.rstart[nruns]);
  const int64_t cta = blockIdx.x;
  const int64_t U0 = cta * U / gridDim.x, U1 = (cta + 1) * U / gridDim.x;
  if (U0 >= U1) return;

  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&m->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int x = 0; x < kSlots; ++x) {
      mbar_init(&m->raw_full[x], 1);
      mbar_init(&m->raw_empty[x], kDequantWarps);
    }
    for (int x = 0; x < 6; ++x) {
      mbar_init(&m->kv_full[x], kDequantWarps);
      mbar_init(&m->kv_empty[x], 1);
    }
    for (int x = 0; x < 3; ++x) {
      mbar_init(&m->s_full[x], 1);
      mbar_init(&m->p_full[x], 128);
    }
    for (int x = 0; x < 4; ++x) mbar_init(&m->o_done[x >> 1][x & 1], 1);
    mbar_init(&m->q_full, 256);
    mbar_init(&m->drain, 1);
    m->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m->tmem;

  if (warp >= 16) {
    fewer_regs<kRegsLast>();              // (one instruction for the whole warpgroup)
    if (warp == kWarpLoad) {
      // ---------------- loader ----------------
      // Batches of up to four tiles, a page per lane; the descriptors of a batch are
      // requested two batches ahead and the live masks one.
      struct Batch {
        int64_t row;                            // first entry of the prefix's lists
        uint64_t desc;
        uint32_t mask;
        int h, tiles;
      };
      int64_t u = U0, t = 0;
      Piece x;
      x.t1 = 0;
      auto fetch = [&]() {
        Batch b;
        b.tiles = 0;
        b.mask = 0;
        b.desc = ~0ull;
        b.row = 0;
        b.h = 0;
        if (t >= x.t1) {
          if (u >= U1) return b;
          x = piece_at(p, nruns, u, U1, cta);
          u += x.t1 - x.t0;
          t = x.t0;
        }
        b.row = (int64_t)x.run.prefix * p.max_blocks;
        b.h = x.h;
        b.tiles = (int)min((int64_t)4, x.t1 - t);
        const int64_t j = t * kTilePages + lane;
        if (lane < b.tiles * kTilePages && j < x.run.pages) b.desc = p.live_list[b.row + j];
        t += b.tiles;
        return b;
      };
      uint32_t seq = 0, head = 0, used = 0, oldest = 0;   // byte ring, in tiles: [oldest, seq) hold it
      uint32_t held = 0;                        // lane l < kSlots: ring bytes of the tile in slot l
      bool ok = true;
      Batch cur, nxt;
      cur.tiles = nxt.tiles = 0;
      nxt.desc = ~0ull;
      for (int ahead = 2; ok && (ahead > 0 || cur.tiles > 0); --ahead) {
        if (nxt.desc != ~0ull) nxt.mask = entry_mask(p.table[nxt.row + live_desc_entry(nxt.desc)]);
        const Batch after = fetch();
        if (cur.tiles == 0) {                   // the first two rounds only fetch
          cur = nxt;
          nxt = after;
          continue;
        }
        const bool page = cur.desc != ~0ull;
        const int c = page ? entry_class(cur.desc) : 0;
        const uint32_t bytes = page ? (uint32_t)p.phb[c] : 0u;
        const uint64_t src = reinterpret_cast<uint64_t>(p.pool[c]) +
                             ((uint64_t)entry_page(cur.desc) * p.Hkv + cur.h) * (uint64_t)p.phb[c];
        uint32_t end = bytes;                   // prefix sums inside each tile's eight lanes
#pragma unroll
        for (int o = 1; o < kTilePages; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, end, o);
          if ((lane & 7) >= o) end += y;
        }
        for (int k = 0; k < cur.tiles; ++k, ++seq) {
          const uint32_t total = __shfl_sync(0xFFFFFFFFu, end, 8 * k + 7), slot = seq % kSlots;
          uint32_t pad;
          bool wrap;
          while (true) {                        // until the slot and enough bytes have been given back
            if (used == 0) head = 0;
            wrap = head + total > (uint32_t)S::ring;
            pad = wrap ? (uint32_t)S::ring - head : 0u;
            if (seq - oldest < (uint32_t)kSlots && used + pad + total <= (uint32_t)S::ring) break;
            if (!(ok = wait_warp(m, &m->raw_empty[oldest % kSlots], (oldest / kSlots) & 1u))) break;
            used -= __shfl_sync(0xFFFFFFFFu, held, oldest % kSlots);
            ++oldest;
          }
          if (!ok) break;
          if (wrap) head = 0;
          const uint32_t at = head + end - bytes;
          if ((lane >> 3) == k) {
            m->slot_off[slot][lane & 7] = at;
            m->slot_bits[slot][lane & 7] = page ? ((uint32_t)p.bits[c] | (cur.mask << 16)) : 0u;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&m->raw_full[slot], total);
          __syncwarp();
          if ((lane >> 3) == k && page)
            bulk_g2s(smem + S::off_ring + at, reinterpret_cast<const void*>(src), bytes, &m->raw_full[slot]);
          if (lane == (int)slot) held = pad + total;
          head += total;
          used += pad + total;
        }
        cur = nxt;
        nxt = after;
      }
      // every block in flight has landed before the CTA ends
      if (lane == 0)
        for (uint32_t y = seq > kSlots ? seq - kSlots : 0; y < seq; ++y)
          mbar_wait_bounded(&m->raw_full[y % kSlots], (y / kSlots) & 1u);
    } else if (warp == kWarpMma) {
      // ---------------- products ----------------
      // The whole warp keeps the books, so that the operands are warp-uniform; one
      // lane issues.
      const uint32_t lead = elect_one();
      uint32_t seq = 0, piece = 0, base = 0;           // tiles, pieces, steps before this piece
      uint32_t odd = 0;                                // bit j: group j's next product has an odd number
      const uint64_t q_desc = operand_desc(smem_u32(smem + S::off_q)), kv_desc = operand_desc(smem_u32(smem + S::off_kv));
      bool ok = true;
      for (int64_t u = U0; ok && u < U1; ++piece) {
        const Piece x = piece_at(p, nruns, u, U1, cta);
        u += x.t1 - x.t0;
        const uint32_t T = __shfl_sync(0xFFFFFFFFu, (uint32_t)(x.t1 - x.t0), 0);
        const uint32_t pair = __shfl_sync(0xFFFFFFFFu, (uint32_t)x.pair, 0);
        const uint32_t steps = T << pair;              // products of one group and one key tile
        ok = wait_warp(m, &m->q_full, piece & 1u);
        constexpr uint32_t NS = S::s_bufs;             // scores are made NS steps ahead of the values
        for (uint32_t s = 0; ok && s < steps + NS; ++s) {
          if (s >= NS) {                               // O_j += P_j V
            const uint32_t r = s - NS, j = r & 1u, pos = 2 * (seq + (r >> pair)) + 1, buf = pos % S::kv_bufs;
            const uint32_t g = base + r, sb = g % NS;
            if (!pair || j == 0) ok = wait_warp(m, &m->kv_full[buf], (pos / S::kv_bufs) & 1u);
            ok = ok && wait_warp(m, &m->p_full[sb], (g / NS) & 1u);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = kv_desc + buf * (S::kv_bytes >> 4);
            const uint32_t d = tmem + S::col_o + j * D, a = tmem + sb * kTile;
            if (lead) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                mma_ts(d, a + k * 8, b + (((k / 4) * (D * 128) + (k % 4) * 32) >> 4), instr_desc(D), r >= 2 || k > 0);
              if (!pair || j == 1) mma_commit(&m->kv_empty[buf]);
              mma_commit(&m->o_done[j][(odd >> j) & 1u]);
            }
            odd ^= 1u << j;
            __syncwarp();
          }
          if (s < steps) {                             // S_j = Q_j K^T
            const uint32_t j = s & 1u, pos = 2 * (seq + (s >> pair)), buf = pos % S::kv_bufs;
            const uint32_t sb = (base + s) % NS;
            if (!pair || j == 0) {
              ok = wait_warp(m, &m->kv_full[buf], (pos / S::kv_bufs) & 1u);
              if (!ok) break;
            }
            tc_fence_after();
            const uint64_t a = q_desc + (pair ? j : 0u) * (S::q_bytes >> 4), b = kv_desc + buf * (S::kv_bytes >> 4);
            const uint32_t d = tmem + sb * kTile;
            if (lead) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k / 4) * (128 * 128) + (k % 4) * 32) >> 4;
                mma_ss(d, a + off, b + off, instr_desc(kTile), k > 0);
              }
              mma_commit(&m->s_full[sb]);
              if (!pair || j == 1) mma_commit(&m->kv_empty[buf]);
            }
            __syncwarp();
          }
        }
        base += steps;
        seq += T;
      }
    }
  } else if (warp >= 8) {
    fewer_regs<kRegsDequant>();
    // ---------------- codes -> fp16 operands ----------------
    const int page = warp - 8;
    uint32_t seq = 0;
    bool ok = true;
    for (int64_t u = U0; ok && u < U1;) {
      const Piece x = piece_at(p, nruns, u, U1, cta);
      u += x.t1 - x.t0;
      for (int64_t t = x.t0; t < x.t1; ++t, ++seq) {
        const uint32_t slot = seq % kSlots;
        if (!(ok = wait_warp(m, &m->raw_full[slot], (seq / kSlots) & 1u))) break;
        const uint32_t info = m->slot_bits[slot][page], bits = info & 0xFFFFu, mask = info >> 16;
        const uint8_t* blk = smem + S::off_ring + m->slot_off[slot][page];
        uint32_t pos = 2 * seq, buf = pos % S::kv_bufs;
        if (!(ok = wait_warp(m, &m->kv_empty[buf], ((pos / S::kv_bufs) & 1u) ^ 1u))) break;
        if (lane == 0) m->mask[seq & 3][page] = (uint16_t)mask;
        if (bits) write_page<D, G, true>(blk, bits, smem + S::off_kv + buf * S::kv_bytes, page, mask);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->kv_full[buf]);
        ++pos;
        buf = pos % S::kv_bufs;
        if (!(ok = wait_warp(m, &m->kv_empty[buf], ((pos / S::kv_bufs) & 1u) ^ 1u))) break;
        if (bits) write_page<D, G, false>(blk, bits, smem + S::off_kv + buf * S::kv_bytes, page, mask);
        else zero_values<D>(smem + S::off_kv + buf * S::kv_bytes, page);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&m->raw_empty[slot]);
          mbar_arrive(&m->kv_full[buf]);
        }
      }
    }
  } else {
    more_regs<kRegsSoftmax>();
    // ---------------- softmax ----------------
    const uint32_t j = warp >> 2;                    // group
    const int row = (warp & 3) * 32 + lane;          // row of the group's tile
    const uint32_t t_row = tmem + ((uint32_t)(warp & 3) << 21), t_o = t_row + S::col_o + j * D;
    uint32_t seq = 0, piece = 0, base = 0, no = 0;   // tiles, pieces, steps, products of the group so far
    // Product i of the group is done.  Two barriers take turns: a wait sees only
    // the parity of the phase, and the product before the awaited one may or may not be done.
    auto wait_product = [&](uint32_t i) { return wait_warp(m, &m->o_done[j][i & 1u], (i >> 1) & 1u); };
    bool ok = true;
    for (int64_t u = U0; ok && u < U1; ++piece) {
      const Piece x = piece_at(p, nruns, u, U1, cta);
      const uint32_t T = (uint32_t)(x.t1 - x.t0);
      u += T;
      // ---- queries: this group's 128 rows (a small block's rows by group 0) ----
      if (x.pair || j == 0) {
        // Rows of consecutive sequences: D/8 lanes a row, eight loads in flight each
        constexpr int RL = D / 8, RS = 128 / RL;        // lanes of a row, rows of a step
        const int c = tid % RL, r0 = (tid & 127) / RL;
        const uint32_t inv = 65536u / (uint32_t)p.Gq + 1;   // lr / Gq for lr < 256, Gq <= 8
        uint8_t* dst = smem + S::off_q + j * S::q_bytes + (c / 8) * (128 * 128);
#pragma unroll 1
        for (int y = 0; y < 128 / RS; y += 8) {
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int lr = j * 128 + r0 + (y + k) * RS;
            v[k] = make_uint4(0, 0, 0, 0);
            if (lr < x.rows) {
              const int in = (int)(((uint32_t)lr * inv) >> 16), hd = x.h * p.Gq + lr - in * p.Gq;
              v[k] = __ldg(reinterpret_cast<const uint4*>(p.q + ((int64_t)(x.first_member + in) * p.Hq + hd) * D) + c);
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = r0 + (y + k) * RS;
            *reinterpret_cast<uint4*>(dst + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = v[k];
          }
        }
        fence_proxy_async_smem();
      }
      mbar_arrive(&m->q_full);
      // Both groups are past the piece before: every earlier phase of the score
      // tiles is over, so that the parities below mean this piece's (and a group
      // without a step arrives in the right phase the next time).
      if (!(ok = wait_warp(m, &m->q_full, piece & 1u))) break;

      float ref = -INFINITY, sum = 0.f;
      const uint32_t steps = x.pair ? 2 * T : T;
      uint32_t done = 0;
      for (uint32_t r = j; r < steps; r += 2, ++done) {
        constexpr uint32_t NS = S::s_bufs;
        const uint32_t t = x.pair ? r >> 1 : r, sb = (base + r) % NS;
        if (!(ok = ok && wait_warp(m, &m->s_full[sb], ((base + r) / NS) & 1u))) break;
        tc_fence_after();
        const uint32_t t_s = t_row + sb * kTile;
        const uint4 live = *reinterpret_cast<const uint4*>(m->mask[(seq + t) & 3]);
        const bool full = (live.x & live.y & live.z & live.w) == 0xFFFFFFFFu;
        // ---- P = 2^(s - ref), packed over the tile's own scores, 32 at a time ----
        float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weigh = [&](uint32_t (&sc)[32], int c, uint32_t live_c) {
          if (!full) hide_dead(sc, live_c);
          const float mx = max32(sc) * p.scale_log2 - kHeadroom;
          // a row whose maximum has outgrown its reference moves it, and what
          // was weighed and summed under it, by a whole power of two
          if (__any_sync(0xFFFFFFFFu, mx > ref + kSlack)) {
            const float to = mx > ref + kSlack ? ceilf(mx) : ref;
            const float f = ref > -INFINITY ? exp2_approx(ref - to) : (to > -INFINITY ? 0.f : 1.f);
            // what is scaled here was stored by this thread (weights of earlier columns,
            // accumulators of an earlier move): a load is not ordered behind such a store
            tc_wait_st();
            if (done > 0) {                      // the group's last product may still be running
              ok = ok && wait_product(no + done - 1);
              tc_fence_after();
              scale_columns<D / 32>(t_o, f);
            }
            for (int x = 0; x < c; ++x) scale_weights(t_s + x * 16, f);
            add[0].x *= f; add[0].y *= f; add[1].x *= f; add[1].y *= f;
            sum *= f;
            ref = to;
          }
          weights32(sc, p.scale_log2, ref > -INFINITY ? ref : 0.f, add, t_s + c * 16);
        };
        uint32_t s0[32], s1[32];                 // the next 32 columns arrive under the present ones
        tmem_ld32(t_s, s0);
        tc_wait_ld_of(s0);
#pragma unroll 1
        for (int c = 0; c < 4; c += 2) {
          tmem_ld32(t_s + c * 32 + 32, s1);
          weigh(s0, c, c ? live.z : live.x);
          tc_wait_ld_of(s1);
          if (c == 0) tmem_ld32(t_s + 64, s0);
          weigh(s1, c + 1, c ? live.w : live.y);
          tc_wait_ld_of(s0);
        }
        sum += (add[0].x + add[0].y) + (add[1].x + add[1].y);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&m->p_full[sb]);
      }
      if (!ok) break;
      seq += T;
      base += steps;
      // ---- the partial rows ----
      const int lr = (x.pair ? j * 128 : 0) + row;
      const int64_t at = x.row + (x.pair ? (int64_t)lr : (int64_t)j * x.rows + lr);
      float4* po = reinterpret_cast<float4*>(p.o + at * D);
      if (done > 0) {
        if (!(ok = wait_product(no + done - 1))) break;
        no += done;
        tc_fence_after();
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (done > 0) {
          tmem_ld32(t_o + c * 32, o);
          tc_wait_ld_of(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (lr < x.rows) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            po[c * 8 + e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                        __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        }
      }
      tc_fence_before();
      if (lr < x.rows) p.ml[at] = make_float2(done > 0 ? ref : -INFINITY, sum);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) {
    if (m->abort) {
      // products may still be in flight: a last commit covers them all
      if (elect_one()) {
        set_status(p.status, THINKV_ERR_TIMEOUT);
        mma_commit(&m->drain);
        mbar_wait_bounded(&m->drain, 0);
      }
      __syncwarp();
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int D, int G>
cudaError_t launch_t(const PrefixParams& p, int grid, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(prefix_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Shape<D>::smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_kernel<D, G>, dim3(grid), dim3(kThreads), (size_t)Shape<D>::smem, stream, p);
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, int D, int G, int grid, cudaStream_t stream) {
  if (D == 128 && G == 64) return launch_t<128, 64>(p, grid, stream);
  if (D == 128 && G == 32) return launch_t<128, 32>(p, grid, stream);
  if (D == 64 && G == 64) return launch_t<64, 64>(p, grid, stream);
  return launch_t<64, 32>(p, grid, stream);
}

}  // namespace thinkv
