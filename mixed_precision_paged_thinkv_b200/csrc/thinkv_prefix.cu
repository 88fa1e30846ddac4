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
// unnormalised row) per row and segment it touched, merged by the combine
// kernel.  Inside a CTA the roles are
//   warp 17      loads page-head blocks into a byte ring (cp.async.bulk);
//   warps 8-15   page p of a tile belongs to warp 8 + p: codes and params
//                become fp16 keys and values, written as the K-major,
//                128-byte-swizzled operands of tcgen05.mma (values transposed:
//                the packed V codes pair two tokens of a channel);
//   warp 16      one thread issues S = Q K^T and O += P V (accumulators and P
//                in tensor memory);
//   warps 0-7    two softmax groups, a thread per row: running maximum, P =
//                2^(s - reference) in fp16, sums in fp32.  The groups alternate, so that
//                one's exponentials run under the other's products: a block of
//                more than 128 rows gives each group its own rows, a smaller one
//                even and odd key tiles.
// The reference exponent trails the running maximum: P may grow to 2^15 before
// the accumulators are rescaled, and starts at 2^7, so that the small weights of
// a long flat row keep fp16's normal precision.
//
// Rounding: keys, values and P enter the products as fp16 (each value is one
// fused multiply-add zero + scale * code, rounded once); sums are fp32.
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
constexpr int kThreads = 18 * 32;
constexpr int kSlots = 32;                    // raw page slots in flight (4 tiles)
constexpr float kHeadroom = 7.f;              // P starts at 2^7 at a row's maximum
constexpr float kSlack = 8.f;                 // and grows by up to 2^8 before a rescale

template <int D>
struct Shape {
  static constexpr int kv_bytes = kTile * D * 2;            // one key or value tile
  static constexpr int q_bytes = 128 * D * 2;               // one query tile
  static constexpr int kv_bufs = D == 128 ? 3 : 6;
  static constexpr int ring = 65536;                        // raw bytes in flight
  static constexpr int off_q = 0;
  static constexpr int off_kv = 2 * q_bytes;
  static constexpr int off_ring = off_kv + kv_bufs * kv_bytes;
  static constexpr int off_misc = off_ring + ring;
  static constexpr int smem = off_misc + 2048 + 1024;       // + alignment of the base
};

struct Misc {
  uint64_t raw_full[kSlots], raw_empty[kSlots];
  uint64_t kv_full[6], kv_empty[6];
  uint64_t s_full[2], p_full[2], o_full[2], q_full, drain;
  uint32_t slot_off[kSlots];                  // where the slot's block lies in the ring
  uint32_t slot_bits[kSlots];                 // its class's bits (0: no page)
  uint32_t slot_size[kSlots];                 // ring bytes it holds (loader's books)
  uint16_t mask[4][kTilePages];               // live masks of the last four tiles
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
__device__ inline void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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

// Waits for a phase for two seconds at most; false when they ran out or another
// role gave up.
constexpr uint64_t kWaitNs = 2000000000ull;
__device__ inline uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ inline bool wait_role(Misc* m, uint64_t* bar, uint32_t parity) {
  if (mbar_test_wait(bar, parity)) return true;
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  while (!m->abort && now_ns() - t0 < kWaitNs)
    for (int it = 0; it < 32; ++it)
      if (mbar_try_wait(bar, parity)) return true;
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
template <int B, int F>
__device__ constexpr float largest_code() {
  return F == 1 ? (B == 8 ? 448.f : B == 4 ? 6.f : 2.f) : (float)((1 << B) - 1);   // (ternary codes: 0..2)
}

// A scale whose largest value zero + scale * code would round past fp16's
// range is lowered to what fits (a value past 65504 + 16 would become inf).
template <int B, int F>
__device__ inline __half2 fitting_scale(__half2 s, __half2 z) {
  const __half2 top = __hfma2(s, __float2half2_rn(largest_code<B, F>()), z);
  if (__hisinf(__low2half(top)) || __hisinf(__high2half(top))) {
    const float2 zf = __half22float2(z), sf = __half22float2(s);
    const float k = 1.f / largest_code<B, F>();
    s = __halves2half2(__float2half_rd(fminf(sf.x, (65504.f - zf.x) * k)),
                       __float2half_rd(fminf(sf.y, (65504.f - zf.y) * k)));
  }
  return s;
}

// Pair k of word w as fp16 values.
template <int B, int F>
__device__ inline uint32_t value_pair(uint32_t w, int k, __half2 s, __half2 z) {
  __half2 c;
  if constexpr (F == 1 && B != 2) {
    const uint32_t x = unpack_float_pair<B>(w, k);
    c = *reinterpret_cast<const __half2*>(&x);
  } else {
    const uint32_t x = hsub2_bits(unpack_pair<B>(w, k), 0x64006400u);
    c = *reinterpret_cast<const __half2*>(&x);
  }
  const __half2 v = __hfma2(c, s, z);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Keys of one page-head: rows page * 16 + slot of the key tile.
template <int D, int G, int B, int F>
__device__ inline void write_keys(const uint8_t* blk, uint8_t* tile, int page) {
  constexpr int NG = D / G, LANE_BYTES = D * B / 16;
  constexpr int PB = G * B / 32, NW = PB >= 4 ? PB / 4 : 1;
  constexpr int U = LANE_BYTES < 16 ? LANE_BYTES : 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t* kpar = reinterpret_cast<const uint32_t*>(blk + 4 * D * B);
  const uint8_t* kbase = blk + lane * U;
  constexpr bool KALL = LANE_BYTES <= 32;
  constexpr int KW = KALL ? LANE_BYTES / 4 : 2 * PB / 4;
  uint32_t kw[KW];
  if constexpr (KALL) lane_words<LANE_BYTES, KW>(kbase, 0, kw);
#pragma unroll
  for (int gr = 0; gr < NG; ++gr) {
    if constexpr (!KALL) lane_words<LANE_BYTES, KW>(kbase, gr * 2 * PB / 4, kw);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t w[NW];
      if constexpr (PB == 2) {
        const uint32_t h16 = (kw[gr] >> (16 * r)) & 0xFFFFu;
        w[0] = (h16 & 0xFFu) | ((h16 & 0xFF00u) << 8);
      } else {
#pragma unroll
        for (int x = 0; x < NW; ++x) w[x] = kw[(KALL ? gr * 2 * NW : 0) + r * NW + x];
      }
      __half2 s = __float2half2_rn(1.f), z = __float2half2_rn(0.f);
      if constexpr (B < 16) {
        const uint32_t par = kpar[gr * 16 + g + 8 * r];
        const __half2 sz = *reinterpret_cast<const __half2*>(&par);
        s = __low2half2(sz);
        z = __high2half2(sz);
        s = fitting_scale<B, F>(s, z);
      }
      constexpr int PAIRS = B == 16 ? 1 : (PB == 2 ? 4 : 16 / B);   // pairs of a word
      const int row = page * kPage + g + 8 * r;
#pragma unroll
      for (int c = 0; c < G / 32; ++c) {               // 16-byte chunks of the piece
        uint32_t v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int u = c * 4 + x;
          if constexpr (B == 16) v[x] = w[u];
          else v[x] = value_pair<B, F>(w[u / PAIRS], u % PAIRS, s, z);
        }
        const int ch = gr * G + t * (G / 4) + c * 8;   // first channel of the chunk
        uint8_t* dst = tile + (ch / 64) * (kTile * 128) + row * 128 + ((((ch % 64) / 8) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

// Values of one page-head, transposed: row = channel, tokens along the row.
template <int D, int G, int B, int F>
__device__ inline void write_values(const uint8_t* blk, uint8_t* tile, int page, uint32_t mask) {
  constexpr int NG = D / G, LANE_BYTES = D * B / 16;
  constexpr int Q = B == 16 ? D / 8 : D * B / 128;     // words per token pair
  constexpr int PER = B == 16 ? 1 : 16 / B;            // codes per half-word
  constexpr int U = LANE_BYTES < 16 ? LANE_BYTES : 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t* vpar = reinterpret_cast<const uint32_t*>(blk + 4 * D * B + 64 * NG);
  const uint8_t* vbase = blk + 2 * D * B + lane * U;
  constexpr bool VALL = LANE_BYTES <= 32;
  uint32_t vall[VALL ? LANE_BYTES / 4 : 1];
  if constexpr (VALL) lane_words<LANE_BYTES, (VALL ? LANE_BYTES / 4 : 1)>(vbase, 0, vall);
  // a dead slot's weight is 0, but what its bytes decode to may not be finite
  const uint32_t tm = mask >> (2 * t);
  const uint32_t dm[2] = {((tm & 1u) ? 0xFFFFu : 0u) | ((tm & 2u) ? 0xFFFF0000u : 0u),
                          ((tm & 0x100u) ? 0xFFFFu : 0u) | ((tm & 0x200u) ? 0xFFFF0000u : 0u)};
  uint8_t* base = tile + (page / 4) * (D * 128) + 4 * t;
#pragma unroll
  for (int P = 0; P < 2; ++P) {
    const int chunk = (page % 4) * 2 + P;
    uint8_t* at = base + g * 128 + ((chunk ^ g) << 4);
    constexpr int HALF = Q >= 2 ? 2 : 1, QH = Q / HALF;
#pragma unroll
    for (int hf = 0; hf < HALF; ++hf) {
      uint32_t vr[QH];
      if constexpr (VALL) {
#pragma unroll
        for (int x = 0; x < QH; ++x) vr[x] = vall[P * Q + hf * QH + x];
      } else {
        lane_words<LANE_BYTES, QH>(vbase, P * Q + hf * QH, vr);
      }
      __half2 s = __float2half2_rn(1.f), z = __float2half2_rn(0.f);
#pragma unroll
      for (int x = 0; x < QH * PER; ++x) {
        const int e = hf * QH * PER + x;               // channel 16 * (e / 2) + g + 8 * (e % 2)
        if constexpr (B < 16) {
          if (x == 0 || (e * 8) % G == 0) {            // the next group's params
            const int gr = e * 8 / G;
            const uint32_t p0 = vpar[gr * 16 + 2 * t + 8 * P], p1 = vpar[gr * 16 + 2 * t + 8 * P + 1];
            const uint32_t sb = __byte_perm(p0, p1, 0x5410), zb = __byte_perm(p0, p1, 0x7632);
            s = *reinterpret_cast<const __half2*>(&sb);
            z = *reinterpret_cast<const __half2*>(&zb);
            s = fitting_scale<B, F>(s, z);
          }
        }
        uint32_t v;
        if constexpr (B == 16) v = vr[x];
        else v = value_pair<B, F>(vr[x / PER], x % PER, s, z);
        *reinterpret_cast<uint32_t*>(at + e * 1024) = v & dm[P];
      }
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

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(PrefixParams p) {
  using S = Shape<D>;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
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
      mbar_init(&m->raw_empty[x], 1);
    }
    for (int x = 0; x < 6; ++x) {
      mbar_init(&m->kv_full[x], kDequantWarps);
      mbar_init(&m->kv_empty[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&m->s_full[x], 1);
      mbar_init(&m->p_full[x], 128);
      mbar_init(&m->o_full[x], 1);
    }
    mbar_init(&m->q_full, 256);
    mbar_init(&m->drain, 1);
    m->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m->tmem;

  if (warp == kWarpLoad) {
    // ---------------- loader ----------------
    uint32_t seq = 0;                           // tiles so far
    uint32_t head = 0, used = 0, oldest = 0;    // byte ring; oldest: first page whose bytes are held
    uint32_t issued = 0;                        // pages handed to the ring
    bool ok = true;
    for (int64_t u = U0; ok && u < U1;) {
      const Piece x = piece_at(p, nruns, u, U1, cta);
      u += x.t1 - x.t0;
      const int64_t row = (int64_t)x.run.prefix * p.max_blocks;
      for (int64_t t = x.t0; ok && t < x.t1; t += 4) {
        // 32 pages: descriptors and masks, a page per lane
        const int64_t j = t * kTilePages + lane;
        const int tiles = (int)min((int64_t)4, x.t1 - t);
        uint64_t src = 0;
        int cls = -1;
        uint32_t mask = 0;
        if (j < x.run.pages && lane < tiles * kTilePages) {
          const uint64_t desc = p.live_list[row + j];
          cls = entry_class(desc);
          src = reinterpret_cast<uint64_t>(p.pool[cls]) +
                ((uint64_t)entry_page(desc) * p.Hkv + x.h) * (uint64_t)p.phb[cls];
          mask = entry_mask(p.table[row + live_desc_entry(desc)]);
        }
        for (int k = 0; ok && k < tiles * kTilePages; ++k) {
          const uint64_t a = __shfl_sync(0xFFFFFFFFu, src, k);
          const int c = __shfl_sync(0xFFFFFFFFu, cls, k);
          const uint32_t mk = __shfl_sync(0xFFFFFFFFu, mask, k);
          if (lane == 0) {
            const uint32_t page = (seq + (k >> 3)) * kTilePages + (k & 7);
            const uint32_t slot = page % kSlots;
            const uint32_t bytes = c < 0 ? 0u : (uint32_t)p.phb[c];
            const bool wrap = head + bytes > (uint32_t)S::ring;    // the rest of the ring is skipped
            const uint32_t pad = wrap ? (uint32_t)S::ring - head : 0u;
            // the slot's last page and enough bytes must have been given back
            while (ok && (page - oldest >= (uint32_t)kSlots || used + pad + bytes > (uint32_t)S::ring)) {
              ok = wait_role(m, &m->raw_empty[oldest % kSlots], (oldest / kSlots) & 1u);
              used -= m->slot_size[oldest % kSlots];
              ++oldest;
            }
            if (ok) {
              if (wrap) head = 0;
              m->slot_size[slot] = pad + bytes;
              m->slot_off[slot] = head;
              m->slot_bits[slot] = c < 0 ? 0u : ((uint32_t)p.bits[c] | (mk << 16));
              if (bytes) {
                mbar_arrive_expect_tx(&m->raw_full[slot], bytes);
                bulk_g2s(smem + S::off_ring + head, reinterpret_cast<const void*>(a), bytes, &m->raw_full[slot]);
              } else {
                mbar_arrive(&m->raw_full[slot]);
              }
              head += bytes;
              used += pad + bytes;
              issued = page + 1;
            }
          }
          ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0);
        }
        seq += tiles;
      }
    }
    // every block in flight has landed before the CTA ends
    if (lane == 0)
      for (uint32_t x = issued > kSlots ? issued - kSlots : 0; x < issued; ++x)
        mbar_wait_bounded(&m->raw_full[x % kSlots], (x / kSlots) & 1u);
  } else if (warp >= 8 && warp < 8 + kDequantWarps) {
    // ---------------- codes -> fp16 operands ----------------
    const int page = warp - 8;
    uint32_t seq = 0;
    bool ok = true;
    for (int64_t u = U0; ok && u < U1;) {
      const Piece x = piece_at(p, nruns, u, U1, cta);
      u += x.t1 - x.t0;
      for (int64_t t = x.t0; t < x.t1; ++t, ++seq) {
        const uint32_t n = seq * kTilePages + page, slot = n % kSlots;
        if (!(ok = wait_warp(m, &m->raw_full[slot], (n / kSlots) & 1u))) break;
        const uint32_t info = m->slot_bits[slot], bits = info & 0xFFFFu, mask = info >> 16;
        const uint8_t* blk = smem + S::off_ring + m->slot_off[slot];
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
  } else if (warp == kWarpMma) {
    // ---------------- products ----------------
    if (lane == 0) {
      uint32_t seq = 0, piece = 0, np[2] = {0, 0};
      const uint32_t q_addr = smem_u32(smem + S::off_q), kv_addr = smem_u32(smem + S::off_kv);
      bool ok = true;
      for (int64_t u = U0; ok && u < U1; ++piece) {
        const Piece x = piece_at(p, nruns, u, U1, cta);
        const uint32_t T = (uint32_t)(x.t1 - x.t0);
        u += T;
        const uint32_t steps = x.pair ? 2 * T : T;   // products of one group and one key tile
        ok = wait_role(m, &m->q_full, piece & 1u);
        tc_fence_after();
        auto qk = [&](uint32_t s) {
          const uint32_t j = s & 1u, kt = x.pair ? s >> 1 : s, pos = 2 * (seq + kt), buf = pos % S::kv_bufs;
          if (!x.pair || j == 0) {
            ok = ok && wait_role(m, &m->kv_full[buf], (pos / S::kv_bufs) & 1u);
            if (!ok) return;
            tc_fence_after();
          }
          const uint32_t a = q_addr + (x.pair ? j : 0u) * S::q_bytes, b = kv_addr + buf * S::kv_bytes;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * (128 * 128) + (k % 4) * 32;
            mma_ss(tmem + j * 128, operand_desc(a + off), operand_desc(b + off), instr_desc(kTile), k > 0);
          }
          mma_commit(&m->s_full[j]);
          if (!x.pair || j == 1) mma_commit(&m->kv_empty[buf]);
        };
        auto pv = [&](uint32_t s) {
          const uint32_t j = s & 1u, kt = x.pair ? s >> 1 : s, pos = 2 * (seq + kt) + 1, buf = pos % S::kv_bufs;
          if (!x.pair || j == 0) ok = ok && wait_role(m, &m->kv_full[buf], (pos / S::kv_bufs) & 1u);
          ok = ok && wait_role(m, &m->p_full[j], np[j] & 1u);
          if (!ok) return;
          ++np[j];
          tc_fence_after();
          const uint32_t b = kv_addr + buf * S::kv_bytes;
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k) {
            const uint32_t off = (k / 4) * (D * 128) + (k % 4) * 32;
            mma_ts(tmem + 256 + j * D, tmem + j * 128 + k * 8, operand_desc(b + off), instr_desc(D),
                   s >= 2 || k > 0);
          }
          if (!x.pair || j == 1) mma_commit(&m->kv_empty[buf]);
          if (s + 2 >= steps) mma_commit(&m->o_full[j]);
        };
        if (ok) qk(0);
        if (ok && steps > 1) qk(1);
        for (uint32_t s = 0; ok && s < steps; ++s) {
          pv(s);
          if (ok && s + 2 < steps) qk(s + 2);
        }
        seq += T;
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---------------- softmax ----------------
    const uint32_t j = warp >> 2;                    // group
    const int row = (warp & 3) * 32 + lane;          // row of the group's tile
    const uint32_t t_s = tmem + j * 128 + ((uint32_t)(warp & 3) << 21);
    const uint32_t t_o = tmem + 256 + j * D + ((uint32_t)(warp & 3) << 21);
    uint32_t seq = 0, ns = 0, no = 0, piece = 0;
    bool ok = true;
    for (int64_t u = U0; ok && u < U1; ++piece) {
      const Piece x = piece_at(p, nruns, u, U1, cta);
      const uint32_t T = (uint32_t)(x.t1 - x.t0);
      u += T;
      // ---- queries: this group's 128 rows (a small block's rows by group 0) ----
      if (x.pair || j == 0) {
        const int lo = j * 128;
        for (int i = tid & 127; i < 128 * (D / 8); i += 128) {
          const int r = i / (D / 8), c = i % (D / 8), lr = lo + r;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (lr < x.rows) {
            const int mem = x.first_member + lr / p.Gq, hd = x.h * p.Gq + lr % p.Gq;
            v = *reinterpret_cast<const uint4*>(p.q + ((int64_t)mem * p.Hq + hd) * D + c * 8);
          }
          *reinterpret_cast<uint4*>(smem + S::off_q + j * S::q_bytes + (c / 8) * (128 * 128) + r * 128 +
                                    (((c % 8) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
      }
      mbar_arrive(&m->q_full);

      float ref = -INFINITY, sum = 0.f;
      const uint32_t first = x.pair ? 0 : j, step = x.pair ? 1 : 2;
      uint32_t done = 0;
      for (uint32_t t = first; t < T; t += step, ++done) {
        if (!(ok = wait_warp(m, &m->s_full[j], ns & 1u))) break;
        ++ns;
        tc_fence_after();
        uint32_t live[4];
        {
          const uint2* mp = reinterpret_cast<const uint2*>(m->mask[(seq + t) & 3]);
          const uint2 m0 = mp[0], m1 = mp[1];
          live[0] = m0.x; live[1] = m0.y; live[2] = m1.x; live[3] = m1.y;
        }
        const bool full = (live[0] & live[1] & live[2] & live[3]) == 0xFFFFFFFFu;
        // ---- the row's maximum over the tile ----
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t s[32];
          tmem_ld32(t_s + c * 32, s);
          tc_wait_ld();
          if (full) {
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(s[e]));
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              mx = fmaxf(mx, (live[c] >> e) & 1u ? __uint_as_float(s[e]) : -INFINITY);
          }
        }
        mx *= p.scale_log2;
        // ---- move the reference where the maximum has outgrown it ----
        const bool move = mx - kHeadroom > ref + kSlack || done == 0;
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float to = move ? mx - kHeadroom : ref;
          const float f = done == 0 ? 0.f : exp2_approx(ref - to);
          if (done > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(t_o + c * 32, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(t_o + c * 32, o);
            }
          }
          sum *= f;
          ref = to;
        }
        // ---- P = 2^(s - ref), packed over the tile's own scores ----
        float add[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t s[32], pk[16];
          tmem_ld32(t_s + c * 32, s);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a = exp2_approx(fmaf(__uint_as_float(s[e]), p.scale_log2, -ref));
            float b = exp2_approx(fmaf(__uint_as_float(s[e + 1]), p.scale_log2, -ref));
            if (!full) {
              a = (live[c] >> e) & 1u ? a : 0.f;
              b = (live[c] >> (e + 1)) & 1u ? b : 0.f;
            }
            add[0] += a;
            add[1] += b;
            pk[e / 2] = pack_half2_rn(a, b);
          }
          tmem_st16(t_s + c * 16, pk);
        }
        sum += add[0] + add[1];
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&m->p_full[j]);
      }
      // a group without a tile waits for the other's queries here: else it would
      // arrive for the next piece in this piece's phase
      if (done == 0) ok = ok && wait_warp(m, &m->q_full, piece & 1u);
      if (!ok) break;
      seq += T;
      // ---- the partial rows ----
      const int lr = (x.pair ? j * 128 : 0) + row;
      const int64_t at = x.row + (x.pair ? (int64_t)lr : (int64_t)j * x.rows + lr);
      float4* po = reinterpret_cast<float4*>(p.o + at * D);
      if (done > 0) {
        if (!(ok = wait_warp(m, &m->o_full[j], no & 1u))) break;
        ++no;
        tc_fence_after();
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (done > 0) {
          tmem_ld32(t_o + c * 32, o);
          tc_wait_ld();
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
      if (lane == 0) {
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
