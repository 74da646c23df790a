// Draft-tree attention on the 5th-generation tensor cores, head_dim 64 to 512.
//
// The rows of one kv head are the nodes times its G q heads, so every key byte
// serves n G rows: at 4 D bytes a key (BF16) and 4 D n G operations the keys'
// bytes bound the kernel up to some 290 rows, and padding the rows to the
// tensor core's 128 costs nothing that matters. What has to hold is that the
// chain scores -> softmax -> weighted values keeps up with the memory.
//
//  * One CTA an SM takes an equal share of all key tiles (tree_plan.cuh). A
//    tile is 128 keys. Two groups of four softmax warps, one thread a row:
//    up to 128 rows the groups take alternate tiles of the same rows and merge
//    at the end; above, each takes 128 rows of every tile. (head_dim 256: one
//    group, 64 keys, see kOneO. head_dim 512: 32 keys, and an item is half of the
//    columns of V and O, so K is read twice, the second time mostly from L2.)
//  * TMEM holds per group S (128 columns fp32), over which P is written as
//    16-bit pairs, and O (D columns). P is then the A operand from TMEM, so
//    shared memory carries K, V and Q only.
//  * The producer warp copies K and V units (128 keys of one head) by TMA into
//    a ring, in the order in which they are used. FP8 and NVFP4 units land raw
//    and four more warps widen them to f16 (exact: every E4M3 value and every
//    E2M1 x E4M3 product is an f16); q is then scaled by a power of two a row
//    (widen_q).
//  * A row's P is taken against a running reference: the largest of the first
//    scores it sees. Floating-point P need no exact maximum, so a tile is read
//    once: the reference moves, and what was computed is rescaled, only where 32
//    keys' P add up to 2^15. Sums, of the unrounded P, and O are fp32. P is rounded
//    to bf16 with BF16 caches, since both operands of a product have one type, else to
//    f16: outputs are 0.0023 of their size from 64 bits with the one (0.0017 with P in
//    fp32) and 0.0017 with the other. The loops over a tile stay rolled: with one or
//    two warps a scheduler, straight-line code for 128 keys runs at the rate of fetches.
//  * V rows that no node sees are zeroed, so stale bytes never meet a weight.
//  * Measured (GB300): single tokens of 32 sequences over 4096 keys 98 us, 6.5 TB/s
//    between a start and a join of 12 us together; 32 trees of 4 to 16 nodes 70 us;
//    2 trees of 64 nodes over 32K keys 85 us (808 TFLOP/s), bound by each group's
//    chain of scores, softmax and weighted values; 64 trees in FP8 180 us, in NVFP4
//    217, by the same chain with the widening in it. Without the softmax the four
//    took 94, 65, 73 and 141 us (FP8), with an eighth of the products 95, 66, 71 and
//    165. head_dim 512, 64 nodes of 8 heads over 28000 keys: 184 us (mma.sync 690).
//  * Every wait is bounded (2 s, that for a piece's first keys by consumer_wait_ns):
//    on time-out the CTA raises PD_DEV_TIMEOUT, waits for its copies and MMAs in
//    flight, frees its TMEM and ends.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cstring>

#pragma nv_diag_suppress 177  // TreeCfg<> defines every constant for every form

#include "mma_common.cuh"
#include "pd_common.cuh"
#include "tree_plan.cuh"
#include "umma_common.cuh"

namespace pd {
namespace {

using namespace ::pd::mma;
using namespace ::pd::umma;
using namespace ::pd::tree;

constexpr float kTreeHigh = 32768.0f; // a row's P add up to less in 32 keys, or its reference moves
// A piece's start and end cost about three tiles (1: 3 to 8% slower with batches of 32
// and 64 sequences); a CTA takes two units at least (1, 3: 14.9 and 15.7 us for one short
// sequence, against 14.2).
constexpr int kTreeSlack = 3;
constexpr int kTreeLeast = 2;
constexpr int kTreeMma = 8;
constexpr int kTreeQ = 9;             // the next piece's q rows and what they see
constexpr int kTreeProd = 10;         // from here on: the copies, units in turn
constexpr int kTreeConv = 12;         // quantised units are widened by warps 12..15
constexpr int kTreeTmemCols = 512;
constexpr int kTreeBadRing = 32;      // tiles whose page masks are kept

template <int FMT, int D, int BS>
struct TreeCfg {
  static constexpr bool kQuant = FMT != PD_KV_BF16;
  // head_dim 256 and up: one O fills half the tensor memory, so a single group of
  // softmax warps takes every tile, its scores in two buffers by turns
  static constexpr bool kOneO = D >= 256;
  // head_dim 512: an item is one half of the columns of V and O, with all of K
  static constexpr int kHalves = D == 512 ? 2 : 1;
  static constexpr int kDV = D / kHalves;
  static constexpr int kKT = D == 512 ? 32 : D == 256 ? 64 : 128;  // keys of a tile
  static constexpr int kQTiles = kOneO ? 1 : 2;
  static constexpr int kSoftWarps = kOneO ? 4 : 8;
  // One thread issues a 2 KB copy about every 100 cycles, a third of the rate at
  // which an SM's share of the memory delivers BF16 units: four producers.
  // Quantised units take half the copies or fewer. (A producer must not come back
  // to a slot whose last but one unit is still in use: no more of them than slots.)
  static constexpr int kProds = kQuant || D == 512 ? 2 : 4;
  static constexpr int kThreads = (kQuant ? kTreeConv + 4 : kTreeProd + kProds) * 32;
  static constexpr int kCopies = kKT / BS;            // pages of a tile
  static constexpr int kQBytes = 128 * D * 2;             // one Q tile, chunk-major
  static constexpr int kUnitBytes = kKT * D * 2;      // one 16-bit K or V unit, chunk-major
  static constexpr int kUnits =
      ((kQuant ? 96 : 160) - (D == 512 ? (kQuant ? 32 : 64) : 0)) * 1024 / kUnitBytes;
  // a raw quantised unit: rows [kKT][row bytes] (FP8: in slabs of 256 columns), then
  // NVFP4 scales [kKT][D / 16]
  static constexpr int kRowBytes = FMT == PD_KV_FP8_E4M3 ? D : D / 2;
  static constexpr int kRawData = kKT * kRowBytes;
  static constexpr int kRawScales = FMT == PD_KV_NVFP4 ? kKT * (D / 16) : 0;
  static constexpr int kRawBytes = kQuant ? (kRawData + kRawScales + 1023) / 1024 * 1024 : 0;
  // NVFP4 pages by gathers of four, while a head's codes of a page fit a box
  static constexpr bool kGather = FMT == PD_KV_NVFP4 && BS == 16 && D <= 128;
  static constexpr int kRaws = kQuant ? (D == 512 ? 32 : 64) * 1024 / kRawBytes : 0;
  static constexpr int kUnitOff = kQTiles * kQBytes;
  static constexpr int kRawOff = kUnitOff + kUnits * kUnitBytes;
  static constexpr int kBarOff = kRawOff + kRaws * kRawBytes;
  // unit full / empty, raw full / empty, s_full[2], p_full[2], o_done[2],
  // ml_full[2], q_full[2], q_empty[2], v_empty, o_free, q_raw[2], fin
  static constexpr int kNumBars = 2 * kUnits + 2 * kRaws + 17;
  // what the piece's nodes see: bits[64], lo[64], any node's bits and lo; the
  // rows' score multipliers [256]; page masks
  static constexpr int kViewOff = kBarOff + (kNumBars + 1) / 2 * 16;
  static constexpr int kMulOff = kViewOff + 64 * 12 + 16;
  static constexpr int kBadOff = kMulOff + 256 * 4;
  static constexpr int kHolderOff = kBadOff + kTreeBadRing * 4;
  static constexpr int kLastOff = kHolderOff + 16;  // the producers' newest units
  static constexpr int kSmemBytes = kLastOff + 16;
  static_assert(kProds <= (kQuant ? kRaws : kUnits) && kProds <= 4, "producers are not lapped");
  static_assert(kUnitBytes % 1024 == 0 && kRawBytes % 1024 == 0, "aligned tiles");
  static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory");
};

// The bounded waits of mma_common.cuh with a suspend-time hint: a warp that waits
// sleeps up to 20 us at a time instead of polling. Six or more warps of a CTA wait
// at any moment; polling, they took half the issue slots of the warps at work.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool sleep_wait(uint32_t bar, uint32_t parity,
                                           const volatile int* abort_flag,
                                           uint64_t limit_ns = kWaitLimitNs) {
  if (limit_ns == 0) return mbar_test_wait(bar, parity);
  if (try_wait_long(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!try_wait_long(bar, parity)) {
    if (*abort_flag != 0 || global_ns() - t0 > limit_ns) return false;
  }
  return true;
}
__device__ __forceinline__ bool warp_sleep_wait(uint32_t bar, uint32_t parity,
                                                const volatile int* abort_flag,
                                                uint64_t limit_ns = kWaitLimitNs) {
  return __all_sync(0xFFFFFFFFu, sleep_wait(bar, parity, abort_flag, limit_ns));
}

// Order in which a piece of T tiles uses its 2 T units: dual (each group has its
// own rows) K0 V0 K1 V1 ..; alternating groups K0 K1 V0 K2 V1 ...
__device__ __forceinline__ void unit_at(int t, int T, bool dual, bool& is_v, int& j) {
  if (dual) {
    is_v = t & 1;
    j = t >> 1;
  } else if (t == 2 * T - 1) {
    is_v = true;
    j = T - 1;
  } else if (t >= 2 && (t & 1) == 0) {
    is_v = true;
    j = (t - 2) >> 1;
  } else {
    is_v = false;
    j = (t + 1) >> 1;
  }
}
__device__ __forceinline__ int v_unit(int j, int T, bool dual) {
  return dual ? 2 * j + 1 : (j == T - 1 ? 2 * T - 1 : 2 * j + 2);
}

// The page mask of a 32-key chunk from the tile's bad pages.
template <int BS>
__device__ __forceinline__ uint32_t bad32(uint32_t bad, int chunk) {
  if constexpr (BS == 32) return ((bad >> chunk) & 1u) ? 0xFFFFFFFFu : 0u;
  return (((bad >> (2 * chunk)) & 1u) ? 0x0000FFFFu : 0u) |
         (((bad >> (2 * chunk + 1)) & 1u) ? 0xFFFF0000u : 0u);
}

// Both 16-bit halves (f16 or bf16) times a.
template <bool F16>
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, float a) {
  if constexpr (!F16) return pack_bf16x2(bf16_lo(w) * a, bf16_hi(w) * a);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_f16x2(x.x * a, x.y * a);
}

// A raw unit widened to f16 in the swizzled operand layout (chunk-major
// 128-byte rows) by four warps; a warp's rows whose `keep` bit is off become
// zeros. Eight lanes take a row, a lane the same 8 elements (a 16-byte f16 piece)
// of every 64-element chunk: eight lanes store eight different pieces of a row.
// Rows that would read from the same banks begin with another chunk.
// COLS of the row's D columns, from 64-column chunk `chunk0` on (FP8: a raw unit
// holds these columns only, in slabs of 256).
template <int FMT, int D, int COLS>
__device__ __forceinline__ void widen_unit(uint32_t raw, uint32_t op, int chunk0, int warp,
                                           int lane, uint32_t keep) {
  constexpr int kKT = D == 512 ? 32 : D == 256 ? 64 : 128;
  constexpr int kRow = FMT == PD_KV_FP8_E4M3 ? (D < 256 ? D : 256) : D / 2;
  constexpr int kSteps = kKT / 4 / 4;
  constexpr int kCh = COLS / 64;
  const int p = lane & 7;
  const int row0 = warp * (kKT / 4) + (lane >> 3);
  const int turn = kCh == 1 ? 0 : (FMT == PD_KV_FP8_E4M3 ? (lane >> 3) & 1 : lane >> 4);
  uint2 w[kSteps][kCh];
  uint32_t sc[kSteps][kCh];
#pragma unroll
  for (int it = 0; it < kSteps; ++it)
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      const int row = row0 + it * 4, ch = k ^ turn;
      if constexpr (FMT == PD_KV_FP8_E4M3) {
        w[it][k] = lds64(raw + (ch >> 2) * (kKT * 256) + row * kRow + (ch & 3) * 64 + p * 8);
      } else {
        const int piece = (chunk0 + ch) * 8 + p;
        w[it][k].x = lds32(raw + row * kRow + piece * 4);
        sc[it][k] = lds_u8(raw + kKT * kRow + row * (D / 16) + piece / 2);
      }
    }
  if (keep != 0xFFFFFFFFu) {
#pragma unroll
    for (int it = 0; it < kSteps; ++it)
      if (!((keep >> ((lane >> 3) + it * 4)) & 1u)) {
#pragma unroll
        for (int k = 0; k < kCh; ++k) {
          w[it][k] = make_uint2(0u, 0u);
          sc[it][k] = 0u;
        }
      }
  }
#pragma unroll
  for (int it = 0; it < kSteps; ++it)
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      const int row = row0 + it * 4;
      uint32_t f[4];
      if constexpr (FMT == PD_KV_FP8_E4M3) {
        f[0] = e4m3x2_f16x2(w[it][k].x & 0xFFFFu);
        f[1] = e4m3x2_f16x2(w[it][k].x >> 16);
        f[2] = e4m3x2_f16x2(w[it][k].y & 0xFFFFu);
        f[3] = e4m3x2_f16x2(w[it][k].y >> 16);
      } else {
        const uint32_t s2 = e4m3x2_f16x2(sc[it][k] | (sc[it][k] << 8));
        e2m1x8_f16x2(w[it][k].x, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = hmul2_u32(f[e], s2);
      }
      sts128(op + (k ^ turn) * (kKT * 128) + swz128(row * 128 + p * 16), f[0], f[1], f[2], f[3]);
    }
}

// A piece's bf16 q rows to f16 times a power of two, in place, by four warps: a
// row's largest |q| into [2^14, 2^15). f16 holds bf16's 8 bits down to 2^-17, 2^-31 of
// the largest; smaller elements are off by at most 2^-39 of it. mul_s[r] becomes row r's
// score multiplier. Rows from `second` on are the second tile's.
template <int D>
__device__ __forceinline__ void widen_q(uint32_t tile, int tile_bytes, int rows, int second,
                                        float mul, float* mul_s, int warp, int lane) {
  constexpr int kLanes = D < 256 ? D / 8 : 32;  // lanes of a row
  constexpr int kPer = D / 8 / kLanes;          // 16-byte pieces of a lane
  constexpr int kStep = 32 / kLanes;            // rows of a step
  constexpr int kBatch = 4;                     // steps whose latencies overlap
  const int c = lane % kLanes;
#pragma unroll 1
  for (int r0 = warp * kBatch * kStep; r0 < rows; r0 += 4 * kBatch * kStep) {
    uint32_t at[kBatch][kPer];
    uint4 x[kBatch][kPer];
    float mq[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = min(r0 + k * kStep + lane / kLanes, rows - 1);
      const int m = r >= second ? r - second : r;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int piece = c + j * kLanes;
        at[k][j] = tile + (r >= second ? tile_bytes : 0) + (piece / 8) * (128 * 128) +
                   swz128(m * 128 + (piece % 8) * 16);
        x[k][j] = lds128(at[k][j]);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      mq[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t y[4] = {x[k][j].x, x[k][j].y, x[k][j].z, x[k][j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mq[k] = fmaxf(mq[k], fmaxf(fabsf(bf16_lo(y[e])), fabsf(bf16_hi(y[e]))));
      }
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        mq[k] = fmaxf(mq[k], __shfl_xor_sync(0xFFFFFFFFu, mq[k], o));
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * kStep + lane / kLanes;
      if (r < rows) {
        const int up = ilog2f(mq[k]);
        const float down = exp2i(14 - up);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          uint32_t y[4] = {x[k][j].x, x[k][j].y, x[k][j].z, x[k][j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = pack_f16x2(bf16_lo(y[e]) * down, bf16_hi(y[e]) * down);
          sts128(at[k][j], y[0], y[1], y[2], y[3]);
        }
        if (c == 0) mul_s[r] = mul * exp2i(up - 14);
      }
    }
  }
}

template <int FMT, int D, int BS>
__global__ void __launch_bounds__(TreeCfg<FMT, D, BS>::kThreads, 1)
    tree_umma_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_ks,
                     const __grid_constant__ CUtensorMap tm_vs,
                     const __grid_constant__ CUtensorMap tm_q, const TreeArgs a,
                     const TreeWork w) {
  using C = TreeCfg<FMT, D, BS>;
  constexpr bool kQuant = C::kQuant;
  constexpr bool kOneO = C::kOneO;
  constexpr int KT = C::kKT;
  constexpr int DV = C::kDV;  // columns of V and O that an item has
  asm volatile("griddepcontrol.launch_dependents;");
  const int G = a.group;
  const int TPG = 128 / G;        // nodes of 128 rows
  const int IN = w.item_nodes;    // nodes of an item: TPG, or with two groups 2 TPG
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t s0 = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* u_full = bars;
  uint64_t* u_empty = u_full + C::kUnits;
  uint64_t* r_full = u_empty + C::kUnits;
  uint64_t* r_empty = r_full + C::kRaws;
  uint64_t* s_full = r_empty + C::kRaws;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* ml_full = o_done + 2;
  uint64_t* q_full = ml_full + 2;
  uint64_t* q_empty = q_full + 2;
  uint64_t* v_empty = q_empty + 2;
  uint64_t* o_free = v_empty + 1;
  uint64_t* q_raw = o_free + 1;
  uint64_t* fin = q_raw + 2;
  uint64_t* bits_s = reinterpret_cast<uint64_t*>(smem + C::kViewOff);  // [64], [64]: any node
  int* lo_s = reinterpret_cast<int*>(bits_s + 65);                     // [64], [64]: any node
  float* mul_s = reinterpret_cast<float*>(smem + C::kMulOff);          // [256]
  uint32_t* bad_s = reinterpret_cast<uint32_t*>(smem + C::kBadOff);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::kHolderOff);
  volatile int* abort_s = reinterpret_cast<volatile int*>(holder + 1);

  if (tid == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      const uint64_t* b = bars + i;
      uint32_t count = 1;
      if (kQuant && b >= u_full && b < u_full + C::kUnits) count = 4;      // widening warps
      if (kQuant && b >= r_empty && b < r_empty + C::kRaws) count = 4;
      if (b == p_full || b == p_full + 1 || b == ml_full || b == ml_full + 1) count = 4;
      if (b >= q_empty && b <= o_free) count = C::kSoftWarps;
      // what rows see, and the copy or the four warps that widen it
      if (b == q_full || b == q_full + 1) count = kQuant ? 5 : 2;
      mbar_init(smem_u32(b), count);
    }
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kTreeMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(holder)),
                 "n"(kTreeTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // what touches global memory waits for the previous work on the stream
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (scratch where Q will be)
  const Share share = make_share(a, IN, KT, kTreeSlack, w.min_units,
                                 reinterpret_cast<ShareScratch*>(smem));
  if (tid == 0) w.records[blockIdx.x] = JoinRecord{0, 0, 0, 0};
  // the swizzled tiles need 1024-byte alignment: refuse, do not guess
  if ((s0 & 1023u) && tid == 0) atomicOr(a.flags, PD_DEV_BAD_SMEM);
  const bool work = share.b >= 0 && (s0 & 1023u) == 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  if (!work) {
    if (warp == kTreeMma)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "n"(kTreeTmemCols)
                   : "memory");
    return;
  }
  // S (and P) of group X at X * 128, O at 256 + X * D. Q: two tiles; while no
  // piece has more than 128 rows they are two buffers, piece by piece
  const int nbuf = !kOneO && w.rows <= 128 ? 2 : 1;
  const uint32_t unit_s = s0 + C::kUnitOff;
  const uint32_t raw_s = s0 + C::kRawOff;
  Walker walk(a, share, IN, KT, kTreeSlack);
  Piece q;
  bool failed = false;
  auto give_up = [&](bool say) {
    if (say) atomicOr(a.flags, PD_DEV_TIMEOUT);
    *abort_s = 1;
    failed = true;
  };

  if (warp >= kTreeProd && warp < kTreeProd + C::kProds) {
    // =========================== producers ================================
    constexpr int kSlots = kQuant ? C::kRaws : C::kUnits;
    uint64_t* full = kQuant ? r_full : u_full;
    uint64_t* empty = kQuant ? r_empty : u_empty;
    const int pool_rows = static_cast<int>(a.num_blocks * BS);
    const int mine = warp - kTreeProd;
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
    int u0 = 0;        // units of the pieces before
    int tile0 = 0;     // tiles before
    int last = -1;     // last unit issued here
    while (!failed && walk.next(q)) {
      if (lane == 0 && mine == 0 && q.begins && !q.whole)
        w.records[blockIdx.x] = JoinRecord{walk.pieces_of_last(q.j1), q.p.s.q0 + q.rt * IN,
                                           min(IN, q.p.s.n - q.rt * IN) | q.half << 16, q.g * G};
      const int nodes = min(IN, q.p.s.n - q.rt * IN);
      const bool dual = nodes > TPG;
      const int T = q.j1 - q.j0;
      const int32_t* bt = a.block_tables + static_cast<int64_t>(q.b) * a.max_blocks_per_seq;
      // block-table entries [win, win + 32) and the 32 after them, one a lane; units
      // go back by two tiles at most, so the window moves on three quarters in
      int win = -(1 << 30), cur = -1, nxt = -1;
      auto load = [&](int e) { return e < a.max_blocks_per_seq ? bt[e] : -1; };
      // this warp's units: u % kProds == mine
      for (int t = (mine - u0) & (C::kProds - 1); t < 2 * T; t += C::kProds) {
        bool is_v;
        int j;
        unit_at(t, T, dual, is_v, j);
        const int t0 = tile_key(q.p, q.j0 + j, KT);
        const int first = t0 / BS;
        if (first < win || first - win >= 64) {
          win = first;
          cur = load(win + lane);
          nxt = load(win + 32 + lane);
        } else if (first - win >= 48) {
          win += 32;
          cur = nxt;
          nxt = load(win + 32 + lane);
        }
        const int at = first - win + lane;
        int pg = __shfl_sync(0xFFFFFFFFu, cur, at & 31);
        if (first - win + C::kCopies > 32) {
          const int far = __shfl_sync(0xFFFFFFFFu, nxt, at & 31);
          if (at >= 32) pg = far;
        }
        const bool in = lane < C::kCopies &&
                        t0 + lane * BS < tile_end(q.p, q.j0 + j, KT, a.num_sinks);
        const bool ok_page = in && pg >= 0 && pg < a.num_blocks;
        const uint32_t bad = __ballot_sync(0xFFFFFFFFu, in && !ok_page);
        if (!ok_page) pg = -1;
        const int u = u0 + t;
        const int slot = u % kSlots;
        if (u >= kSlots && !warp_sleep_wait(smem_u32(&empty[slot]), ((u / kSlots) - 1) & 1, abort_s)) {
          give_up(lane == 0);
          break;
        }
        const uint32_t fb = smem_u32(&full[slot]);
        const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
        if (lane == 0) {
          if (bad) atomicOr(a.flags, PD_DEV_BAD_PAGE);
          bad_s[(tile0 + j) % kTreeBadRing] = bad;  // K and V of a tile: the same word
        }
        // one lane issues all copies: a copy a lane would be issued one after
        // another all the same, with a loop over the lanes around it
        if constexpr (FMT != PD_KV_NVFP4) {
          // pages that are not read land as zeros, from past the pool
          const int z = pg >= 0 ? pg * BS : pool_rows;
          int zs[C::kCopies];
#pragma unroll
          for (int k = 0; k < C::kCopies; ++k) zs[k] = __shfl_sync(0xFFFFFFFFu, z, k);
          if (lane == 0) {
            if constexpr (FMT == PD_KV_BF16) {
              const int chunks = C::kHalves > 1 && is_v ? DV / 64 : D / 64;
              const int x0 = C::kHalves > 1 && is_v ? q.half * DV : 0;
              mbar_arrive_expect_tx(fb, KT * 128 * chunks);
              const uint32_t dst = unit_s + slot * C::kUnitBytes;
#pragma unroll
              for (int k = 0; k < C::kCopies; ++k)
#pragma unroll
                for (int ch = 0; ch < D / 64; ++ch)
                  if (C::kHalves == 1 || ch < chunks)
                    tma_load_3d(dst + ch * (KT * 128) + k * (BS * 128), tm, x0 + ch * 64, q.g,
                                zs[k], fb);
            } else {
              // a box is 256 columns at most
              constexpr int kBox = D < 256 ? D : 256;
              const int boxes = C::kHalves > 1 && is_v ? 1 : D / kBox;
              const int x0 = C::kHalves > 1 && is_v ? q.half * DV : 0;
              mbar_arrive_expect_tx(fb, KT * kBox * boxes);
              const uint32_t dst = raw_s + slot * C::kRawBytes;
#pragma unroll
              for (int k = 0; k < C::kCopies; ++k)
#pragma unroll
                for (int h = 0; h < D / kBox; ++h)
                  if (h < boxes)
                    tma_load_3d(dst + h * (KT * kBox) + k * (BS * kBox), tm, x0 + h * kBox, q.g,
                                zs[k], fb);
            }
          }
        } else if constexpr (C::kGather) {
          // gathers of four pages, their codes and their scales
          constexpr int kSlabWords = 16 * (D / 2) / 4, kScaleWords = 16 * (D / 16) / 4;
          const int z = pg >= 0 ? pg : static_cast<int>(a.num_blocks);
          int zs[C::kCopies];
#pragma unroll
          for (int k = 0; k < C::kCopies; ++k) zs[k] = __shfl_sync(0xFFFFFFFFu, z, k);
          if (lane == 0) {
            mbar_arrive_expect_tx(fb, C::kRawData + C::kRawScales);
            const CUtensorMap* ts = is_v ? &tm_vs : &tm_ks;
            const uint32_t dst = raw_s + slot * C::kRawBytes;
            const int x = static_cast<int>(a.data_bytes / 4) + q.g * kScaleWords;
#pragma unroll
            for (int h = 0; h < C::kCopies; h += 4) {
              tma_gather4(dst + h * (16 * (D / 2)), tm, q.g * kSlabWords, zs[h], zs[h + 1],
                          zs[h + 2], zs[h + 3], fb);
              tma_gather4(dst + C::kRawData + h * (16 * (D / 16)), ts, x, zs[h], zs[h + 1],
                          zs[h + 2], zs[h + 3], fb);
            }
          }
        } else {
          constexpr uint32_t db = BS * (D / 2), sb = BS * (D / 16);
          const uint32_t have = __ballot_sync(0xFFFFFFFFu, pg >= 0);
          if (lane == 0) mbar_arrive_expect_tx(fb, __popc(have) * (db + sb));
          __syncwarp();
          if (pg >= 0) {
            const uint8_t* src = (is_v ? a.v_cache : a.k_cache) + pg * a.page_bytes;
            const int64_t line = static_cast<int64_t>(q.g) * BS;
            const uint32_t dst = raw_s + slot * C::kRawBytes;
            bulk_load(dst + lane * db, src + line * (D / 2), db, fb);
            bulk_load(dst + C::kRawData + lane * sb, src + a.data_bytes + line * (D / 16), sb, fb);
          }
        }
        __syncwarp();
        last = u;
      }
      u0 += 2 * T;
      tile0 += T;
    }
    // every copy issued lands before the CTA can end: each slot's newest unit, whose
    // producer waits for it (an older unit has landed, and its phase could not be
    // told from the next but one)
    volatile int* last_s = reinterpret_cast<volatile int*>(smem + C::kLastOff);
    if (lane == 0) last_s[mine] = last;
    asm volatile("bar.sync 1, %0;" ::"n"(C::kProds * 32) : "memory");
    for (int u = last; u >= 0 && u > last - kSlots; u -= C::kProds)
      if (u + kSlots > last_s[(u + kSlots) & (C::kProds - 1)])
        (void)mbar_wait(smem_u32(&full[u % kSlots]), (u / kSlots) & 1);
  } else if (warp == kTreeQ) {
    // =========================== q rows ===================================
    int piece = 0;
    bool armed = false;  // this piece's copy is on its way, its views are not written
    while (!failed && walk.next(q)) {
      const TreeSeq& s = q.p.s;
      const int node0 = q.rt * IN;
      const int nodes = min(IN, s.n - node0);
      const int buf = piece % nbuf;
      const bool dual = nodes > TPG;
      if (piece >= nbuf &&
          !warp_sleep_wait(smem_u32(&q_empty[buf]), (piece / nbuf - 1) & 1, abort_s)) {
        give_up(lane == 0);
        break;
      }
      // one box a chunk: TPG tokens of G heads, rows in (node, head) order
      const uint32_t q_bar = smem_u32(kQuant ? &q_raw[buf] : &q_full[buf]);
      armed = true;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_bar, (dual ? 2 : 1) * static_cast<uint32_t>(TPG * G * D * 2));
        for (int x = 0; x < (dual ? 2 : 1); ++x)
#pragma unroll
          for (int ch = 0; ch < D / 64; ++ch)
            tma_load_3d(s0 + (buf + x) * C::kQBytes + ch * (128 * 128), &tm_q, ch * 64, q.g * G,
                        s.q0 + node0 + x * TPG, q_bar);
      }
      const RowView any = any_view(a, s, lane);
      RowView v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (lane + 32 * k < nodes) v[k] = row_view(a, s, node0 + lane + 32 * k);
      if (piece > 0 && !warp_sleep_wait(smem_u32(v_empty), (piece - 1) & 1, abort_s)) {
        give_up(lane == 0);
        break;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (lane + 32 * k < nodes) {
          bits_s[lane + 32 * k] = v[k].bits;
          lo_s[lane + 32 * k] = v[k].lo;
        }
      if (lane == 0) {
        bits_s[64] = any.bits;
        lo_s[64] = any.lo;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&q_full[buf]));
      ++piece;
      armed = false;
    }
    // every copy issued lands before the CTA can end, whoever gave up
    if (armed) {
      if (!kQuant && lane == 0) mbar_arrive(smem_u32(&q_full[piece % nbuf]));
      ++piece;
    }
    __syncwarp();
    for (int p = piece - 1; p >= 0 && p >= piece - nbuf; --p)
      (void)mbar_wait(smem_u32(kQuant ? &q_raw[p % nbuf] : &q_full[p % nbuf]), (p / nbuf) & 1);
  } else if (warp == kTreeMma) {
    // =========================== products =================================
    // (A second warp for the second group, both issuing at once, was slower at 256
    // rows, 103 us against 92: the groups' products then share the tensor core, and
    // a group waits twice as long for its own.)
    if (lane == 0) {
      constexpr uint32_t idS = kQuant ? umma_idesc_f16(128, KT, 0) : umma_idesc(128, KT, 0);
      constexpr uint32_t idO = kQuant ? umma_idesc_f16(128, DV, 1) : umma_idesc(128, DV, 1);
      const uint64_t dq0 = umma_desc(s0, 16, 1024);
      const uint64_t dk0 = umma_desc(unit_s, 16, 1024);
      const uint64_t dv0 = umma_desc(unit_s, KT * 128, 1024);
      int piece = 0, slot = 0;
      uint32_t turn = 0;   // parity of the ring's turn
      int c0 = 0, c1 = 0;  // tiles of the groups before this piece
      bool ok = true;
      auto wait = [&](const uint64_t* bar, int parity) {
        return sleep_wait(smem_u32(bar), parity & 1, abort_s);
      };
      // the next unit, once it has landed: units come in the order of use
      auto take = [&](int& s) -> bool {
        s = slot;
        const uint32_t ph = turn;
        if (++slot == C::kUnits) {
          slot = 0;
          turn ^= 1u;
        }
        return sleep_wait(smem_u32(&u_full[s]), ph, abort_s);
      };
      while (ok && walk.next(q)) {
        const int nodes = min(IN, q.p.s.n - q.rt * IN);
        const bool dual = nodes > TPG;
        const int T = q.j1 - q.j0;
        const int n0 = dual ? T : (T + 1) / 2, n1 = dual ? T : T / 2;
        const int buf = piece % nbuf;
        // q has landed; the products that read the last P are done; the first keys are there
        // (the one wait for copies that takes the test's limit: in the loop over the tiles
        // it cost 3 to 7% above 128 rows)
        if (!(ok = wait(&q_full[buf], piece / nbuf) && (c0 == 0 || wait(&o_done[0], c0 - 1)) &&
                   (c1 == 0 || wait(&o_done[1], c1 - 1)) &&
                   (kQuant ||
                    sleep_wait(smem_u32(&u_full[slot]), turn, abort_s, a.consumer_wait_ns))))
          break;
        tc_fence_after();
        int ks = 0, vs = 0;  // the last K and V unit; dual pieces use each twice
        auto issue_s = [&](int X) -> bool {
          if (!(dual && X == 1) && !take(ks)) return false;
          tc_fence_after();
          const uint64_t qa = dq0 + static_cast<uint64_t>((buf + (dual ? X : 0)) * (C::kQBytes >> 4));
          const uint64_t kb = dk0 + static_cast<uint64_t>((ks * C::kUnitBytes) >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t qoff = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
            const uint32_t koff = ((k >> 2) * (KT * 128) + (k & 3) * 32) >> 4;
            umma_f16(tmem + X * 128, qa + qoff, kb + koff, idS, k > 0 ? 1u : 0u);
          }
          umma_commit(smem_u32(&s_full[X]));
          if (!dual || X == 1) umma_commit(smem_u32(&u_empty[ks]));
          return true;
        };
        ok = issue_s(0);
        if (ok && n1 > 0) ok = issue_s(1);
        // the last piece's O has been read
        if (ok && piece > 0) ok = wait(o_free, piece - 1);
        for (int i = 0; i < n0 && ok; ++i) {
          for (int X = 0; X < 2; ++X) {
            if (X == 1 && i >= n1) continue;
            const int c = (X ? c1 : c0) + i;  // this tile is the group's c-th
            if (!(dual && X == 1) && !(ok = take(vs))) break;
            const uint64_t vb = dv0 + static_cast<uint64_t>((vs * C::kUnitBytes) >> 4);
            const uint32_t o_tm = tmem + 256 + (kOneO ? 0 : X * D);
            const bool more = (kOneO ? i + X : i) > 0;
            if (!(ok = wait(&p_full[X], c))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < KT / 16; ++k)
              umma_f16_ts(o_tm, tmem + X * 128 + k * 8, vb + ((k * 2048) >> 4), idO,
                          more || k > 0 ? 1u : 0u);
            umma_commit(smem_u32(&o_done[X]));
            if (!dual || X == 1) umma_commit(smem_u32(&u_empty[vs]));
            if (i + 1 < (X ? n1 : n0)) {
              // the next scores overwrite P: the product that reads it is done first
              if (!(ok = wait(&o_done[X], c))) break;
              if (!(ok = issue_s(X))) break;
            }
          }
        }
        c0 += n0;
        c1 += n1;
        ++piece;
      }
      if (!ok) give_up(true);
      // every product issued has completed before TMEM is freed
      umma_commit(smem_u32(fin));
      (void)mbar_wait(smem_u32(fin), 0);
    }
    __syncwarp();
  } else if (kQuant && warp >= kTreeConv) {
    // =========================== widening warps ===========================
    if constexpr (kQuant) {
      const int cw = warp - kTreeConv;
      int tile0 = 0, piece = 0;
      int rs = 0, us = 0;               // raw unit, and its place as an operand
      uint32_t r_turn = 0, u_turn = 1;  // their rings' parities: an operand's first turn is free
      while (!failed && walk.next(q)) {
        const int nodes = min(IN, q.p.s.n - q.rt * IN);
        const bool dual = nodes > TPG;
        const int T = q.j1 - q.j0;
        const RowView any = any_view(a, q.p.s, lane);
        const int buf = piece % nbuf;
        if (!warp_sleep_wait(smem_u32(&q_raw[buf]), (piece / nbuf) & 1, abort_s) ||
            (piece > 0 && !warp_sleep_wait(smem_u32(v_empty), (piece - 1) & 1, abort_s)) ||
            !warp_sleep_wait(smem_u32(&r_full[rs]), r_turn, abort_s, a.consumer_wait_ns)) {
          give_up(lane == 0);
          break;
        }
        widen_q<D>(s0 + buf * C::kQBytes, C::kQBytes, nodes * G, TPG * G,
                   a.scale_log2 * (FMT == PD_KV_FP8_E4M3 ? a.k_scale : 1.0f), mul_s, cw, lane);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&q_full[buf]));
        ++piece;
        int next_k = 0, next_v = 0;
        for (int t = 0; t < 2 * T; ++t) {
          const bool is_v = next_k == T || (dual ? t & 1 : next_k - next_v == 2);  // as unit_at
          const int j = is_v ? next_v++ : next_k++;
          if (!warp_sleep_wait(smem_u32(&r_full[rs]), r_turn, abort_s) ||
              !warp_sleep_wait(smem_u32(&u_empty[us]), u_turn, abort_s)) {
            give_up(lane == 0);
            break;
          }
          const int t0 = tile_key(q.p, q.j0 + j, KT);
          const uint32_t bad = bad_s[(tile0 + j) % kTreeBadRing];
          const int row0 = cw * (KT / 4);  // this warp's first row
          uint32_t keep = 0xFFFFFFFFu;
          if (bad != 0u || t0 < any.lo || t0 + KT > any.prefix)
            keep = (seen32(any, t0 + row0 / 32 * 32) & ~bad32<BS>(bad, row0 / 32)) >> (row0 % 32);
          const uint32_t raw = raw_s + rs * C::kRawBytes, op = unit_s + us * C::kUnitBytes;
          if (C::kHalves > 1 && is_v)
            widen_unit<FMT, D, DV>(raw, op, q.half * (DV / 64), cw, lane, keep);
          else
            widen_unit<FMT, D, D>(raw, op, 0, cw, lane, keep);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&u_full[us]));
            mbar_arrive(smem_u32(&r_empty[rs]));
          }
          if (++rs == C::kRaws) {
            rs = 0;
            r_turn ^= 1u;
          }
          if (++us == C::kUnits) {
            us = 0;
            u_turn ^= 1u;
          }
        }
        tile0 += T;
      }
    }
  } else if (warp < C::kSoftWarps) {
    // =========================== softmax warps ============================
    const int X = warp >> 2;  // the group
    const int m = (warp & 3) * 32 + lane;  // row of the group's tile = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_tm = tmem + lane_base + 256;  // + group * D
    const float vmul = FMT == PD_KV_FP8_E4M3 ? a.v_scale : 1.0f;
    int u0 = 0, tile0 = 0, piece = 0, merges = 0;
    int c0 = 0, c1 = 0;  // tiles the groups have finished
    while (!failed && walk.next(q)) {
      const TreeSeq& s = q.p.s;
      const int node0 = q.rt * IN;
      const int nodes = min(IN, s.n - node0);
      const bool dual = nodes > TPG;
      const int T = q.j1 - q.j0;
      const int n0 = dual ? T : (T + 1) / 2, n1 = dual ? T : T / 2;
      const int nX = kOneO ? T : (X ? n1 : n0);
      const int buf = piece % nbuf;
      // ---- this row: node, head, what it sees ----
      const int i = m / G + (dual ? X * TPG : 0);
      const bool rvalid = m < TPG * G && i < nodes;
      const int qh = q.g * G + m % G;
      const int64_t qrow = static_cast<int64_t>(s.q0 + node0 + (rvalid ? i : 0));
      const int r = (dual ? X * TPG * G : 0) + m;  // row of the item
      if (!warp_sleep_wait(smem_u32(&q_full[buf]), (piece / nbuf) & 1, abort_s)) {
        give_up(lane == 0);
        break;
      }
      RowView any, view;
      any.prefix = s.L - s.n;
      any.sinks = a.sliding_window > 0 ? min(a.num_sinks, any.prefix) : 0;
      any.lo = lo_s[64];
      any.bits = bits_s[64];
      view = any;
      if (rvalid) {
        view.lo = lo_s[i];
        view.bits = bits_s[i];
      }
      const float sl2 = kQuant ? (rvalid ? mul_s[r] : 0.0f) : a.scale_log2;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(v_empty));
      // a padding row runs along as a full one against reference 0
      float m_run = rvalid ? -INFINITY : 0.0f, l_run = 0.0f;
      // warps whose 32 rows are all padding only keep the barriers going
      const bool idle = !__any_sync(0xFFFFFFFFu, rvalid);
      for (int jl = 0; jl < nX; ++jl) {
        const int j = dual || kOneO ? jl : 2 * jl + X;
        const int sx = kOneO ? jl & 1 : X;  // score buffer
        const uint32_t s_tm = tmem + lane_base + sx * 128;
        const int t0 = tile_key(q.p, q.j0 + j, KT);
        const int cnt = (sx ? c1 : c0) + (kOneO ? jl >> 1 : jl);
        if (!warp_sleep_wait(smem_u32(&s_full[sx]), cnt & 1, abort_s)) {
          give_up(lane == 0);
          break;
        }
        tc_fence_after();
        const uint32_t bad = bad_s[(tile0 + j) % kTreeBadRing];
        if constexpr (!kQuant) {
          // V rows no node sees: zeros, by the group that uses the tile first
          if ((bad != 0u || t0 < any.lo || t0 + KT > any.prefix) && (!dual || X == 0) && m < KT) {
            const uint32_t keep = seen32(any, t0 + (warp & 3) * 32) & ~bad32<BS>(bad, warp & 3);
            if (keep != 0xFFFFFFFFu) {
              const int vu = u0 + v_unit(j, T, dual), vslot = vu % C::kUnits;
              if (!warp_sleep_wait(smem_u32(&u_full[vslot]), (vu / C::kUnits) & 1, abort_s)) {
                give_up(lane == 0);
                break;
              }
              if (!((keep >> lane) & 1u)) {
                const uint32_t vrow = unit_s + vslot * C::kUnitBytes;
#pragma unroll
                for (int p = 0; p < DV / 8; ++p)
                  sts128(vrow + (p / 8) * (KT * 128) + swz128(m * 128 + (p % 8) * 16), 0u, 0u,
                         0u, 0u);
              }
              fence_async_smem();
            }
          }
        }
        if (!idle) {
          // the chunk's keys this row sees (a padding row: all, its scores are
          // whatever its stale q gives and go nowhere)
          const bool open = bad == 0u && t0 >= view.lo && t0 + KT <= view.prefix;
          const bool all_open = __all_sync(0xFFFFFFFFu, open || !rvalid);
          auto seen = [&](int c) -> uint32_t {
            if (open || !rvalid) return 0xFFFFFFFFu;
            return seen32(view, t0 + 32 * c) & ~bad32<BS>(bad, c);
          };
          // ---- P, written over the scores behind the reads: the chunk's 16
          // columns lie in a chunk that has been read ----
          bool lost = false;
          // (scores past 2^24 round by whole steps of the reference: no end of moves)
          int c = 0, moves = 0;
          for (;;) {
            const float nref = m_run == -INFINITY ? 0.0f : -m_run;
            // rows that need another reference: at the first keys they see, and
            // where the chunk's sum shows a P that f16 might not hold
            bool move = false;
#pragma unroll 1
            for (; c < KT / 32; ++c) {
              uint32_t v[32], pk[16];
              float ls[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              tmem_ld32(s_tm + c * 32, v);
              tmem_wait_ld();
              if (all_open) {
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                  const float px = ex2(fmaf(__uint_as_float(v[k]), sl2, nref));
                  const float py = ex2(fmaf(__uint_as_float(v[k + 1]), sl2, nref));
                  ls[(k >> 1) & 1] += px;
                  ls[2 + ((k >> 1) & 1)] += py;
                  pk[k / 2] = kQuant ? pack_f16x2(px, py) : pack_bf16x2(px, py);
                }
                move = m_run == -INFINITY;
              } else {
                const uint32_t vw = seen(c);
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                  float px = ex2(fmaf(__uint_as_float(v[k]), sl2, nref));
                  float py = ex2(fmaf(__uint_as_float(v[k + 1]), sl2, nref));
                  px = (vw >> k) & 1u ? px : 0.0f;
                  py = (vw >> (k + 1)) & 1u ? py : 0.0f;
                  ls[(k >> 1) & 1] += px;
                  ls[2 + ((k >> 1) & 1)] += py;
                  pk[k / 2] = kQuant ? pack_f16x2(px, py) : pack_bf16x2(px, py);
                }
                move = m_run == -INFINITY && vw != 0u;
              }
              const float sum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
              move = rvalid && (move || sum > kTreeHigh);
              if (__any_sync(0xFFFFFFFFu, move) && moves < KT / 16) break;
              l_run += sum;
              tmem_st16(s_tm + c * 16, pk);
            }
            if (c == KT / 32) break;
            ++moves;
            // ---- the chunk's largest score as the reference; what was computed
            // against the last one is rescaled ----
            float mx = -INFINITY, alpha = 1.0f;
            {
              uint32_t v[32];
              tmem_ld32(s_tm + c * 32, v);
              tmem_wait_ld();
              const uint32_t vw = seen(c);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                mx = fmaxf(mx, (vw >> k) & 1u ? __uint_as_float(v[k]) * sl2 : -INFINITY);
            }
            if (move) {
              mx = fmaxf(floorf(mx), -3.0e38f);  // a whole number: the rescaling is exact
              alpha = m_run == -INFINITY ? 0.0f : ex2(m_run - mx);
              m_run = mx;
              l_run *= alpha;
            }
            tmem_wait_st();
#pragma unroll 1
            for (int h = 0; h < c; ++h) {
              uint32_t v[16];
              tmem_ld16(s_tm + h * 16, v);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = scale_pair<kQuant>(v[k], alpha);
              tmem_st16(s_tm + h * 16, v);
            }
            if (jl == 0) continue;
            // O, once the previous product is done (with an O for each group,
            // these scores were issued after it)
            if constexpr (kOneO) {
              const int last = (sx ? c0 : c1) + ((jl - 1) >> 1);
              if (!warp_sleep_wait(smem_u32(&o_done[1 - sx]), last & 1, abort_s)) {
                lost = true;
                break;
              }
              tc_fence_after();
            }
#pragma unroll 1
            for (int h = 0; h < DV / 16; ++h) {
              uint32_t v[16];
              tmem_ld16(o_tm + (kOneO ? 0 : X * D) + h * 16, v);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
              tmem_st16(o_tm + (kOneO ? 0 : X * D) + h * 16, v);
            }
          }
          tmem_wait_st();  // (before a CTA that gives up frees the columns, too)
          if (lost) {
            give_up(lane == 0);
            break;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[sx]));
      }
      if (failed) break;
      // ---- end of the piece: this group's products, the other's (m, l) ----
      c0 += n0;
      c1 += n1;
      if (((kOneO || X == 0 || n1 == 0) && !warp_sleep_wait(smem_u32(&o_done[0]), (c0 - 1) & 1, abort_s)) ||
          ((kOneO || X == 1) && n1 > 0 &&
           !warp_sleep_wait(smem_u32(&o_done[1]), (c1 - 1) & 1, abort_s))) {
        give_up(lane == 0);
        break;
      }
      // (m, l) are exchanged where the piece's Q was: a group's last product is
      // issued after the other's last scores, so that nothing reads it any more
      // (a second group without tiles waits for the first's)
      float2* ml_s = reinterpret_cast<float2*>(smem + buf * C::kQBytes);  // [2][128]
      const bool merge = !dual && !kOneO;  // two groups hold tiles of the same rows
      if (merge) {
        ml_s[X * 128 + m] = make_float2(m_run, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ml_full[X]));
        if (!warp_sleep_wait(smem_u32(&ml_full[1 - X]), merges & 1, abort_s)) {
          give_up(lane == 0);
          break;
        }
        ++merges;
      }
      tc_fence_after();
      const bool both = merge && n1 > 0;
      float f_own = 1.0f, f_other = 0.0f, M = m_run, L = l_run;
      if (merge) {
        const float2 o = ml_s[(1 - X) * 128 + m];
        M = fmaxf(m_run, o.x);
        f_own = m_run == -INFINITY ? 0.0f : ex2(m_run - M);
        f_other = o.x == -INFINITY ? 0.0f : ex2(o.x - M);
        if (X == 1 && n1 == 0) f_own = 0.0f;
        L = l_run * f_own + o.y * f_other;
      }
      const float f0 = X ? f_other : f_own, f1 = X ? f_own : f_other;
      const float mul = q.whole ? vmul / fmaxf(L, 1e-20f) : vmul;
      uint16_t* orow = a.out + qrow * a.out_stride + static_cast<int64_t>(qh) * D + q.half * DV;
      float* part = w.o + (static_cast<int64_t>(q.slot) * (DV / 4) * w.rows + r) * 4;
      const int cols = merge ? DV / 2 : DV, col0 = merge ? X * (D / 2) : 0;
      if (!idle) {
        for (int cg = 0; cg < cols; cg += 16) {
          uint32_t va[16], vb[16];
          tmem_ld16(o_tm + (dual ? X * D : 0) + col0 + cg, va);
          if (both) tmem_ld16(o_tm + D + col0 + cg, vb);
          tmem_wait_ld();
          float x[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            x[k] = __uint_as_float(va[k]) * (merge ? f0 : 1.0f);
            if (both) x[k] = fmaf(__uint_as_float(vb[k]), f1, x[k]);
            x[k] *= mul;
          }
          if (rvalid) {
            if (q.whole) {
              uint32_t y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
              uint4* dst = reinterpret_cast<uint4*>(orow + col0 + cg);
              dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
              dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(part + static_cast<int64_t>((col0 + cg) / 4 + k) *
                                                      w.rows * 4) =
                    make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
            }
          }
        }
        if (rvalid && !q.whole && (!merge || X == 0))
          w.ml[static_cast<int64_t>(q.slot) * w.rows + r] = make_float2(M, L);
      }
      tc_fence_before();
      fence_async_smem();  // the next copy lands where (m, l) were
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(o_free));
        mbar_arrive(smem_u32(&q_empty[buf]));
      }
      u0 += 2 * T;
      tile0 += T;
      ++piece;
    }
  }

  // ---- free the TMEM columns once every warp is done with them ----
  tc_fence_before();
  __syncthreads();
  if (warp == kTreeMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "n"(kTreeTmemCols)
                 : "memory");
  }
}

// 3-D map over the q rows: dims (d, q head, row), box (64, G, 128 / G): a tile's
// rows in (node, head) order, 128-byte swizzled. Rows past total_q land as zeros.
bool encode_q_map(CUtensorMap* m, const TreeArgs& a, int D) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.num_q_heads),
                              static_cast<cuuint64_t>(a.total_q)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2,
                                 static_cast<cuuint64_t>(a.q_stride) * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(a.group),
                             static_cast<cuuint32_t>(128 / a.group)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t*>(a.q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int D, int BS>
cudaError_t launch_umma_cfg(const TreeArgs& a, const TreeWork& w, cudaStream_t st) {
  using C = TreeCfg<FMT, D, BS>;
  CUtensorMap tk, tv, tks, tvs;
  std::memset(&tk, 0, sizeof(tk));
  std::memset(&tv, 0, sizeof(tv));
  std::memset(&tks, 0, sizeof(tks));
  std::memset(&tvs, 0, sizeof(tvs));
  const int64_t rows = a.num_blocks * BS;
  if constexpr (FMT == PD_KV_NVFP4) {
    if constexpr (C::kGather) {
      constexpr int kSlab = 16 * (D / 2), kScales = 16 * (D / 16);
      if (!encode_nvfp4_gather_map(&tk, a.k_cache, a.page_bytes, a.num_blocks, kSlab) ||
          !encode_nvfp4_gather_map(&tv, a.v_cache, a.page_bytes, a.num_blocks, kSlab) ||
          !encode_nvfp4_gather_map(&tks, a.k_cache, a.page_bytes, a.num_blocks, kScales) ||
          !encode_nvfp4_gather_map(&tvs, a.v_cache, a.page_bytes, a.num_blocks, kScales))
        return cudaErrorInvalidValue;
    }
  } else {
    constexpr int kInner = FMT == PD_KV_BF16 ? 64 : (D < 256 ? D : 256);
    constexpr bool kSwz = FMT == PD_KV_BF16;
    if (!encode_cache_map(&tk, a.k_cache, FMT, D, a.num_kv_heads, rows, kInner, BS, kSwz) ||
        !encode_cache_map(&tv, a.v_cache, FMT, D, a.num_kv_heads, rows, kInner, BS, kSwz))
      return cudaErrorInvalidValue;
  }
  CUtensorMap tq;
  if (!encode_q_map(&tq, a, D)) return cudaErrorInvalidValue;
  auto kern = tree_umma_kernel<FMT, D, BS>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {};  // per device; setting it twice is harmless
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  e = launch_dependent(dim3(w.ctas), C::kThreads, C::kSmemBytes, st, kern, tk, tv, tks, tvs, tq, a, w);
  if (e != cudaSuccess) return e;
  return launch_tree_join(a, w, D, st);
}

template <int FMT, int D>
cudaError_t launch_umma_bs(const TreeArgs& a, const TreeWork& w, cudaStream_t st) {
  return a.block_size == 16 ? launch_umma_cfg<FMT, D, 16>(a, w, st)
                            : launch_umma_cfg<FMT, D, 32>(a, w, st);
}

template <int FMT>
cudaError_t launch_umma_fmt(const TreeArgs& a, const TreeWork& w, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_umma_bs<FMT, 64>(a, w, st);
    case 128: return launch_umma_bs<FMT, 128>(a, w, st);
    case 256: return launch_umma_bs<FMT, 256>(a, w, st);
    default: return launch_umma_bs<FMT, 512>(a, w, st);
  }
}

}  // namespace

size_t tree_umma_workspace(int max_q_len, int group, int head_dim, int num_sms, TreeWork* w,
                           void* workspace) {
  const int item_nodes = (head_dim >= 256 ? 1 : 2) * (128 / group);
  const int nodes = max_q_len < item_nodes ? (max_q_len < 1 ? 1 : max_q_len) : item_nodes;
  const int rows = (nodes * group + 7) / 8 * 8;
  const WorkLayout l = work_layout(num_sms, rows, head_dim > 256 ? 256 : head_dim);
  if (w) {
    uint8_t* p = static_cast<uint8_t*>(workspace);
    w->records = reinterpret_cast<JoinRecord*>(p);
    w->ml = reinterpret_cast<float2*>(p + l.ml);
    w->o = reinterpret_cast<float*>(p + l.o);
    w->ctas = num_sms;
    w->rows = rows;
    w->item_nodes = item_nodes;
    w->min_units = kTreeLeast;
  }
  return l.bytes;
}

cudaError_t launch_tree_umma(const TreeArgs& a, const TreeWork& w, int head_dim, int kv_dtype,
                             cudaStream_t st) {
  switch (kv_dtype) {
    case PD_KV_BF16: return launch_umma_fmt<PD_KV_BF16>(a, w, head_dim, st);
    case PD_KV_FP8_E4M3: return launch_umma_fmt<PD_KV_FP8_E4M3>(a, w, head_dim, st);
    default: return launch_umma_fmt<PD_KV_NVFP4>(a, w, head_dim, st);
  }
}

}  // namespace pd
