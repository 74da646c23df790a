// Chunks of prompts over INT8 pages (pd_prefill) on tcgen05, head_dim 64 and 128:
// the persistent kernel of prefill_packed.cu with widening warps between the copies and
// the tensor core.
//
//   t_j = scale * kscale(j) * (q . kcode_j) + log2 vscale(j),  w_j = 2^(t_j - m + 7)
//   out = sum w_j vcode_j / sum (w_j / vscale(j))
//
// Codes of 8 bits are exact in bf16 and in f16: K goes in as bf16, beside q as it is,
// V as f16, beside weights rounded to f16. Value scales ride in the exponent as in the
// decode kernel; a page's two scales cost half a fused multiply-add a score. A masked
// key has weight zero and any byte is a finite code: nothing is cleared.
//
// Warps: 8 for the softmax of two 128-row query tiles (one thread a row), 6 that
// widen (and bring Q, row by row: its last row is known on the device only), one that
// finds the items and copies, one that issues MMAs. K and V tiles of 128
// keys come as codes into a raw ring, one bulk copy a page, and go widened, swizzled,
// into the operand ring. A pair of codes takes four instructions as bf16 (128 + (c mod
// 128), less 128, or 256 for a negative code), two as f16 (int8_tile.cuh), all exact.
//
// Measured: 8 chunks of 512 tokens over 4096 keys, 32/8 heads of 128, 276 us (930
// TFLOP/s, floor 134; a BF16 cache's kernel 420, mma.sync tiles 1930), head_dim 64 198
// (floor 67). Issue slots 43%, tensor pipe 38% (head_dim 64: 49%, 25%): the chain of a
// tile bounds it, copy, widen, scores, softmax, product (with four widening warps 315 us
// where six took 297; seven eighths of the widening left out 226). Three operand slots
// are what fits at head_dim 128; four with a raw ring of two, or a raw ring of four,
// change nothing. 16 tokens over 8000 keys take 106 us, 44 times the 2.4 us of their
// bytes: keys are not divided among CTAs, and 8 of the 152 work (mma.sync tiles 415;
// there is no size from 1 token on at which those were faster).
//
// Every wait is bounded (2 s); a role that gives up says so, and the copying warp
// and the MMA warp wait for what they issued before the CTA ends.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstring>

#include "int8_tile.cuh"
#include "prompt_items.cuh"
#include "prompt_roles.cuh"
#include "serve_common.cuh"

namespace pd {
namespace {

using namespace ::pd::mma;
using namespace ::pd::umma;

// Weights 2^(t - m + kLift) against a reference m that the maximum passes by 2^8 at
// most: they stay below 2^15, and the largest is 2^7 or more, so that what f16 loses
// (below 2^-25) is below 2^-32 of it.
constexpr float kMoveLog2 = 8.0f, kLift = kWeightLog2 - kMoveLog2;
constexpr int kKT = 128;           // keys of a tile
constexpr int kMaxGroups = kKT / 16;

template <int D>
struct ChCfg {
  static constexpr int kQBytes = 128 * 2 * D;      // one query tile
  static constexpr int kSlotBytes = kKT * 2 * D;   // one tile of K or of V as bf16
  static constexpr int kRawBytes = kKT * D;        // and as codes
  static constexpr int kOutBytes = 8 * 2048;       // a warp's 32 rows x 32 outputs
  static constexpr int kSlots = D == 128 ? 3 : 6;
  static constexpr int kRaw = D == 128 ? 3 : 6;
  static constexpr int kRingOff = 2 * kQBytes;
  static constexpr int kRawOff = kRingOff + kSlots * kSlotBytes;
  static constexpr int kOutOff = kRawOff + kRaw * kRawBytes;
  static constexpr int kRawScaleOff = kOutOff + kOutBytes;
  static constexpr int kScaleBytes = kMaxGroups * static_cast<int>(sizeof(I8Scales));
  static constexpr int kScaleOff = kRawScaleOff + kRaw * kScaleBytes;
  static constexpr int kBarOff = kScaleOff + kSlots * kScaleBytes;
  // raw_full, raw_empty [raw]; kv_full, kv_empty [slots]; q_full, q_empty; item_full,
  // item_empty [2]; per query tile s_full, p_full, o_done, p_half; fin
  static constexpr int kNumBars = 2 * kRaw + 2 * kSlots + 2 + 4 + 2 * 4 + 1;
  static constexpr int kItemOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kHolderOff = kItemOff + 2 * 64;
  static constexpr int kSearchOff = kHolderOff + 16;  // words of the item search
  static constexpr int kSmemBytes = kSearchOff + 2 * 32 * 4;
  static constexpr int kWidenWarp = 8, kProdWarp = 12, kMmaWarp = 13;
  static constexpr int kWideners = 6;  // warps 8 to 11, 14 and 15
  static constexpr int kThreads = 16 * 32;
  static constexpr int kOCol = 2 * kKT;  // scores of tile X at column 128 X, O behind
  static constexpr int kTmemCols = 512;
  static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory");
};

struct alignas(16) Item {
  int q0, n;       // the sequence's first row and its new tokens
  int b, L;        // the sequence and its keys
  int tok0;        // the pair's first token
  int g;           // kv head; -1: no more items
  int k_lo, k_hi;  // the first key of the first tile (a page's first); behind the last
  int ntiles, jA1, jB0, jB1;  // tile A works on key tiles [0, jA1), B on [jB0, jB1)
};
static_assert(sizeof(Item) <= 64, "an item's place");

// Key positions of token t of an item's sequence.
__device__ __forceinline__ int pos_of(const Item& it, int causal, int t) {
  return causal ? it.L - it.n + t : it.L - 1;
}
__device__ __forceinline__ void set_tiles(Item& it, int tpc, int causal, int W, int bs) {
  auto lo = [&](int t) {
    const int p = pos_of(it, causal, t);
    return (W > 0 && p >= W) ? p + 1 - W : 0;
  };
  const int a0 = it.tok0, a1 = min(a0 + tpc, it.n);
  const int b0 = a0 + tpc, b1 = min(b0 + tpc, it.n);
  const bool has_b = b1 > b0;
  it.k_lo = lo(a0) / bs * bs;
  const int hi_a = pos_of(it, causal, a1 - 1) + 1;
  const int hi_b = has_b ? pos_of(it, causal, b1 - 1) + 1 : 0;
  it.k_hi = has_b ? hi_b : hi_a;
  it.ntiles = (it.k_hi - it.k_lo + kKT - 1) / kKT;
  it.jA1 = (hi_a - it.k_lo + kKT - 1) / kKT;
  it.jB0 = has_b ? (lo(b0) - it.k_lo) / kKT : 0;
  it.jB1 = has_b ? (hi_b - it.k_lo + kKT - 1) / kKT : 0;
}

// New tokens of a sequence, none where its counts do not fit.
struct ChunkCounts {
  struct Raw {
    int q0, q1, L;
  };
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int* flags;
  int max_q_len, max_keys;
  __device__ __forceinline__ Raw load(int b) const {
    return Raw{cu_q[b], cu_q[b + 1], seq_lens[b]};
  }
  __device__ __forceinline__ int tokens(const Raw& r, bool tell) const {
    const int n = r.q1 - r.q0;
    if (n > max_q_len || (n > 0 && (r.L < n || r.L > max_keys))) {
      if (tell) atomicOr(flags, PD_DEV_BAD_SEQ_LEN);
      return 0;
    }
    return max(n, 0);
  }
};

// Codes 2 i, 2 i + 1 (SEL 0x4140) or 2 i + 2, 2 i + 3 (0x4342) of a word as bf16.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t i8x2_bf16x2(uint32_t w) {
  const uint32_t c = __byte_perm(w, 0u, SEL);
  const uint32_t up = (c & 0x007F007Fu) | 0x43004300u, down = (c & 0x00800080u) | 0x43004300u;
  __nv_bfloat162 x, y;
  memcpy(&x, &up, 4);
  memcpy(&y, &down, 4);
  const __nv_bfloat162 r = __hsub2(x, y);
  uint32_t o;
  memcpy(&o, &r, 4);
  return o;
}

// A lane's pieces of a tile, `n` of them STEP rows apart: codes at `from` as operand
// elements at `to` and, the second eight of a piece, `odd` bytes behind.
template <int D, int STEP, bool V>
__device__ __forceinline__ void widen_tile(uint32_t from, uint32_t to, uint32_t odd, int n) {
#pragma unroll
  for (int i = 0; i < (kKT + STEP - 1) / STEP; ++i) {
    if (i >= n) break;  // warp-uniform
    const uint4 w = lds128(from + i * STEP * D);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (V) {
        const uint32_t x = u[q] ^ 0x80808080u;
        o[2 * q] = i8x2_f16x2<0x4140>(x);
        o[2 * q + 1] = i8x2_f16x2<0x4342>(x);
      } else {
        o[2 * q] = i8x2_bf16x2<0x4140>(u[q]);
        o[2 * q + 1] = i8x2_bf16x2<0x4342>(u[q]);
      }
    }
    sts128(to + i * STEP * 128, o[0], o[1], o[2], o[3]);
    sts128(to + odd + i * STEP * 128, o[4], o[5], o[6], o[7]);
  }
}

template <int D, int BS>
__global__ void __launch_bounds__(ChCfg<D>::kThreads, 1)
    prefill_int8_kernel(const PrefillArgs a, const int max_q_len, const int64_t page_bytes,
                        const int64_t data_bytes) {
  using C = ChCfg<D>;
  constexpr int NG = kKT / BS;  // pages of a tile
  asm volatile("griddepcontrol.launch_dependents;");
  const int G = a.group;
  const int tpc = 128 / G;  // tokens of a query tile
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw;
  const uint32_t s0 = smem_u32(smem);
  if (s0 & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (tid == 0) atomicOr(a.flags, PD_DEV_BAD_SMEM);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* raw_full = bars;
  uint64_t* raw_empty = raw_full + C::kRaw;
  uint64_t* kv_full = raw_empty + C::kRaw;
  uint64_t* kv_empty = kv_full + C::kSlots;
  uint64_t* q_full = kv_empty + C::kSlots;
  uint64_t* q_empty = q_full + 1;
  uint64_t* item_full = q_full + 2;
  uint64_t* item_empty = q_full + 4;
  uint64_t* tile_bars = q_full + 6;
  uint64_t* fin_bar = tile_bars + 8;
  auto s_full = [&](int X) { return smem_u32(tile_bars + X * 4); };
  auto p_full = [&](int X) { return smem_u32(tile_bars + X * 4 + 1); };
  auto o_done = [&](int X) { return smem_u32(tile_bars + X * 4 + 2); };
  auto p_half = [&](int X) { return smem_u32(tile_bars + X * 4 + 3); };
  I8Scales* raw_scales = reinterpret_cast<I8Scales*>(smem + C::kRawScaleOff);
  I8Scales* scales = reinterpret_cast<I8Scales*>(smem + C::kScaleOff);
  Item* items = reinterpret_cast<Item*>(smem + C::kItemOff);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::kHolderOff);
  volatile int* abort_s = reinterpret_cast<volatile int*>(holder + 1);

  if (tid == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      // several warps arrive at some: the widening ones, the softmax's of a tile, an
      // item's readers
      const uint64_t* bar = bars + i;
      uint32_t count = 1;
      if ((bar >= raw_empty && bar < kv_empty) || bar == q_full) count = C::kWideners;
      for (int X = 0; X < 2; ++X)
        if (smem_u32(bar) == p_full(X) || smem_u32(bar) == p_half(X)) count = 4;
      if (bar == item_empty || bar == item_empty + 1) count = 8 + C::kWideners + 1;
      mbar_init(smem_u32(bar), count);
    }
    *abort_s = 0;
    holder[2] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(holder)),
                 "n"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int W = a.sliding_window;
  bool failed = false;
  const volatile int* no_abort = reinterpret_cast<const volatile int*>(holder + 2);  // stays 0

  // registers dealt by warpgroup (4 x 128 at launch: 2 x 80 and 2 x 176)
  if (warp >= C::kWidenWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == C::kProdWarp) {
      // ============================ copying warp ============================
      const int span = 2 * tpc;  // tokens of an item
      const ChunkCounts counts{a.cu_q, a.seq_lens, a.flags, max_q_len, a.max_blocks_per_seq * BS};
      ItemSearch<ChunkCounts> search(counts, lane, a.num_seqs, span, a.num_kv_heads,
                                     blockIdx.x == 0,
                                     reinterpret_cast<int(*)[32]>(smem + C::kSearchOff));
      auto find = [&]() {  // this CTA's next item; g = -1: none left
        const auto at = search.next();
        Item it = {};
        it.g = at.g;
        if (at.g < 0) return it;
        it.n = at.n;
        it.b = at.b;
        it.q0 = a.cu_q[at.b];
        it.L = a.seq_lens[at.b];
        it.tok0 = at.tok0;
        set_tiles(it, tpc, a.causal, W, BS);
        return it;
      };
      // item kk for the others to read
      auto publish = [&](const Item& it, int kk) {
        const int is = kk & 1;
        if (kk >= 2 && !warp_wait(smem_u32(item_empty + is), ((kk >> 1) - 1) & 1, abort_s)) {
          failed = true;
          return;
        }
        if (lane == 0) {
          items[is] = it;
          mbar_arrive(smem_u32(item_full + is));
        }
        __syncwarp();
      };
      const uint8_t* kc = static_cast<const uint8_t*>(a.k_cache);
      const uint8_t* vc = static_cast<const uint8_t*>(a.v_cache);
      int raw = 0;  // raw slots filled so far
      Item it = find();
      publish(it, 0);
      for (int k = 0; it.g >= 0 && !failed; ++k) {
        const int32_t* bt = a.block_tables + static_cast<int64_t>(it.b) * a.max_blocks_per_seq;
        const int pages = (it.k_hi + BS - 1) / BS;
        // lane x: entry base + x of the table and its page's two scales, and the same
        // of the 32 entries that follow
        struct Entry {
          int page;
          float ks, vs;
        };
        auto entry_at = [&](int e) {
          Entry r{-1, 0.0f, 1.0f};
          if (e < pages) {
            r.page = bt[e];
            if (r.page >= 0 && r.page < a.num_blocks) {
              const int64_t at = r.page * page_bytes + data_bytes + 4 * it.g;
              r.ks = *reinterpret_cast<const float*>(kc + at);
              r.vs = *reinterpret_cast<const float*>(vc + at);
            } else {
              r.page = -1;
            }
          }
          return r;
        };
        int base = it.k_lo / BS;
        Entry cur = entry_at(base + lane), nxt = entry_at(base + 32 + lane);
        for (int j = 0; j < max(it.ntiles, 3) && !failed; ++j) {
          if (j == 2) publish(find(), k + 1);
          if (failed || j >= it.ntiles) continue;
          const int first = it.k_lo / BS + j * NG;  // a tile's pages: NG divides 32
          if (first - base >= 32) {
            base += 32;
            cur = nxt;
            nxt = entry_at(base + 32 + lane);
          }
          const int src = first - base + (lane < NG ? lane : 0);
          const int page = __shfl_sync(0xFFFFFFFFu, cur.page, src);
          const float ks = __shfl_sync(0xFFFFFFFFu, cur.ks, src);
          const float vs = __shfl_sync(0xFFFFFFFFu, cur.vs, src);
          const bool mine = lane < NG && first + lane < pages;
          const bool copies = mine && page >= 0;
          if (mine && !copies) atomicOr(a.flags, PD_DEV_BAD_PAGE);
          const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, copies));
          const int64_t at = page * page_bytes + static_cast<int64_t>(it.g) * (BS * D);
#pragma unroll
          for (int part = 0; part < 2; ++part, ++raw) {
            const int rs = raw % C::kRaw;
            if (raw >= C::kRaw &&
                !warp_wait(smem_u32(raw_empty + rs), ((raw / C::kRaw) - 1) & 1, abort_s)) {
              failed = true;
              break;
            }
            const uint32_t fb = smem_u32(raw_full + rs);
            if (copies)
              bulk_load(s0 + C::kRawOff + rs * C::kRawBytes + lane * (BS * D),
                        (part ? vc : kc) + at, BS * D, fb);
            if (part == 1 && lane < NG)
              raw_scales[rs * kMaxGroups + lane] =
                  copies ? I8Scales{ks, __log2f(vs), __fdividef(1.0f, vs), 0.0f}
                         : I8Scales{0.0f, -INFINITY, 0.0f, 0.0f};
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(fb, n * (BS * D));
            __syncwarp();
          }
        }
        if (failed) break;
        it = items[(k + 1) & 1];
      }
      if (failed) {
        if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
        *abort_s = 1;
      }
      // the copies already issued land before the block can exit
      for (int t = max(0, raw - C::kRaw); t < raw; ++t)
        (void)mbar_wait(smem_u32(raw_full + t % C::kRaw), (t / C::kRaw) & 1);
    } else if (warp == C::kMmaWarp) {
      // ============================= MMA warp ================================
      const uint32_t lead = elect_one();
      constexpr uint32_t idS = umma_idesc(128, kKT, 0);
      constexpr uint32_t idO = umma_idesc_f16(128, D, 1);
      const uint32_t q_lo = desc_lo(s0, 16), k_lo = desc_lo(s0 + C::kRingOff, 16);
      const uint32_t v_lo = desc_lo(s0 + C::kRingOff, kKT * 128);
      Ring<C::kSlots> kr, vr;  // the next tile of K, and of V
      vr.next();
      uint32_t p_par[2] = {0u, 0u};  // of the next weights
      bool ok = true;
      int nt = 0, jA1 = 0, jB0 = 0, jB1 = 0;
      int nt1 = 0, jA1_1 = 0, jB0_1 = 0, jB1_1 = 0;
      auto look = [&](int kk) {  // item kk's tiles; none at the end (or a failed wait)
        nt1 = 0;
        if (!(ok = warp_wait(smem_u32(item_full + (kk & 1)), (kk >> 1) & 1, abort_s))) return;
        const Item it = items[kk & 1];
        __syncwarp();
        arrive_if(lead, smem_u32(item_empty + (kk & 1)));
        nt1 = __shfl_sync(0xFFFFFFFFu, it.g < 0 ? 0 : it.ntiles, 0);
        jA1_1 = __shfl_sync(0xFFFFFFFFu, it.jA1, 0);
        jB0_1 = __shfl_sync(0xFFFFFFFFu, it.jB0, 0);
        jB1_1 = __shfl_sync(0xFFFFFFFFu, it.jB1, 0);
      };
      look(0);
      for (int k = 0; ok && nt1 > 0; ++k) {
        nt = nt1;
        jA1 = jA1_1;
        jB0 = jB0_1;
        jB1 = jB1_1;
        if (!(ok = warp_wait(smem_u32(q_full), k & 1, abort_s))) break;
        auto in = [&](int X, int j) { return X ? (j >= jB0 && j < jB1) : j < jA1; };
        auto last = [&](int X, int j) { return j == (X ? jB1 : jA1) - 1; };
        auto scores = [&](int X) {
          const uint32_t b = k_lo + kr.at * (C::kSlotBytes >> 4);
          const uint32_t q = q_lo + X * (C::kQBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ss(tmem + X * kKT, q + (((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4),
                   b + (((ks >> 2) * (kKT * 128) + (ks & 3) * 32) >> 4), idS, ks > 0, lead);
          commit_if(lead, s_full(X));
        };
        auto product = [&](int X, bool first) {
          const uint32_t b = v_lo + vr.at * (C::kSlotBytes >> 4);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!warp_wait(half ? p_full(X) : p_half(X), p_par[X], abort_s)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = half * (kKT / 32); kk < (half + 1) * (kKT / 32); ++kk)
              mma_ts(tmem + C::kOCol + X * D, tmem + X * kKT + kk * 8, b + ((kk * 2048) >> 4), idO,
                     !first || kk > 0, lead);
          }
          p_par[X] ^= 1u;
          return true;
        };
        auto wait_k = [&]() { return warp_wait(smem_u32(kv_full + kr.at), kr.parity, abort_s); };
        auto wait_v = [&]() { return warp_wait(smem_u32(kv_full + vr.at), vr.parity, abort_s); };
        auto pass_k = [&](int j) {  // K's tile j handed back behind its scores
          commit_if(lead, smem_u32(kv_empty + kr.at));
          if (j == nt - 1) commit_if(lead, smem_u32(q_empty));
          kr.next();
          kr.next();
        };
        if (!(ok = wait_k())) break;
        tc_fence_after();
#pragma unroll
        for (int X = 0; X < 2; ++X)
          if (in(X, 0)) scores(X);
        pass_k(0);
        if (nt == 1) look(k + 1);
        for (int j = 0; ok && j < nt; ++j) {
          const bool more = j + 1 < nt;
          if (!(ok = wait_v())) break;
#pragma unroll
          for (int X = 0; X < 2; ++X) {
            if (in(X, j)) {
              if (!(ok = product(X, X == 1 ? j == jB0 : j == 0))) break;
              if (last(X, j)) commit_if(lead, o_done(X));
            }
            if (X == 0 && more && !(ok = wait_k())) break;
            // the next scores go over these weights, behind the product that reads them
            // in the tensor core's order
            if (more && in(X, j + 1)) scores(X);
          }
          if (!ok) break;
          commit_if(lead, smem_u32(kv_empty + vr.at));
          vr.next();
          vr.next();
          if (more) {
            pass_k(j + 1);
            if (j + 2 == nt) look(k + 1);
          }
        }
      }
      if (!ok) {
        if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
        *abort_s = 1;
      }
      // every MMA issued has completed before TMEM is freed
      commit_if(lead, smem_u32(fin_bar));
      (void)warp_wait(smem_u32(fin_bar), 0, no_abort);
    } else {
      // =========================== widening warps ===========================
      const int ww = warp < C::kProdWarp ? warp - C::kWidenWarp : warp - C::kWidenWarp - 2;
      const int wt = ww * 32 + lane;  // 0 .. 191
      // A warp takes units of four rows (head_dim 64: eight), every sixth, a lane a piece
      // of 16 codes. Eight lanes of an access meet eight places of 128 bytes: four pieces
      // of an even row and four of the next, at head_dim 128 of the other half of it
      constexpr int kUnit = D == 128 ? 4 : 8;
      const int urow = D == 128 ? 2 * (lane >> 4) + ((lane >> 2) & 1) : lane >> 2;
      const int ch = D == 128 ? ((lane >> 2) ^ (lane >> 3)) & 1 : 0;
      int slot = 0;                             // slots filled so far, of both rings
      for (int k = 0; !failed; ++k) {
        if (!warp_wait(smem_u32(item_full + (k & 1)), (k >> 1) & 1, abort_s)) {
          failed = true;
          break;
        }
        const Item it = items[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(item_empty + (k & 1)));
        if (it.g < 0) break;
        // ---- Q: rows (token, head) of the two tiles, swizzled; no token: zeros ----
        if (k >= 1 && !warp_wait(smem_u32(q_empty), (k - 1) & 1, abort_s)) {
          failed = true;
          break;
        }
        const int parts = it.jB1 > 0 ? 2 : 1;
        for (int X = 0; X < parts; ++X) {
#pragma unroll 4
          for (int e = wt; e < 128 * D / 8; e += C::kWideners * 32) {
            const int m = e / (D / 8), pc = e % (D / 8);
            const int mt = m / G, mh = m - mt * G;
            const int t = it.tok0 + X * tpc + mt;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (mt < tpc && t < it.n)
              v = *reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(it.q0 + t) * a.q_stride +
                                                  static_cast<int64_t>(it.g * G + mh) * D + pc * 8);
            sts128(s0 + X * C::kQBytes + (pc >> 3) * (128 * 128) + swz128(m * 128 + (pc & 7) * 16),
                   v.x, v.y, v.z, v.w);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(q_full));
        // ---- K and V tiles, in the order the MMA warp takes them ----
        for (int j = 0; j < 2 * it.ntiles; ++j, ++slot) {
          const int rs = slot % C::kRaw, st = slot % C::kSlots;
          if (!warp_wait(smem_u32(raw_full + rs), (slot / C::kRaw) & 1, abort_s) ||
              (slot >= C::kSlots &&
               !warp_wait(smem_u32(kv_empty + st), ((slot / C::kSlots) - 1) & 1, abort_s))) {
            failed = true;
            break;
          }
          const uint32_t src = s0 + C::kRawOff + rs * C::kRawBytes;
          const uint32_t dst = s0 + C::kRingOff + st * C::kSlotBytes;
          if ((j & 1) && wt < NG) scales[st * kMaxGroups + wt] = raw_scales[rs * kMaxGroups + wt];
          // two warps have a unit more: others at V than at K
          const int first = (j & 1) ? (ww < 2 ? ww + 4 : ww - 2) : ww;
          const int key = first * kUnit + urow;
          const uint32_t from = src + key * D + (ch * 4 + (lane & 3)) * 16;
          const uint32_t to0 = swz128(key * 128 + (lane & 3) * 32);
          const uint32_t odd = swz128(key * 128 + (lane & 3) * 32 + 16) - to0;
          const uint32_t to = dst + ch * (kKT * 128) + to0;
          const int units = (kKT / kUnit - first + C::kWideners - 1) / C::kWideners;
          if (j & 1) widen_tile<D, C::kWideners * kUnit, true>(from, to, odd, units);
          else widen_tile<D, C::kWideners * kUnit, false>(from, to, odd, units);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(raw_empty + rs));
            mbar_arrive(smem_u32(kv_full + st));
          }
        }
      }
      if (failed) {
        if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
        *abort_s = 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    // =========================== softmax warps ============================
    const int X = warp >> 2;
    const int m = (warp & 3) * 32 + lane;  // row of the query tile: token m / G, head m % G
    const int mt = m / G, mh = m % G;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_tm = tmem + lane_base + C::kOCol + X * D;
    const uint32_t s_tm = tmem + lane_base + X * kKT;
    int slot = 0, done = 0;  // ring slots and key tiles before the item
    int runs = 0;            // items this query tile had part in
    for (int k = 0; !failed; ++k) {
      if (!warp_wait(smem_u32(item_full + (k & 1)), (k >> 1) & 1, abort_s)) {
        failed = true;
        break;
      }
      const Item it = items[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(item_empty + (k & 1)));
      if (it.g < 0) break;
      const int t = it.tok0 + X * tpc + mt;
      const bool rvalid = mt < tpc && t < it.n;
      // keys this row sees: [rlo, rhi); rows of no token count as seeing all
      const int rpos = pos_of(it, a.causal, t);
      const int rhi = rvalid ? rpos + 1 : INT32_MAX;
      const int rlo = (rvalid && W > 0 && rpos >= W) ? rpos + 1 - W : 0;
      const int j0 = X ? it.jB0 : 0, j1 = X ? it.jB1 : it.jA1;
      float m_run = -INFINITY, l_run = 0.0f;
      for (int j = j0; j < j1; ++j) {
        const int c = done + j - j0;
        const int key0 = it.k_lo + j * kKT;
        const int vs = slot + 2 * j + 1, vst = vs % C::kSlots;
        // the tile's scales come with its V
        if (!warp_wait(s_full(X), c & 1, abort_s) ||
            !warp_wait(smem_u32(kv_full + vst), (vs / C::kSlots) & 1, abort_s)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const I8Scales* sc = scales + vst * kMaxGroups;
        const int lo = rlo - key0, hi = rhi - key0;  // this tile's keys [lo, hi)
        const bool open = __all_sync(0xFFFFFFFFu, !rvalid || (lo <= 0 && hi >= kKT));
        uint32_t v[kKT / 32][32];
#pragma unroll
        for (int ch = 0; ch < kKT / 32; ++ch) tmem_ld32(s_tm + ch * 32, v[ch]);
        tmem_wait_ld32(v[0]);
#pragma unroll
        for (int ch = 1; ch < kKT / 32; ++ch) after_wait32(v[ch]);
        // scores in log2 units, the value scale's logarithm with them
#pragma unroll
        for (int ch = 0; ch < kKT / 32; ++ch)
#pragma unroll
          for (int p = 0; p < 32 / BS; ++p) {
            const float4 f = *reinterpret_cast<const float4*>(sc + ch * (32 / BS) + p);
            const float mul = a.scale_log2 * f.x;
#pragma unroll
            for (int i = p * BS; i < (p + 1) * BS; i += 2) {
              const float2 x = fma2(v[ch][i], v[ch][i + 1], mul, f.y);
              v[ch][i] = __float_as_uint(x.x);
              v[ch][i + 1] = __float_as_uint(x.y);
            }
          }
        if (!open) {
#pragma unroll
          for (int ch = 0; ch < kKT / 32; ++ch) {
            const uint32_t keep = bits_below(hi - ch * 32) & ~bits_below(lo - ch * 32);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[ch][i] = (keep & (1u << i)) ? v[ch][i] : 0xFF800000u;  // -inf
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int ch = 0; ch < kKT / 32; ++ch)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], __uint_as_float(v[ch][i]),
                                     __uint_as_float(v[ch][i + 1]));
        const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]);
        float mn = m_run;
        if (mx != -INFINITY && (mx > m_run + kMoveLog2 || m_run == -INFINITY)) mn = mx;
        const float alpha = (mn == m_run || m_run == -INFINITY) ? 1.0f : ex2(m_run - mn);
        m_run = mn;
        // O is rescaled behind the product before: these scores came behind it
        if (j > j0 && __any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
#pragma unroll 1
          for (int h = 0; h < D / 16; ++h) {
            uint32_t o[16];
            tmem_ld16(o_tm + h * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(o_tm + h * 16, o);
          }
        }
        // ---- weights over this row's scores, each half told of when it is there ----
        const float ref = mn == -INFINITY ? 0.0f : kLift - mn;
        l_run *= alpha;
#pragma unroll
        for (int ch = 0; ch < kKT / 32; ++ch) {
          uint32_t w[16];
#pragma unroll
          for (int p = 0; p < 32 / BS; ++p) {
            float2 sum = {0.0f, 0.0f};
#pragma unroll
            for (int i = p * BS / 2; i < (p + 1) * BS / 2; ++i) {
              const float2 x = add2(
                  float2{__uint_as_float(v[ch][2 * i]), __uint_as_float(v[ch][2 * i + 1])},
                  float2{ref, ref});
              const float2 e = {ex2(x.x), ex2(x.y)};
              sum = add2(sum, e);
              w[i] = pack_f16x2(e.x, e.y);
            }
            // the row sum is of the weights without the value scale
            l_run = fmaf(sum.x + sum.y, sc[ch * (32 / BS) + p].v_inv, l_run);
          }
          tmem_st16(s_tm + ch * 16, w);
          if ((ch + 1) % (kKT / 64) == 0) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ch + 1 == kKT / 32 ? p_full(X) : p_half(X));
          }
        }
      }
      if (failed) break;
      slot += 2 * it.ntiles;
      if (j1 > j0) {
        done += j1 - j0;
        ++runs;
        if (!warp_wait(o_done(X), (runs - 1) & 1, abort_s)) {
          failed = true;
          break;
        }
        tc_fence_after();
        // out by way of shared memory, 32 outputs of the warp's 32 rows at a time: a
        // row's four 16-byte pieces swizzled, eight rows a store
        uint16_t* orow = a.out + static_cast<int64_t>(it.q0 + t) * a.out_stride +
                         static_cast<int64_t>(it.g * G + mh) * D;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, rvalid);
        const float inv = 1.0f / fmaxf(l_run, 1e-20f);
        const uint32_t stage = s0 + C::kOutOff + warp * 2048;
        uint64_t at[4];  // the rows this lane stores a piece of
#pragma unroll
        for (int i = 0; i < 4; ++i)
          at[i] = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(orow), 8 * i + (lane >> 2));
#pragma unroll 1
        for (int h = 0; h < D / 32; ++h) {
          uint32_t o[32];
          tmem_ld32(o_tm + h * 32, o);
          tmem_wait_ld32(o);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(o[q * 8 + 2 * i]) * inv,
                                 __uint_as_float(o[q * 8 + 2 * i + 1]) * inv);
            sts128(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) * 16), w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2);
            const uint4 w = lds128(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) * 16));
            if ((valid >> row) & 1u)
              *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(at[i]) + h * 32 +
                                        (lane & 3) * 8) = w;
          }
          __syncwarp();
        }
        tc_fence_before();
      }
    }
    if (failed) {
      if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
      *abort_s = 1;
    }
  }

  // ---- free the TMEM columns once every warp is done with them ----
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "n"(C::kTmemCols)
                 : "memory");
  }
}

template <int D, int BS>
cudaError_t launch_chunk(const PrefillArgs& a, int max_q_len, int num_sms, cudaStream_t st) {
  using C = ChCfg<D>;
  auto kern = prefill_int8_kernel<D, BS>;
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
  const int span = 2 * (128 / a.group);
  const int64_t most = (static_cast<int64_t>(max_q_len) + span - 1) / span * a.num_seqs *
                       a.num_kv_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most < num_sms ? most : num_sms));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(
      &cfg, kern, a, max_q_len, any_page_bytes(PD_KV_INT8, BS, a.num_kv_heads, D),
      int8_data_bytes(BS, a.num_kv_heads, D));
}

}  // namespace

cudaError_t launch_prefill_int8(const PrefillArgs& a, int head_dim, int max_q_len, int num_sms,
                                cudaStream_t st) {
  const bool bs16 = a.block_size == 16;
  if (head_dim == 64)
    return bs16 ? launch_chunk<64, 16>(a, max_q_len, num_sms, st)
                : launch_chunk<64, 32>(a, max_q_len, num_sms, st);
  if (head_dim == 128)
    return bs16 ? launch_chunk<128, 16>(a, max_q_len, num_sms, st)
                : launch_chunk<128, 32>(a, max_q_len, num_sms, st);
  return cudaErrorInvalidValue;
}

}  // namespace pd
