// Attention of packed prompts over their own rows (pd_prefill_packed) on
// tcgen05. out = softmax(scale Q K^T) V per (token, q head), fp32 scores and
// sums, bf16 weights.
//
// The tensor core is what should bound it: per 128 x 128 tile and head_dim 128
// the two products take 2 x 512 cycles of it, 16384 exponentials about as many
// of the special-function units. So:
//
//  * A query tile is 128 (token, q head) rows of one GQA group (128 / G tokens):
//    fewer tokens than rows, so the causal edge wastes little, and K and V are
//    read once a group. At head_dim 64 / 128 a CTA works on two of them in turn:
//    while one tile's softmax runs the tensor core has the other's products.
//  * Scores of a 128-key tile lie in TMEM (128 columns a query tile), the weights
//    go back over them as bf16 and are the A operand of the second product from
//    there. The next scores of the same tile are issued behind that product:
//    the tensor core takes the instructions of one thread in order.
//  * One thread a row: maximum, exponentials and sum need no exchange. Weights
//    are 2^(s - m) against a reference m that moves only when a tile passes it by
//    2^8; O is rescaled in TMEM then.
//  * CTAs stay. All (sequence, pair of tiles, kv head) items are ranked by the
//    pair's place in its sequence, last first: with a causal mask that is
//    costliest first, whatever the lengths. CTA c takes ranks c, 2 N - 1 - c,
//    2 N + c ... of N CTAs. The copying warp finds the items (prompt_items.cuh) and
//    loads the next item's Q, K and V while the last one's softmax and output are
//    under way. It seeks an item while the ring is full: sought before the loads, 16
//    ragged prompts took 185 us instead of 167.
//  * Copies are TMA boxes (tokens x heads x 64 of head_dim, 128-byte swizzle), K
//    and V in a ring of their own slots. Rows past a sequence's end come along in
//    its last tile: as keys they are masked, as V rows zeroed in shared memory.
//
// head_dim 256: one query tile a CTA (O alone takes half of TMEM), 64-key tiles,
// the scores in two buffers one tile ahead. The same at head_dim 64 (there with two
// tiles a CTA): 48.9 us where two tiles of 128 keys take 40.7 (six prompts of 1500 to
// 4096 tokens, 8/2 heads, window 1024); four tiles of 64 keys, 48: the softmax's
// fixed part is paid for half the keys.
//
// Measured, 32/8 heads of 128, causal: one prompt of 8192 tokens 315 to 350 us (1750 to
// 1570 TFLOP/s: the card's power limit; tensor pipe 74% of the time, the exponentials'
// unit 39%, issue slots 43%); 16 prompts of 64 to 2048 tokens 161 us with the rows of
// the call before in L2, 178 without (1280, 1160): half-masked tiles and the change of
// items. head_dim 64, 8192 tokens, 257 us (1070): a tile's chain scores, softmax,
// product, whose parts are each half busy. head_dim 256, 8/4 heads, 4096 tokens, 58 to
// 66 us by the card (1190 to 1040). Many short prompts pay for whole tiles: 256 of 128
// tokens 126 us, 1024 of 32 tokens 199 us.
//
// Every wait is bounded (2 s); a role that gives up says so, and the copying warp
// and the MMA warp wait for what they issued before the CTA ends.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "prompt_items.cuh"
#include "prompt_roles.cuh"
#include "serve_common.cuh"

namespace pd {
namespace {

using namespace ::pd::mma;
using namespace ::pd::umma;

constexpr float kMoveLog2 = 8.0f;  // weights stay below 2^8

template <int D>
struct PkCfg {
  static constexpr int kTiles = D <= 128 ? 2 : 1;      // query tiles of a CTA
  static constexpr int kKT = D <= 128 ? 128 : 64;      // keys of a tile
  static constexpr int kBufs = kTiles == 2 ? 1 : 2;    // score buffers of a query tile
  static constexpr int kDCH = D / 64;                  // 128-byte chunks of a row
  static constexpr int kQBytes = 128 * 2 * D;          // one query tile
  static constexpr int kSlotBytes = kKT * 2 * D;       // one tile of K or of V
  static constexpr int kOutBytes = kTiles * 4 * 4096;  // a warp's 32 rows x 64 outputs
  static constexpr int kSlots = (224 * 1024 - kTiles * kQBytes - kOutBytes) / kSlotBytes;
  static constexpr int kRingOff = kTiles * kQBytes;
  static constexpr int kOutOff = kRingOff + kSlots * kSlotBytes;
  static constexpr int kBarOff = kOutOff + kOutBytes;
  // kv_full, kv_empty [slots]; q_full, q_empty; item_full, item_empty [2]; per tile
  // s_full[bufs], p_full, o_done, p_half; fin
  static constexpr int kTileBars = kBufs + 3;
  static constexpr int kNumBars = 2 * kSlots + 2 + 4 + kTiles * kTileBars + 1;
  static constexpr int kItemOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kHolderOff = kItemOff + 2 * 48;
  static constexpr int kSearchOff = kHolderOff + 16;  // words of the item search
  static constexpr int kSmemBytes = kSearchOff + 2 * 32 * 4;
  static constexpr int kSoftWarps = 4 * kTiles;
  static constexpr int kProdWarp = kSoftWarps;
  static constexpr int kMmaWarp = kSoftWarps + 1;
  static constexpr int kThreads = (kSoftWarps + 4) * 32;  // two warps of the last four idle
  // TMEM: scores of (tile, buffer) at 128 * tile + kKT * buffer, O of tile X behind
  static constexpr int kOCol = kTiles * kBufs * kKT;
  static constexpr int kTmemCols = 512;
  static_assert(kOCol + kTiles * D <= kTmemCols, "TMEM columns");
  static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory");
  static_assert(kSlots >= 3, "K and V in use and one on its way");
};

// A box of a tensor map into L2.
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}
// An item, as the copying warp leaves it for the others: tokens tok0 .. of query
// tile A, tok0 + 128 / G .. of B, key tiles from k_lo on; A works on tiles [0, jA1),
// B on [jB0, jB1) (none: 0, 0).
struct alignas(16) Item {
  int q0, n;    // the sequence's first row and its tokens
  int tok0;     // the pair's first token
  int g;        // kv head; -1: no more items
  int k_lo, ntiles, jA1, jB0, jB1;
  int pad[3];
};
template <int KT, int TILES>
__device__ __forceinline__ void set_tiles(Item& it, int tpc, int causal, int W) {
  auto pos = [&](int t) { return causal ? t : it.n - 1; };
  auto lo = [&](int t) { return (W > 0 && pos(t) >= W) ? pos(t) + 1 - W : 0; };
  const int a0 = it.tok0, a1 = min(a0 + tpc, it.n);
  const int b0 = a0 + tpc, b1 = min(b0 + tpc, it.n);
  const bool has_b = TILES == 2 && b1 > b0;
  it.k_lo = lo(a0);
  const int hi_a = pos(a1 - 1) + 1, hi_b = has_b ? pos(b1 - 1) + 1 : 0;
  it.ntiles = ((has_b ? hi_b : hi_a) - it.k_lo + KT - 1) / KT;
  it.jA1 = (hi_a - it.k_lo + KT - 1) / KT;
  it.jB0 = has_b ? (lo(b0) - it.k_lo) / KT : 0;
  it.jB1 = has_b ? (hi_b - it.k_lo + KT - 1) / KT : 0;
}

// Tokens of a sequence, none where its counts do not fit the batch.
struct PromptCounts {
  struct Raw {
    int q0, q1;
  };
  const int32_t* cu_q;
  int* flags;
  int total_q, max_q_len;
  __device__ __forceinline__ Raw load(int b) const { return Raw{cu_q[b], cu_q[b + 1]}; }
  __device__ __forceinline__ int tokens(const Raw& r, bool tell) const {
    const int n = r.q1 - r.q0;
    if (r.q0 < 0 || n < 0 || r.q1 > total_q || n > max_q_len) {
      if (tell) atomicOr(flags, PD_DEV_BAD_SEQ_LEN);
      return 0;
    }
    return n;
  }
};

template <int D>
__global__ void __launch_bounds__(PkCfg<D>::kThreads, 1)
    prefill_packed_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const PackedArgs a) {
  using C = PkCfg<D>;
  constexpr int KT = C::kKT;
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
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = bars + C::kSlots;
  uint64_t* q_full = bars + 2 * C::kSlots;
  uint64_t* q_empty = q_full + 1;
  uint64_t* item_full = q_full + 2;
  uint64_t* item_empty = q_full + 4;
  uint64_t* tile_bars = q_full + 6;
  uint64_t* fin_bar = tile_bars + C::kTiles * C::kTileBars;
  auto s_full = [&](int X, int i) { return smem_u32(tile_bars + X * C::kTileBars + i); };
  auto p_full = [&](int X) { return smem_u32(tile_bars + X * C::kTileBars + C::kBufs); };
  auto o_done = [&](int X) { return smem_u32(tile_bars + X * C::kTileBars + C::kBufs + 1); };
  auto p_half = [&](int X) { return smem_u32(tile_bars + X * C::kTileBars + C::kBufs + 2); };
  Item* items = reinterpret_cast<Item*>(smem + C::kItemOff);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::kHolderOff);
  volatile int* abort_s = reinterpret_cast<volatile int*>(holder + 1);

  if (tid == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      const uint32_t bar = smem_u32(bars + i);
      uint32_t count = 1;
      for (int X = 0; X < C::kTiles; ++X)
        if (bar == p_full(X) || bar == p_half(X)) count = 4;
      // an item's readers: the softmax warps and the MMA thread
      if (bars + i == item_empty || bars + i == item_empty + 1) count = C::kSoftWarps + 1;
      mbar_init(bar, count);
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
  if (warp == C::kProdWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int W = a.sliding_window;
  bool failed = false;
  const volatile int* no_abort = reinterpret_cast<const volatile int*>(holder + 2);  // stays 0

  // registers dealt by warpgroup (two tiles: 3 x 168 at launch, then 72 and 2 x 216)
  if (warp >= C::kSoftWarps) {
    if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == C::kProdWarp) {
      // ============================ copying warp ============================
      const int span = C::kTiles * tpc;  // tokens of an item
      ItemSearch<PromptCounts> search(PromptCounts{a.cu_q, a.flags, a.total_q, a.max_q_len}, lane,
                                      a.num_seqs, span, a.num_kv_heads, blockIdx.x == 0,
                                      reinterpret_cast<int(*)[32]>(smem + C::kSearchOff));
      auto find = [&]() {  // this CTA's next item; g = -1: none left
        const auto at = search.next();
        Item it = {};
        it.g = at.g;
        if (at.g < 0) return it;
        it.n = at.n;
        it.q0 = a.cu_q[at.b];
        it.tok0 = at.tok0;
        set_tiles<KT, C::kTiles>(it, tpc, a.causal, W);
        return it;
      };
      // item kk for the others to read; its Q into L2
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
        if (it.g >= 0 && lane < C::kDCH * (it.jB1 > 0 ? 2 : 1))
          prefetch_3d(&tm_q, lane % C::kDCH * 64, it.g * G,
                      it.q0 + it.tok0 + lane / C::kDCH * tpc);
      };
      // Q of item kk: tokens x G heads x 64 of head_dim a copy
      int q_loads = 0;
      auto load_q = [&](const Item& it, int kk) {
        if (kk >= 1 && !warp_wait(smem_u32(q_empty), (kk - 1) & 1, abort_s)) {
          failed = true;
          return;
        }
        if (lane == 0) {
          const uint32_t box = static_cast<uint32_t>(tpc) * G * 128;
          const int parts = it.jB1 > 0 ? 2 : 1;
          mbar_arrive_expect_tx(smem_u32(q_full), box * C::kDCH * parts);
          for (int X = 0; X < parts; ++X)
#pragma unroll
            for (int ch = 0; ch < C::kDCH; ++ch)
              tma_load_3d(s0 + X * C::kQBytes + ch * (128 * 128), &tm_q, ch * 64, it.g * G,
                          it.q0 + it.tok0 + X * tpc, smem_u32(q_full));
        }
        ++q_loads;
        __syncwarp();
      };
      int slot = 0;  // ring slots filled so far
      Item it = find();
      publish(it, 0);
      for (int k = 0; it.g >= 0 && !failed; ++k) {
        // K and V tiles go in the order the MMA warp takes them. Q's buffer is the
        // last item's until its last scores are there: the first K and V tile, whose
        // slots are free before that, go ahead of it. The next item is sought while
        // the ring is full
        const int loads = 2 * it.ntiles;
        const int q_at = k == 0 ? 0 : 2;
        for (int j = 0; j < max(loads, 5); ++j) {
          if (j == q_at) load_q(it, k);
          if (j == 4) publish(find(), k + 1);
          if (failed) break;
          if (j >= loads) continue;
          const int st = slot % C::kSlots;
          if (slot >= C::kSlots &&
              !warp_wait(smem_u32(kv_empty + st), ((slot / C::kSlots) - 1) & 1, abort_s)) {
            failed = true;
            break;
          }
          if (lane == 0) {
            const uint32_t fb = smem_u32(kv_full + st);
            mbar_arrive_expect_tx(fb, C::kSlotBytes);
            const uint32_t dst = s0 + C::kRingOff + st * C::kSlotBytes;
#pragma unroll
            for (int ch = 0; ch < C::kDCH; ++ch)
              tma_load_3d(dst + ch * (KT * 128), (j & 1) ? &tm_v : &tm_k, ch * 64, it.g,
                          it.q0 + it.k_lo + (j >> 1) * KT, fb);
          }
          __syncwarp();
          ++slot;
        }
        if (failed) break;
        it = items[(k + 1) & 1];
      }
      if (failed) {
        if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
        *abort_s = 1;
      }
      // the copies already issued land before the block can exit
      for (int t = max(0, slot - C::kSlots); t < slot; ++t)
        (void)mbar_wait(smem_u32(kv_full + t % C::kSlots), (t / C::kSlots) & 1);
      if (q_loads > 0) (void)mbar_wait(smem_u32(q_full), (q_loads - 1) & 1);
    } else if (warp == C::kMmaWarp) {
      // ============================= MMA warp ================================
      // One lane issues; the whole warp runs the loop, so that descriptors stay in
      // uniform registers and nothing is computed between two instructions
      const uint32_t lead = elect_one();
      constexpr uint32_t idS = umma_idesc(128, KT, 0);
      constexpr uint32_t idO = umma_idesc(128, D, 1);
      const uint32_t q_lo = desc_lo(s0, 16), k_lo = desc_lo(s0 + C::kRingOff, 16);
      const uint32_t v_lo = desc_lo(s0 + C::kRingOff, KT * 128);
      Ring<C::kSlots> kr, vr;  // the next tile of K, and of V
      vr.next();
      int buf = 0;                        // one query tile: the next scores' buffer
      uint32_t p_par[2] = {0u, 0u};       // of the next weights
      int pbuf = 0;
      bool ok = true;
      int nt = 0, jA1 = 0, jB0 = 0, jB1 = 0;
      // item kk's tiles, in uniform registers; false at the end (or a failed wait)
      int nt1 = 0, jA1_1 = 0, jB0_1 = 0, jB1_1 = 0;
      auto look = [&](int kk) {
        nt1 = 0;
        if (!(ok = warp_wait(smem_u32(item_full + (kk & 1)), (kk >> 1) & 1, abort_s))) return;
        const Item it = items[kk & 1];
        __syncwarp();
        arrive_if(lead, smem_u32(item_empty + (kk & 1)));
        nt1 = __shfl_sync(0xFFFFFFFFu, it.ntiles, 0);
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
        // scores of K's next tile for query tile X
        auto scores = [&](int X) {
          const uint32_t b = k_lo + kr.at * (C::kSlotBytes >> 4);
          const uint32_t d = tmem + X * 128 + (C::kBufs == 2 ? buf * KT : 0);
          const uint32_t q = q_lo + X * (C::kQBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ss(d, q + (((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4),
                   b + (((ks >> 2) * (KT * 128) + (ks & 3) * 32) >> 4), idS, ks > 0, lead);
          commit_if(lead, s_full(X, C::kBufs == 2 ? buf : 0));
        };
        // O_X += weights V's next tile
        auto product = [&](int X, bool first) {
          const uint32_t b = v_lo + vr.at * (C::kSlotBytes >> 4);
          const uint32_t p = tmem + X * 128 + (C::kBufs == 2 ? pbuf * KT : 0);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!warp_wait(half ? p_full(X) : p_half(X), p_par[X], abort_s)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = half * (KT / 32); kk < (half + 1) * (KT / 32); ++kk)
              mma_ts(tmem + C::kOCol + X * D, p + kk * 8, b + ((kk * 2048) >> 4), idO,
                     !first || kk > 0, lead);
          }
          p_par[X] ^= 1u;
          return true;
        };
        // the next item is looked up behind this one's last scores, while their
        // softmax is under way
        auto wait_k = [&]() { return warp_wait(smem_u32(kv_full + kr.at), kr.parity, abort_s); };
        auto wait_v = [&]() { return warp_wait(smem_u32(kv_full + vr.at), vr.parity, abort_s); };
        auto pass_k = [&](int j) {  // K's tile j handed back behind its scores
          commit_if(lead, smem_u32(kv_empty + kr.at));
          if (j == nt - 1) commit_if(lead, smem_u32(q_empty));
          kr.next();
          kr.next();
          if constexpr (C::kBufs == 2) buf ^= 1;
        };
        if (!(ok = wait_k())) break;
        tc_fence_after();
#pragma unroll
        for (int X = 0; X < C::kTiles; ++X)
          if (in(X, 0)) scores(X);
        pass_k(0);
        if (nt == 1) look(k + 1);
        for (int j = 0; ok && j < nt; ++j) {
          const bool more = j + 1 < nt;
          if (C::kTiles == 1 && more) {  // two score buffers: the next scores go ahead
            if (!(ok = wait_k())) break;
            tc_fence_after();
            scores(0);
            pass_k(j + 1);
            if (j + 2 == nt) look(k + 1);
            if (!ok) break;
          }
          if (!(ok = wait_v())) break;
          if (C::kTiles == 2 && more && !(ok = wait_k())) break;
#pragma unroll
          for (int X = 0; X < C::kTiles; ++X) {
            if (in(X, j)) {
              if (!(ok = product(X, X == 1 ? j == jB0 : j == 0))) break;
              // two score buffers: each tile's weights wait for it; one: the scores
              // that follow tell of it, but behind the last
              if (C::kBufs == 2 || last(X, j)) commit_if(lead, o_done(X));
            }
            // one buffer: the next scores go over these weights, behind the product
            // that reads them in the tensor core's order
            if (C::kTiles == 2 && more && in(X, j + 1)) scores(X);
          }
          if (!ok) break;
          commit_if(lead, smem_u32(kv_empty + vr.at));
          vr.next();
          vr.next();
          if constexpr (C::kBufs == 2) pbuf ^= 1;
          if (C::kTiles == 2 && more) {
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
    }
  } else {
    if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // =========================== softmax warps ============================
    const int X = warp >> 2;
    const int m = (warp & 3) * 32 + lane;  // row of the query tile: token m / G, head m % G
    const int mt = m / G, mh = m % G;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_tm = tmem + lane_base + C::kOCol + X * D;
    // a masked score is -inf before it is multiplied: never by zero
    const float sl2 = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);
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
      const int rpos = a.causal ? t : it.n - 1;
      const int rhi = rvalid ? rpos + 1 : INT32_MAX;
      const int rlo = (rvalid && W > 0 && rpos >= W) ? rpos + 1 - W : 0;
      const int j0 = X ? it.jB0 : 0, j1 = X ? it.jB1 : it.jA1;
      float m_run = -INFINITY, l_run = 0.0f;
      for (int j = j0; j < j1; ++j) {
        const int c = done + j - j0;
        const uint32_t s_tm = tmem + lane_base + X * 128 + (c % C::kBufs) * KT;
        const int key0 = it.k_lo + j * KT;
        if (!warp_wait(s_full(X, c % C::kBufs), (c / C::kBufs) & 1, abort_s)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const int lo = rlo - key0, hi = rhi - key0;  // this tile's keys [lo, hi)
        const bool open = __all_sync(0xFFFFFFFFu, !rvalid || (lo <= 0 && hi >= KT));
        // ---- the row's scores, their maximum, the reference ----
        uint32_t v[KT / 32][32];
#pragma unroll
        for (int ch = 0; ch < KT / 32; ++ch) tmem_ld32(s_tm + ch * 32, v[ch]);
        tmem_wait_ld32(v[0]);
#pragma unroll
        for (int ch = 1; ch < KT / 32; ++ch) after_wait32(v[ch]);
        if (a.scale_log2 < 0.0f) {  // the largest product is the smallest score's
#pragma unroll
          for (int ch = 0; ch < KT / 32; ++ch)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[ch][i] ^= 0x80000000u;
        }
        if (!open) {
#pragma unroll
          for (int ch = 0; ch < KT / 32; ++ch) {
            const uint32_t keep = bits_below(hi - ch * 32) & ~bits_below(lo - ch * 32);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[ch][i] = (keep & (1u << i)) ? v[ch][i] : 0xFF800000u;  // -inf
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int ch = 0; ch < KT / 32; ++ch)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], __uint_as_float(v[ch][i]),
                                     __uint_as_float(v[ch][i + 1]));
        const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]);
        float mn = m_run;
        if (mx != -INFINITY) {  // some key seen
          const float ms = mx * sl2;
          if (ms > m_run + kMoveLog2 || m_run == -INFINITY) mn = ms;
        }
        const float alpha = (mn == m_run || m_run == -INFINITY) ? 1.0f : ex2(m_run - mn);
        m_run = mn;

        // V rows past the sequence's end belong to others: zeroed before the
        // weights are released, by the first query tile that uses the tile
        const bool zeroer = X == 0 || j >= it.jA1;
        const bool ragged = key0 + KT > it.n;
        const int vs = slot + 2 * j + 1;
        if (zeroer && ragged) {
          if (!warp_wait(smem_u32(kv_full + vs % C::kSlots), (vs / C::kSlots) & 1, abort_s)) {
            failed = true;
            break;
          }
          const uint32_t vst = s0 + C::kRingOff + (vs % C::kSlots) * C::kSlotBytes;
          const int first = it.n - key0;  // >= 1
          for (int pc = first * 8 + m; pc < KT * 8; pc += 128)
#pragma unroll
            for (int ch = 0; ch < C::kDCH; ++ch)
              sts128(vst + ch * (KT * 128) + swz128(pc * 16), 0u, 0u, 0u, 0u);
          fence_async_smem();
        }
        // O may be rescaled once the product before has been added: with one score
        // buffer these scores came behind it. With two its barrier says so, and
        // these weights wait for it in any case, so that no barrier here runs a
        // phase ahead of its readers
        const bool rescale = j > j0 && __any_sync(0xFFFFFFFFu, alpha != 1.0f);
        if (C::kBufs == 2 && j > j0) {
          if (!warp_wait(o_done(X), (c - 1) & 1, abort_s)) {
            failed = true;
            break;
          }
          tc_fence_after();
        }
        if (rescale) {
#pragma unroll 1
          for (int h = 0; h < D / 16; ++h) {
            uint32_t v[16];
            tmem_ld16(o_tm + h * 16, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
            tmem_st16(o_tm + h * 16, v);
          }
        }
        // ---- weights over this row's scores, each half told of when it is there ----
        const float ref = mn == -INFINITY ? 0.0f : -mn;
        float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
        for (int ch = 0; ch < KT / 32; ++ch) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = fma2(v[ch][2 * i], v[ch][2 * i + 1], sl2, ref);
            const float2 e = {ex2(x.x), ex2(x.y)};
            sum[i & 1] = add2(sum[i & 1], e);
            w[i] = pack_bf16x2(e.x, e.y);
          }
          tmem_st16(s_tm + ch * 16, w);
          if ((ch + 1) % (KT / 64) == 0) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ch + 1 == KT / 32 ? p_full(X) : p_half(X));
          }
        }
        l_run = l_run * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
      }
      if (failed) break;
      slot += 2 * it.ntiles;
      if (j1 > j0) {
        done += j1 - j0;
        ++runs;
        if (!warp_wait(o_done(X), ((C::kBufs == 2 ? done : runs) - 1) & 1, abort_s)) {
          failed = true;
          break;
        }
        tc_fence_after();
        // Out by way of shared memory: a lane holds a whole row, but stores that
        // touch a line a lane take a cycle a line. 64 outputs of the warp's 32 rows
        // at a time, 16-byte pieces swizzled; four rows a store
        uint16_t* orow = a.out + static_cast<int64_t>(it.q0 + t) * a.out_stride +
                         static_cast<int64_t>(it.g * G + mh) * D;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, rvalid);
        const float inv = 1.0f / fmaxf(l_run, 1e-20f);
        const uint32_t stage = s0 + C::kOutOff + warp * 4096;
        // (head_dim 256 in two parts: a whole row takes too many registers)
        constexpr int kCols = D <= 128 ? D : 128;
#pragma unroll 1
        for (int part = 0; part < D / kCols; ++part) {
          uint32_t v[kCols / 32][32];
#pragma unroll
          for (int ch = 0; ch < kCols / 32; ++ch) tmem_ld32(o_tm + part * kCols + ch * 32, v[ch]);
          uint64_t at[8];  // the rows this lane stores a piece of
#pragma unroll
          for (int i = 0; i < 8; ++i)
            at[i] = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(orow), 4 * i + (lane >> 3));
          tmem_wait_ld32(v[0]);
#pragma unroll
          for (int ch = 1; ch < kCols / 32; ++ch) after_wait32(v[ch]);
#pragma unroll
          for (int h = 0; h < kCols / 64; ++h) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16x2(__uint_as_float(v[2 * h + (q >> 2)][(q & 3) * 8 + 2 * i]) * inv,
                                   __uint_as_float(v[2 * h + (q >> 2)][(q & 3) * 8 + 2 * i + 1]) *
                                       inv);
              sts128(stage + swz128(lane * 128 + q * 16), w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            uint4 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = lds128(stage + swz128((4 * i + (lane >> 3)) * 128 + (lane & 7) * 16));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if ((valid >> (4 * i + (lane >> 3))) & 1u)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(at[i]) + part * kCols + h * 64 +
                                          (lane & 7) * 8) = w[i];
            __syncwarp();
          }
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

// 3-D map over rows of heads: (head_dim, head, row), box (64, heads, rows).
bool encode_rows_map(CUtensorMap* m, const void* base, int D, int heads, int64_t rows,
                     int64_t row_stride, int box_heads, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2,
                                 static_cast<cuuint64_t>(row_stride) * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_heads),
                             static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_packed(const PackedArgs& a, int num_sms, cudaStream_t st) {
  using C = PkCfg<D>;
  CUtensorMap tq, tk, tv;
  const int tpc = 128 / a.group;
  if (!encode_rows_map(&tq, a.q, D, a.num_q_heads, a.total_q, a.q_stride, a.group, tpc) ||
      !encode_rows_map(&tk, a.k, D, a.num_kv_heads, a.total_q, a.k_stride, 1, C::kKT) ||
      !encode_rows_map(&tv, a.v, D, a.num_kv_heads, a.total_q, a.v_stride, 1, C::kKT))
    return cudaErrorInvalidValue;
  auto kern = prefill_packed_kernel<D>;
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
  // no more CTAs than there can be items: whole spans, and a last part a sequence
  const int span = C::kTiles * tpc;
  const int64_t most = (static_cast<int64_t>(a.total_q) / span + a.num_seqs) * a.num_kv_heads;
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
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_prefill_packed(const PackedArgs& a, int head_dim, int num_sms,
                                  cudaStream_t st) {
  switch (head_dim) {
    case 64: return launch_packed<64>(a, num_sms, st);
    case 128: return launch_packed<128>(a, num_sms, st);
    case 256: return launch_packed<256>(a, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pd
