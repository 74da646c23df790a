// Decode attention over INT8 pages (one scale per page and kv head): the
// split-KV partial kernel of every pd_decode* call for this form.
//
//   s_j = scale * kscale(j) * (q . kcode_j),  w_j = 2^(s_j + log2 vscale(j) - m + 15)
//   O = sum w_j vcode_j,  l = sum w_j / vscale(j),  out = O / l
//
// with s in log2 units and m the running maximum of s_j + log2 vscale(j): the
// value scale rides in the exponent, so the weights stay in (0, 2^15] for f16, the
// codes enter the tensor cores as they are, and a page's two scales cost two
// fused multiply-adds a score. Codes are widened to f16 exactly by integer
// operations (c + 128 as mantissa bits of 1024, less 1152): 1.25 (K) and 1.5 (V)
// instructions an element. A masked key has weight zero, and any byte is a
// finite code, so nothing in the stages needs clearing.
//
// CTA: warp 4 copies, warps 0-3 compute on mma.sync with keys on M and the q
// heads of the GQA group on N (int8_tile.cuh). A page's slab of one kv head is
// [block][dim] codes, one 128-byte-swizzled tensor copy per 128 bytes of
// head_dim; the copying lanes load the page's two scales beside it, 32 block-
// table entries at a time, and leave them in the stage's record. The CTA's work
// is one (sequence, kv head, split), or the pieces of a balanced plan.
//
// head_dim 64 / 128: warps 0 and 1 take 32 keys each of the even 64-key stages, 2
// and 3 of the odd ones, each with its own softmax state, merged at the end of a
// piece through the stage of its last tile. head_dim 256 / 512: the warps share
// head_dim and sum their scores through shared memory per 32-key stage. A warp's chain
// of a tile is long and few warps are there to hide it, so whatever is not widening is
// kept small: 32 keys an update, ring places counted up, a maximum sought over the lanes
// only when one moves.
//
// Measured: 64 sequences of 512 to 16384 keys, 64/8 heads of 128, balanced: 79.7 us
// with the merge of its partials, 390 MB (4.9 TB/s; floor 57.5); this kernel alone
// 76 us, DRAM 67% of its rate, integer pipe 45%, issue slots 44%: nothing is saturated,
// the chain copy, widen, scores, softmax, product waits for itself. Equal lengths, 64 x
// 4096 keys, 32/8 heads: 96 us, 5.6 TB/s. 16 keys an update, all warps on each stage:
// 90.8 us for the first; scales before the copies: 80.7.
//
// The other forms, 32 sequences of 4096 keys, floors in brackets: head_dim 64, 8 kv
// heads, 35.6 us (20): a page is 1 KB, half of head_dim 128's, at the same instructions
// a key for masks, softmax and barriers; DRAM 50%, integer pipe 43%, issue slots 44%.
// head_dim 256, 4 kv heads, 54 (40), 16 q heads 61; the warps meet every 32 keys (DRAM
// 65%, issue slots 52%). head_dim 512, 2 kv heads, 51 (40) with four q heads a kv
// head, 55 with seven, 71 with eight, whose q rows no longer leave room for a second
// CTA an SM. 16 q heads a kv head (two column tiles): head_dim 64 67 (20), 128 73 (40);
// 2048 keys, head_dim 256, 4 kv heads, 48 (20), 512, 8 kv heads, 137 (80): twice the
// softmax and state a key, at 168 registers (head_dim 128 spills 20 to 100 bytes) and
// two CTAs an SM; DRAM 38 to 49%, issue slots 34 to 39%.
//
// Waits are bounded (2 s): a warp that gives up raises the CTA's abort word and
// PD_DEV_TIMEOUT; the copying warp then issues nothing more and waits for what
// it issued.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cstring>
#include <mutex>
#include <type_traits>

#include "int8_tile.cuh"
#include "mma_common.cuh"
#include "serve_common.cuh"

namespace pd {
namespace {

using namespace ::pd::mma;

constexpr int kMaxCopies = 4;  // copies of a stage and cache: 64 keys of 16-row pages

// A piece of work, as the copying warp leaves it with the piece's q rows.
struct Piece {
  int b, g;              // sequence and kv head
  int t_base;            // key index of the first tile's first row
  int t_begin, t_end;    // the keys that count
  int ntiles;            // 0: no more pieces
  int direct;            // all of its (sequence, head): write the output
  int pad;
  int64_t ws_row;        // its first row in the workspace
};
struct StageScales {
  I8Scales copy[kMaxCopies];
};

template <int D, int NT, int BS>
struct I8Cfg {
  static constexpr bool kF16 = true;
  static constexpr int kDSplit = D <= 128 ? 1 : 4;       // warps sharing head_dim
  static constexpr int kDS = D / kDSplit;                // head_dim of a warp
  static constexpr int kKSteps = kDS / 16;
  static constexpr int kU = 2;                           // 16-key m-tiles of a warp per stage
  // head_dim <= 128: 64-key stages, warps 0 / 1 take the even ones' halves, 2 / 3 the
  // odd ones'. Else all warps take all of a 32-key stage
  static constexpr int kKT = kDSplit == 1 ? 64 : 32;
  static constexpr int kOwners = kDSplit == 1 ? 2 : 4;   // warps that work on a stage
  static constexpr int kBR = kKT < BS ? kKT : BS;        // rows per copy
  static constexpr int kNCopy = kKT / kBR;
  static constexpr int kCRB = D < 128 ? D : 128;         // bytes of a row chunk
  static constexpr int kDCH = D / kCRB;
  static constexpr bool kSwizzle = kCRB == 128;
  static constexpr int kCacheStageBytes = kKT * D;
  static constexpr int kStageBytes = 2 * kCacheStageBytes;
  // Stages in flight against CTAs (and registers) an SM. Up to eight heads a group, 32
  // sequences of 4096 keys of 8 heads of 64 / 128 (64 sequences) / 4 of 256 / 2 of 512:
  // 35.5 / 96.2 / 54.6 / 51.1 us; the rings a step smaller 35.2 / 108.7 / 54.8 / 53.5, a
  // step larger 40.6 / 112.0 / 61.1 / 68.8. Sixteen heads a group hold twice the state:
  // head_dim 128 at two CTAs of 96 KB 30.7, three of 64 KB 40.6; head_dim 512 at 64 KB
  // 139 (8 kv heads, 2048 keys), 96 KB 169
  static constexpr int kRing =
      (D == 64 ? 48 : D == 128 ? (NT == 1 ? 64 : 96) : D == 256 ? 64 : (NT == 1 ? 96 : 64)) * 1024;
  static constexpr int kStages = kRing / kStageBytes > 8 ? 8 : kRing / kStageBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kRedBytes = kDSplit == 4 ? 2 * 4 * kU * 32 * 4 * NT * 4 : 0;
  static constexpr int kQMaxBytes = kDSplit == 4 ? NT * 4 * 8 * 4 : 0;
  static constexpr int kHW = 8 * NT;
  static constexpr int kMergeBytes = kDSplit == 1 ? 2 * 2 * 4 * kHW * 4 : 0;  // m, l by parity
  static constexpr int kQSlots = kDSplit == 1 ? 2 : 1;
  static constexpr int kMergeOffset = kRingBytes + kRedBytes + kQMaxBytes;
  static constexpr int kScaleOffset = (kMergeOffset + kMergeBytes + 15) / 16 * 16;
  static constexpr int kPieceOffset = kScaleOffset + kStages * static_cast<int>(sizeof(StageScales));
  static constexpr int kBarOffset = kPieceOffset + kQSlots * static_cast<int>(sizeof(Piece));
  static constexpr int kNumBars = 2 * kStages + 2 * kQSlots + 1;
  static constexpr int kAbortOffset = kBarOffset + kNumBars * 8;
  static constexpr int kQOffset = (kAbortOffset + 16 + 127) / 128 * 128;
  static constexpr uint32_t kCopyBytes = kBR * D;
  static_assert(kNCopy <= kMaxCopies, "a stage's record holds the scales of four copies");
  static_assert(kDSplit == 4 || 4 * 8 * D * 4 <= kStageBytes, "eight heads' merge fits a stage");
  // a stage always belongs to the same warps: they see every phase of its barriers
  static_assert(kDSplit == 4 || kStages % 2 == 0, "even and odd tiles keep to their stages");
  static_assert(sizeof(Piece) % 8 == 0, "the barriers behind the records are 8-byte aligned");
  static constexpr int smem_bytes(int G) { return kQOffset + kQSlots * G * D * 2 + 1024; }
};

// Consumer-warp barrier on an mbarrier (one arrival a warp, bounded wait).
struct ConsumerSync {
  uint32_t bar, parity;
  volatile int* abort_flag;
  __device__ __forceinline__ bool operator()(int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    const bool ok = warp_wait(bar, parity, abort_flag);
    parity ^= 1u;
    if (!ok) *abort_flag = 1;
    return ok;
  }
};

template <int D, int NT, int BS, bool PLAN>
__global__ void __launch_bounds__(kMmaThreads,
                                  partial_min_blocks(I8Cfg<D, NT, BS>::smem_bytes(8 * NT), NT))
    decode_int8_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const DecodeArgs a) {
  using C = I8Cfg<D, NT, BS>;
  asm volatile("griddepcontrol.launch_dependents;");
  const int G = a.group;
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;  // fragment row group, column pair
  const uint32_t q_bytes = static_cast<uint32_t>(G) * D * 2;

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* ring = smem;
  float* red = reinterpret_cast<float*>(smem + C::kRingBytes);
  float* qmax_s = reinterpret_cast<float*>(smem + C::kRingBytes + C::kRedBytes);
  float* mrec = reinterpret_cast<float*>(smem + C::kMergeOffset);  // [2][4][kHW]
  float* lrec = mrec + 2 * 4 * C::kHW;
  StageScales* scales = reinterpret_cast<StageScales*>(smem + C::kScaleOffset);
  Piece* pieces = reinterpret_cast<Piece*>(smem + C::kPieceOffset);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty_bar = full_bar + C::kStages;
  uint64_t* qfull_bar = empty_bar + C::kStages;
  uint64_t* qempty_bar = qfull_bar + C::kQSlots;
  uint64_t* cons_bar = qempty_bar + C::kQSlots;
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + C::kAbortOffset);
  unsigned char* qslots = smem + C::kQOffset;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&empty_bar[i]), C::kOwners);
    }
    for (int i = 0; i < C::kQSlots; ++i) {
      mbar_init(smem_u32(&qfull_bar[i]), 1);
      mbar_init(smem_u32(&qempty_bar[i]), kConsumerWarps);
    }
    mbar_init(smem_u32(cons_bar), kConsumerWarps);
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == kConsumerWarps * 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
  }
  __syncthreads();
  // a programmatic dependent of the work before it: nothing global until then
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this CTA's work ----
  int p_begin, p_end;
  int4 split = make_int4(0, 0, 0, 0);  // the one piece of a split
  if constexpr (PLAN) {
    p_begin = a.plan_cta[blockIdx.x];
    p_end = a.plan_cta[blockIdx.x + 1];
    if (p_begin < 0 || p_end > a.plan_num_pieces || p_end < p_begin) {
      if (tid == 0) atomicOr(a.flags, PD_DEV_BAD_PLAN);
      p_begin = p_end = 0;
    }
  } else {
    const int g = blockIdx.x, s = blockIdx.y, b = blockIdx.z;
    int L = a.seq_lens[b];
    const int cap = a.max_blocks_per_seq * BS;
    if (L < 0 || L > cap) {
      if (tid == 0) atomicOr(a.flags, PD_DEV_BAD_SEQ_LEN);
      L = L < 0 ? 0 : cap;
    }
    const int lo = window_lo(L, a.sliding_window);
    const int P = num_key_pages(L, a.sliding_window, BS);
    if (s * a.chunk >= P) {                // no key of the sequence falls in this split
      if (a.direct && P == 0 && s == 0) {  // an empty sequence: zero output rows
        uint16_t* o = a.out + static_cast<int64_t>(b) * a.out_stride + g * G * D;
        for (int e = tid; e < G * D; e += blockDim.x) o[e] = 0;
      }
      return;
    }
    const int n_act = (P + a.chunk - 1) / a.chunk;
    const int first = lo / BS + s * a.chunk, last = min(lo / BS + P, first + a.chunk);
    split = make_int4(b * a.num_kv_heads + g, max(lo, first * BS), min(L, last * BS),
                      a.direct && n_act == 1 ? 1 : 0);
    p_begin = 0;
    p_end = 1;
  }
  // rows of the workspace between two heads of a piece
  const int64_t head_rows = PLAN ? 1 : a.num_splits;

  // =========================== copying warp ===============================
  if (warp == kConsumerWarps) {
    int desc_base = p_begin;
    int4 my_desc = make_int4(0, 0, 0, 0);
    if constexpr (PLAN) {
      if (p_begin + lane < p_end) my_desc = a.plan_pieces[p_begin + lane];
    }
    int i = 0;   // tiles issued
    int st = 0;  // the next one's stage, and the parity of its fill
    uint32_t parity = 0;
    int k = 0;   // pieces started
    bool ok = true;
    // piece k's record and q rows into its slot
    auto start = [&](int kk, const Piece& pc) {
      const int slot = kk % C::kQSlots;
      if (kk >= C::kQSlots &&
          !warp_wait(smem_u32(&qempty_bar[slot]), ((kk / C::kQSlots) - 1) & 1, abort_s))
        return false;
      if (lane == 0) {
        const uint32_t qb = smem_u32(&qfull_bar[slot]);
        pieces[slot] = pc;
        mbar_arrive_expect_tx(qb, pc.ntiles ? q_bytes : 0u);
        if (pc.ntiles)
          bulk_load(smem_u32(qslots + slot * q_bytes),
                    a.q + static_cast<int64_t>(pc.b) * a.q_stride + pc.g * G * D, q_bytes, qb);
      }
      __syncwarp();
      return true;
    };
    for (int piece = p_begin; piece < p_end && ok; ++piece) {
      int4 d = split;
      if constexpr (PLAN) {
        if (piece - desc_base >= 32) {
          desc_base = piece;
          my_desc = piece + lane < p_end ? a.plan_pieces[piece + lane] : make_int4(0, 0, 0, 0);
        }
        const int src = piece - desc_base;
        d.x = __shfl_sync(0xFFFFFFFFu, my_desc.x, src);
        d.y = __shfl_sync(0xFFFFFFFFu, my_desc.y, src);
        d.z = __shfl_sync(0xFFFFFFFFu, my_desc.z, src);
        d.w = __shfl_sync(0xFFFFFFFFu, my_desc.w, src);
        if (d.x < 0 || d.x >= a.num_seqs * a.num_kv_heads || d.y < 0 || d.z <= d.y ||
            d.z > a.max_blocks_per_seq * BS) {  // not a piece this plan can hold: skipped
          if (lane == 0) atomicOr(a.flags, PD_DEV_BAD_PLAN);
          continue;
        }
      }
      const int t_begin = d.y, t_end = d.z;
      const int b = d.x / a.num_kv_heads, g = d.x - b * a.num_kv_heads;
      const int64_t ws_row =
          PLAN ? static_cast<int64_t>(piece) * G
               : (static_cast<int64_t>(b) * a.num_q_heads + g * G) * a.num_splits + blockIdx.y;
      const int32_t* bt = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
      const int first_page = t_begin / BS, pages = (t_end + BS - 1) / BS;
      // lane x: entry cached_base + x of the table, and its page's two scales
      int cached_base = first_page, my_entry = -1;
      float my_ks = 0.0f, my_vs = 1.0f;
      auto refill = [&](int base) {
        cached_base = base;
        my_entry = base + lane < pages ? bt[base + lane] : -1;
        if (my_entry >= 0 && my_entry < a.num_blocks) {
          const int64_t at = my_entry * a.page_bytes + a.data_bytes + 4 * g;
          my_ks = *reinterpret_cast<const float*>(a.k_cache + at);
          my_vs = *reinterpret_cast<const float*>(a.v_cache + at);
        }
      };
      refill(first_page);
      const int t_base = first_page * BS;
      const int ntiles = (t_end - t_base + C::kKT - 1) / C::kKT;
      if (!start(k, Piece{b, g, t_base, t_begin, t_end, ntiles, d.w & 1, 0, ws_row})) {
        ok = false;
        break;
      }
      ++k;
      for (int j = 0; j < ntiles; ++j) {
        if (i >= C::kStages && !warp_wait(smem_u32(&empty_bar[st]), parity ^ 1u, abort_s)) {
          ok = false;
          break;
        }
        // lane jj < kNCopy makes copy jj of K and of V
        const int t0 = t_base + j * C::kKT;
        const int last_page = (min(t0 + C::kKT, t_end) - 1) / BS;
        if (last_page - cached_base >= 32) refill(t0 / BS);  // warp-uniform
        const int tt = t0 + lane * C::kBR;
        const bool mine = lane < C::kNCopy && tt < t_end;
        const int src = mine ? tt / BS - cached_base : 0;
        const int page = __shfl_sync(0xFFFFFFFFu, my_entry, src);
        const bool copies = mine && page >= 0 && page < a.num_blocks;
        const uint32_t fb = smem_u32(&full_bar[st]);
        // the copies first: the scales may still be on their way (the barrier's phase
        // ends with the arrival below at the earliest)
        if (copies) {
          const uint32_t kst = smem_u32(ring + st * C::kStageBytes);
          const int line = g * BS + tt % BS;
#pragma unroll
          for (int ch = 0; ch < C::kDCH; ++ch) {
            const uint32_t off = ch * (C::kKT * C::kCRB) + lane * (C::kBR * C::kCRB);
            tma_load_3d(kst + off, &tm_k, ch * C::kCRB, line, page, fb);
            tma_load_3d(kst + C::kCacheStageBytes + off, &tm_v, ch * C::kCRB, line, page, fb);
          }
        }
        const float ks = __shfl_sync(0xFFFFFFFFu, my_ks, src);
        const float vs = __shfl_sync(0xFFFFFFFFu, my_vs, src);
        const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, copies));
        if (lane < C::kNCopy)
          scales[st].copy[lane] = copies ? I8Scales{ks, __log2f(vs), __fdividef(1.0f, vs), 0.0f}
                                         : I8Scales{0.0f, -INFINITY, 0.0f, 0.0f};
        if (mine && !copies) atomicOr(a.flags, PD_DEV_BAD_PAGE);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(fb, 2u * C::kCopyBytes * n);
        __syncwarp();
        ++i;
        if (++st == C::kStages) {
          st = 0;
          parity ^= 1u;
        }
      }
    }
    // the end: a piece of no tiles
    if (ok) ok = start(k, Piece{0, 0, 0, 0, 0, 0, 0, 0, 0});
    if (ok) ++k;
    if (!ok) {
      if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
      *abort_s = 1;
    }
    // every copy issued lands before the block can exit
    for (int t = max(0, i - C::kStages); t < i; ++t)
      (void)mbar_wait(smem_u32(&full_bar[t % C::kStages]), (t / C::kStages) & 1);
    for (int t = max(0, k - C::kQSlots); t < k; ++t)
      (void)mbar_wait(smem_u32(&qfull_bar[t % C::kQSlots]), (t / C::kQSlots) & 1);
    return;
  }

  // =========================== computing warps ============================
  const int d0 = C::kDSplit == 4 ? warp * C::kDS : 0;
  ConsumerSync csync{smem_u32(cons_bar), 0u, abort_s};
  // head_dim index of accumulator element (m-tile md, row half hh)
  auto drow = [&](int md, int hh) { return d0 + r * (C::kDS / 8) + hh * C::kKSteps + md; };
  const ThreadPlace tp{warp, lane, r, c, d0};
  const int first = C::kDSplit == 1 ? (warp & 1) * 32 : 0;  // the warp's first key of a stage
  const I8Place<C> at(first, d0, r, c);
  // waits for a barrier's phase; false (for all warps alike where they share
  // barriers) if the wait ran out
  auto await = [&](uint64_t* bar, uint32_t par) {
    bool ok = warp_wait(smem_u32(bar), par, abort_s, a.consumer_wait_ns);
    if constexpr (C::kDSplit == 4) ok = consumers_vote(ok);
    if (!ok) {
      if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
      *abort_s = 1;
    }
    return ok;
  };
  int st = 0, red_buf = 0, ip = 0;
  uint32_t parity = 0;   // of stage st's fill
  uint32_t turn = 0;     // the tile's number, even or odd
  for (int k = 0;; ++k) {
    const int qslot = k % C::kQSlots;
    if (!await(&qfull_bar[qslot], (k / C::kQSlots) & 1)) break;
    const Piece pc = pieces[qslot];
    if (pc.ntiles == 0) break;
    const int b = pc.b, g = pc.g, t_begin = pc.t_begin, t_end = pc.t_end;
    const int64_t ws_row = pc.ws_row;
    const bool direct = pc.direct != 0;
    TileState<C, NT> ts;
    load_q_fragments<PD_KV_INT8, D, NT>(
        ts, reinterpret_cast<const uint16_t*>(qslots + qslot * q_bytes), G, a.scale_log2, 1.0f, tp,
        qmax_s);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&qempty_bar[qslot]));
    reset_state(ts);
    auto& acc = ts.acc;
    auto& m_run = ts.m_run;
    auto& l_run = ts.l_run;
    bool gave_up = false;
    int held = 0;  // the last tile's stage, and whether this warp worked on it
    bool held_own = false;
    int key0 = pc.t_base + first;
    for (int j = 0; j < pc.ntiles; ++j, key0 += C::kKT) {
      const bool own = C::kDSplit == 4 || turn == static_cast<uint32_t>(warp >> 1);
      const bool last = j == pc.ntiles - 1;
      if (own) {
        if (!await(&full_bar[st], parity)) {
          gave_up = true;
          break;
        }
        const uint32_t kst = smem_u32(ring + st * C::kStageBytes);
        consume_int8_tile<D, NT>(ts, at, kst, kst + C::kCacheStageBytes, key0, t_begin, t_end,
                                 scales[st].copy + first / C::kBR, tp, red, red_buf);
        if constexpr (C::kDSplit == 4) red_buf ^= 1;
        __syncwarp();
        // head_dim <= 128: the piece's last stage is handed back after the merge
        if (lane == 0 && !(C::kDSplit == 1 && last)) mbar_arrive(smem_u32(&empty_bar[st]));
      }
      held = st;
      held_own = own;
      turn ^= 1u;
      if (++st == C::kStages) {
        st = 0;
        parity ^= 1u;
      }
    }
    if (gave_up) break;

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          l_run[nt][j] += __shfl_xor_sync(0xFFFFFFFFu, l_run[nt][j], o);
    const int64_t orow0 = static_cast<int64_t>(b) * a.out_stride + g * G * D;  // head 0's row
    if constexpr (C::kDSplit == 4) {
      // every warp holds the same (m, l) and its own part of O's head_dim
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int h = nt * 8 + 2 * c + j;
          if (h >= G) continue;
          const float inv = 1.0f / fmaxf(l_run[nt][j], 1e-20f);
          const int64_t row = ws_row + h * head_rows;
#pragma unroll
          for (int md = 0; md < C::kKSteps; ++md)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float v = acc[md][nt][2 * hh + j] * inv;
              if (direct) a.out[orow0 + static_cast<int64_t>(h) * D + drow(md, hh)] = f32_to_bf16(v);
              else a.ws_o[row * D + drow(md, hh)] = v;
            }
          if (!direct && warp == 0 && r == 0)
            a.ws_ml[row] = make_float2(m_run[nt][j] - kWeightLog2, l_run[nt][j]);
        }
    } else {
      // the four warps' m and l by piece parity (a warp can reach the next
      // piece's merge while another still reads this one's), then eight heads at
      // a time their O in the held stage, element (d = 16 r' + e) of head h at
      // word (8 e + r') ^ 8 (h / 2 mod 4) of row (warp, h): no two lanes of a
      // store meet in a bank
      float* mr = mrec + ip * 4 * C::kHW;
      float* lr = lrec + ip * 4 * C::kHW;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (r == 0) {
            mr[warp * C::kHW + nt * 8 + 2 * c + j] = m_run[nt][j];
            lr[warp * C::kHW + nt * 8 + 2 * c + j] = l_run[nt][j];
          }
      float* orec = reinterpret_cast<float*>(ring + held * C::kStageBytes);
      constexpr int kE = D / 8;  // elements of d per fragment row group
      bool ok = true;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // every warp is done with the stage's keys, or with the heads before
        if (!(ok = csync(lane))) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float* row = orec + (warp * 8 + 2 * c + j) * D;
#pragma unroll
          for (int md = 0; md < C::kKSteps; ++md)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              row[((hh * C::kKSteps + md) * 8 + r) ^ (c * 8)] = acc[md][nt][2 * hh + j];
        }
        if (!(ok = csync(lane))) break;
        const int h_n = min(8, G - nt * 8);
        for (int e = tid; e < h_n * D; e += kConsumerWarps * 32) {
          const int hl = e / D, d = e % D, h = nt * 8 + hl;
          const int at = ((d % kE) * 8 + d / kE) ^ (((hl >> 1) & 3) * 8);
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) M = fmaxf(M, mr[w * C::kHW + h]);
          float lsum = 0.0f, o = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float mw = mr[w * C::kHW + h];
            const float f = (mw == -INFINITY) ? 0.0f : ex2(mw - M);
            lsum += lr[w * C::kHW + h] * f;
            o += orec[(w * 8 + hl) * D + at] * f;
          }
          const float v = o / fmaxf(lsum, 1e-20f);
          if (direct) {
            a.out[orow0 + static_cast<int64_t>(h) * D + d] = f32_to_bf16(v);
          } else {
            const int64_t row = ws_row + h * head_rows;
            a.ws_o[row * D + d] = v;
            if (d == 0) a.ws_ml[row] = make_float2(M - kWeightLog2, lsum);
          }
        }
      }
      if (!ok) break;
      // all warps are done with the stage, and their stores come before the copies
      // into it that follow
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (!csync(lane)) break;
      if (lane == 0 && held_own) mbar_arrive(smem_u32(&empty_bar[held]));
      ip ^= 1;
    }
  }
}

// Host: 3-D map over a cache of INT8 pages: (head_dim, kv head x row, page),
// box (chunk, rows, 1).
bool encode_int8_map(CUtensorMap* m, const void* base, int D, int lines, int64_t pages,
                     int64_t page_bytes, int chunk, int rows, bool swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(lines),
                              static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(page_bytes)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(chunk), static_cast<cuuint32_t>(rows), 1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, int BS, bool PLAN>
cudaError_t launch_cfg(const DecodeArgs& a, cudaStream_t st) {
  using C = I8Cfg<D, NT, BS>;
  CUtensorMap tk, tv;
  std::memset(&tk, 0, sizeof(tk));
  std::memset(&tv, 0, sizeof(tv));
  const int lines = a.num_kv_heads * BS;
  if (!encode_int8_map(&tk, a.k_cache, D, lines, a.num_blocks, a.page_bytes, C::kCRB, C::kBR,
                       C::kSwizzle) ||
      !encode_int8_map(&tv, a.v_cache, D, lines, a.num_blocks, a.page_bytes, C::kCRB, C::kBR,
                       C::kSwizzle))
    return cudaErrorInvalidValue;
  auto kern = decode_int8_kernel<D, NT, BS, PLAN>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {};  // per device; setting it twice is harmless
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::smem_bytes(8 * NT));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = PLAN ? dim3(a.plan_num_ctas) : dim3(a.num_kv_heads, a.num_splits, a.num_seqs);
  cfg.blockDim = dim3(kMmaThreads);
  cfg.dynamicSmemBytes = C::smem_bytes(a.group);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, a);
}

template <int D, int NT, int BS>
cudaError_t launch_src(const DecodeArgs& a, cudaStream_t st) {
  return a.plan_cta ? launch_cfg<D, NT, BS, true>(a, st) : launch_cfg<D, NT, BS, false>(a, st);
}

template <int D>
cudaError_t launch_dim(const DecodeArgs& a, cudaStream_t st) {
  if (a.group <= 8)
    return a.block_size == 16 ? launch_src<D, 1, 16>(a, st) : launch_src<D, 1, 32>(a, st);
  return a.block_size == 16 ? launch_src<D, 2, 16>(a, st) : launch_src<D, 2, 32>(a, st);
}

}  // namespace

int int8_ctas_per_sm(int head_dim, int group) {
  const bool two = group > 8;
  int smem = 0;
  switch (head_dim) {
    case 64: smem = two ? I8Cfg<64, 2, 16>::smem_bytes(group) : I8Cfg<64, 1, 16>::smem_bytes(group); break;
    case 128: smem = two ? I8Cfg<128, 2, 16>::smem_bytes(group) : I8Cfg<128, 1, 16>::smem_bytes(group); break;
    case 256: smem = two ? I8Cfg<256, 2, 16>::smem_bytes(group) : I8Cfg<256, 1, 16>::smem_bytes(group); break;
    default: smem = two ? I8Cfg<512, 2, 16>::smem_bytes(group) : I8Cfg<512, 1, 16>::smem_bytes(group); break;
  }
  const int n = (228 * 1024) / (smem + 1024);
  return n < 1 ? 1 : (n > 4 ? 4 : n);
}

cudaError_t launch_decode_int8(const DecodeArgs& a, int head_dim, cudaStream_t st) {
  if (a.num_seqs == 0 || (a.plan_cta && a.plan_num_ctas == 0)) return cudaSuccess;
  switch (head_dim) {
    case 64: return launch_dim<64>(a, st);
    case 128: return launch_dim<128>(a, st);
    case 256: return launch_dim<256>(a, st);
    case 512: return launch_dim<512>(a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pd
