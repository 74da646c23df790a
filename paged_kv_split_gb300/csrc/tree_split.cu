// Draft-tree attention at head_dim 256 and 512 in few rows, where the tcgen05 kernel
// would widen, score and weight for a nearly empty tile (and at 512 go over the keys
// twice): mma.sync tiles with keys on M and 8 or 16 rows (nodes times q
// heads) on N, head_dim split over four consumer warps, as decode_balanced.cu
// has them (mma_tile.cuh). More rows than that are further node tiles, which
// run side by side and find the keys in L2. Single tokens of 8 sequences over 8192
// keys, 16 / 2 heads of 512: 54 us in BF16 (floor 40), 41 in FP8 (20), 44 in NVFP4
// (11), the quantised forms bound by widening in registers.
//
// Keys are dealt by the device plan of tree_plan.cuh in 16-key tiles; a warp
// produces (TMA copies for BF16 and FP8, bulk copies for NVFP4, one page a tile)
// and four consume. All warps walk the plan themselves. Waits are bounded as in
// decode_balanced.cu, the consumers' for a piece's first copies by consumer_wait_ns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "mma_common.cuh"
#include "mma_tile.cuh"
#include "pd_common.cuh"
#include "tree_plan.cuh"

// Cfg<> defines every layout constant for every form; some forms ignore some.
#pragma nv_diag_suppress 177

namespace pd {
namespace {

using namespace ::pd::mma;
using namespace ::pd::tree;

constexpr int kSplitKT = 16;     // keys of a tile
constexpr int kSplitSlack = 4;   // units a piece costs beside its tiles
constexpr int kSplitBadRing = 16;

template <int FMT, int D, int NT>
struct SplitCfg {
  static constexpr bool kF16 = FMT != PD_KV_BF16;
  static constexpr int kDSplit = 4;
  static constexpr int kDS = D / 4;                 // head_dim slice of a warp
  static constexpr int kKSteps = kDS / 16;
  static constexpr int kWM = 1;
  static constexpr int kKT = kSplitKT;
  static constexpr int kMT = 1;
  static constexpr int kBR = 16;
  static constexpr int kRowBytes = FMT == PD_KV_BF16 ? 2 * D : (FMT == PD_KV_FP8_E4M3 ? D : D / 2);
  static constexpr int kCRB = FMT == PD_KV_NVFP4 ? D / 2 : 128;
  static constexpr int kDCH = kRowBytes / kCRB;
  static constexpr int kCopyElems = FMT == PD_KV_BF16 ? kCRB / 2 : kCRB;
  static constexpr bool kSwizzle = kCRB == 128 && FMT != PD_KV_NVFP4;
  static constexpr int kDataBytes = kKT * kRowBytes;
  static constexpr int kScaleBytes = FMT == PD_KV_NVFP4 ? kKT * (D / 16) : 0;
  static constexpr int kCacheStageBytes = (kDataBytes + kScaleBytes + 1023) / 1024 * 1024;
  static constexpr int kStageBytes = 2 * kCacheStageBytes;
  static constexpr int kStagesRaw = PD_MMA_RING_BYTES_LARGE_D / kStageBytes;
  static constexpr int kStages = kStagesRaw < 2 ? 2 : (kStagesRaw > 8 ? 8 : kStagesRaw);
  static constexpr int kRedBytes = 2 * 4 * 32 * 4 * NT * 4;
  static constexpr int kQMaxBytes = NT * 4 * 8 * 4;
  static constexpr int kRows = 8 * NT;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kRedOffset = kStages * kStageBytes;
  static constexpr int kQMaxOffset = kRedOffset + kRedBytes;
  static constexpr int kQOffset = (kQMaxOffset + kQMaxBytes + 127) / 128 * 128;
  static constexpr int kBarOffset = kQOffset + kQBytes;
  // full / empty [kStages], q full, q empty
  static constexpr int kBadOffset = kBarOffset + (2 * kStages + 2) * 8;
  static constexpr int kAbortOffset = kBadOffset + kSplitBadRing * 4;
  static constexpr int kSmemBytes = kAbortOffset + 16 + 1024;  // slack to align the ring
  static constexpr int kCopyBytes = kBR * kRowBytes + kScaleBytes;
  static constexpr int kPerSm =
      (228 * 1024) / (kSmemBytes + 1024) > 3 ? 3 : (228 * 1024) / (kSmemBytes + 1024);
};

// What the thread's four (or two) columns see, for consume_tile.
template <int NT>
struct TreeMask {
  RowView col[NT][2];
  RowView all;       // any column
  int open_lo;       // every column sees [open_lo, prefix)
  __device__ __forceinline__ static bool in(const RowView& v, int key) {
    if (key < v.prefix) return key >= v.lo || key < v.sinks;
    return key - v.prefix < 64 && ((v.bits >> (key - v.prefix)) & 1u);
  }
  __device__ __forceinline__ bool open(int key0) const {
    return key0 >= open_lo && key0 + 16 <= all.prefix;
  }
  __device__ __forceinline__ bool sees(int nt, int j, int key) const { return in(col[nt][j], key); }
  __device__ __forceinline__ bool any(int key) const { return in(all, key); }
};

template <int FMT, int D, int NT, int BS>
__global__ void __launch_bounds__(kMmaThreads, (SplitCfg<FMT, D, NT>::kPerSm))
    tree_split_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const TreeArgs a,
                      const TreeWork w) {
  using C = SplitCfg<FMT, D, NT>;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int G = a.group;
  const int TPC = w.item_nodes;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int r = lane >> 2;  // fragment row group
  const int c = lane & 3;   // fragment column pair

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // (scratch where the ring will be)
  const Share share = make_share(a, TPC, C::kKT, kSplitSlack, w.min_units,
                                 reinterpret_cast<ShareScratch*>(smem));
  if (tid == 0) w.records[blockIdx.x] = JoinRecord{0, 0, 0, 0};
  if (share.b < 0) return;
  float* red = reinterpret_cast<float*>(smem + C::kRedOffset);
  float* qmax_s = reinterpret_cast<float*>(smem + C::kQMaxOffset);
  unsigned char* q_s = smem + C::kQOffset;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty_bar = full_bar + C::kStages;
  uint64_t* q_full = empty_bar + C::kStages;
  uint64_t* q_empty = q_full + 1;
  uint32_t* bad_s = reinterpret_cast<uint32_t*>(smem + C::kBadOffset);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + C::kAbortOffset);
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&empty_bar[i]), kConsumerWarps);
    }
    mbar_init(smem_u32(q_full), 1);
    mbar_init(smem_u32(q_empty), kConsumerWarps);
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  Walker walk(a, share, TPC, C::kKT, kSplitSlack);
  Piece q;
  int i = 0;      // tiles so far
  int piece = 0;  // pieces whose q rows were copied, or used

  // =========================== producer warp ===============================
  if (warp == kConsumerWarps) {
    bool ok = true;
    while (ok && walk.next(q)) {
      if (lane == 0 && q.begins && !q.whole)
        w.records[blockIdx.x] =
            JoinRecord{walk.pieces_of_last(q.j1), q.p.s.q0 + q.rt * TPC,
                       min(TPC, q.p.s.n - q.rt * TPC), q.g * G};
      const int node0 = q.rt * TPC;
      const int nodes = min(TPC, q.p.s.n - node0);
      // the rows' q: the group's heads of a node are contiguous
      if (piece > 0 && !warp_wait(smem_u32(q_empty), (piece - 1) & 1, abort_s)) {
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(q_full), nodes * G * D * 2);
      __syncwarp();
      if (lane < nodes)
        bulk_load(smem_u32(q_s + lane * G * D * 2),
                  a.q + static_cast<int64_t>(q.p.s.q0 + node0 + lane) * a.q_stride +
                      static_cast<int64_t>(q.g) * G * D,
                  G * D * 2, smem_u32(q_full));
      ++piece;
      const int32_t* bt = a.block_tables + static_cast<int64_t>(q.b) * a.max_blocks_per_seq;
      int base = -(1 << 30), entry = -1, ahead = -1;  // entries [base, base + 32), the next 32
      auto load = [&](int e) { return e < a.max_blocks_per_seq ? bt[e] : -1; };
      for (int j = q.j0; j < q.j1; ++j, ++i) {
        const int t0 = tile_key(q.p, j, C::kKT);
        const int e = t0 / BS;
        if (e - base >= 32 && e - base < 64) {
          base += 32;
          entry = ahead;
          ahead = load(base + 32 + lane);
        } else if (e < base || e - base >= 64) {
          base = e;
          entry = load(base + lane);
          ahead = load(base + 32 + lane);
        }
        const int pg = __shfl_sync(0xFFFFFFFFu, entry, e - base);
        const bool good = pg >= 0 && pg < a.num_blocks;
        const int st = i % C::kStages;
        if (i >= C::kStages &&
            !warp_wait(smem_u32(&empty_bar[st]), ((i / C::kStages) - 1) & 1, abort_s)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t fb = smem_u32(&full_bar[st]);
          bad_s[i % kSplitBadRing] = good ? 0u : 1u;
          if (!good) atomicOr(a.flags, PD_DEV_BAD_PAGE);
          mbar_arrive_expect_tx(fb, good ? 2u * C::kCopyBytes : 0u);
          if (good) {
            const uint32_t kst = smem_u32(smem + st * C::kStageBytes);
            const uint32_t vst = kst + C::kCacheStageBytes;
            const int row0 = t0 % BS;
            if constexpr (FMT == PD_KV_NVFP4) {
              const int64_t line = static_cast<int64_t>(q.g) * BS + row0;
              const uint8_t* kp = a.k_cache + pg * a.page_bytes;
              const uint8_t* vp = a.v_cache + pg * a.page_bytes;
              constexpr uint32_t db = C::kBR * (D / 2), sb = C::kBR * (D / 16);
              bulk_load(kst, kp + line * (D / 2), db, fb);
              bulk_load(vst, vp + line * (D / 2), db, fb);
              bulk_load(kst + C::kDataBytes, kp + a.data_bytes + line * (D / 16), sb, fb);
              bulk_load(vst + C::kDataBytes, vp + a.data_bytes + line * (D / 16), sb, fb);
            } else {
              const int z = pg * BS + row0;
#pragma unroll
              for (int ch = 0; ch < C::kDCH; ++ch) {
                const uint32_t off = ch * (C::kKT * C::kCRB);
                tma_load_3d(kst + off, &tm_k, ch * C::kCopyElems, q.g, z, fb);
                tma_load_3d(vst + off, &tm_v, ch * C::kCopyElems, q.g, z, fb);
              }
            }
          }
        }
        __syncwarp();
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
      *abort_s = 1;
    }
    // every copy issued lands before the block can exit, the q rows of a piece
    // that was given up among them
    for (int t = max(0, i - C::kStages); t < i; ++t)
      (void)mbar_wait(smem_u32(&full_bar[t % C::kStages]), (t / C::kStages) & 1);
    if (piece > 0) (void)mbar_wait(smem_u32(q_full), (piece - 1) & 1);
    return;
  }

  // =========================== consumer warps ==============================
  const int d0 = warp * C::kDS;  // this warp's head_dim slice
  const float vmul = FMT == PD_KV_FP8_E4M3 ? a.v_scale : 1.0f;
  // head_dim index of accumulator element (m-tile md, row half hh: 0 -> r, 1 -> r+8)
  auto drow = [&](int md, int hh) -> int {
    if constexpr (FMT == PD_KV_BF16) return d0 + md * 16 + r + 8 * hh;
    return d0 + r * (C::kDS / 8) + hh * C::kKSteps + md;
  };
  const ThreadPlace tp{warp, lane, r, c, d0};
  // the warps meet at named barriers every tile, so they agree on every wait
  auto agree = [&](bool ok) {
    ok = consumers_vote(ok);
    if (!ok) {
      if (lane == 0) atomicOr(a.flags, PD_DEV_TIMEOUT);
      *abort_s = 1;
    }
    return ok;
  };
  int red_buf = 0;
  while (walk.next(q)) {
    const TreeSeq& s = q.p.s;
    const int node0 = q.rt * TPC;
    const int nodes = min(TPC, s.n - node0);
    const int rows = nodes * G;
    // ---- what the columns see ----
    TreeMask<NT> mask;
    mask.all = any_view(a, s, lane);
    int open_lo = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int h = nt * 8 + 2 * c + j;
        mask.col[nt][j] = row_view(a, s, node0 + (h < rows ? h / G : 0));
        open_lo = max(open_lo, mask.col[nt][j].lo);
      }
    mask.open_lo = __reduce_max_sync(0xFFFFFFFFu, open_lo);
    // ---- q fragments ----
    // (the first keys are waited for here, too: these two waits take the test's limit,
    // which in the loop over the tiles cost 2% in 32 rows)
    if (!agree(warp_wait(smem_u32(q_full), piece & 1, abort_s, a.consumer_wait_ns) &&
               warp_wait(smem_u32(&full_bar[i % C::kStages]), (i / C::kStages) & 1, abort_s,
                         a.consumer_wait_ns)))
      return;
    TileState<C, NT> ts;
    load_q_fragments<FMT, D, NT>(ts, reinterpret_cast<const uint16_t*>(q_s), rows, a.scale_log2,
                                 a.k_scale, tp, qmax_s);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(q_empty));
    reset_state(ts);
    for (int j = q.j0; j < q.j1; ++j, ++i) {
      const int st = i % C::kStages;
      if (!agree(warp_wait(smem_u32(&full_bar[st]), (i / C::kStages) & 1, abort_s))) return;
      const uint32_t kst = smem_u32(smem + st * C::kStageBytes);
      const int t0 = tile_key(q.p, j, C::kKT);
      consume_tile<FMT, D, NT>(
          ts, StageView{kst, kst + C::kCacheStageBytes, t0, 0, s.L, bad_s[i % kSplitBadRing]}, tp,
          red, red_buf, mask);
      red_buf ^= 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty_bar[st]));
    }
    // ---- end of the piece: full row sums; every warp holds the same (m, l)
    // and its own head_dim slice of O ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float l = ts.l_run[nt][j];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        const int h = nt * 8 + 2 * c + j;
        if (h >= rows) continue;
        if (q.whole) {
          const float inv = vmul / fmaxf(l, 1e-20f);
          uint16_t* o = a.out + static_cast<int64_t>(s.q0 + node0 + h / G) * a.out_stride +
                        static_cast<int64_t>(q.g * G + h % G) * D;
#pragma unroll
          for (int md = 0; md < C::kKSteps; ++md) {
            o[drow(md, 0)] = f32_to_bf16(ts.acc[md][nt][j] * inv);
            o[drow(md, 1)] = f32_to_bf16(ts.acc[md][nt][2 + j] * inv);
          }
        } else {
          float* o = w.o + (static_cast<int64_t>(q.slot) * (D / 4) * w.rows + h) * 4;
#pragma unroll
          for (int md = 0; md < C::kKSteps; ++md)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int d = drow(md, hh);
              o[static_cast<int64_t>(d / 4) * w.rows * 4 + d % 4] = ts.acc[md][nt][2 * hh + j] * vmul;
            }
          if (warp == 0 && r == 0)
            w.ml[static_cast<int64_t>(q.slot) * w.rows + h] = make_float2(ts.m_run[nt][j], l);
        }
      }
    ++piece;
  }
}

template <int FMT, int D, int NT, int BS>
cudaError_t launch_split_cfg(const TreeArgs& a, const TreeWork& w, cudaStream_t st) {
  using C = SplitCfg<FMT, D, NT>;
  CUtensorMap tk, tv;
  std::memset(&tk, 0, sizeof(tk));
  std::memset(&tv, 0, sizeof(tv));
  if constexpr (FMT != PD_KV_NVFP4) {
    const int64_t rows = a.num_blocks * BS;
    if (!encode_cache_map(&tk, a.k_cache, FMT, D, a.num_kv_heads, rows, C::kCopyElems, C::kBR,
                          C::kSwizzle) ||
        !encode_cache_map(&tv, a.v_cache, FMT, D, a.num_kv_heads, rows, C::kCopyElems, C::kBR,
                          C::kSwizzle))
      return cudaErrorInvalidValue;
  }
  auto kern = tree_split_kernel<FMT, D, NT, BS>;
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
  e = launch_dependent(dim3(w.ctas), kMmaThreads, C::kSmemBytes, st, kern, tk, tv, a, w);
  if (e != cudaSuccess) return e;
  return launch_tree_join(a, w, D, st);
}

// head_dim 256 comes here in up to 8 rows only.
template <int FMT>
cudaError_t launch_split_nt(const TreeArgs& a, const TreeWork& w, int head_dim, cudaStream_t st) {
  const bool one = w.item_nodes * a.group <= 8;
  if (head_dim == 256)
    return a.block_size == 16 ? launch_split_cfg<FMT, 256, 1, 16>(a, w, st)
                              : launch_split_cfg<FMT, 256, 1, 32>(a, w, st);
  if (a.block_size == 16)
    return one ? launch_split_cfg<FMT, 512, 1, 16>(a, w, st)
               : launch_split_cfg<FMT, 512, 2, 16>(a, w, st);
  return one ? launch_split_cfg<FMT, 512, 1, 32>(a, w, st)
             : launch_split_cfg<FMT, 512, 2, 32>(a, w, st);
}

template <int FMT>
int split_per_sm(bool one, int head_dim) {
  if (head_dim == 256) return SplitCfg<FMT, 256, 1>::kPerSm;
  return one ? SplitCfg<FMT, 512, 1>::kPerSm : SplitCfg<FMT, 512, 2>::kPerSm;
}

}  // namespace

size_t tree_split_workspace(int max_q_len, int group, int head_dim, int kv_dtype, int num_sms,
                            TreeWork* w, void* workspace) {
  // 8 rows where they hold every node of the batch, else 16
  const bool one = (max_q_len < 1 ? 1 : max_q_len) * group <= 8;
  const int item_nodes = (one ? 8 : 16) / group;
  const int rows = one ? 8 : 16;
  const int per_sm = kv_dtype == PD_KV_BF16       ? split_per_sm<PD_KV_BF16>(one, head_dim)
                     : kv_dtype == PD_KV_FP8_E4M3 ? split_per_sm<PD_KV_FP8_E4M3>(one, head_dim)
                                                  : split_per_sm<PD_KV_NVFP4>(one, head_dim);
  const int ctas = num_sms * per_sm;
  const WorkLayout l = work_layout(ctas, rows, head_dim);
  if (w) {
    uint8_t* p = static_cast<uint8_t*>(workspace);
    w->records = reinterpret_cast<JoinRecord*>(p);
    w->ml = reinterpret_cast<float2*>(p + l.ml);
    w->o = reinterpret_cast<float*>(p + l.o);
    w->ctas = ctas;
    w->rows = rows;
    w->item_nodes = item_nodes;
    w->min_units = 8;
  }
  return l.bytes;
}

cudaError_t launch_tree_split(const TreeArgs& a, const TreeWork& w, int head_dim, int kv_dtype,
                              cudaStream_t st) {
  switch (kv_dtype) {
    case PD_KV_BF16: return launch_split_nt<PD_KV_BF16>(a, w, head_dim, st);
    case PD_KV_FP8_E4M3: return launch_split_nt<PD_KV_FP8_E4M3>(a, w, head_dim, st);
    default: return launch_split_nt<PD_KV_NVFP4>(a, w, head_dim, st);
  }
}

}  // namespace pd
