// How draft-tree attention is dealt to CTAs, worked out on the device.
//
// An item is (sequence, kv head, tile of the sequence's nodes); its keys are a
// line of key tiles: the tiles that hold the first tokens that stay visible,
// then those from the window's first page on (or all of them). All items, laid
// end to end (sequence, then kv head, then node tile: the node tiles of a head
// run side by side and share its keys in L2), make one line of units, a unit a
// key tile, with `ov` units of slack after each item for what a piece costs
// beside its tiles. CTA c takes units [c S, (c + 1) S). So every CTA streams the
// same number of tiles whatever the lengths, an item cut by a share's end
// becomes pieces whose partials a second kernel joins, and at most one item
// begins in a CTA and goes on in the next: the partials need two slots a CTA.
// Every CTA sums the line from cu_q and seq_lens itself, so the host needs no
// lengths and a captured graph follows them.
#pragma once

#include "pd_common.cuh"

namespace pd {
namespace tree {

// One sequence's tiles.
struct SeqPlan {
  TreeSeq s;
  int nst;   // leading tiles, from key 0, for the first tokens
  int base;  // first key of the other tiles (page aligned)
  int nt;    // tiles
  int rts;   // node tiles (times two where V's columns come in halves)
};
__device__ __forceinline__ SeqPlan seq_plan(const TreeArgs& a, int b, int tpc, int kt, int* flags) {
  SeqPlan p;
  p.s = tree_seq(a.cu_q, a.seq_lens, b, a.total_q, a.max_q_len, a.max_blocks_per_seq, a.block_size,
                 flags);
  p.nst = p.base = p.nt = p.rts = 0;
  if (p.s.n == 0) return p;
  const int prefix = p.s.L - p.s.n;
  if (a.sliding_window > 0) {
    const int lo = max(0, prefix + 1 - a.sliding_window);  // a node of depth 0 sees the most
    p.base = lo / a.block_size * a.block_size;
    p.nst = (min(a.num_sinks, p.s.L) + kt - 1) / kt;
    if (p.base <= p.nst * kt) p.nst = p.base = 0;  // the two ranges meet
  }
  p.nt = p.nst + (p.s.L - p.base + kt - 1) / kt;
  p.rts = (p.s.n + tpc - 1) / tpc << a.half_bits;
  return p;
}
// First key of tile j.
__device__ __forceinline__ int tile_key(const SeqPlan& p, int j, int kt) {
  return j < p.nst ? j * kt : p.base + (j - p.nst) * kt;
}
// Keys of tile j end here (the first tokens' last tile stops at num_sinks).
__device__ __forceinline__ int tile_end(const SeqPlan& p, int j, int kt, int sinks) {
  return j < p.nst ? min((j + 1) * kt, sinks) : min(p.base + (j - p.nst + 1) * kt, p.s.L);
}

// Non-negative 64-bit quotients that are nearly always 32-bit ones.
__device__ __noinline__ inline long long quotient64(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long quotient_of(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return quotient64(a, b);
}

// A CTA's share of the line.
struct Share {
  long long units;  // S
  long long x0;     // first unit
  int b, k, off;    // its sequence, item there and unit in the item; b < 0: nothing
  SeqPlan p;        // of that sequence
};
struct ShareScratch {
  long long warp_sum[32];
  long long units;
  int b, k, off;
};
// The start of the share [x0, ..) among the sequences [b0, b1), whose units begin at `at`.
__device__ __forceinline__ void find_start(const TreeArgs& a, int tpc, int kt, int ov, int b0, int b1,
                                           long long at, Share* r) {
  for (int b = b0; b < b1; ++b) {
    const SeqPlan p = seq_plan(a, b, tpc, kt, nullptr);
    const long long cost = static_cast<long long>(p.rts) * a.num_kv_heads * (p.nt + ov);
    if (r->x0 < at + cost) {
      const int item = p.nt + ov;
      r->b = b;
      r->k = static_cast<int>(quotient_of(r->x0 - at, item));
      r->off = static_cast<int>(r->x0 - at - static_cast<long long>(r->k) * item);
      r->p = p;
      return;
    }
    at += cost;
  }
}
// Up to kWarpPlan sequences every warp works the share out for itself, without
// barriers (one short sequence 14.1 -> 13.8 us, 64 sequences in FP8 181 -> 179);
// beyond that a lane would have more than four in turn.
constexpr int kWarpPlan = 128;
__device__ __forceinline__ Share warp_share(const TreeArgs& a, int tpc, int kt, int ov,
                                            int per_cta_min) {
  const int lane = threadIdx.x & 31;
  const int per = (a.num_seqs + 31) / 32;
  const int b0 = min(lane * per, a.num_seqs), b1 = min(b0 + per, a.num_seqs);
  int* flags = blockIdx.x == 0 && threadIdx.x < 32 ? a.flags : nullptr;
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqPlan p = seq_plan(a, b, tpc, kt, flags);
    sum += static_cast<long long>(p.rts) * a.num_kv_heads * (p.nt + ov);
  }
  long long incl = sum;
  for (int o = 1; o < 32 && o * per < a.num_seqs; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  const long long total = __shfl_sync(0xFFFFFFFFu, incl, max(a.num_seqs - 1, 0) / max(per, 1));
  Share r;
  r.units = quotient_of(total + gridDim.x - 1, gridDim.x);
  if (r.units < per_cta_min) r.units = per_cta_min;
  r.x0 = r.units * blockIdx.x;
  r.b = -1;
  r.k = r.off = 0;
  r.p.s.q0 = r.p.s.n = r.p.s.L = r.p.nst = r.p.base = r.p.nt = r.p.rts = 0;
  const bool mine = r.x0 >= incl - sum && r.x0 < incl;
  if (mine) find_start(a, tpc, kt, ov, b0, b1, incl - sum, &r);
  const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine);
  if (who == 0u) return r;
  const int src = __ffs(who) - 1;
  int* const field[] = {&r.b, &r.k, &r.off, &r.p.s.q0, &r.p.s.n, &r.p.s.L, &r.p.nst, &r.p.base,
                        &r.p.nt, &r.p.rts};
#pragma unroll
  for (int i = 0; i < 10; ++i) *field[i] = __shfl_sync(0xFFFFFFFFu, *field[i], src);
  return r;
}
// Called by all threads of the CTA. `per_cta_min`: a share is at least that long.
__device__ __forceinline__ Share make_share(const TreeArgs& a, int tpc, int kt, int ov,
                                            int per_cta_min, ShareScratch* sh) {
  if (a.num_seqs <= kWarpPlan) return warp_share(a, tpc, kt, ov, per_cta_min);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthreads = blockDim.x;
  const int per = (a.num_seqs + nthreads - 1) / nthreads;
  const int b0 = min(tid * per, a.num_seqs), b1 = min(b0 + per, a.num_seqs);
  int* flags = blockIdx.x == 0 ? a.flags : nullptr;
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqPlan p = seq_plan(a, b, tpc, kt, flags);
    sum += static_cast<long long>(p.rts) * a.num_kv_heads * (p.nt + ov);
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  if (tid == 0) sh->b = -1;
  __syncthreads();
  long long before = 0, total = 0;
  const int warps = nthreads >> 5;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) before = total;
    total += sh->warp_sum[w];
  }
  Share r;
  r.units = quotient_of(total + gridDim.x - 1, gridDim.x);
  if (r.units < per_cta_min) r.units = per_cta_min;
  r.x0 = r.units * blockIdx.x;
  long long at = before + incl - sum;  // first unit of this thread's sequences
  if (r.x0 >= at && r.x0 < at + sum) {
    find_start(a, tpc, kt, ov, b0, b1, at, &r);
    sh->b = r.b;
    sh->k = r.k;
    sh->off = r.off;
  }
  __syncthreads();
  r.b = sh->b;
  r.k = sh->k;
  r.off = sh->off;
  if (r.b >= 0) r.p = seq_plan(a, r.b, tpc, kt, nullptr);
  return r;
}

// A CTA's part of one item.
struct Piece {
  SeqPlan p;
  int b, g, rt, half;
  int j0, j1;     // its tiles
  bool begins;    // holds the item's first tile
  bool whole;     // and its last: writes the output itself
  int slot;       // else its partial's slot
};
// Goes through a share's pieces; every warp role that needs them runs its own.
struct Walker {
  const TreeArgs& a;
  int tpc, kt, ov;
  long long units, x, end;
  int b, k, off;
  SeqPlan p;

  __device__ __forceinline__ Walker(const TreeArgs& args, const Share& s, int tpc_, int kt_, int ov_)
      : a(args), tpc(tpc_), kt(kt_), ov(ov_), units(s.units), x(s.x0), end(s.x0 + s.units), b(s.b),
        k(s.k), off(s.off), p(s.p) {}
  __device__ __forceinline__ bool next(Piece& q) {
    while (x < end && b < a.num_seqs) {
      const int items = p.rts * a.num_kv_heads;
      if (k >= items) {
        k = 0;
        if (++b < a.num_seqs) p = seq_plan(a, b, tpc, kt, nullptr);
        continue;
      }
      const int take = static_cast<int>(min(static_cast<long long>(p.nt + ov - off), end - x));
      const int j0 = off, j1 = min(off + take, p.nt);
      x += take;
      q.g = k / p.rts;
      q.rt = k % p.rts;
      q.half = q.rt & ((1 << a.half_bits) - 1);
      q.rt >>= a.half_bits;
      if (off + take == p.nt + ov) {
        ++k;
        off = 0;
      } else {
        off += take;
      }
      if (j0 >= j1) continue;  // slack only
      q.p = p;
      q.b = b;
      q.j0 = j0;
      q.j1 = j1;
      q.begins = j0 == 0;
      q.whole = j0 == 0 && j1 == p.nt;
      q.slot = 2 * static_cast<int>(blockIdx.x) + (q.begins ? 1 : 0);
      return true;
    }
    return false;
  }
  // pieces of the item whose first j1 tiles end this share
  __device__ __forceinline__ int pieces_of_last(int j1) const {
    const long long s = end - j1;  // the item's first unit
    return static_cast<int>(quotient_of(s + p.nt - 1, units) - static_cast<int>(blockIdx.x)) + 1;
  }
};

// What a CTA leaves for the join: the item that begins in it and goes on (its
// first query row, nodes (bit 16: the second half of head_dim), first q head), or
// pieces = 0.
struct JoinRecord {
  int pieces, row0, nodes, head0;
};

// Workspace: records [ctas], then (m, l) [2 ctas][rows], then O
// [2 ctas][D / 4][rows][4] fp32, rows the padded rows of an item. m in log2
// units, l and O not divided.
struct WorkLayout {
  size_t ml, o, bytes;
};
__host__ __device__ inline WorkLayout work_layout(int ctas, int rows, int d) {
  WorkLayout w;
  w.ml = (static_cast<size_t>(ctas) * sizeof(JoinRecord) + 255) / 256 * 256;
  w.o = w.ml + (static_cast<size_t>(2) * ctas * rows * sizeof(float2) + 255) / 256 * 256;
  w.bytes = w.o + static_cast<size_t>(2) * ctas * rows * d * sizeof(float);
  return w;
}

// The workspace as the kernels see it.
}  // namespace tree
struct TreeWork {
  tree::JoinRecord* records;  // [ctas]
  float2* ml;
  float* o;
  int ctas, rows, item_nodes, min_units;
};
// Launch as a programmatic dependent of the previous work on the stream.
template <class... A>
inline cudaError_t launch_dependent(dim3 grid, int threads, int smem, cudaStream_t st, void (*kern)(A...),
                             const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_tree_join(const TreeArgs& a, const TreeWork& w, int head_dim, cudaStream_t st);
// On tcgen05 or, where it says so, on mma.sync. The workspace functions return
// its size and, with w, lay it out.
// head_dim 512 in up to 32 rows (nodes times q heads of a kv head) runs on mma.sync,
// 16 rows a pass over the keys; on tcgen05 128 rows take two passes. 16 / 2 heads, 8
// sequences over 8192 keys, mma.sync against tcgen05 in us, BF16 / FP8 / NVFP4: 32
// rows 112 / 119 / 114 against 109 / 123 / 139, 64 rows 213 / 220 / 200 against 114 /
// 129 / 141. head_dim 256 in up to 8 rows does too: 8 / 4 heads, 16 sequences over
// 4096 keys 53 / 41 / 44 against 58 / 59 / 58; 16 rows 97 / 70 / 69 against 59 / 60 /
// 60. At 128 in 8 rows a batch takes as long on either (93.5 / 91 against 93.5 / 89.5),
// one short sequence would take 12.3 against 14.2; but the FP8 form of mma.sync tiles
// at that width gave wrong outputs, from a cause not found, and there is none.
inline bool tree_on_umma(int max_q_len, int group, int head_dim) {
  return head_dim <= 128 || max_q_len * group > (head_dim == 256 ? 8 : 32);
}
size_t tree_split_workspace(int max_q_len, int group, int head_dim, int kv_dtype, int num_sms,
                            TreeWork* w, void* workspace);
cudaError_t launch_tree_split(const TreeArgs& a, const TreeWork& w, int head_dim, int kv_dtype,
                              cudaStream_t st);
size_t tree_umma_workspace(int max_q_len, int group, int head_dim, int num_sms, TreeWork* w,
                           void* workspace);
cudaError_t launch_tree_umma(const TreeArgs& a, const TreeWork& w, int head_dim, int kv_dtype,
                             cudaStream_t st);
namespace tree {

// Which cached rows and nodes a node (or, merged, any node) sees.
struct RowView {
  int lo, prefix, sinks;  // rows [lo, prefix) and [0, sinks), sinks <= prefix
  uint64_t bits;
};
// Bits [a, b) of a word.
__device__ __forceinline__ uint32_t range32(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  return (b - a == 32 ? 0xFFFFFFFFu : ((1u << (b - a)) - 1u)) << a;
}
// Bit i: row k0 + i is seen.
__device__ __forceinline__ uint32_t seen32(const RowView& v, int k0) {
  uint32_t w = range32(v.lo - k0, v.prefix - k0) | range32(-k0, v.sinks - k0);
  const int s = k0 - v.prefix;
  if (s >= 0) {
    if (s < 64) w |= static_cast<uint32_t>(v.bits >> s);
  } else if (s > -32) {
    w |= static_cast<uint32_t>(v.bits << -s);
  }
  return w;
}
__device__ __forceinline__ RowView row_view(const TreeArgs& a, const TreeSeq& s, int i) {
  const NodeView n = node_view(a.tree_mask, s, i, a.sliding_window, a.num_sinks);
  RowView v;
  v.prefix = s.L - s.n;
  v.lo = min(n.lo, v.prefix);
  v.sinks = a.sliding_window > 0 ? min(a.num_sinks, v.prefix) : 0;
  v.bits = n.bits;
  return v;
}
// What any node of the sequence sees (all lanes of a warp together).
__device__ __forceinline__ RowView any_view(const TreeArgs& a, const TreeSeq& s, int lane) {
  RowView u;
  u.prefix = s.L - s.n;
  u.lo = u.prefix;
  u.sinks = a.sliding_window > 0 ? min(a.num_sinks, u.prefix) : 0;
  u.bits = 0;
  for (int i = lane; i < s.n; i += 32) {
    const RowView v = row_view(a, s, i);
    u.lo = min(u.lo, v.lo);
    u.bits |= v.bits;
  }
  u.lo = __reduce_min_sync(0xFFFFFFFFu, u.lo);
  const uint32_t lo32 = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(u.bits));
  const uint32_t hi32 = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(u.bits >> 32));
  u.bits = (static_cast<uint64_t>(hi32) << 32) | lo32;
  return u;
}

}  // namespace tree
}  // namespace pd
