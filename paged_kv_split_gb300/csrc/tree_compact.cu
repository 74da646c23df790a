// Moving the K and V rows of a draft tree's accepted nodes to consecutive
// positions: row prefix + i <- row prefix + accepted[i], in every layer's
// caches, and the new sequence lengths.
//
// accepted is strictly increasing, so accepted[i] >= i and a row is never
// overwritten before it is read when rows move in order. One CTA takes one
// (sequence, layer, K or V): a thread owns fixed bytes of the row and moves
// them for all accepted rows, kBatch loads ahead of kBatch stores, so no
// thread waits for another. Bytes moved are a few rows a sequence: the call is
// bound by latency (block table, then rows, then stores), which the
// (sequence, layer) CTAs overlap, each with its sequence's lookups: 2.9 us for 32
// sequences in 4 layers, 7.2 us for 64 in 32 (FP8; 12.7 MB, a quarter of the copy
// rate; BF16 8.2, NVFP4 9.4).
#include "pd_common.cuh"

namespace pd {
namespace {

constexpr int kCompactThreads = 128;
constexpr int kBatch = 8;

struct Place {
  int page, row;
};

// Moves unit U of every row of the list; at(place) is the unit's byte offset.
template <class U, class At>
__device__ __forceinline__ void move_rows(uint8_t* cache, const Place* src, const Place* dst, int n,
                                          At at) {
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    U v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k < n) v[k] = *reinterpret_cast<const U*>(cache + at(src[i0 + k]));
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k < n) *reinterpret_cast<U*>(cache + at(dst[i0 + k])) = v[k];
  }
}

template <bool NVFP4>
__global__ void __launch_bounds__(kCompactThreads) compact_tree_kernel(const CompactArgs a) {
  // a programmatic dependent of the previous work on the stream: nothing
  // global is touched before that grid has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x;
  const int layer = blockIdx.y;
  const bool first = layer == 0 && blockIdx.z == 0;  // the CTA that reports for the sequence
  const int tid = threadIdx.x;
  const int bs = a.block_size;
  __shared__ Place src_s[kMaxTreeNodes], dst_s[kMaxTreeNodes];  // the rows that move
  __shared__ int moves_s;

  const TreeSeq s = tree_seq(a.cu_q, a.seq_lens, b, 0x7FFFFFFF, 0x7FFFFFFF, a.max_blocks_per_seq,
                             bs, first && tid == 0 ? a.flags : nullptr);
  const int num = a.num_accepted[b];
  const int32_t* acc = a.accepted + static_cast<int64_t>(b) * a.max_accepted;
  bool ok = num >= 0 && num <= a.max_accepted && num <= s.n;
  if (ok && tid < num) {
    const int x = acc[tid];
    ok = x >= 0 && x < s.n && (tid == 0 || x > acc[tid - 1]);
  }
  ok = __syncthreads_and(ok);
  const int prefix = s.L - s.n;
  if (first && tid == 0) {
    if (!ok) atomicOr(a.flags, PD_DEV_BAD_TREE);
    a.new_seq_lens[b] = min(max(prefix, 0), a.max_blocks_per_seq * bs) + (ok ? num : 0);
  }
  if (!ok) return;
  if (tid < 32) {
    const int32_t* bt = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
    int moves = 0;
    for (int i0 = 0; i0 < num; i0 += 32) {
      const int i = i0 + tid;
      bool move = i < num && acc[i] != i;
      Place sp{0, 0}, dp{0, 0};
      if (move) {
        const int from = prefix + acc[i], to = prefix + i;
        sp = Place{bt[from / bs], from % bs};
        dp = Place{bt[to / bs], to % bs};
        move = sp.page >= 0 && sp.page < a.num_blocks && dp.page >= 0 && dp.page < a.num_blocks;
        if (!move && first) atomicOr(a.flags, PD_DEV_BAD_PAGE);
      }
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, move);
      if (move) {
        const int k = moves + __popc(m & ((1u << tid) - 1u));
        src_s[k] = sp;
        dst_s[k] = dp;
      }
      moves += __popc(m);
    }
    if (tid == 0) moves_s = moves;
  }
  __syncthreads();
  const int n = moves_s;
  if (n == 0) return;
  uint8_t* cache = (blockIdx.z ? a.v_caches : a.k_caches) + layer * a.layer_bytes;
  const int64_t pb = a.page_bytes;
  if constexpr (!NVFP4) {
    // a row's bytes are contiguous in its page
    const int row_bytes = static_cast<int>(pb / bs);
    for (int u = tid * 16; u < row_bytes; u += kCompactThreads * 16)
      move_rows<uint4>(cache, src_s, dst_s, n, [&](const Place& p) {
        return p.page * pb + static_cast<int64_t>(p.row) * row_bytes + u;
      });
  } else {
    // per head a row of D / 2 code bytes, and D / 16 scale bytes behind them all
    const int db = a.head_dim / 2, sb = a.head_dim / 16;
    for (int u = tid * 16; u < a.num_kv_heads * db; u += kCompactThreads * 16)
      move_rows<uint4>(cache, src_s, dst_s, n, [&](const Place& p) {
        return p.page * pb + (static_cast<int64_t>(u / db) * bs + p.row) * db + u % db;
      });
    for (int u = tid * 4; u < a.num_kv_heads * sb; u += kCompactThreads * 4)
      move_rows<uint32_t>(cache, src_s, dst_s, n, [&](const Place& p) {
        return p.page * pb + a.data_bytes + (static_cast<int64_t>(u / sb) * bs + p.row) * sb +
               u % sb;
      });
  }
}

}  // namespace

cudaError_t launch_compact_tree(const CompactArgs& a, cudaStream_t st) {
  if (a.num_seqs == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_seqs, a.num_layers, 2);
  cfg.blockDim = dim3(kCompactThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.kv_dtype == PD_KV_NVFP4 ? cudaLaunchKernelEx(&cfg, compact_tree_kernel<true>, a)
                                   : cudaLaunchKernelEx(&cfg, compact_tree_kernel<false>, a);
}

}  // namespace pd
