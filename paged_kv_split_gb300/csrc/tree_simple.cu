// Draft-tree attention on CUDA cores: one CTA per (node, q head), the keys dealt
// to its four warps, one online softmax a warp, merged at the end. It reads
// nothing that its node does not see. The cross-check of the tensor-core
// kernels (pd_decode_tree_crosscheck).
#include "pd_common.cuh"

namespace pd {
namespace {

constexpr int kSimpleWarps = 4;

// Element d of a key or value row (page, row, head).
template <int FMT, int D>
__device__ __forceinline__ float cache_elem(const uint8_t* cache, int64_t page, int row, int h,
                                            int hkv, int bs, int64_t page_bytes,
                                            int64_t data_bytes, int d) {
  const uint8_t* pg = cache + page * page_bytes;
  if constexpr (FMT == PD_KV_BF16) {
    return bf16_to_f32(
        reinterpret_cast<const uint16_t*>(pg)[(static_cast<int64_t>(row) * hkv + h) * D + d]);
  } else if constexpr (FMT == PD_KV_FP8_E4M3) {
    return e4m3_decode(pg[(static_cast<int64_t>(row) * hkv + h) * D + d]);
  } else {
    const int64_t line = static_cast<int64_t>(h) * bs + row;
    const uint32_t w = pg[line * (D / 2) + d / 2];
    return e2m1_decode((d & 1) ? w >> 4 : w & 15u) *
           e4m3_decode(pg[data_bytes + line * (D / 16) + d / 16]);
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kSimpleWarps * 32) tree_simple_kernel(const TreeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kE = D / 32;  // elements of a lane: lane + 32 k
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = a.block_size;
  const TreeSeq s = tree_seq(a.cu_q, a.seq_lens, b, a.total_q, a.max_q_len, a.max_blocks_per_seq,
                             bs, threadIdx.x == 0 ? a.flags : nullptr);
  if (i >= s.n) return;
  const NodeView v = node_view(a.tree_mask, s, i, a.sliding_window, a.num_sinks);
  const int prefix = s.L - s.n;
  const int g = h / a.group;
  const int32_t* bt = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
  const uint16_t* q = a.q + static_cast<int64_t>(s.q0 + i) * a.q_stride + static_cast<int64_t>(h) * D;
  const float kmul = a.scale_log2 * (FMT == PD_KV_FP8_E4M3 ? a.k_scale : 1.0f);
  float qe[kE], o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    qe[e] = bf16_to_f32(q[lane + 32 * e]);
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int r = warp; r < s.L; r += kSimpleWarps) {
    const bool seen = r < prefix ? (r >= v.lo || r < a.num_sinks) : ((v.bits >> (r - prefix)) & 1u);
    if (!seen) continue;
    const int page = bt[r / bs];
    if (page < 0 || page >= a.num_blocks) {
      if (lane == 0) atomicOr(a.flags, PD_DEV_BAD_PAGE);
      continue;
    }
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      dot += qe[e] * cache_elem<FMT, D>(a.k_cache, page, r % bs, g, a.num_kv_heads, bs,
                                        a.page_bytes, a.data_bytes, lane + 32 * e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
    const float x = dot * kmul;
    const float mn = fmaxf(m, x);
    const float alpha = m == -INFINITY ? 0.0f : exp2f(m - mn);
    const float p = mn == -INFINITY ? 0.0f : exp2f(x - mn);
    m = mn;
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      o[e] = o[e] * alpha +
             p * cache_elem<FMT, D>(a.v_cache, page, r % bs, g, a.num_kv_heads, bs, a.page_bytes,
                                    a.data_bytes, lane + 32 * e);
  }
  __shared__ float o_s[kSimpleWarps][D], m_s[kSimpleWarps], l_s[kSimpleWarps];
#pragma unroll
  for (int e = 0; e < kE; ++e) o_s[warp][lane + 32 * e] = o[e];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kSimpleWarps; ++w) M = fmaxf(M, m_s[w]);
  uint16_t* out = a.out + static_cast<int64_t>(s.q0 + i) * a.out_stride + static_cast<int64_t>(h) * D;
  float f[kSimpleWarps];
  for (int w = 0; w < kSimpleWarps; ++w) {
    f[w] = m_s[w] == -INFINITY ? 0.0f : exp2f(m_s[w] - M);
    sum += l_s[w] * f[w];
  }
  const float inv = (FMT == PD_KV_FP8_E4M3 ? a.v_scale : 1.0f) / fmaxf(sum, 1e-20f);
  for (int d = threadIdx.x; d < D; d += kSimpleWarps * 32) {
    float acc = 0.0f;
    for (int w = 0; w < kSimpleWarps; ++w) acc += o_s[w][d] * f[w];
    out[d] = f32_to_bf16(acc * inv);
  }
}

template <int FMT, int D>
cudaError_t launch_simple(const TreeArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.max_q_len, a.num_q_heads, a.num_seqs);
  cfg.blockDim = dim3(kSimpleWarps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_simple_kernel<FMT, D>, a);
}

template <int FMT>
cudaError_t launch_simple_fmt(const TreeArgs& a, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_simple<FMT, 64>(a, st);
    case 128: return launch_simple<FMT, 128>(a, st);
    case 256: return launch_simple<FMT, 256>(a, st);
    case 512: return launch_simple<FMT, 512>(a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_tree_simple(const TreeArgs& a, int head_dim, int kv_dtype, cudaStream_t st) {
  if (a.num_seqs == 0 || a.max_q_len == 0) return cudaSuccess;
  switch (kv_dtype) {
    case PD_KV_BF16: return launch_simple_fmt<PD_KV_BF16>(a, head_dim, st);
    case PD_KV_FP8_E4M3: return launch_simple_fmt<PD_KV_FP8_E4M3>(a, head_dim, st);
    default: return launch_simple_fmt<PD_KV_NVFP4>(a, head_dim, st);
  }
}

}  // namespace pd
