// The join of draft-tree attention's partials.
#include "mma_common.cuh"
#include "pd_common.cuh"
#include "tree_plan.cuh"

namespace pd {
namespace {

using namespace ::pd::mma;
using namespace ::pd::tree;

// The items that were cut: out = sum_p O_p 2^(m_p - M) / sum_p l_p 2^(m_p - M),
// the pieces in key order. A warp takes 4 rows x 32 head_dim columns, so that
// partials are read and outputs written in whole 64-byte pieces.
template <int D>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeArgs a, const TreeWork w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinRecord rec = w.records[blockIdx.x];
  if (rec.pieces == 0) return;
  constexpr int kColBlocks = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d4 = (blockIdx.y % kColBlocks) * 8 + (lane & 7);
  const int r = (blockIdx.y / kColBlocks) * 32 + warp * 4 + (lane >> 3);
  const int q0 = a.cu_q[rec.b], n = a.cu_q[rec.b + 1] - q0;
  const int node = rec.rt * w.item_nodes + r / a.group;
  if (r >= w.item_nodes * a.group || node >= n) return;
  auto slot = [&](int p) {
    return 2 * (static_cast<int64_t>(blockIdx.x) + p) + (p == 0 ? 1 : 0);
  };
  float M = -INFINITY;
  for (int p = 0; p < rec.pieces; ++p) M = fmaxf(M, w.ml[slot(p) * w.rows + r].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.0f;
#pragma unroll 4
  for (int p = 0; p < rec.pieces; ++p) {
    const float2 ml = w.ml[slot(p) * w.rows + r];
    const float4 o = *reinterpret_cast<const float4*>(
        w.o + ((slot(p) * (D / 4) + d4) * w.rows + r) * 4);
    const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - M);
    l = fmaf(ml.y, f, l);
    acc.x = fmaf(o.x, f, acc.x);
    acc.y = fmaf(o.y, f, acc.y);
    acc.z = fmaf(o.z, f, acc.z);
    acc.w = fmaf(o.w, f, acc.w);
  }
  const float inv = 1.0f / fmaxf(l, 1e-20f);
  const int qh = rec.g * a.group + r % a.group;
  uint16_t* out = a.out + static_cast<int64_t>(q0 + node) * a.out_stride +
                  static_cast<int64_t>(qh) * D + d4 * 4;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace

cudaError_t launch_tree_join(const TreeArgs& a, const TreeWork& w, int head_dim, cudaStream_t st) {
  const dim3 grid(w.ctas, (w.rows + 31) / 32 * (head_dim / 32));
  switch (head_dim) {
    case 64: return launch_dependent(grid, 256, 0, st, tree_join_kernel<64>, a, w);
    case 128: return launch_dependent(grid, 256, 0, st, tree_join_kernel<128>, a, w);
    case 256: return launch_dependent(grid, 256, 0, st, tree_join_kernel<256>, a, w);
    default: return launch_dependent(grid, 256, 0, st, tree_join_kernel<512>, a, w);
  }
}

}  // namespace pd
