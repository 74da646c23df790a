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
// partials are read and outputs written in whole 64-byte pieces. What it costs
// is latency (record, then partials), so kBatch pieces are read at once.
// D columns of a head's HD.
template <int D, int HD>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeArgs a, const TreeWork w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinRecord rec = w.records[blockIdx.x];
  constexpr int kBatch = 8;
  constexpr int kColBlocks = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d4 = (blockIdx.y % kColBlocks) * 8 + (lane & 7);
  const int r = (blockIdx.y / kColBlocks) * 32 + warp * 4 + (lane >> 3);
  const int nodes = rec.nodes & 0xFFFF, col0 = (rec.nodes >> 16) * D;
  if (rec.pieces == 0 || r >= nodes * a.group) return;
  // the first piece is its CTA's second slot, the others their CTAs' first
  const int64_t slot0 = 2 * static_cast<int64_t>(blockIdx.x);
  const float2* ml = w.ml + slot0 * w.rows + r;
  const float* o = w.o + (slot0 * (D / 4) + d4) * w.rows * 4 + r * 4;
  const int64_t ml_step = 2 * w.rows, o_step = 2ll * (D / 4) * w.rows * 4;
  float M = -INFINITY, l = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < rec.pieces; p0 += kBatch) {
    float2 x[kBatch];
    float4 y[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int p = p0 + k;
      x[k] = make_float2(-INFINITY, 0.0f);
      y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < rec.pieces) {
        x[k] = ml[p == 0 ? w.rows : p * ml_step];
        y[k] = *reinterpret_cast<const float4*>(o + (p == 0 ? o_step / 2 : p * o_step));
      }
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, x[k].x);
    if (top == -INFINITY) continue;  // nothing seen yet
    const float f0 = M == -INFINITY ? 0.0f : ex2(M - top);
    M = top;
    l *= f0;
    acc.x *= f0;
    acc.y *= f0;
    acc.z *= f0;
    acc.w *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float f = x[k].x == -INFINITY ? 0.0f : ex2(x[k].x - top);
      l = fmaf(x[k].y, f, l);
      acc.x = fmaf(y[k].x, f, acc.x);
      acc.y = fmaf(y[k].y, f, acc.y);
      acc.z = fmaf(y[k].z, f, acc.z);
      acc.w = fmaf(y[k].w, f, acc.w);
    }
  }
  const float inv = 1.0f / fmaxf(l, 1e-20f);
  const int node = r / a.group;
  uint16_t* out = a.out + static_cast<int64_t>(rec.row0 + node) * a.out_stride +
                  static_cast<int64_t>(rec.head0 + r - node * a.group) * HD + col0 + d4 * 4;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace

cudaError_t launch_tree_join(const TreeArgs& a, const TreeWork& w, int head_dim, cudaStream_t st) {
  const int cols = head_dim >> a.half_bits;
  const dim3 grid(w.ctas, (w.rows + 31) / 32 * (cols / 32));
  switch (head_dim) {
    case 64: return launch_dependent(grid, 256, 0, st, tree_join_kernel<64, 64>, a, w);
    case 128: return launch_dependent(grid, 256, 0, st, tree_join_kernel<128, 128>, a, w);
    case 256: return launch_dependent(grid, 256, 0, st, tree_join_kernel<256, 256>, a, w);
    default:
      return a.half_bits ? launch_dependent(grid, 256, 0, st, tree_join_kernel<256, 512>, a, w)
                         : launch_dependent(grid, 256, 0, st, tree_join_kernel<512, 512>, a, w);
  }
}

}  // namespace pd
