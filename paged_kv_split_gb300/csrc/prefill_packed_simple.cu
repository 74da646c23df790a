// Attention of packed prompts over their own rows on CUDA cores: the plain
// form behind pd_prefill_packed_crosscheck. One warp per (token, q head), lanes
// over head_dim, an online softmax key by key in fp32.
#include "serve_common.cuh"

namespace pd {
namespace {

constexpr int kWarpsPerCta = 8;

template <int D>
__global__ void __launch_bounds__(kWarpsPerCta * 32)
    prefill_packed_simple_kernel(const PackedArgs a) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  const int g = h / a.group;
  const int b = blockIdx.z;
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
  const int n = q1 - q0;
  if (q0 < 0 || n < 0 || q1 > a.total_q || n > a.max_q_len) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) atomicOr(a.flags, PD_DEV_BAD_SEQ_LEN);
    return;
  }
  const int i = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  if (i >= n) return;
  const int pos = a.causal ? i : n - 1;
  const int lo = (a.sliding_window > 0 && pos >= a.sliding_window) ? pos + 1 - a.sliding_window : 0;
  const uint16_t* q = a.q + static_cast<int64_t>(q0 + i) * a.q_stride + static_cast<int64_t>(h) * D;
  float qr[kPer], acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    qr[k] = bf16_to_f32(q[lane + 32 * k]);
    acc[k] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = lo; j <= pos; ++j) {
    const int64_t r = q0 + j;
    const uint16_t* kp = a.k + r * a.k_stride + static_cast<int64_t>(g) * D;
    const uint16_t* vp = a.v + r * a.v_stride + static_cast<int64_t>(g) * D;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) s = fmaf(qr[k], bf16_to_f32(kp[lane + 32 * k]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float al = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = fmaf(p, bf16_to_f32(vp[lane + 32 * k]), acc[k] * al);
  }
  uint16_t* o = a.out + static_cast<int64_t>(q0 + i) * a.out_stride + static_cast<int64_t>(h) * D;
  const float inv = 1.0f / fmaxf(l, 1e-20f);
#pragma unroll
  for (int k = 0; k < kPer; ++k) o[lane + 32 * k] = f32_to_bf16(acc[k] * inv);
}

}  // namespace

cudaError_t launch_prefill_packed_simple(const PackedArgs& a, int head_dim, cudaStream_t st) {
  const dim3 grid((a.max_q_len + kWarpsPerCta - 1) / kWarpsPerCta, a.num_q_heads, a.num_seqs);
  switch (head_dim) {
    case 64: prefill_packed_simple_kernel<64><<<grid, kWarpsPerCta * 32, 0, st>>>(a); break;
    case 128: prefill_packed_simple_kernel<128><<<grid, kWarpsPerCta * 32, 0, st>>>(a); break;
    case 256: prefill_packed_simple_kernel<256><<<grid, kWarpsPerCta * 32, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace pd
