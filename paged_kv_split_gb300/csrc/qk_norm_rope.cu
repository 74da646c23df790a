// Per-head RMS norm of q and k, the position rotation and the cache write of K
// and V in one pass over fused QKV rows, and the cosine / sine table it reads.
//
// For one head x of D elements, every step an fp32 operation rounded once:
//   ms = (sum of x_i^2) / D, the sum a balanced binary tree over neighbours
//        (x_i^2 is exact in fp32: x is bf16)
//   y_i = (x_i * (1 / sqrt(ms + eps))) * (offset + w_i)
//   a pair (a, b) of the first rot_dim elements becomes
//   (a cos - b sin, b cos + a sin), products rounded before the sum (no fma)
// and one rounding to bf16. The order is part of the definition, so the cache
// codes that K is quantised to afterwards are reproducible bit for bit.
//
// The pass reads each fused row once and writes each q row and cache row once;
// instructions weigh as much as memory in it: so a lane
// holds two 8-element chunks of a head half a head apart, where a full rotation
// finds its partners without shuffles; the weights lie in shared memory; and
// CTAs stay, each with a run of (token, head group) items, the next item's rows
// on their way while one is computed. Measured: 8192 rows of 32 + 2 x 8 heads of
// 128 in 41.7 us, 74% of the copy rate, with 72% of the issue slots and 45% of the
// DRAM rate taken (writes stay in L2): neither is full, one item ahead is 24 KB an SM
// in flight (one chunk a lane, partners by shuffle: 77 us; 4 or 8 resident CTAs: 49 and
// 51). Into FP8 49.4 us, into NVFP4 71.0. 832 rows of 64 + 2 x 8 heads into FP8 10.0
// us, four or five items a CTA one after another; 8 rows 2.3 us, a chain of latencies.
#include "pd_common.cuh"

namespace pd {
namespace {

#ifndef PD_ROPE_CTAS
#define PD_ROPE_CTAS 6  // CTAs an SM holds
#endif
constexpr int kRopeThreads = 128;

template <int D>
struct RopeShape {
  static constexpr int kLanes = D / 16;                 // lanes of one head
  static constexpr int kHeads = kRopeThreads / kLanes;  // heads of an item
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = bf16_lo(u[k]);
    x[2 * k + 1] = bf16_hi(u[k]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    u[k] = static_cast<uint32_t>(f32_to_bf16(x[2 * k])) |
           (static_cast<uint32_t>(f32_to_bf16(x[2 * k + 1])) << 16);
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Two values to E4M3 codes, the first in the low byte: nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2_of(float first, float second) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(second), "f"(first));
  return r;
}

// One lane's 8 consecutive elements (bf16 bits) of a K or V head into the
// cache, in its form. NVFP4: neighbouring lanes hold a 16-element group.
template <int FMT, int D>
__device__ __forceinline__ void store_cache(uint8_t* page, const uint4& bits, int h, int row,
                                            int chunk, int hkv, int bs, int64_t data_bytes,
                                            float scale, bool on) {
  if constexpr (FMT == PD_KV_BF16) {
    if (on)
      *reinterpret_cast<uint4*>(page + ((static_cast<int64_t>(row) * hkv + h) * D + chunk * 8) * 2) =
          bits;
  } else {
    if (!__any_sync(0xFFFFFFFFu, on)) return;
    float x[8];
    unpack8(bits, x);
    if constexpr (FMT == PD_KV_FP8_E4M3) {
      uint32_t o[2] = {0u, 0u};
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const uint32_t pair = e4m3x2_of(__fdiv_rn(x[k], scale), __fdiv_rn(x[k + 1], scale));
        o[k >> 2] |= pair << (8 * (k & 2));
      }
      bool nan = false;
#pragma unroll
      for (int k = 0; k < 8; ++k) nan = nan || x[k] != x[k];
      if (nan) {  // a NaN's code takes the input's sign
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (x[k] != x[k]) {
            const uint32_t code = 0x7Fu | ((__float_as_uint(x[k]) >> 24) & 0x80u);
            o[k >> 2] = (o[k >> 2] & ~(0xFFu << (8 * (k & 3)))) | (code << (8 * (k & 3)));
          }
      }
      if (on)
        *reinterpret_cast<uint2*>(page + (static_cast<int64_t>(row) * hkv + h) * D + chunk * 8) =
            make_uint2(o[0], o[1]);
    } else {
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(x[k]));  // fmaxf drops NaN
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      const uint32_t sc = e4m3_encode(__fdiv_rn(amax, 6.0f));
      const float sdec = e4m3_decode(sc);
      uint32_t o = 0u;
      if (sdec != 0.0f) {
#pragma unroll
        for (int k = 0; k < 8; ++k) o |= e2m1_encode(quotient(x[k], sdec)) << (4 * k);
      }
      if (on) {
        const int64_t line = static_cast<int64_t>(h) * bs + row;
        *reinterpret_cast<uint32_t*>(page + line * (D / 2) + chunk * 4) = o;
        if ((chunk & 1) == 0)
          page[data_bytes + line * (D / 16) + chunk / 2] = static_cast<uint8_t>(sc);
      }
    }
  }
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// How pairs lie: elements (i, i + D / 2) of a full rotation, (i, i + rot / 2) of a
// part, or neighbours.
enum RopePairs { kHalves, kPartHalves, kNeighbours };

template <int FMT, int D, int PAIRS>
__global__ void __launch_bounds__(kRopeThreads, PD_ROPE_CTAS) qk_norm_rope_kernel(const NormRopeArgs a) {
  using S = RopeShape<D>;
  // a programmatic dependent of the previous work on the stream: nothing
  // global is touched before that grid has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int l = tid % S::kLanes;  // this lane's place in its head: chunks l and l + kLanes
  const int head_lane0 = (tid & 31) - l;
  const int rot = a.rot_dim, half = rot / 2;
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int heads = hq + 2 * hkv;
  const int groups = (heads + S::kHeads - 1) / S::kHeads;
  const bool norm = a.q_weight != nullptr;

  // offset + w of q and k
  __shared__ __align__(16) float g_s[2][D];
  if (norm) {
    for (int i = tid; i < D; i += kRopeThreads) {
      g_s[0][i] = __fadd_rn(bf16_to_f32(a.q_weight[i]), a.weight_offset);
      g_s[1][i] = __fadd_rn(bf16_to_f32(a.k_weight[i]), a.weight_offset);
    }
  }
  // this CTA's items
  const int64_t items = static_cast<int64_t>(a.num_tokens) * groups;
  const int64_t it0 = items * blockIdx.x / gridDim.x, it1 = items * (blockIdx.x + 1) / gridDim.x;
  if (it0 >= it1) return;
  int t = static_cast<int>(it0 / groups), hg = static_cast<int>(it0 % groups);
  uint4 raw[2];
  auto load_rows = [&](int tt, int gg) {
    int h = gg * S::kHeads + tid / S::kLanes;
    if (h >= heads) h = heads - 1;
    const uint16_t* src =
        a.qkv + static_cast<int64_t>(tt) * a.qkv_stride + static_cast<int64_t>(h) * D + l * 8;
    raw[0] = *reinterpret_cast<const uint4*>(src);
    raw[1] = *reinterpret_cast<const uint4*>(src + D / 2);
  };
  load_rows(t, hg);
  __syncthreads();

  // cosine and signed sine of this lane's elements: out = own * c + partner * s
  float c[2][8], s[2][8];
  uint8_t* kpage = nullptr;
  uint8_t* vpage = nullptr;
  int row = 0;
  bool in_pool = false;
  int pos_raw = a.positions[t], slot_raw = a.slots[t];
  bool fresh = true;
  for (int64_t it = it0; it < it1; ++it) {
    if (fresh) {  // a new token: its table row and place in the cache
      fresh = false;
      int pos = pos_raw;
      if (pos < 0 || pos >= a.max_position) {
        if (tid == 0) atomicOr(a.flags, PD_DEV_BAD_POSITION);
        pos = pos < 0 ? 0 : a.max_position - 1;
      }
      const int64_t slot = slot_raw;
      in_pool = slot >= 0 && slot < a.num_blocks * a.block_size;
      if (slot >= 0 && !in_pool && tid == 0) atomicOr(a.flags, PD_DEV_BAD_SLOT);
      const int64_t page = in_pool ? slot / a.block_size : 0;
      row = in_pool ? static_cast<int>(slot % a.block_size) : 0;
      kpage = a.k_cache + page * a.page_bytes;
      vpage = a.v_cache + page * a.page_bytes;
      const float* cs = a.cos_sin + static_cast<int64_t>(pos) * rot;
      if constexpr (PAIRS == kHalves) {
        load8(cs + l * 8, c[0]);
        load8(cs + half + l * 8, s[1]);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e0 = (l + k * S::kLanes) * 8;
          if (e0 >= rot) continue;
          if constexpr (PAIRS == kNeighbours) {
            const float4 cc = *reinterpret_cast<const float4*>(cs + e0 / 2);
            const float4 ss = *reinterpret_cast<const float4*>(cs + half + e0 / 2);
            c[k][0] = cc.x; c[k][1] = cc.y; c[k][2] = cc.z; c[k][3] = cc.w;
            s[k][0] = ss.x; s[k][1] = ss.y; s[k][2] = ss.z; s[k][3] = ss.w;
          } else {
            const bool low = e0 < half;
            const int i0 = low ? e0 : e0 - half;
            load8(cs + i0, c[k]);
            load8(cs + half + i0, s[k]);
#pragma unroll
            for (int p = 0; p < 8; ++p) s[k][p] = low ? -s[k][p] : s[k][p];
          }
        }
      }
    }
    const uint4 own[2] = {raw[0], raw[1]};
    const int h = hg * S::kHeads + tid / S::kLanes;
    const int tt = t;
    if (it + 1 < it1) {  // the next item's rows, and its token's place
      if (++hg == groups) {
        hg = 0;
        ++t;
        fresh = true;
        pos_raw = a.positions[t];
        slot_raw = a.slots[t];
      }
      load_rows(t, hg);
    }
    const bool on = h < heads;
    const bool is_v = h >= hq + hkv;
    const bool is_k = !is_v && h >= hq;
    float y[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) unpack8(own[k], y[k]);
    if (norm) {
      float ss[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float q[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) q[p] = __fmul_rn(y[k][p], y[k][p]);
        ss[k] = __fadd_rn(__fadd_rn(__fadd_rn(q[0], q[1]), __fadd_rn(q[2], q[3])),
                          __fadd_rn(__fadd_rn(q[4], q[5]), __fadd_rn(q[6], q[7])));
#pragma unroll
        for (int o = 1; o < S::kLanes; o <<= 1)
          ss[k] = __fadd_rn(ss[k], __shfl_xor_sync(0xFFFFFFFFu, ss[k], o));
      }
      const float sum = __fadd_rn(ss[0], ss[1]);
      const float inv =
          __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / static_cast<float>(D)), a.eps)));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float g[8];
        load8(&g_s[is_k ? 1 : 0][(l + k * S::kLanes) * 8], g);
#pragma unroll
        for (int p = 0; p < 8; ++p) y[k][p] = __fmul_rn(__fmul_rn(y[k][p], inv), g[p]);
      }
    }
    // rotation
    float z[2][8];
    if constexpr (PAIRS == kHalves) {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        z[0][p] = __fsub_rn(__fmul_rn(y[0][p], c[0][p]), __fmul_rn(y[1][p], s[1][p]));
        z[1][p] = __fadd_rn(__fmul_rn(y[1][p], c[0][p]), __fmul_rn(y[0][p], s[1][p]));
      }
    } else if constexpr (PAIRS == kNeighbours) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool turned = (l + k * S::kLanes) * 8 < rot;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float x0 = y[k][2 * p], x1 = y[k][2 * p + 1];
          z[k][2 * p] = turned ? __fsub_rn(__fmul_rn(x0, c[k][p]), __fmul_rn(x1, s[k][p])) : x0;
          z[k][2 * p + 1] = turned ? __fadd_rn(__fmul_rn(x1, c[k][p]), __fmul_rn(x0, s[k][p])) : x1;
        }
      }
    } else {
      // the partner of chunk e0 / 8 is half / 8 chunks on or back
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int chunk = l + k * S::kLanes;
        const bool turned = chunk * 8 < rot;
        const int pc = !turned ? chunk : (chunk * 8 < half ? chunk + half / 8 : chunk - half / 8);
        const int src = head_lane0 + pc % S::kLanes;
        const bool second = pc >= S::kLanes;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const float a0 = __shfl_sync(0xFFFFFFFFu, y[0][p], src);
          const float a1 = __shfl_sync(0xFFFFFFFFu, y[1][p], src);
          z[k][p] = turned ? __fadd_rn(__fmul_rn(y[k][p], c[k][p]),
                                       __fmul_rn(second ? a1 : a0, s[k][p]))
                           : y[k][p];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int chunk = l + k * S::kLanes;
      const uint4 bits = is_v ? own[k] : pack8(z[k]);
      if (on && !is_v && !is_k)
        *reinterpret_cast<uint4*>(a.q_out + static_cast<int64_t>(tt) * a.q_out_stride +
                                  static_cast<int64_t>(h) * D + chunk * 8) = bits;
      store_cache<FMT, D>(is_v ? vpage : kpage, bits, is_v ? h - hq - hkv : h - hq, row, chunk, hkv,
                          a.block_size, a.data_bytes, is_v ? a.v_scale : a.k_scale,
                          on && in_pool && (is_v || is_k));
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");
}

// angle = position * base^(-2 i / rot_dim), its cosine and sine in 64 bits
// (an fp32 angle is off by 2^-24 of itself: 8e-3 at position 131072)
__global__ void __launch_bounds__(256)
    rope_table_kernel(float* __restrict__ cos_sin, int64_t n, int half, double step) {
  for (int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; k < n;
       k += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t pos = k / half;
    const int i = static_cast<int>(k % half);
    double sn, cn;
    sincos(static_cast<double>(pos) * exp2(static_cast<double>(i) * step), &sn, &cn);
    float* row = cos_sin + pos * 2 * half;
    row[i] = static_cast<float>(cn);
    row[half + i] = static_cast<float>(sn);
  }
}

template <int FMT, int D>
cudaError_t launch_rope(const NormRopeArgs& a, int num_sms, cudaStream_t st) {
  const int groups = (a.num_q_heads + 2 * a.num_kv_heads + RopeShape<D>::kHeads - 1) /
                     RopeShape<D>::kHeads;
  const int64_t items = static_cast<int64_t>(a.num_tokens) * groups;
  const int64_t most = static_cast<int64_t>(num_sms) * PD_ROPE_CTAS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items < most ? items : most));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.interleaved) return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<FMT, D, kNeighbours>, a);
  if (a.rot_dim == D) return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<FMT, D, kHalves>, a);
  return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<FMT, D, kPartHalves>, a);
}

template <int FMT>
cudaError_t launch_rope_fmt(const NormRopeArgs& a, int D, int num_sms, cudaStream_t st) {
  switch (D) {
    case 64: return launch_rope<FMT, 64>(a, num_sms, st);
    case 128: return launch_rope<FMT, 128>(a, num_sms, st);
    case 256: return launch_rope<FMT, 256>(a, num_sms, st);
    case 512: return launch_rope<FMT, 512>(a, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope_cache(const NormRopeArgs& a, int head_dim, int kv_dtype,
                                      int num_sms, cudaStream_t st) {
  if (a.num_tokens == 0) return cudaSuccess;
  switch (kv_dtype) {
    case PD_KV_BF16: return launch_rope_fmt<PD_KV_BF16>(a, head_dim, num_sms, st);
    case PD_KV_FP8_E4M3: return launch_rope_fmt<PD_KV_FP8_E4M3>(a, head_dim, num_sms, st);
    default: return launch_rope_fmt<PD_KV_NVFP4>(a, head_dim, num_sms, st);
  }
}

cudaError_t launch_rope_table(float* cos_sin, int max_position, int rot_dim, double base,
                              cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(max_position) * (rot_dim / 2);
  if (n == 0) return cudaSuccess;
  int64_t blocks = (n + 255) / 256;
  if (blocks > 65535) blocks = 65535;
  const double step = -2.0 / rot_dim * log2(base);
  rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(cos_sin, n, rot_dim / 2, step);
  return cudaGetLastError();
}

}  // namespace pd
