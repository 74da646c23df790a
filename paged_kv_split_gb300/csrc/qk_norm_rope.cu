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
// about 8 operations an element leave it bound by memory. One CTA takes one
// token (its table row is then read once, into registers) and 256 / (D / 8)
// heads at a time, 8 elements (16 bytes) a lane; few tokens spread their heads
// over more CTAs instead.
#include "pd_common.cuh"

namespace pd {
namespace {

constexpr int kRopeThreads = 256;

template <int D>
struct RopeShape {
  static constexpr int kLanes = D / 8 < 32 ? D / 8 : 32;  // lanes of one head
  static constexpr int kChunks = D / 8 / kLanes;          // 8-element chunks of a lane
  static constexpr int kHeads = kRopeThreads / kLanes;    // heads of one CTA pass
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

// One lane's 8 consecutive elements (bf16 bits) of a K or V head into the
// cache, in its form. NVFP4: two neighbouring lanes hold a 16-element group
// and must both be here.
template <int FMT, int D>
__device__ __forceinline__ void store_cache(uint8_t* page, const uint4& bits, int h, int row,
                                            int chunk, int hkv, int bs, int64_t data_bytes,
                                            float scale, bool on) {
  if constexpr (FMT == PD_KV_BF16) {
    if (on)
      *reinterpret_cast<uint4*>(page + ((static_cast<int64_t>(row) * hkv + h) * D + chunk * 8) * 2) =
          bits;
  } else {
    float x[8];
    unpack8(bits, x);
    if constexpr (FMT == PD_KV_FP8_E4M3) {
      uint32_t o[2] = {0u, 0u};
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k >> 2] |= e4m3_encode(quotient(x[k], scale)) << (8 * (k & 3));
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

template <int FMT, int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const NormRopeArgs a) {
  using S = RopeShape<D>;
  // a programmatic dependent of the previous work on the stream: nothing
  // global is touched before that grid has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = blockIdx.x;
  const int tid = threadIdx.x;
  const int l = tid % S::kLanes;  // this lane's place in its head
  const int lane = tid & 31;
  const int head_lane0 = lane - l;  // first lane of the head in the warp
  const int rot = a.rot_dim, half = rot / 2;

  int pos = a.positions[t];
  if (pos < 0 || pos >= a.max_position) {
    if (tid == 0 && blockIdx.y == 0) atomicOr(a.flags, PD_DEV_BAD_POSITION);
    pos = pos < 0 ? 0 : a.max_position - 1;
  }
  const int64_t slot = a.slots[t];
  const bool in_pool = slot >= 0 && slot < a.num_blocks * a.block_size;
  if (slot >= 0 && !in_pool && tid == 0 && blockIdx.y == 0) atomicOr(a.flags, PD_DEV_BAD_SLOT);
  const int64_t page = in_pool ? slot / a.block_size : 0;
  const int row = in_pool ? static_cast<int>(slot % a.block_size) : 0;

  // cosine and signed sine of this lane's elements: out = own * c + partner * s
  float c[S::kChunks][8], s[S::kChunks][8];
  int psrc[S::kChunks], pchunk[S::kChunks];  // partner chunk: its lane and index there
  const float* cs = a.cos_sin + static_cast<int64_t>(pos) * rot;
#pragma unroll
  for (int k = 0; k < S::kChunks; ++k) {
    const int e0 = (l + k * S::kLanes) * 8;
    psrc[k] = lane;
    pchunk[k] = k;
    if (e0 < rot) {
      if (a.interleaved) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float cc = cs[e0 / 2 + p], ss = cs[half + e0 / 2 + p];
          c[k][2 * p] = c[k][2 * p + 1] = cc;
          s[k][2 * p] = -ss;
          s[k][2 * p + 1] = ss;
        }
      } else {
        const bool low = e0 < half;
        const int i0 = low ? e0 : e0 - half;
        const int pc = (low ? e0 + half : e0 - half) / 8;
        psrc[k] = head_lane0 + pc % S::kLanes;
        pchunk[k] = pc / S::kLanes;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          c[k][p] = cs[i0 + p];
          const float ss = cs[half + i0 + p];
          s[k][p] = low ? -ss : ss;
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < 8; ++p) c[k][p] = s[k][p] = 0.0f;
    }
  }

  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int heads = hq + 2 * hkv;
  const uint16_t* src = a.qkv + static_cast<int64_t>(t) * a.qkv_stride;
  const bool norm = a.q_weight != nullptr;
  for (int h0 = blockIdx.y * S::kHeads; h0 < heads; h0 += gridDim.y * S::kHeads) {
    const int h = h0 + tid / S::kLanes;
    const bool on = h < heads;
    const int hh = on ? h : heads - 1;
    const bool is_v = hh >= hq + hkv;
    const bool is_k = !is_v && hh >= hq;
    float y[S::kChunks][8];
    uint4 raw[S::kChunks];
#pragma unroll
    for (int k = 0; k < S::kChunks; ++k)
      raw[k] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(hh) * D +
                                               (l + k * S::kLanes) * 8);
#pragma unroll
    for (int k = 0; k < S::kChunks; ++k) unpack8(raw[k], y[k]);
    if (norm) {
      float ss[S::kChunks];
#pragma unroll
      for (int k = 0; k < S::kChunks; ++k) {
        float q[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) q[p] = __fmul_rn(y[k][p], y[k][p]);
        ss[k] = __fadd_rn(__fadd_rn(__fadd_rn(q[0], q[1]), __fadd_rn(q[2], q[3])),
                          __fadd_rn(__fadd_rn(q[4], q[5]), __fadd_rn(q[6], q[7])));
#pragma unroll
        for (int o = 1; o < S::kLanes; o <<= 1)
          ss[k] = __fadd_rn(ss[k], __shfl_xor_sync(0xFFFFFFFFu, ss[k], o));
      }
      float sum = ss[0];
      if constexpr (S::kChunks == 2) sum = __fadd_rn(ss[0], ss[1]);
      const float inv =
          __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / static_cast<float>(D)), a.eps)));
      const uint16_t* w = is_k ? a.k_weight : a.q_weight;
#pragma unroll
      for (int k = 0; k < S::kChunks; ++k) {
        float g[8];
        unpack8(*reinterpret_cast<const uint4*>(w + (l + k * S::kLanes) * 8), g);
#pragma unroll
        for (int p = 0; p < 8; ++p)
          y[k][p] = __fmul_rn(__fmul_rn(y[k][p], inv), __fadd_rn(g[p], a.weight_offset));
      }
    }
    // rotation
    float z[S::kChunks][8];
#pragma unroll
    for (int k = 0; k < S::kChunks; ++k) {
      const bool turned = (l + k * S::kLanes) * 8 < rot;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        float partner;
        if (a.interleaved) {
          partner = y[k][p ^ 1];
        } else {
          partner = __shfl_sync(0xFFFFFFFFu, y[0][p], psrc[k]);
          if constexpr (S::kChunks == 2) {
            const float far = __shfl_sync(0xFFFFFFFFu, y[1][p], psrc[k]);
            if (pchunk[k] == 1) partner = far;
          }
        }
        z[k][p] = turned ? __fadd_rn(__fmul_rn(y[k][p], c[k][p]), __fmul_rn(partner, s[k][p]))
                         : y[k][p];
      }
    }
#pragma unroll
    for (int k = 0; k < S::kChunks; ++k) {
      const int chunk = l + k * S::kLanes;
      const uint4 bits = is_v ? raw[k] : pack8(z[k]);
      if (on && !is_v && !is_k)
        *reinterpret_cast<uint4*>(a.q_out + static_cast<int64_t>(t) * a.q_out_stride +
                                  static_cast<int64_t>(hh) * D + chunk * 8) = bits;
      uint8_t* pg = (is_v ? a.v_cache : a.k_cache) + page * a.page_bytes;
      store_cache<FMT, D>(pg, bits, is_v ? hh - hq - hkv : hh - hq, row, chunk, hkv, a.block_size,
                          a.data_bytes, is_v ? a.v_scale : a.k_scale,
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
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int passes = (heads + RopeShape<D>::kHeads - 1) / RopeShape<D>::kHeads;
  cudaLaunchConfig_t cfg = {};
  // few tokens: a token's heads over as many CTAs as it takes to fill the SMs
  int split = a.num_tokens < 4 * num_sms ? passes : 1;
  cfg.gridDim = dim3(a.num_tokens, split);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<FMT, D>, a);
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
