// The per-tile work of the INT8 decode kernel's computing warps: for one stage
// of keys the scores S^T = K Q^T, one online-softmax update and O^T += V^T P^T
// on mma.sync, keys on M and the q heads of the GQA group on N, as mma_tile.cuh
// does for the other forms (whose q fragments and running state it shares).
//
// Codes become f16 by integer operations. f16 1024 + n (n < 1024) is 0x6400 + n,
// so c + 128, the code with its top bit flipped, goes in as the low byte, and
// 1152 is subtracted: exact.
#pragma once

#include "mma_tile.cuh"

namespace pd {
namespace mma {

__device__ __forceinline__ uint32_t hsub2_u32(uint32_t x, uint32_t y) {
  __half2 hx, hy;
  memcpy(&hx, &x, 4);
  memcpy(&hy, &y, 4);
  const __half2 hr = __hsub2(hx, hy);
  uint32_t r;
  memcpy(&r, &hr, 4);
  return r;
}
// Two of four codes with flipped top bits, the low two (SEL 0x4140) or the high
// two (0x4342).
template <uint32_t SEL>
__device__ __forceinline__ uint32_t i8x2_f16x2(uint32_t flipped) {
  return hsub2_u32(__byte_perm(flipped, 0x64646464u, SEL), 0x64806480u);
}
// Code J of word x and code J of word y, as they are.
template <int J>
__device__ __forceinline__ uint32_t i8_pair_f16x2(uint32_t x, uint32_t y) {
  constexpr uint32_t kSel = J * 0x11u | (J + 4) * 0x1100u;
  return hsub2_u32((__byte_perm(x, y, kSel) & 0x00FF00FFu) ^ 0x64806480u, 0x64806480u);
}

// Weights are 2^(t - m + kWeightLog2) for scores t (the value scale's logarithm in
// them) with maximum m. f16 holds 2^-14 to 65504 in full and loses what is below
// 2^-25: with the largest weight at 2^15 that is 2^-40 of it, with the largest at 1
// pages whose value scales lie 2^25 apart would lose the smaller one's values.
constexpr float kWeightLog2 = 15.0f;

// What a copy (a page, or half of one) brings beside its codes: the key scale,
// log2 of the value scale and its reciprocal. A copy that was not made (past the
// keys, a page outside the pool) has log2 = -inf, which masks its keys.
struct alignas(16) I8Scales {
  float k, v_log2, v_inv, pad;
};

// A warp's place in a stage: byte offsets of its first K rows (per 16-byte piece)
// and V rows, which rows 8 on keep (the swizzle repeats every 8 rows).
template <class C>
struct I8Place {
  uint32_t k[C::kKSteps / 4], v[2];
  __device__ __forceinline__ I8Place(int key0, int d0, int r, int c) {
    constexpr int kVB = C::kDS / 8;
    const int kb = d0 + c * (C::kDS / 4), vb = d0 + r * kVB;
#pragma unroll
    for (int q4 = 0; q4 < C::kKSteps / 4; ++q4)
      k[q4] = swz<C::kSwizzle>((kb / C::kCRB) * (C::kKT * C::kCRB) + (key0 + r) * C::kCRB +
                               kb % C::kCRB + 16 * q4);
#pragma unroll
    for (int odd = 0; odd < 2; ++odd)
      v[odd] = swz<C::kSwizzle>((vb / C::kCRB) * (C::kKT * C::kCRB) +
                                (key0 + 2 * c + odd) * C::kCRB + vb % C::kCRB);
  }
};

// The warp's C::kU x 16 keys of a stage: those from index key0 (of the sequence) on,
// of which [t_begin, t_end) count. sc: the scales of the stage's copies, from the
// warp's first on.
template <int D, int NT, class C>
__device__ __forceinline__ void consume_int8_tile(TileState<C, NT>& s, const I8Place<C>& at,
                                                  uint32_t kst, uint32_t vst, int key0, int t_begin,
                                                  int t_end, const I8Scales* sc,
                                                  const ThreadPlace& tp, float* red, int red_buf) {
  const int warp = tp.warp, lane = tp.lane, r = tp.r;
  constexpr int kU = C::kU;
  float p[kU][NT][4];
  // ---- scores: keys 16 u + r, + 8; bytes d in [c DS / 4, (c + 1) DS / 4) ----
#pragma unroll
  for (int u = 0; u < kU; ++u) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) p[u][nt][0] = p[u][nt][1] = p[u][nt][2] = p[u][nt][3] = 0.0f;
    uint32_t wa[C::kKSteps], wb[C::kKSteps];
#pragma unroll
    for (int q4 = 0; q4 < C::kKSteps / 4; ++q4) {
      lds_words<16>(kst + at.k[q4] + 16 * u * C::kCRB, wa + 4 * q4);
      lds_words<16>(kst + at.k[q4] + (16 * u + 8) * C::kCRB, wb + 4 * q4);
    }
#pragma unroll
    for (int ks = 0; ks < C::kKSteps; ++ks) {
      const uint32_t xa = wa[ks] ^ 0x80808080u, xb = wb[ks] ^ 0x80808080u;
      uint32_t af[4];
      af[0] = i8x2_f16x2<0x4140>(xa);
      af[1] = i8x2_f16x2<0x4140>(xb);
      af[2] = i8x2_f16x2<0x4342>(xa);
      af[3] = i8x2_f16x2<0x4342>(xb);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma16816<true>(p[u][nt], af, s.qf[ks][nt][0], s.qf[ks][nt][1]);
    }
  }
  if constexpr (C::kDSplit == 4) {  // sum the warps' parts of head_dim
    float* mine = red + (red_buf * 4 + warp) * (kU * NT * 32 * 4);
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float4*>(mine + ((u * NT + nt) * 32 + lane) * 4) =
            make_float4(p[u][nt][0], p[u][nt][1], p[u][nt][2], p[u][nt][3]);
    consumers_sync();
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(
              red + (red_buf * 4 + w) * (kU * NT * 32 * 4) + ((u * NT + nt) * 32 + lane) * 4);
          t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
        }
        p[u][nt][0] = t.x; p[u][nt][1] = t.y; p[u][nt][2] = t.z; p[u][nt][3] = t.w;
      }
  }

  // ---- one online-softmax update ----
  // the weight 2^(score - m) times the value scale, whose logarithm joins the
  // score: the running maximum m is that of both
  float v_inv[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const I8Scales f = sc[16 * u / C::kBR];
    v_inv[u] = f.v_inv;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float f0 = s.qmul[nt][0] * f.k, f1 = s.qmul[nt][1] * f.k;
      p[u][nt][0] = fmaf(p[u][nt][0], f0, f.v_log2);
      p[u][nt][1] = fmaf(p[u][nt][1], f1, f.v_log2);
      p[u][nt][2] = fmaf(p[u][nt][2], f0, f.v_log2);
      p[u][nt][3] = fmaf(p[u][nt][3], f1, f.v_log2);
    }
  }
  if (key0 < t_begin || key0 + 16 * kU > t_end) {  // warp-uniform
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int ka = key0 + 16 * u + r, kb = ka + 8;
      const bool va = ka >= t_begin && ka < t_end, vb = kb >= t_begin && kb < t_end;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (!va) p[u][nt][0] = p[u][nt][1] = -INFINITY;
        if (!vb) p[u][nt][2] = p[u][nt][3] = -INFINITY;
      }
    }
  }
  uint32_t pbf[kU][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      mx0 = fmaxf(mx0, fmaxf(p[u][nt][0], p[u][nt][2]));
      mx1 = fmaxf(mx1, fmaxf(p[u][nt][1], p[u][nt][3]));
    }
    // a column's maximum moved in some lane: then all lanes find it, and rescale
    if (__any_sync(0xFFFFFFFFu, mx0 > s.m_run[nt][0] || mx1 > s.m_run[nt][1])) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, o));
      }
      const float mn0 = fmaxf(s.m_run[nt][0], mx0), mn1 = fmaxf(s.m_run[nt][1], mx1);
      const float al0 = (mn0 == -INFINITY) ? 1.0f : ex2(s.m_run[nt][0] - mn0);
      const float al1 = (mn1 == -INFINITY) ? 1.0f : ex2(s.m_run[nt][1] - mn1);
      s.l_run[nt][0] *= al0;
      s.l_run[nt][1] *= al1;
#pragma unroll
      for (int md = 0; md < C::kKSteps; ++md) {
        s.acc[md][nt][0] *= al0;
        s.acc[md][nt][1] *= al1;
        s.acc[md][nt][2] *= al0;
        s.acc[md][nt][3] *= al1;
      }
      s.m_run[nt][0] = mn0;
      s.m_run[nt][1] = mn1;
    }
    const float r0 = s.m_run[nt][0] == -INFINITY ? 0.0f : s.m_run[nt][0] - kWeightLog2;
    const float r1 = s.m_run[nt][1] == -INFINITY ? 0.0f : s.m_run[nt][1] - kWeightLog2;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float p0 = ex2(p[u][nt][0] - r0), p1 = ex2(p[u][nt][1] - r1);
      const float p2 = ex2(p[u][nt][2] - r0), p3 = ex2(p[u][nt][3] - r1);
      // the row sum is of the weights without the value scale
      s.l_run[nt][0] = fmaf(p0 + p2, v_inv[u], s.l_run[nt][0]);
      s.l_run[nt][1] = fmaf(p1 + p3, v_inv[u], s.l_run[nt][1]);
      pbf[u][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
      pbf[u][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
    }
  }

  // ---- O^T += V^T P^T: bytes d in [r DS / 8, (r + 1) DS / 8) of keys 2c, 2c + 1,
  // 2c + 8, 2c + 9; byte j is head_dim row (m-tile j, r) for j < DS / 16, else
  // (m-tile j - DS / 16, r + 8). A masked key's weight is zero and any byte is a
  // finite code ----
  constexpr int kVB = C::kDS / 8;  // 16 or 8
  constexpr int kHalf = kVB / 8;   // words of the first half of the bytes
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    uint32_t v[4][kVB / 4];
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4)
      lds_words<kVB>(vst + at.v[k4 & 1] + (16 * u + 8 * (k4 >> 1)) * C::kCRB, v[k4]);
    auto m_tile = [&](auto jj, const int w) {
      constexpr int J = decltype(jj)::value;
      uint32_t af[4];
      af[0] = i8_pair_f16x2<J>(v[0][w], v[1][w]);
      af[1] = i8_pair_f16x2<J>(v[0][w + kHalf], v[1][w + kHalf]);
      af[2] = i8_pair_f16x2<J>(v[2][w], v[3][w]);
      af[3] = i8_pair_f16x2<J>(v[2][w + kHalf], v[3][w + kHalf]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma16816<true>(s.acc[w * 4 + J][nt], af, pbf[u][nt][0], pbf[u][nt][1]);
    };
#pragma unroll
    for (int w = 0; w < kHalf; ++w) {
      m_tile(std::integral_constant<int, 0>{}, w);
      m_tile(std::integral_constant<int, 1>{}, w);
      m_tile(std::integral_constant<int, 2>{}, w);
      m_tile(std::integral_constant<int, 3>{}, w);
    }
  }
}

}  // namespace mma
}  // namespace pd
