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

// One stage: K and V codes in shared memory, the key index of its first row, the
// key range that counts, the copies whose pages were outside the pool, and per
// copy the key scale, log2 of the value scale and its reciprocal (three runs of
// kNCopy floats).
struct I8Stage {
  uint32_t kst, vst;
  int t0, t_begin, t_end;
  uint32_t bad;
  const float* scales;
};

template <int D, int NT, class C>
__device__ __forceinline__ void consume_int8_tile(TileState<C, NT>& s, const I8Stage& sv,
                                                  const ThreadPlace& tp, float* red, int red_buf) {
  const int warp = tp.warp, lane = tp.lane, r = tp.r, c = tp.c, d0 = tp.d0;
  // the 16 keys this warp takes: its own (keys split over the warps) or the
  // stage's (head_dim split)
  const int key0 = C::kDSplit == 1 ? warp * 16 : 0;
  float sc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;

  // ---- scores: keys key0 + r, + 8; bytes d in [c DS / 4, (c + 1) DS / 4) ----
  {
    const int dbyte = d0 + c * (C::kDS / 4);
    const uint32_t base = (dbyte / C::kCRB) * (C::kKT * C::kCRB) + (dbyte % C::kCRB);
    uint32_t wa[C::kKSteps], wb[C::kKSteps];
#pragma unroll
    for (int q4 = 0; q4 < C::kKSteps / 4; ++q4) {
      const uint32_t offa = base + (key0 + r) * C::kCRB + 16 * q4;
      lds_words<16>(sv.kst + swz<C::kSwizzle>(offa), wa + 4 * q4);
      lds_words<16>(sv.kst + swz<C::kSwizzle>(offa + 8 * C::kCRB), wb + 4 * q4);
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
        mma16816<true>(sc[nt], af, s.qf[ks][nt][0], s.qf[ks][nt][1]);
    }
  }
  if constexpr (C::kDSplit == 4) {  // sum the warps' parts of head_dim
    float* mine = red + (red_buf * 4 + warp) * (NT * 32 * 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      *reinterpret_cast<float4*>(mine + (nt * 32 + lane) * 4) =
          make_float4(sc[nt][0], sc[nt][1], sc[nt][2], sc[nt][3]);
    consumers_sync();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(
            red + (red_buf * 4 + w) * (NT * 32 * 4) + (nt * 32 + lane) * 4);
        t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
      }
      sc[nt][0] = t.x; sc[nt][1] = t.y; sc[nt][2] = t.z; sc[nt][3] = t.w;
    }
  }

  // ---- one online-softmax update; fragment rows r, r + 8 are keys key0 + r, + 8 ----
  const int copy = key0 / C::kBR;
  const float kf = sv.scales[copy], vl = sv.scales[C::kNCopy + copy];
  const float vi = sv.scales[2 * C::kNCopy + copy];
  const int k0 = sv.t0 + key0;
  bool va = true, vb = true;
  if (k0 < sv.t_begin || k0 + 16 > sv.t_end || ((sv.bad >> copy) & 1u)) {  // warp-uniform
    const bool page = !((sv.bad >> copy) & 1u);
    va = page && k0 + r >= sv.t_begin && k0 + r < sv.t_end;
    vb = page && k0 + r + 8 >= sv.t_begin && k0 + r + 8 < sv.t_end;
  }
  uint32_t pbf[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    // the weight 2^(score - m) times the value scale, whose logarithm joins the
    // score: the running maximum m is that of both
    const float f0 = s.qmul[nt][0] * kf, f1 = s.qmul[nt][1] * kf;
    float p0 = va ? fmaf(sc[nt][0], f0, vl) : -INFINITY;
    float p1 = va ? fmaf(sc[nt][1], f1, vl) : -INFINITY;
    float p2 = vb ? fmaf(sc[nt][2], f0, vl) : -INFINITY;
    float p3 = vb ? fmaf(sc[nt][3], f1, vl) : -INFINITY;
    float mx0 = fmaxf(p0, p2), mx1 = fmaxf(p1, p3);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, o));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, o));
    }
    const float mn0 = fmaxf(s.m_run[nt][0], mx0), mn1 = fmaxf(s.m_run[nt][1], mx1);
    // no column's maximum moved: every factor is exactly 1, skip the rescale
    if (__any_sync(0xFFFFFFFFu, mn0 > s.m_run[nt][0] || mn1 > s.m_run[nt][1])) {
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
    p0 = (mn0 == -INFINITY) ? 0.0f : ex2(p0 - mn0);
    p1 = (mn1 == -INFINITY) ? 0.0f : ex2(p1 - mn1);
    p2 = (mn0 == -INFINITY) ? 0.0f : ex2(p2 - mn0);
    p3 = (mn1 == -INFINITY) ? 0.0f : ex2(p3 - mn1);
    // the row sum is of the weights without the value scale
    s.l_run[nt][0] = fmaf(p0 + p2, vi, s.l_run[nt][0]);
    s.l_run[nt][1] = fmaf(p1 + p3, vi, s.l_run[nt][1]);
    pbf[nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
    pbf[nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
  }

  // ---- O^T += V^T P^T: bytes d in [r DS / 8, (r + 1) DS / 8) of keys 2c, 2c + 1,
  // 2c + 8, 2c + 9; byte j is head_dim row (m-tile j, r) for j < DS / 16, else
  // (m-tile j - DS / 16, r + 8). A masked key's weight is zero and any byte is a
  // finite code ----
  constexpr int kVB = C::kDS / 8;  // 16 or 8
  constexpr int kHalf = kVB / 8;   // words of the first half of the bytes
  const int dbyte = d0 + r * kVB;
  const uint32_t base = (dbyte / C::kCRB) * (C::kKT * C::kCRB) + (dbyte % C::kCRB);
  uint32_t v[4][kVB / 4];
#pragma unroll
  for (int k4 = 0; k4 < 4; ++k4) {
    const int key = key0 + 2 * c + (k4 & 1) + 8 * (k4 >> 1);
    lds_words<kVB>(sv.vst + swz<C::kSwizzle>(base + key * C::kCRB), v[k4]);
  }
  auto m_tile = [&](auto jj, const int w) {
    constexpr int J = decltype(jj)::value;
    uint32_t af[4];
    af[0] = i8_pair_f16x2<J>(v[0][w], v[1][w]);
    af[1] = i8_pair_f16x2<J>(v[0][w + kHalf], v[1][w + kHalf]);
    af[2] = i8_pair_f16x2<J>(v[2][w], v[3][w]);
    af[3] = i8_pair_f16x2<J>(v[2][w + kHalf], v[3][w + kHalf]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma16816<true>(s.acc[w * 4 + J][nt], af, pbf[nt][0], pbf[nt][1]);
  };
#pragma unroll
  for (int w = 0; w < kHalf; ++w) {
    m_tile(std::integral_constant<int, 0>{}, w);
    m_tile(std::integral_constant<int, 1>{}, w);
    m_tile(std::integral_constant<int, 2>{}, w);
    m_tile(std::integral_constant<int, 3>{}, w);
  }
}

}  // namespace mma
}  // namespace pd
