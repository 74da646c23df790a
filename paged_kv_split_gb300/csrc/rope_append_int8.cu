// Rotation of new tokens' q and k heads and the append of K and V to INT8
// pages with one scale per page and kv head (pd_rope_append_int8).
//
// A rotated pair is (a cos - b sin, b cos + a sin), every operation an fp32
// operation rounded once (no fma). For the rows R that a page gets and one kv
// head of K or V:
//   want  = clamp(max |x| over R / 127, 2^-60, 2^60)
//   scale = want if row 0 is in R, else max(old scale, want)
//   code  = rint(x * (1 / scale)) for R, and, where the scale grew,
//           rint(code * (old scale / scale)) for the page's earlier rows
// A (page, head) is one CTA's or one lane group's alone, so nothing is atomic.
//
// Two kernels. A prompt's page takes 16 or 32 rows: one CTA per page and run of
// heads holds a head's rows in registers (kLanes lanes a row, 16 elements a lane),
// finds the maximum over the block, and writes the codes: one pass over memory,
// which bounds it. 8945 rows of 32/8 heads of 128, 245 MB with the output rows: 47.1
// us, 5.2 TB/s, of it 199 MB from and to DRAM (the rest stays in L2).
//
// A decode step (max_q_len 1) has one row a page. It is a chain of memory latencies
// (counts, table, scale and rows) that no bandwidth shortens, and in most steps
// some page's scale grows. There a warp takes a kv head: its lane groups all work
// the new row out, without a block barrier, and hold the page's earlier rows, read
// beside the scale, in case it grows. 64 sequences of 32/8 heads of 128, every page
// a step fuller than in the call before: 3.8 us; one lane group a kv head, which
// reads the rows once the scale is known, 13.0.
#include "mma_common.cuh"
#include "serve_common.cuh"

namespace pd {
namespace {

using ::pd::mma::pack_bf16x2;

constexpr int kAppendThreads = 128;
constexpr float kScaleMin = 8.673617379884035e-19f;  // 2^-60
constexpr float kScaleMax = 1.152921504606847e18f;   // 2^60

// A lane's 16 elements of a head: two 8-element chunks that are each other's
// partners where they are rotated (cosines and sines at [8 l, 8 l + 8) of the
// table's halves, in either pairing), or 16 neighbours.
struct LaneChunks {
  int c0, c1;
  bool turned;
};
__device__ __forceinline__ LaneChunks lane_chunks(int l, int rot, bool inter) {
  LaneChunks k;
  k.turned = l * 16 < rot;
  const bool halves = k.turned && !inter;
  k.c0 = halves ? l * 8 : l * 16;
  k.c1 = halves ? rot / 2 + l * 8 : l * 16 + 8;
  return k;
}

__device__ __forceinline__ void unpack16(const uint4 (&w)[2], float (&x)[16]) {
  const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(u[i]);
    x[2 * i + 1] = bf16_hi(u[i]);
  }
}
__device__ __forceinline__ void pack16(const float (&x)[16], uint4 (&w)[2]) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    u[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  w[0] = make_uint4(u[0], u[1], u[2], u[3]);
  w[1] = make_uint4(u[4], u[5], u[6], u[7]);
}
__device__ __forceinline__ void rotate16(float (&x)[16], const float (&c)[8], const float (&s)[8],
                                         bool inter) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = inter ? x[2 * i] : x[i];
    const float b = inter ? x[2 * i + 1] : x[8 + i];
    const float y0 = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
    const float y1 = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
    (inter ? x[2 * i] : x[i]) = y0;
    (inter ? x[2 * i + 1] : x[8 + i]) = y1;
  }
}
// the largest finite |x|
__device__ __forceinline__ float finite_max(const float (&x)[16], float m) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = fabsf(x[i]);
    m = (v > m && v < INFINITY) ? v : m;
  }
  return m;
}
__device__ __forceinline__ float wanted_scale(float amax) {
  return fminf(fmaxf(__fdiv_rn(amax, 127.0f), kScaleMin), kScaleMax);
}
// rint(x * f) clamped to +-127; NaN gives 0
__device__ __forceinline__ int int8_code(float x, float f) {
  const int q = __float2int_rn(__fmul_rn(x, f));
  return q > 127 ? 127 : (q < -127 ? -127 : q);
}
__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i >> 2] |= (static_cast<uint32_t>(int8_code(x[i], inv)) & 0xFFu) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}
// Codes of 16 bytes times a ratio <= 1: c + 128 as the low byte of 2^23 gives the
// code as a float exactly, and adding 1.5 * 2^23 rounds the product to the nearest
// even integer, whose low byte is the new code.
__device__ __forceinline__ uint4 rescale16(const uint4& v, float ratio) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t flipped = u[w] ^ 0x80808080u;
    uint32_t n[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = __uint_as_float(__byte_perm(flipped, 0x4B000000u, 0x7440u + i)) - 8388736.0f;
      n[i] = __float_as_uint(__fadd_rn(__fmul_rn(c, ratio), 12582912.0f));
    }
    o[w] = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// A lane's part of rows first, first + step .. below n of a head, N of them at a
// time: all of a batch is on its way before the first is needed.
template <int N>
struct OldRows {
  uint4 v[N];
  __device__ __forceinline__ void load(const uint8_t* at, int row_bytes, int first, int step,
                                       int n) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (first + k * step < n)
        v[k] = *reinterpret_cast<const uint4*>(at + (first + k * step) * row_bytes);
  }
  __device__ __forceinline__ void store(uint8_t* at, int row_bytes, int first, int step, int n,
                                        float ratio) const {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (first + k * step < n)
        *reinterpret_cast<uint4*>(at + (first + k * step) * row_bytes) = rescale16(v[k], ratio);
  }
};

// A sequence's rows in the batch and in its cache; n = 0 where its counts do
// not fit.
struct AppendSeq {
  int q0, n, first;  // first: the first new row's index in the sequence
};
__device__ __forceinline__ AppendSeq append_seq(const AppendArgs& a, int b, bool tell) {
  AppendSeq s;
  s.q0 = a.cu_q[b];
  const int q1 = a.cu_q[b + 1];
  const int L = a.seq_lens[b];
  s.n = q1 - s.q0;
  s.first = L - s.n;
  if (s.q0 < 0 || q1 < s.q0 || q1 > a.total_q || s.n > a.max_q_len || L < s.n ||
      L > a.max_blocks_per_seq * a.block_size) {
    if (tell) atomicOr(a.flags, PD_DEV_BAD_SEQ_LEN);
    s.n = 0;
  }
  return s;
}
__device__ __forceinline__ int table_row(const AppendArgs& a, int row, int pos, bool tell) {
  if (a.positions) pos = a.positions[row];
  if (pos < 0 || pos >= a.max_position) {
    if (tell) atomicOr(a.flags, PD_DEV_BAD_POSITION);
    pos = pos < 0 ? 0 : a.max_position - 1;
  }
  return pos;
}
__device__ __forceinline__ void load_turn(const AppendArgs& a, int pos, int l, float (&c)[8],
                                          float (&s)[8]) {
  const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim + l * 8;
  const float4 c0 = *reinterpret_cast<const float4*>(cs);
  const float4 c1 = *reinterpret_cast<const float4*>(cs + 4);
  const float4 s0 = *reinterpret_cast<const float4*>(cs + a.rot_dim / 2);
  const float4 s1 = *reinterpret_cast<const float4*>(cs + a.rot_dim / 2 + 4);
  c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
  c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
  s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
  s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
}

// ---------------------------------------------------------------------------
// Pages of several rows: CTA (page u of sequence b's new rows, head group z).
// Where a lane has one row, seven CTAs an SM (72 registers; 8945 rows: 47.7 us, six
// CTAs 49.6, eight 48.7, ten, with spills, 56); with more rows what the compiler takes.
template <int D, int BS, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, D * BS <= 2048 ? 7 : 0)
    append_pages_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kLanes = D / 16;                        // lanes of a row
  constexpr int kSlots = kAppendThreads / kLanes;       // rows at a time
  constexpr int kRows = (BS + kSlots - 1) / kSlots;     // rows of a lane
  constexpr bool kKeepTurn = kRows <= 2;                // cosines and sines stay in registers
  const int tid = threadIdx.x;
  const int b = blockIdx.y;
  const int h0 = blockIdx.z * a.heads_per_cta;
  const AppendSeq sq = append_seq(a, b, tid == 0 && blockIdx.x == 0 && blockIdx.z == 0);
  if (sq.n <= 0) return;
  const int page_index = sq.first / BS + blockIdx.x;
  const int L = sq.first + sq.n;
  if (page_index * BS >= L) return;
  const int r_lo = max(sq.first - page_index * BS, 0);   // the page's new rows
  const int r_hi = min(L - page_index * BS, BS);
  const int64_t page =
      a.block_tables[static_cast<int64_t>(b) * a.max_blocks_per_seq + page_index];
  const bool in_pool = page >= 0 && page < a.num_blocks;
  if (!in_pool && tid == 0 && blockIdx.z == 0) atomicOr(a.flags, PD_DEV_BAD_PAGE);
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int heads = hq + 2 * hkv;
  const int l = tid % kLanes, slot = tid / kLanes;
  const LaneChunks ch = lane_chunks(l, a.rot_dim, INTER);
  __shared__ float red[2][kAppendThreads / 32];

  // rows slot + j * kSlots of the page; row_of: their row of the batch
  bool on[kRows];
  int64_t row_of[kRows];
  int pos_of[kRows];
  float c[kKeepTurn ? kRows : 1][8], s[kKeepTurn ? kRows : 1][8];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int r = slot + j * kSlots;
    on[j] = r >= r_lo && r < r_hi;
    const int pos = page_index * BS + r;
    row_of[j] = on[j] ? sq.q0 + pos - sq.first : sq.q0;
    pos_of[j] = table_row(a, static_cast<int>(row_of[j]), on[j] ? pos : 0,
                          on[j] && l == 0 && blockIdx.z == 0);
    if constexpr (kKeepTurn) {
      if (ch.turned) load_turn(a, pos_of[j], l, c[j], s[j]);
    }
  }
  uint4 raw[kRows][2];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const uint16_t* src = a.qkv + row_of[j] * a.qkv_stride + static_cast<int64_t>(h) * D;
      raw[j][0] = *reinterpret_cast<const uint4*>(src + ch.c0);
      raw[j][1] = *reinterpret_cast<const uint4*>(src + ch.c1);
    }
  };
  const int h1 = min(h0 + a.heads_per_cta, heads);
  int turn = 0;  // buffer of the block's maxima
  load(h0);
  for (int h = h0; h < h1; ++h) {
    const bool is_v = h >= hq + hkv, is_k = !is_v && h >= hq;
    float x[kRows][16];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      unpack16(raw[j], x[j]);
      if (!is_v && ch.turned) {
        if constexpr (kKeepTurn) {
          rotate16(x[j], c[j], s[j], INTER);
        } else {
          load_turn(a, pos_of[j], l, c[0], s[0]);
          rotate16(x[j], c[0], s[0], INTER);
        }
      }
    }
    if (h + 1 < h1) load(h + 1);
    if (!is_v && (!is_k || a.k_out)) {
      uint16_t* dst0 = is_k ? a.k_out : a.q_out;
      const int64_t stride = is_k ? a.k_out_stride : a.q_out_stride;
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        if (!on[j]) continue;
        uint4 w[2];
        pack16(x[j], w);
        uint16_t* dst = dst0 + row_of[j] * stride + static_cast<int64_t>(is_k ? h - hq : h) * D;
        *reinterpret_cast<uint4*>(dst + ch.c0) = w[0];
        *reinterpret_cast<uint4*>(dst + ch.c1) = w[1];
      }
    }
    if (h < hq || !in_pool) continue;
    const int g = is_v ? h - hq - hkv : h - hq;
    uint8_t* base = (is_v ? a.v_cache : a.k_cache) + page * a.page_bytes;
    float* scale_p = reinterpret_cast<float*>(base + a.data_bytes) + g;
    const float have = r_lo > 0 ? *scale_p : 0.0f;
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (on[j]) m = finite_max(x[j], m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((tid & 31) == 0) red[turn][tid >> 5] = m;
    __syncthreads();  // and every thread has read the old scale
    m = fmaxf(fmaxf(red[turn][0], red[turn][1]), fmaxf(red[turn][2], red[turn][3]));
    turn ^= 1;
    const float want = wanted_scale(m);
    const bool grown = r_lo > 0 && want > have;
    const float scale = (r_lo == 0 || grown) ? want : have;
    const float inv = __fdiv_rn(1.0f, scale);
    uint8_t* lines = base + static_cast<int64_t>(g) * BS * D;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (!on[j]) continue;
      uint8_t* dst = lines + (slot + j * kSlots) * D;
      *reinterpret_cast<uint2*>(dst + ch.c0) = codes8(x[j], inv);
      *reinterpret_cast<uint2*>(dst + ch.c1) = codes8(x[j] + 8, inv);
    }
    if (r_lo == 0 || grown) {
      if (tid == 0) *scale_p = scale;
      if (grown) {
        const float ratio = __fdiv_rn(have, scale);
        for (int r = slot; r < r_lo; r += kSlots) {
          uint4* p = reinterpret_cast<uint4*>(lines + r * D + l * 16);
          *p = rescale16(*p, ratio);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// One row a sequence. A kv head of K or V is a warp's, each of whose lane groups
// of kLanes works the new row out; the page's earlier rows are dealt among them.
// A q head is a lane group's.
template <int D, int BS, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) append_step_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kLanes = D / 16;
  constexpr int kWarps = kAppendThreads / 32, kSlots = 32 / kLanes;
  // a lane's earlier rows, at most 16 (64 registers) at a time: BS / kSlots are all
  constexpr int kAhead = BS / kSlots < 16 ? BS / kSlots : 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % kLanes, slot = lane / kLanes;
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int b = blockIdx.y;
  const int kv_blocks = (2 * hkv + kWarps - 1) / kWarps;
  const bool is_q = blockIdx.x >= kv_blocks;
  // the head's place in the row
  const int h = is_q ? ((blockIdx.x - kv_blocks) * kWarps + warp) * kSlots + slot
                     : hq + blockIdx.x * kWarps + warp;
  if (h >= (is_q ? hq : hq + 2 * hkv)) return;  // kv heads: a whole warp leaves
  const bool is_v = h >= hq + hkv;
  const bool teller = h == hq && lane == 0;
  const AppendSeq sq = append_seq(a, b, teller);
  if (sq.n <= 0) return;
  const LaneChunks ch = lane_chunks(l, a.rot_dim, INTER);
  const int64_t row = sq.q0;
  const uint16_t* src = a.qkv + row * a.qkv_stride + static_cast<int64_t>(h) * D;
  const uint4 raw[2] = {*reinterpret_cast<const uint4*>(src + ch.c0),
                        *reinterpret_cast<const uint4*>(src + ch.c1)};
  float x[16];
  unpack16(raw, x);
  if (!is_v) {
    const int pos = table_row(a, static_cast<int>(row), sq.first, teller);
    if (ch.turned) {
      float c[8], s[8];
      load_turn(a, pos, l, c, s);
      rotate16(x, c, s, INTER);
    }
  }
  auto put = [&](uint16_t* dst) {
    uint4 w[2];
    pack16(x, w);
    *reinterpret_cast<uint4*>(dst + ch.c0) = w[0];
    *reinterpret_cast<uint4*>(dst + ch.c1) = w[1];
  };
  if (is_q) {
    put(a.q_out + row * a.q_out_stride + static_cast<int64_t>(h) * D);
    return;
  }
  const int page_index = sq.first / BS, r = sq.first % BS;
  const int64_t page =
      a.block_tables[static_cast<int64_t>(b) * a.max_blocks_per_seq + page_index];
  const bool in_pool = page >= 0 && page < a.num_blocks;
  if (!in_pool && teller) atomicOr(a.flags, PD_DEV_BAD_PAGE);
  const int g = is_v ? h - hq - hkv : h - hq;
  uint8_t* base = (is_v ? a.v_cache : a.k_cache) + (in_pool ? page * a.page_bytes : 0);
  float* scale_p = reinterpret_cast<float*>(base + a.data_bytes) + g;
  uint8_t* lines = base + static_cast<int64_t>(g) * BS * D;
  // the earlier rows come with the scale: a page that grows waits no second time
  const int have_rows = in_pool ? r : 0;
  const float have = have_rows > 0 ? *scale_p : 0.0f;
  OldRows<kAhead> old;
  old.load(lines + l * 16, D, slot, kSlots, have_rows);
  float m = finite_max(x, 0.0f);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  // every lane has read the row (k_out may be the row itself) and the old scale
  __syncwarp();
  if (!is_v && a.k_out && slot == 0)
    put(a.k_out + row * a.k_out_stride + static_cast<int64_t>(g) * D);
  if (!in_pool) return;
  const float want = wanted_scale(m);
  const bool grown = r > 0 && want > have;
  const float scale = (r == 0 || grown) ? want : have;
  if (slot == 0) {
    const float inv = __fdiv_rn(1.0f, scale);
    *reinterpret_cast<uint2*>(lines + r * D + ch.c0) = codes8(x, inv);
    *reinterpret_cast<uint2*>(lines + r * D + ch.c1) = codes8(x + 8, inv);
  }
  if (r == 0 || grown) {
    if (lane == 0) *scale_p = scale;
    if (grown) {
      const float ratio = __fdiv_rn(have, scale);
      old.store(lines + l * 16, D, slot, kSlots, r, ratio);
      if constexpr (kAhead * kSlots < BS) {  // head_dim 512, 32 rows
        old.load(lines + l * 16, D, slot + kAhead * kSlots, kSlots, r);
        old.store(lines + l * 16, D, slot + kAhead * kSlots, kSlots, r, ratio);
      }
    }
  }
}

template <typename K>
cudaError_t launch(K kern, dim3 grid, const AppendArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kAppendThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D>
cudaError_t launch_append(AppendArgs a, int num_sms, cudaStream_t st) {
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int bs = a.block_size;
  const bool inter = a.interleaved != 0;
  // One new row a sequence: the step kernel (64 sequences of 32/8 heads of 128 in
  // pages that grow as they fill, 3.8 us; the pages kernel, a CTA a head and page,
  // 10.0; 1024 sequences 13.9 and 72)
  if (a.max_q_len == 1) {
    constexpr int kWarps = kAppendThreads / 32, kSlots = kAppendThreads / (D / 16);
    const dim3 grid((2 * a.num_kv_heads + kWarps - 1) / kWarps +
                        (a.num_q_heads + kSlots - 1) / kSlots,
                    a.num_seqs);
    if (bs == 16)
      return inter ? launch(append_step_kernel<D, 16, true>, grid, a, st)
                   : launch(append_step_kernel<D, 16, false>, grid, a, st);
    return inter ? launch(append_step_kernel<D, 32, true>, grid, a, st)
                 : launch(append_step_kernel<D, 32, false>, grid, a, st);
  }
  // the most pages a sequence's new rows touch
  const int pages = (a.max_q_len + bs - 2) / bs + 1;
  // runs of heads long enough to reuse the cosines, short enough to fill the SMs
  // (8945 rows of 48 heads of 128, six CTAs at a time: 32 an SM 49.5 us, 8 58, 16 51,
  // 64 51.5)
  const int64_t units = (static_cast<int64_t>(a.total_q) + bs - 1) / bs + a.num_seqs;
  int64_t groups = (static_cast<int64_t>(num_sms) * 32 + units - 1) / units;
  if (groups > heads) groups = heads;
  a.heads_per_cta = static_cast<int>((heads + groups - 1) / groups);
  const dim3 grid(pages, a.num_seqs, (heads + a.heads_per_cta - 1) / a.heads_per_cta);
  if (bs == 16)
    return inter ? launch(append_pages_kernel<D, 16, true>, grid, a, st)
                 : launch(append_pages_kernel<D, 16, false>, grid, a, st);
  return inter ? launch(append_pages_kernel<D, 32, true>, grid, a, st)
               : launch(append_pages_kernel<D, 32, false>, grid, a, st);
}

}  // namespace

cudaError_t launch_rope_append_int8(AppendArgs a, int head_dim, int num_sms, cudaStream_t st) {
  switch (head_dim) {
    case 64: return launch_append<64>(a, num_sms, st);
    case 128: return launch_append<128>(a, num_sms, st);
    case 256: return launch_append<256>(a, num_sms, st);
    case 512: return launch_append<512>(a, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pd
