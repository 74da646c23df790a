// What serving from an INT8 cache adds to pd_common.cuh: the page geometry of the
// form and the argument blocks and launchers of its kernels.
#pragma once

#include "pd_common.cuh"

namespace pd {

// ---------------------------------------------------------------------------
// Cache geometry of every form. INT8: codes [hkv][bs][d], then a scale a head.
__host__ __device__ __forceinline__ int64_t int8_data_bytes(int bs, int hkv, int d) {
  return static_cast<int64_t>(bs) * hkv * d;
}
__host__ __device__ __forceinline__ int64_t any_page_bytes(int kv_dtype, int bs, int hkv, int d) {
  if (kv_dtype != PD_KV_INT8) return page_bytes_of(kv_dtype, bs, hkv, d);
  return (int8_data_bytes(bs, hkv, d) + 4 * static_cast<int64_t>(hkv) + 127) / 128 * 128;
}

// ---------------------------------------------------------------------------
// Kernel argument blocks.
// Rotation of new tokens and their append to INT8 pages (pd_rope_append_int8).
struct AppendArgs {
  const uint16_t* qkv;
  int64_t qkv_stride;
  const int32_t* cu_q;           // [B + 1]
  const int32_t* seq_lens;       // [B], the new rows included
  const int32_t* positions;      // [total_q], or null: the row in the sequence
  const float* cos_sin;          // [max_position][rot_dim]: cosines, then sines
  uint16_t* q_out;
  int64_t q_out_stride;
  uint16_t* k_out;               // null: not wanted
  int64_t k_out_stride;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int32_t* block_tables;   // [B][MBS]
  int* flags;
  int64_t num_blocks, page_bytes, data_bytes;
  int num_seqs, total_q, max_q_len, num_q_heads, num_kv_heads, block_size, max_blocks_per_seq;
  int max_position, rot_dim, interleaved;
  int heads_per_cta;
};

// Attention of packed prompts over their own rows (pd_prefill_packed).
struct PackedArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  int64_t q_stride, k_stride, v_stride, out_stride;
  const int32_t* cu_q;           // [B + 1]
  int* flags;
  int num_seqs, total_q, max_q_len, num_q_heads, num_kv_heads, group;
  int causal, sliding_window;
  float scale_log2;              // scale * log2(e)
};

cudaError_t launch_rope_append_int8(AppendArgs a, int head_dim, int num_sms, cudaStream_t st);
// Decode over INT8 pages: splits, or a plan where a.plan_cta is set.
cudaError_t launch_decode_int8(const DecodeArgs& a, int head_dim, cudaStream_t st);
// Resident CTAs per SM of launch_decode_int8's kernel (host only).
int int8_ctas_per_sm(int head_dim, int group);
// pd_prefill over INT8 pages on tcgen05, head_dim 64 and 128.
cudaError_t launch_prefill_int8(const PrefillArgs& a, int head_dim, int max_q_len, int num_sms,
                                cudaStream_t st);
cudaError_t launch_prefill_packed(const PackedArgs& a, int head_dim, int num_sms,
                                  cudaStream_t st);
cudaError_t launch_prefill_packed_simple(const PackedArgs& a, int head_dim, cudaStream_t st);

}  // namespace pd
