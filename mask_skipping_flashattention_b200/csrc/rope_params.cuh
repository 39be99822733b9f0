// Parameters of the rotary kernel (filled on the host, passed by value).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace bfa {

// One launch rotates queries (out of place or in place) and, when it fills a
// cache, rotates the new keys and copies the new values into their pages.
struct RopeParams {
  int32_t D;            // head dim (a multiple of 8)
  int32_t rotary;       // leading values of a head that turn (a multiple of 16, 0: none)
  int32_t interleaved;  // 1: pairs (2i, 2i + 1); 0: pairs (i, i + rotary / 2)
  float amplitude;      // factor of cos and sin
  float sign;           // -1: the inverse rotation
  const double* inv_freq;  // [rotary / 2] radians per position
  int64_t tokens;       // rows of q (batched: B * S)
  int32_t S;            // batched: tokens per batch row (packed: = tokens)
  int32_t H, Hkv;       // heads of q (0: none), of k and v (0: none)
  int32_t heads_per_block, tokens_per_block;
  const __nv_bfloat16* q;
  int64_t q_sb, q_ss, q_sh;
  __nv_bfloat16* q_out;
  int64_t qo_sb, qo_ss, qo_sh;
  // positions given: one per (batch row, token)
  const void* positions;
  int32_t positions64;
  int64_t pos_sb;
  // or taken from a ragged batch's lengths (positions == nullptr), with the cache
  const int32_t* cu_seqlens;  // [n_seq + 1]
  const int32_t* seqused_k;   // [n_seq] keys of each sequence, the new ones included
  int32_t n_seq;
  const __nv_bfloat16* k;
  int64_t k_ss, k_sh;
  const __nv_bfloat16* v;
  int64_t v_ss, v_sh;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  int64_t c_sp, c_st, c_sh;  // cache strides: page, token, head
  int64_t num_pages;
  int32_t page_size, pages_per_seq;
  const int32_t* block_table;
  uint32_t* err;  // status word of the chunk kernels (written by the checked build's index checks)
};

cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t s);

}  // namespace bfa
