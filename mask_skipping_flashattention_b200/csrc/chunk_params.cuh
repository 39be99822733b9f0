// Parameters of the chunk kernels: attention of the newest tokens of each
// sequence over a paged cache (filled on the host, passed by value).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "score.cuh"

namespace bfa {

constexpr int kChunkTileRows = 256;  // rows of a unit of launch_chunk_tiles
constexpr int kChunkRows = 16;       // rows of a unit of launch_chunk_rows
constexpr int kChunkCutBytes = 24;   // a note of a cut (chunk_split.cuh)

struct ChunkParams {
  int32_t D, H, Hkv, G;  // G = H / Hkv query heads a kv head
  int32_t B;             // sequences
  int32_t total_q;       // rows of q (the last sequence may end before)
  const __nv_bfloat16* q;
  int64_t q_ss, q_sh;
  __nv_bfloat16* out;
  int64_t o_ss, o_sh;
  float* lse;            // [H, total_q] or nullptr
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  int64_t c_sp, c_st, c_sh;  // cache strides: page, token, head
  int64_t num_pages;
  int32_t page_size, pages_per_seq;
  const int32_t* block_table;  // [B, pages_per_seq]
  const int32_t* cu_seqlens;   // [B + 1]
  const int32_t* seqused_k;    // [B]
  int32_t window;              // keys with 0 <= position - key < window; -1: all
  float scale_log2;            // softmax scale * log2(e)
  ScoreParams score;
  // which sequences this launch serves: rows = new tokens * G in (rows_lo, rows_hi]
  int32_t rows_lo, rows_hi;
  // split of the work (chunk_split.cuh): blocks, the least share of one, and the length
  // that starting a unit counts, in key tiles
  int32_t slots, min_share, start_cost;
  float* ws_o;   // [2 slots, rows of a unit, D] partial outputs, unnormalised
  float2* ws_ml; // [2 slots, rows of a unit] reference maximum (log2) and sum
  void* ws_cuts; // [slots] Cut
  uint64_t wait_ns;
  uint32_t* err;
};

// many rows a kv head: 256 rows a unit
cudaError_t launch_chunk_tiles(const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& p, cudaStream_t s);
// few rows: 16 rows a unit; `after_tiles`: launched behind the tile kernel, whose
// last blocks it may overlap
cudaError_t launch_chunk_rows(const ChunkParams& p, bool after_tiles, cudaStream_t s);
// joins the cut units of both (slots = 0: that one was not launched)
cudaError_t launch_chunk_join(const ChunkParams& row, const ChunkParams& tile, cudaStream_t s);


}  // namespace bfa
