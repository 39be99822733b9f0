// Parameters of the chunk kernels: attention of the newest tokens of each
// sequence over a paged cache (filled on the host, passed by value).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "score.cuh"

namespace bfa {

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
  int64_t rows_lo, rows_hi;
  // split of the keys: about `slots` pieces of at least `min_tiles` key tiles
  int32_t slots, min_tiles;
  int32_t max_segs;   // pieces the grid and the workspace have room for
  int32_t max_units;  // (sequence, kv head, row tile) units there can be
  float* ws_o;        // [max_segs, rows of a tile, D] partial outputs, unnormalised
  float2* ws_ml;      // [max_segs, rows of a tile] reference maximum (log2) and sum
  uint64_t wait_ns;
  uint32_t* err;
};

// few rows a kv head: 16 or 32 rows a unit (row_tiles 1, 2); with the join
cudaError_t launch_chunk_rows(const ChunkParams& p, int row_tiles, cudaStream_t s);
// many rows: 256 rows a unit; with the join
cudaError_t launch_chunk_tiles(const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& p, cudaStream_t s);
// joins the pieces of units of `rows` rows and key tiles of `keys`
cudaError_t launch_chunk_join(const ChunkParams& p, int rows, int keys, cudaStream_t s);

constexpr int kChunkTileRows = 256;  // rows of a unit of launch_chunk_tiles

}  // namespace bfa
