// Attention of the newest tokens of each sequence over a paged cache, for few
// query rows a kv head (single tokens, short chunks):
//   out_i = sum_j softmax_j(z_ij) v_j,  z = the shaped score of score.cuh,
// query token t of a sequence with kv keys at position kv - q_len + t, keys
// 0 <= j <= position (and position - j < window).
//
// Bound by HBM: a key and its value are 4 D bytes a kv head and meet only G query
// heads of a token.  A block runs one piece of the keys (chunk_split.cuh) for 16
// or 32 query rows of one kv head (rows = tokens x the G heads, so the group shares
// every byte).  Its four warps take 16 keys of a 64-key tile each, with a ring of
// asynchronous copies of their own, their own online softmax and no barrier
// between them until they are merged at the end; both products run on
// mma.sync m16n8k16 (bf16, fp32 sums), which at 16 rows is far from its limit.
// Units of several pieces leave unnormalised fp32 sums, joined by k_chunk_join.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "chunk_params.cuh"
#include "chunk_split.cuh"
#include "device_once.cuh"
#include "plan_types.cuh"
#include "ptx.cuh"
#include "score.cuh"

namespace bfa {

using namespace ptx;

namespace {

constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kRowKeys = 16 * kRowWarps;  // keys of a tile: 16 a warp
constexpr int kRowStages = 3;             // per-warp ring of 16-key slices

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// final value of a row's lse from its reference maximum (log2) and sum
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// four consecutive values of a row of the output
__device__ __forceinline__ void store4(const ChunkParams& p, int64_t tok, int h, int col, float4 v) {
  __nv_bfloat16* o = p.out + tok * p.o_ss + static_cast<int64_t>(h) * p.o_sh + col;
  *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

template <int D, int MT>
struct RowCfg {
  static constexpr int kRows = 16 * MT;
  static constexpr int kSlice = 16 * D * 2;                        // bytes of 16 keys (or values)
  static constexpr int kRing = kRowWarps * kRowStages * 2 * kSlice;  // also holds the warps' sums at the end
  static constexpr int kSums = kRowWarps * kRows * D * 4;
  static constexpr int kSmem = kRing > kSums ? kRing : kSums;
};

}  // namespace

template <int D, int MT, bool kScore>
__global__ void __launch_bounds__(kRowThreads, 2) k_chunk_rows(const ChunkParams p) {
  using C = RowCfg<D, MT>;
  extern __shared__ __align__(1024) uint8_t smem_rows[];
  __shared__ Piece pc_s;
  __shared__ int64_t warp_sums[kRowWarps];
  __shared__ float2 ml_s[kRowWarps][C::kRows];
  if (!find_piece<C::kRows, kRowKeys>(p, blockIdx.x, false, &pc_s, warp_sums)) return;
  const Piece& pc = pc_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q_len = pc.sp.q_len, kv = pc.sp.kv, q0 = pc.sp.q0;
  const int rows = q_len * p.G;  // served sequences: fits
  const int row0 = pc.rt * C::kRows;
  // keys that some row of the tile sees
  const int tok_a = row0 / p.G, tok_b = min(row0 + C::kRows, rows) - 1;
  const int pos_a = kv - q_len + tok_a, pos_b = kv - q_len + tok_b / p.G;
  const int lo_u = p.window >= 0 ? max(0, pos_a - p.window + 1) : 0, hi_u = min(kv, pos_b + 1);

  // this thread's rows: g + 8 i of each 16-row block
  int pos[MT][2], hi[MT][2], lo[MT][2];
  float slope[MT][2];
  uint32_t qf[MT][D / 16][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const __nv_bfloat16* qr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row0 + mt * 16 + (lane >> 2) + 8 * i;
      const bool in = r < rows;
      const int t = in ? r / p.G : 0;
      const int h = pc.hk * p.G + (in ? r - t * p.G : 0);
      pos[mt][i] = kv - q_len + t;
      hi[mt][i] = in ? min(kv, pos[mt][i] + 1) : 0;
      lo[mt][i] = p.window >= 0 ? max(0, pos[mt][i] - p.window + 1) : 0;
      slope[mt][i] = (kScore && p.score.slopes) ? __ldg(p.score.slopes + h) * kLog2e : 0.f;
      qr[i] = in ? p.q + (static_cast<int64_t>(q0) + t) * p.q_ss + static_cast<int64_t>(h) * p.q_sh : nullptr;
    }
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const int c = kk * 16 + (lane & 3) * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qf[mt][kk][i] = qr[i] ? *reinterpret_cast<const uint32_t*>(qr[i] + c) : 0u;
        qf[mt][kk][2 + i] = qr[i] ? *reinterpret_cast<const uint32_t*>(qr[i] + c + 8) : 0u;
      }
    }
  }

  // ring of this warp: stage st holds 16 keys, then their values
  uint8_t* const ring = smem_rows + warp * (kRowStages * 2 * C::kSlice);
  const uint32_t ring_u = smem_u32(ring);
  const int n = pc.t1 - pc.t0;
  const int kb0 = pc.t0 * kRowKeys + warp * 16;  // first key of slice 0
  const int32_t* bt = p.block_table + static_cast<int64_t>(pc.s) * p.pages_per_seq;
  constexpr int kChunks = D / 8;          // 16-byte chunks of a row
  constexpr int kPer = 32 / kChunks;      // rows a copy instruction covers
  // place in the cache of the lane's key of slice t (lanes 16..31 repeat), -1: none
  auto place = [&](int t) -> int64_t {
    const int key = kb0 + t * kRowKeys + (lane & 15);
    if (t >= n || key < lo_u || key >= hi_u) return -1;
    const int pi = key / p.page_size;
    const int64_t page = __ldg(bt + pi);
    if (page < 0 || page >= p.num_pages) return -1;
    return page * p.c_sp + static_cast<int64_t>(key - pi * p.page_size) * p.c_st;
  };
  auto issue = [&](int64_t at, int st) {
    const uint32_t dk = ring_u + st * 2 * C::kSlice, dv = dk + C::kSlice;
    const int64_t head = static_cast<int64_t>(pc.hk) * p.c_sh;
#pragma unroll
    for (int it = 0; it < 16 / kPer; ++it) {
      const int row = it * kPer + lane / kChunks, ch = lane % kChunks;
      const int64_t o = __shfl_sync(0xffffffffu, at, row);
      const uint32_t d = row * (D * 2) + ((ch ^ (row & 7)) << 4);
      const int64_t e = (o < 0 ? 0 : o) + head + ch * 8;
      cp_async16(dk + d, p.k_cache + e, o >= 0);
      cp_async16(dv + d, p.v_cache + e, o >= 0);
    }
  };

  float acc[MT][D / 8][4];
  float m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int d = 0; d < D / 8; ++d) acc[mt][d][0] = acc[mt][d][1] = acc[mt][d][2] = acc[mt][d][3] = 0.f;
    m[mt][0] = m[mt][1] = -INFINITY;
    l[mt][0] = l[mt][1] = 0.f;
  }
#pragma unroll
  for (int t = 0; t < kRowStages - 1; ++t) {
    if (t < n) issue(place(t), t);
    cp_async_commit();
  }
  int64_t at_next = place(kRowStages - 1);

  int st = 0;
  for (int t = 0; t < n; ++t) {
    cp_async_wait<kRowStages - 2>();
    __syncwarp();
    {  // refill the stage that the previous slice left
      const int tn = t + kRowStages - 1;
      const int sn = st == 0 ? kRowStages - 1 : st - 1;
      if (tn < n) issue(at_next, sn);
      cp_async_commit();
      at_next = place(tn + 1);
    }
    const uint32_t sk = ring_u + st * 2 * C::kSlice, sv = sk + C::kSlice;
    st = st + 1 == kRowStages ? 0 : st + 1;
    const int kb = kb0 + t * kRowKeys;
    if (kb >= hi_u || kb + 16 <= lo_u) continue;  // no row sees any of these keys

    // S = Q K^T: 16 keys in two blocks of 8
    float s[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 2; ++j) s[mt][j][0] = s[mt][j][1] = s[mt][j][2] = s[mt][j][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const int key = ((lane >> 4) << 3) + (lane & 7), ch = kk * 2 + ((lane >> 3) & 1);
      uint32_t b[4];
      ldsm4(sk + key * (D * 2) + ((ch ^ (key & 7)) << 4), b);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma16816(s[mt][0], qf[mt][kk], b[0], b[1]);
        mma16816(s[mt][1], qf[mt][kk], b[2], b[3]);
      }
    }
    uint32_t pf[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // shaped scores in log2 units; masked ones -inf
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e >> 1, key = kb + j * 8 + (lane & 3) * 2 + (e & 1);
          float z = s[mt][j][e];
          if constexpr (kScore) {
            z = p.score.c1 != 0.f ? p.score.c1 * tanh_any(z * p.score.c0) : z * p.scale_log2;
            z = fmaf(-slope[mt][i], static_cast<float>(pos[mt][i] - key), z);
          } else {
            z *= p.scale_log2;
          }
          s[mt][j][e] = (key >= lo[mt][i] && key < hi[mt][i]) ? z : -INFINITY;
        }
      float alpha[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmaxf(s[mt][0][2 * i], s[mt][0][2 * i + 1]), fmaxf(s[mt][1][2 * i], s[mt][1][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mnew = fmaxf(m[mt][i], mx);
        alpha[i] = mnew == m[mt][i] ? 1.f : ex2_approx(m[mt][i] - mnew);  // 0 from -inf
        m[mt][i] = mnew;
        const float mref = mnew == -INFINITY ? 0.f : mnew;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p0 = ex2_approx(s[mt][j][2 * i] - mref), p1 = ex2_approx(s[mt][j][2 * i + 1] - mref);
          sum += p0 + p1;
          pf[mt][2 * j + i] = pack_bf16x2(p0, p1);  // A fragment of P (rounded to bf16 as V is; the sum is not)
        }
        l[mt][i] = l[mt][i] * alpha[i] + sum;
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          acc[mt][d][0] *= alpha[0];
          acc[mt][d][1] *= alpha[0];
          acc[mt][d][2] *= alpha[1];
          acc[mt][d][3] *= alpha[1];
        }
      }
    }
    // O += P V
#pragma unroll
    for (int d2 = 0; d2 < D / 16; ++d2) {
      const int key = (((lane >> 3) & 1) << 3) + (lane & 7), ch = d2 * 2 + (lane >> 4);
      uint32_t b[4];
      ldsm4_t(sv + key * (D * 2) + ((ch ^ (key & 7)) << 4), b);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma16816(acc[mt][2 * d2], pf[mt], b[0], b[1]);
        mma16816(acc[mt][2 * d2 + 1], pf[mt], b[2], b[3]);
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();
  __syncthreads();  // every ring is done with: the warps' sums go over them

  float* const sums = reinterpret_cast<float*>(smem_rows) + static_cast<int64_t>(warp) * C::kRows * D;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[mt][i];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = mt * 16 + (lane >> 2) + 8 * i;
      if ((lane & 3) == 0) ml_s[warp][r] = make_float2(m[mt][i], sum);
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        *reinterpret_cast<float2*>(sums + r * D + d * 8 + (lane & 3) * 2) =
            make_float2(acc[mt][d][2 * i], acc[mt][d][2 * i + 1]);
    }
  __syncthreads();
  // merge the warps: thread -> (row, four columns)
  constexpr int kCols = D / 4;
  const float* const all = reinterpret_cast<const float*>(smem_rows);
  const int64_t seg = pc.seg0 + static_cast<int64_t>(pc.i) * pc.sp.rts;
  for (int e = threadIdx.x; e < C::kRows * kCols; e += kRowThreads) {
    const int r = e / kCols, c4 = (e % kCols) * 4;
    if (row0 + r >= rows) break;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, ml_s[w][r].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      const float2 ml = ml_s[w][r];
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
      const float4 a = *reinterpret_cast<const float4*>(all + (static_cast<int64_t>(w) * C::kRows + r) * D + c4);
      o.x = fmaf(a.x, f, o.x);
      o.y = fmaf(a.y, f, o.y);
      o.z = fmaf(a.z, f, o.z);
      o.w = fmaf(a.w, f, o.w);
      L = fmaf(ml.y, f, L);
    }
    if (pc.nseg == 1) {
      const int t = (row0 + r) / p.G, h = pc.hk * p.G + (row0 + r) - t * p.G;
      const float inv = L > 0.f ? 1.f / L : 0.f;
      store4(p, static_cast<int64_t>(q0) + t, h, c4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
      if (p.lse && c4 == 0) p.lse[static_cast<int64_t>(h) * p.total_q + q0 + t] = lse_of(M, L);
    } else if (seg < p.max_segs) {
      *reinterpret_cast<float4*>(p.ws_o + (seg * C::kRows + r) * D + c4) = o;
      if (c4 == 0) p.ws_ml[seg * C::kRows + r] = make_float2(M, L);
    }
  }
}

// Join the pieces of a unit: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,
// always in the order of the pieces.  A block takes 16 rows (blockIdx.y) of one unit.
template <int D, int R, int T>
__global__ void __launch_bounds__(128) k_chunk_join(const ChunkParams p) {
  __shared__ Piece pc_s;
  __shared__ int64_t warp_sums[4];
  if (!find_piece<R, T>(p, blockIdx.x, true, &pc_s, warp_sums)) return;
  const Piece& pc = pc_s;
  if (pc.nseg == 1) return;  // written by its only piece
  const int rows = pc.sp.q_len * p.G, row0 = pc.rt * R;
  constexpr int kCols = D / 4;
  for (int e = threadIdx.x; e < 16 * kCols; e += 128) {
    const int r = blockIdx.y * 16 + e / kCols, c4 = (e % kCols) * 4;
    if (row0 + r >= rows) break;
    float M = -INFINITY;
    for (int i = 0; i < pc.nseg; ++i) {
      const int64_t seg = pc.seg0 + static_cast<int64_t>(i) * pc.sp.rts;
      if (seg < p.max_segs) M = fmaxf(M, p.ws_ml[seg * R + r].x);
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
#pragma unroll 4
    for (int i = 0; i < pc.nseg; ++i) {
      const int64_t seg = pc.seg0 + static_cast<int64_t>(i) * pc.sp.rts;
      if (seg >= p.max_segs) break;
      const float2 ml = p.ws_ml[seg * R + r];
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
      const float4 a = *reinterpret_cast<const float4*>(p.ws_o + (seg * R + r) * D + c4);
      o.x = fmaf(a.x, f, o.x);
      o.y = fmaf(a.y, f, o.y);
      o.z = fmaf(a.z, f, o.z);
      o.w = fmaf(a.w, f, o.w);
      L = fmaf(ml.y, f, L);
    }
    const int t = (row0 + r) / p.G, h = pc.hk * p.G + (row0 + r) - t * p.G;
    const float inv = L > 0.f ? 1.f / L : 0.f;
    store4(p, static_cast<int64_t>(pc.sp.q0) + t, h, c4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (p.lse && c4 == 0) p.lse[static_cast<int64_t>(h) * p.total_q + pc.sp.q0 + t] = lse_of(M, L);
  }
}

// ----------------------------------------------------------------------------
// launchers (host)
// ----------------------------------------------------------------------------
cudaError_t launch_chunk_join(const ChunkParams& p, int rows, int keys, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.max_units), static_cast<unsigned>(rows / 16));
  const bool wide = p.D == 128;
  if (rows == 16 && keys == kRowKeys) {
    if (wide) k_chunk_join<128, 16, kRowKeys><<<grid, 128, 0, s>>>(p);
    else k_chunk_join<64, 16, kRowKeys><<<grid, 128, 0, s>>>(p);
  } else if (rows == 32 && keys == kRowKeys) {
    if (wide) k_chunk_join<128, 32, kRowKeys><<<grid, 128, 0, s>>>(p);
    else k_chunk_join<64, 32, kRowKeys><<<grid, 128, 0, s>>>(p);
  } else if (rows == kChunkTileRows && keys == kTile) {
    if (wide) k_chunk_join<128, kChunkTileRows, kTile><<<grid, 128, 0, s>>>(p);
    else k_chunk_join<64, kChunkTileRows, kTile><<<grid, 128, 0, s>>>(p);
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <int D, int MT, bool kScore>
static cudaError_t launch_rows_one(const ChunkParams& p, cudaStream_t s) {
  using C = RowCfg<D, MT>;
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(k_chunk_rows<D, MT, kScore>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (e != cudaSuccess) return e;
  k_chunk_rows<D, MT, kScore><<<p.max_segs, kRowThreads, C::kSmem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_chunk_join(p, C::kRows, kRowKeys, s);
}

template <int D, int MT>
static cudaError_t launch_rows_mt(const ChunkParams& p, cudaStream_t s) {
  return (p.score.c1 != 0.f || p.score.slopes) ? launch_rows_one<D, MT, true>(p, s)
                                               : launch_rows_one<D, MT, false>(p, s);
}

cudaError_t launch_chunk_rows(const ChunkParams& p, int row_tiles, cudaStream_t s) {
  if (p.max_segs <= 0 || p.max_units <= 0) return cudaSuccess;
  if (p.D == 64) return row_tiles == 1 ? launch_rows_mt<64, 1>(p, s) : launch_rows_mt<64, 2>(p, s);
  return row_tiles == 1 ? launch_rows_mt<128, 1>(p, s) : launch_rows_mt<128, 2>(p, s);
}

}  // namespace bfa
