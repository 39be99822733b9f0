// Attention of the newest tokens of each sequence over a paged cache, for few
// query rows a kv head (single tokens, short chunks):
//   out_i = sum_j softmax_j(z_ij) v_j,  z = the shaped score of score.cuh,
// query token t of a sequence with kv keys at position kv - q_len + t, keys
// 0 <= j <= position (and position - j < window).
//
// Bound by HBM: a key and its value are 4 D bytes a kv head and meet only G query
// heads of a token.  A block runs one piece of the keys (chunk_split.cuh) for 16
// query rows of one kv head (rows = tokens x the G heads, so the group shares every
// byte).  Its four warps take 16 keys of a 64-key tile each, with a ring of
// asynchronous copies of their own, their own online softmax and no barrier
// between them until they are merged at the end; both products run on
// mma.sync m16n8k16 (bf16, fp32 sums), which at 16 rows is far from its limit.
// Cut units leave unnormalised fp32 sums, joined by k_chunk_join.
// Measured, 32 / 8 heads, D 128: 64 sequences of up to 8192 keys 170 us for the 1.074 GB of
// their keys and values (6.3 TB/s, 0.96 of the measured copy rate; 3 stages of 16 keys
// a warp and two blocks a SM keep 128 KB in flight); one sequence of 500 keys 9 us with
// the join, which is the latency of two launches, three dependent reads and the merge.
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

// four consecutive values of a row of the output
__device__ __forceinline__ void store4(const ChunkParams& p, int64_t tok, int h, int col, float4 v) {
  BFA_CHECK(h >= 0 && h < p.H, p.err);
  __nv_bfloat16* o = p.out + tok * p.o_ss + static_cast<int64_t>(h) * p.o_sh + col;
  *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

template <int D>
struct RowCfg {
  static constexpr int kSlice = 16 * D * 2;                          // bytes of 16 keys (or values)
  static constexpr int kRing = kRowWarps * kRowStages * 2 * kSlice;  // also holds the warps' sums at the end
  static constexpr int kSums = kRowWarps * kChunkRows * D * 4;
  static constexpr int kSmem = kRing > kSums ? kRing : kSums;
};

}  // namespace

template <int D, bool kScore>
__global__ void __launch_bounds__(kRowThreads, 2) k_chunk_rows(const ChunkParams p) {
  using C = RowCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_rows[];
  __shared__ Piece pc_s;
  __shared__ int have_s;
  __shared__ float2 ml_s[kRowWarps][kChunkRows];
  grid_trigger();  // the join may take the place of blocks that are done
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // warp 0 walks this block's share of the line (warp 1 leaves the note of its first cut)
  Walk walk;
  int64_t left = 0;
  bool more = false;
  if (warp <= 1) {
    const Line ln = line_of<kChunkRows, kRowKeys>(p);
    const int64_t pos = ln.start(blockIdx.x);
    left = ln.start(blockIdx.x + 1) - pos;
    more = left > 0;
    if (more) walk = walk_to<kChunkRows, kRowKeys>(p, pos);
    if (warp == 1 && lane == 0) note_cut(p, walk, ln, blockIdx.x, more);
  }
  for (;;) {
    if (warp == 0) {
      if (more) {
        const int64_t x1 = min(walk.w, walk.x + left);
        const Piece pc = piece_of<kChunkRows, kRowKeys>(p, walk, x1, blockIdx.x);
        left -= x1 - walk.x;
        if (lane == 0) pc_s = pc;
      }
      if (lane == 0) have_s = more;
      more = more && left > 0 && walk.template next<kChunkRows, kRowKeys>(p);
    }
    __syncthreads();
    if (!have_s) break;
    const Piece pc = pc_s;
    const int q_len = pc.sp.q_len, kv = pc.sp.kv, q0 = pc.sp.q0;
    const int rows = q_len * p.G;  // served sequences: fits
    const int row0 = pc.rt * kChunkRows;
    const int lo_u = pc.lo, hi_u = pc.hi;  // keys that some row of the unit sees

    // ring of this warp: stage st holds 16 keys, then their values
    const uint32_t ring_u = smem_u32(smem_rows + warp * (kRowStages * 2 * C::kSlice));
    const int n = pc.t1 - pc.t0;
    const int kb0 = pc.t0 * kRowKeys + warp * 16;  // first key of slice 0
    const int32_t* bt = p.block_table + static_cast<int64_t>(pc.s) * p.pages_per_seq;
    constexpr int kChunks = D / 8;      // 16-byte chunks of a row
    constexpr int kPer = 32 / kChunks;  // rows a copy instruction covers
    // place in the cache of the lane's key of slice t (lanes 16..31 repeat), -1: none
    auto place = [&](int t) -> int64_t {
      const int key = kb0 + t * kRowKeys + (lane & 15);
      if (t >= n || key < lo_u || key >= hi_u) return -1;
      const int pi = key / p.page_size;
      const int64_t page = __ldg(bt + BFA_IDX(pi, p.pages_per_seq, p.err));
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
    // the first copies go out before anything else is read
    int64_t at[kRowStages];
#pragma unroll
    for (int t = 0; t < kRowStages; ++t) at[t] = place(t);
#pragma unroll
    for (int t = 0; t < kRowStages - 1; ++t) {
      if (t < n) issue(at[t], t);
      cp_async_commit();
    }
    int64_t at_next = at[kRowStages - 1];

    // this thread's rows: lane / 4 + 8 i
    int pos[2], hi[2], lo[2];
    float slope[2];
    uint32_t qf[D / 16][4];
    {
      const __nv_bfloat16* qr[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row0 + (lane >> 2) + 8 * i;
        const bool in = r < rows;
        const int t = in ? r / p.G : 0;
        const int h = pc.hk * p.G + (in ? r - t * p.G : 0);
        pos[i] = kv - q_len + t;
        hi[i] = in ? min(kv, pos[i] + 1) : 0;
        lo[i] = p.window >= 0 ? max(0, pos[i] - p.window + 1) : 0;
        slope[i] = (kScore && p.score.slopes) ? __ldg(p.score.slopes + h) * kLog2e : 0.f;
        qr[i] = in ? p.q + BFA_IDX(static_cast<int64_t>(q0) + t, p.total_q, p.err) * p.q_ss + static_cast<int64_t>(h) * p.q_sh : nullptr;
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int c = kk * 16 + (lane & 3) * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qf[kk][i] = qr[i] ? *reinterpret_cast<const uint32_t*>(qr[i] + c) : 0u;
          qf[kk][2 + i] = qr[i] ? *reinterpret_cast<const uint32_t*>(qr[i] + c + 8) : 0u;
        }
      }
    }

    float acc[D / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < D / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;

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
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int key = ((lane >> 4) << 3) + (lane & 7), ch = kk * 2 + ((lane >> 3) & 1);
        uint32_t b[4];
        ldsm4(sk + key * (D * 2) + ((ch ^ (key & 7)) << 4), b);
        mma16816(s[0], qf[kk], b[0], b[1]);
        mma16816(s[1], qf[kk], b[2], b[3]);
      }
      // shaped scores in log2 units; masked ones -inf
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e >> 1, key = kb + j * 8 + (lane & 3) * 2 + (e & 1);
          float z = s[j][e];
          if constexpr (kScore) {
            z = p.score.c1 != 0.f ? capped_any(z, p.score) : z * p.scale_log2;
            z = fmaf(-slope[i], static_cast<float>(pos[i] - key), z);
          } else {
            z *= p.scale_log2;
          }
          s[j][e] = (key >= lo[i] && key < hi[i]) ? z : -INFINITY;
        }
      uint32_t pf[4];
      float alpha[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mnew = fmaxf(m[i], mx);
        alpha[i] = mnew == m[i] ? 1.f : ex2_approx(m[i] - mnew);  // 0 from -inf
        m[i] = mnew;
        const float mref = mnew == -INFINITY ? 0.f : mnew;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p0 = ex2_approx(s[j][2 * i] - mref), p1 = ex2_approx(s[j][2 * i + 1] - mref);
          sum += p0 + p1;
          pf[2 * j + i] = pack_bf16x2(p0, p1);  // A fragment of P (rounded to bf16 as V is; the sum is not)
        }
        l[i] = l[i] * alpha[i] + sum;
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          acc[d][0] *= alpha[0];
          acc[d][1] *= alpha[0];
          acc[d][2] *= alpha[1];
          acc[d][3] *= alpha[1];
        }
      }
      // O += P V
#pragma unroll
      for (int d2 = 0; d2 < D / 16; ++d2) {
        const int key = (((lane >> 3) & 1) << 3) + (lane & 7), ch = d2 * 2 + (lane >> 4);
        uint32_t b[4];
        ldsm4_t(sv + key * (D * 2) + ((ch ^ (key & 7)) << 4), b);
        mma16816(acc[2 * d2], pf, b[0], b[1]);
        mma16816(acc[2 * d2 + 1], pf, b[2], b[3]);
      }
      __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();  // every ring is done with: the warps' sums go over them

    float* const sums = reinterpret_cast<float*>(smem_rows) + warp * kChunkRows * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[i];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = (lane >> 2) + 8 * i;
      if ((lane & 3) == 0) ml_s[warp][r] = make_float2(m[i], sum);
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        *reinterpret_cast<float2*>(sums + r * D + d * 8 + (lane & 3) * 2) = make_float2(acc[d][2 * i], acc[d][2 * i + 1]);
    }
    __syncthreads();
    // merge the warps: thread -> (row, four columns)
    constexpr int kCols = D / 4;
    const float* const all = reinterpret_cast<const float*>(smem_rows);
    for (int e = threadIdx.x; e < kChunkRows * kCols; e += kRowThreads) {
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
        const float4 a = *reinterpret_cast<const float4*>(all + (w * kChunkRows + r) * D + c4);
        o.x = fmaf(a.x, f, o.x);
        o.y = fmaf(a.y, f, o.y);
        o.z = fmaf(a.z, f, o.z);
        o.w = fmaf(a.w, f, o.w);
        L = fmaf(ml.y, f, L);
      }
      if (pc.whole) {
        const int t = (row0 + r) / p.G, h = pc.hk * p.G + (row0 + r) - t * p.G;
        const float inv = L > 0.f ? 1.f / L : 0.f;
        store4(p, BFA_IDX(static_cast<int64_t>(q0) + t, p.total_q, p.err), h, c4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (p.lse && c4 == 0) p.lse[BFA_IDX(static_cast<int64_t>(h) * p.total_q + q0 + t, static_cast<int64_t>(p.H) * p.total_q, p.err)] = lse_of(M, L);
      } else {
        const int64_t at = BFA_IDX(static_cast<int64_t>(pc.place) * kChunkRows + r, 2LL * p.slots * kChunkRows, p.err);
        *reinterpret_cast<float4*>(p.ws_o + at * D + c4) = o;
        if (c4 == 0) p.ws_ml[at] = make_float2(M, L);
      }
    }
    __syncthreads();  // the sums and the piece are read
  }
  // Nothing here reads what the tile kernel before this one writes, but the join
  // behind waits for this kernel only: so this one does not end before that one.
  grid_wait();
}

// Join the pieces of the cut units: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// A unit of P pieces has P - 1 cuts, and each takes its share of the unit's rows (so
// every cut has about as much to join); `part` of `parts` blocks of a cut takes some of
// those.  It is all latency, so rows or pieces go side by side: four rows a warp at up to
// four pieces, a row a warp at up to 32 (lane i holds piece i's maximum), and beyond
// (a long sequence has hundreds) the block's warps share the pieces of a row.  The order
// of the sums depends on the number of pieces alone.
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;

template <int D>
struct JoinShared {
  float o[kJoinWarps][D];
  float l[kJoinWarps];
};

template <int D, int R>
__device__ __forceinline__ void join_cut(const ChunkParams& p, int cut, int part, int parts, JoinShared<D>* sh) {
  const Cut c = static_cast<const Cut*>(p.ws_cuts)[BFA_IDX(cut, p.slots, p.err)];
  if (c.pieces == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kV = D / 32;  // columns a lane
  const int row0 = c.rt * R, n = min(R, c.rows - row0), cuts = c.pieces - 1;
  const int first = cut - 1 - c.index;  // the block that starts the unit (its odd place); the others' even ones
  const int ra = n * c.index / cuts, rb = n * (c.index + 1) / cuts;
  BFA_CHECK(c.index >= 0 && c.index < cuts && first >= 0 && first + cuts < p.slots && n > 0, p.err);
  auto place = [&](int i, int r) {
    return static_cast<int64_t>(BFA_IDX(static_cast<int64_t>(i == 0 ? 2 * first + 1 : 2 * (first + i)) * R + r,
                                        2LL * p.slots * R, p.err));
  };
  // the lane's columns of a workspace row; the tile kernel's rows have their 16-byte chunks
  // swizzled by the row's place among 32
  auto load = [&](int64_t at, float (&a)[kV]) {
    const int mix = R == kChunkTileRows ? static_cast<int>(at) & (D / 4 - 1) & 31 : 0;
    if constexpr (kV == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p.ws_o + at * D + (lane ^ mix) * 4);
      a[0] = v.x; a[1] = v.y; a[2] = v.z; a[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p.ws_o + at * D + (((lane >> 1) ^ mix) << 2) + (lane & 1) * 2);
      a[0] = v.x; a[1] = v.y;
    }
  };
  auto store = [&](int r, const float (&o)[kV], float M, float L) {
    const int t = (row0 + r) / p.G, h = c.hk * p.G + (row0 + r) - t * p.G;
    const int64_t tok = BFA_IDX(static_cast<int64_t>(c.q0) + t, p.total_q, p.err);
    BFA_CHECK(h >= 0 && h < p.H, p.err);
    const float inv = L > 0.f ? 1.f / L : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + tok * p.o_ss + static_cast<int64_t>(h) * p.o_sh + lane * kV);
    if constexpr (kV == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
      *dst = pack_bf16x2(o[0] * inv, o[1] * inv);
    if (p.lse && lane == 0) p.lse[static_cast<int64_t>(h) * p.total_q + tok] = lse_of(M, L);
  };
  if (c.pieces <= 4) {
    for (int r4 = ra + (part * kJoinWarps + warp) * 4; r4 < rb; r4 += parts * kJoinWarps * 4) {
      // lane 8 r + i holds the maximum and sum of row r4 + r, piece i; a piece that saw no key
      // of a row left zeros
      const int lr = lane >> 3, li = lane & 7;
      const bool in = r4 + lr < rb && li < c.pieces;
      const float2 ml = in ? p.ws_ml[place(li, r4 + lr)] : make_float2(-INFINITY, 0.f);
      float a[4][4][kV];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r4 + r < rb && i < c.pieces) load(place(i, r4 + r), a[r][i]);
      float M = ml.x;
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float o[kV] = {}, L = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float fi = __shfl_sync(0xffffffffu, f, 8 * r + i);
          L = fmaf(__shfl_sync(0xffffffffu, ml.y, 8 * r + i), fi, L);
          if (r4 + r < rb && i < c.pieces) {
#pragma unroll
            for (int v = 0; v < kV; ++v) o[v] = fmaf(a[r][i][v], fi, o[v]);
          }
        }
        const float Mr = __shfl_sync(0xffffffffu, M, 8 * r);
        if (r4 + r < rb) store(r4 + r, o, Mr, L);
      }
    }
    return;
  }
  if (c.pieces <= 32) {
    constexpr int kSide = 8;
    for (int r = ra + part * kJoinWarps + warp; r < rb; r += parts * kJoinWarps) {
      const float2 ml = lane < c.pieces ? p.ws_ml[place(lane, r)] : make_float2(-INFINITY, 0.f);
      float o[kV] = {}, L = 0.f, M = ml.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
      for (int i0 = 0; i0 < c.pieces; i0 += kSide) {
        float a[kSide][kV];
#pragma unroll
        for (int i = 0; i < kSide; ++i)
          if (i0 + i < c.pieces) load(place(i0 + i, r), a[i]);
#pragma unroll
        for (int i = 0; i < kSide; ++i) {
          const float fi = __shfl_sync(0xffffffffu, f, (i0 + i) & 31);
          const float li = __shfl_sync(0xffffffffu, ml.y, (i0 + i) & 31);
          if (i0 + i < c.pieces) {
            L = fmaf(li, fi, L);
#pragma unroll
            for (int v = 0; v < kV; ++v) o[v] = fmaf(a[i][v], fi, o[v]);
          }
        }
      }
      store(r, o, M, L);
    }
    return;
  }
  for (int r = ra + part; r < rb; r += parts) {
    float M = -INFINITY, L = 0.f;
    float o[kV] = {};
    for (int i = lane; i < c.pieces; i += 32) M = fmaxf(M, p.ws_ml[place(i, r)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
#pragma unroll 8
    for (int i = warp; i < c.pieces; i += kJoinWarps) {
      const int64_t at = place(i, r);
      const float2 ml = p.ws_ml[at];
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
      float a[kV];
      load(at, a);
#pragma unroll
      for (int v = 0; v < kV; ++v) o[v] = fmaf(a[v], f, o[v]);
      L = fmaf(ml.y, f, L);
    }
    __syncthreads();  // the sums of the row before are read
#pragma unroll
    for (int v = 0; v < kV; ++v) sh->o[warp][lane * kV + v] = o[v];
    if (lane == 0) sh->l[warp] = L;
    __syncthreads();
    if (warp == 0) {
      L = 0.f;
#pragma unroll
      for (int v = 0; v < kV; ++v) o[v] = 0.f;
#pragma unroll
      for (int x = 0; x < kJoinWarps; ++x) {
        L += sh->l[x];
#pragma unroll
        for (int v = 0; v < kV; ++v) o[v] += sh->o[x][lane * kV + v];
      }
      store(r, o, M, L);
    }
  }
}

// Blocks [0, tile_blocks) join the tile kernel's units, the others the row kernel's.
constexpr int kJoinTileParts = 8, kJoinRowParts = 1;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    k_chunk_join(const ChunkParams row, const ChunkParams tile, int tile_blocks) {
  __shared__ JoinShared<D> sh;
  grid_wait();  // every block: what follows this kernel relies on the ones before it
  const int b = blockIdx.x, c = b - tile_blocks;
  if (b < tile_blocks) join_cut<D, kChunkTileRows>(tile, 1 + b / kJoinTileParts, b % kJoinTileParts, kJoinTileParts, &sh);
  else join_cut<D, kChunkRows>(row, 1 + c / kJoinRowParts, c % kJoinRowParts, kJoinRowParts, &sh);
}

// ----------------------------------------------------------------------------
// launchers (host)
// ----------------------------------------------------------------------------
// A launch that may start while the kernel before it still runs (grid_trigger).
template <typename K, typename... A>
static cudaError_t launch_dependent(K kernel, unsigned grid, int threads, int smem, bool dependent, cudaStream_t s,
                                    const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_chunk_join(const ChunkParams& row, const ChunkParams& tile, cudaStream_t s) {
  const int tile_blocks = tile.slots > 1 ? (tile.slots - 1) * kJoinTileParts : 0;
  const int row_blocks = row.slots > 1 ? (row.slots - 1) * kJoinRowParts : 0;
  if (tile_blocks + row_blocks == 0) return cudaSuccess;
  const unsigned blocks = static_cast<unsigned>(tile_blocks + row_blocks);
  if (row.D == 64) return launch_dependent(k_chunk_join<64>, blocks, kJoinThreads, 0, true, s, row, tile, tile_blocks);
  return launch_dependent(k_chunk_join<128>, blocks, kJoinThreads, 0, true, s, row, tile, tile_blocks);
}

template <int D, bool kScore>
static cudaError_t launch_rows_one(const ChunkParams& p, bool after_tiles, cudaStream_t s) {
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(k_chunk_rows<D, kScore>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                RowCfg<D>::kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_dependent(k_chunk_rows<D, kScore>, static_cast<unsigned>(p.slots), kRowThreads, RowCfg<D>::kSmem,
                          after_tiles, s, p);
}

cudaError_t launch_chunk_rows(const ChunkParams& p, bool after_tiles, cudaStream_t s) {
  const bool shaped = p.score.mode() != kScorePlain;
  if (p.D == 64) return shaped ? launch_rows_one<64, true>(p, after_tiles, s) : launch_rows_one<64, false>(p, after_tiles, s);
  return shaped ? launch_rows_one<128, true>(p, after_tiles, s) : launch_rows_one<128, false>(p, after_tiles, s);
}

}  // namespace bfa
