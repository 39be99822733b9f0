// How the chunk kernels divide a ragged batch, computed by every block from the
// lengths on the device, so that the host needs none of them.
//
// A unit is (sequence, kv head, row tile): R rows of the sequence's new tokens x
// the G heads of the kv head (row r = token r / G, head r % G).  Its keys, the
// tiles from the first that any new token sees to the last, are cut into pieces of
// nearly equal length; a block computes one piece.  The piece length is the
// batch's whole work over `slots`, so that few long sequences fill the machine as
// many short ones do.  Pieces are numbered by sequence, kv head, piece, row tile
// (the row tiles of one key range run together and share it in L2).
#pragma once

#include <cstdint>

#include "chunk_params.cuh"

namespace bfa {

struct SeqSpan {
  int32_t q0, q_len;   // rows of q
  int32_t kv;          // keys
  int32_t t_lo, n;     // first key tile and tiles (at least 1) of the whole chunk
  int32_t rts;         // row tiles; 0: not served by this launch
};

struct Piece {
  SeqSpan sp;
  int32_t s, hk, rt;
  int32_t t0, t1;      // key tiles
  int32_t nseg, i;     // pieces of the unit, this one's index
  int64_t seg0;        // piece i of the unit is number seg0 + i * sp.rts
};

template <int R, int T>
__device__ __forceinline__ SeqSpan seq_span(const ChunkParams& p, int s) {
  SeqSpan sp;
  // lengths outside their arrays are cut to them
  int a = min(max(__ldg(p.cu_seqlens + s), 0), p.total_q);
  int b = min(max(__ldg(p.cu_seqlens + s + 1), a), p.total_q);
  sp.q0 = a;
  sp.q_len = b - a;
  const int64_t room = static_cast<int64_t>(p.pages_per_seq) * p.page_size;
  sp.kv = static_cast<int>(min(static_cast<int64_t>(max(__ldg(p.seqused_k + s), 0)), room));
  const int64_t rows = static_cast<int64_t>(sp.q_len) * p.G;
  sp.rts = (rows > p.rows_lo && rows <= p.rows_hi) ? static_cast<int>((rows + R - 1) / R) : 0;
  int lo = p.window >= 0 ? max(0, sp.kv - sp.q_len - p.window + 1) : 0;
  lo = min(lo, sp.kv);
  sp.t_lo = lo / T;
  sp.n = max(1, (sp.kv + T - 1) / T - sp.t_lo);
  return sp;
}

// Inclusive scan over the block's threads (a multiple of 32, at most 512).
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += x;
  }
  __syncthreads();  // the sums of a scan before may still be read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int w = 0; w < warps; ++w) {
    const int64_t x = warp_sums[w];
    if (w < warp) before += x;
    total += x;
  }
  return v + before;
}

// The piece `want` (or, with `units`, the unit `want` as a piece with i = 0) into
// shared memory; false when there is none.  Called by the whole block.
template <int R, int T>
__device__ bool find_piece(const ChunkParams& p, int64_t want, bool units, Piece* out, int64_t* warp_sums) {
  const int tid = threadIdx.x, nt = blockDim.x;
  int64_t work = 0, total = 0;
  SeqSpan sp;
  for (int base = 0; base < p.B; base += nt) {
    int64_t w = 0;
    if (base + tid < p.B) {
      sp = seq_span<R, T>(p, base + tid);
      w = static_cast<int64_t>(sp.n) * sp.rts * p.Hkv;
    }
    block_scan(w, warp_sums, total);
    work += total;
  }
  const int64_t per = max(static_cast<int64_t>(p.min_tiles), (work + p.slots - 1) / p.slots);
  int64_t done_units = 0, done_segs = 0;
  __shared__ int found;
  if (tid == 0) found = 0;
  for (int base = 0; base < p.B; base += nt) {
    int64_t nu = 0, ns = 0;
    int nseg = 1;
    if (base + tid < p.B) {
      if (p.B > nt) sp = seq_span<R, T>(p, base + tid);
      nseg = static_cast<int>((sp.n + per - 1) / per);
      nu = static_cast<int64_t>(sp.rts) * p.Hkv;
      ns = nu * nseg;
    }
    int64_t units_here, segs_here;
    const int64_t eu = done_units + block_scan(nu, warp_sums, units_here) - nu;
    const int64_t es = done_segs + block_scan(ns, warp_sums, segs_here) - ns;
    const int64_t e = units ? eu : es, cnt = units ? nu : ns;
    if (want >= e && want < e + cnt) {
      Piece pc;
      pc.sp = sp;
      pc.s = base + tid;
      pc.nseg = nseg;
      const int64_t local = want - e;
      pc.rt = static_cast<int>(local % sp.rts);
      const int64_t rest = local / sp.rts;
      pc.i = units ? 0 : static_cast<int>(rest % nseg);
      pc.hk = static_cast<int>(units ? rest : rest / nseg);
      pc.t0 = sp.t_lo + static_cast<int>(static_cast<int64_t>(sp.n) * pc.i / nseg);
      pc.t1 = sp.t_lo + static_cast<int>(static_cast<int64_t>(sp.n) * (pc.i + 1) / nseg);
      pc.seg0 = es + (static_cast<int64_t>(pc.hk) * nseg) * sp.rts + pc.rt;
      *out = pc;
      found = 1;
    }
    done_units += units_here;
    done_segs += segs_here;
    if (want < (units ? done_units : done_segs)) break;  // the same for every thread
  }
  __syncthreads();
  return found != 0;
}

}  // namespace bfa
