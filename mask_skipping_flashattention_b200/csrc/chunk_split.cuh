// How the chunk kernels divide a ragged batch, computed on the device from the
// lengths there, so that the host needs none of them.
//
// A unit is (sequence, kv head, row tile): R rows of the sequence's new tokens x
// the G heads of the kv head (row r = token r / G, head r % G), with the key tiles
// (T keys) that some row of it sees.  The units in order (row tiles fastest) make
// one line of work, a unit's length being its key tiles plus a constant for starting
// it; block b of `slots` resident ones takes the b-th of equal shares, at least
// min_share long.  So every block has the same work whatever the batch looks like (one
// long sequence, many short ones, a causal triangle), and at most slots - 1 units are
// cut.  A block's part of a cut unit goes to the workspace: place 2 b if it starts
// inside the unit, 2 b + 1 if it starts it; and block b leaves a note of the cut in
// front of it, by which the join finds what to do.
// Measured on single tokens (32 / 8 heads, D 128): 64 ragged sequences of up to 8192 keys
// 170 us (0.96 of the measured copy rate), one of 32768 keys 34 us.  Before, with blocks that
// each looked up one of many pieces, no fixed number served both: 2 a SM took 199 and 40 us,
// 3 took 178 and 50, 8 took 178 and 88; a length chosen by a cost model took 203 and 46
// (every block paid for the search).
//
// The order along a unit's line only has to be the same everywhere, so lengths are a
// closed form of the row tile (line_before) and a cut at x of w falls on key tile
// n x / w of the unit's own n.
#pragma once

#include <cstdint>

#include "chunk_params.cuh"
#include "plan_types.cuh"

namespace bfa {

struct SeqSpan {
  int32_t q0, q_len;  // rows of q
  int32_t kv;         // keys
  int32_t rts;        // row tiles; 0: not served by this launch
};

struct Piece {
  SeqSpan sp;
  int32_t s, hk, rt;
  int32_t lo, hi;     // keys some row of the unit sees
  int32_t t0, t1;     // key tiles of the piece
  int32_t whole;      // the piece is its unit
  int32_t place;      // its place in the workspace otherwise
};

// The cut between blocks b - 1 and b, for the join.
struct Cut {
  int32_t pieces;      // pieces of the unit it goes through; 0: it goes through none
  int32_t index;       // number of this cut among the unit's
  int32_t hk, rt, q0;  // the unit; first row of its sequence in q
  int32_t rows;        // rows of its sequence's chunk (a kv head)
};
static_assert(sizeof(Cut) == kChunkCutBytes, "workspace size");

template <int R>
__device__ __forceinline__ SeqSpan seq_span(const ChunkParams& p, int s0) {
  SeqSpan sp;
  const int s = static_cast<int>(BFA_IDX(s0, p.B, p.err));
  // lengths outside their arrays are cut to them
  const int a = min(max(__ldg(p.cu_seqlens + s), 0), p.total_q);
  const int b = min(max(__ldg(p.cu_seqlens + s + 1), a), p.total_q);
  sp.q0 = a;
  sp.q_len = b - a;
  sp.kv = min(max(__ldg(p.seqused_k + s), 0), p.pages_per_seq * p.page_size);  // below 2^30
  const int rows = sp.q_len * p.G;                                              // below 2^23
  sp.rts = (rows > p.rows_lo && rows <= p.rows_hi) ? (rows + R - 1) / R : 0;
  return sp;
}

// length of the line before row tile rt of a sequence's kv head
template <int R, int T>
__device__ __forceinline__ int64_t line_before(const ChunkParams& p, const SeqSpan& sp, unsigned rt) {
  if (R == kChunkRows || p.window >= 0) {  // every unit alike: the window and its own tokens, or all keys
    const unsigned reach = p.window >= 0 ? min(sp.kv, p.window + min(sp.q_len, R / p.G + 1)) : sp.kv;
    return static_cast<int64_t>(rt) * (reach / T + 1 + p.start_cost);
  }
  // causal: unit i sees the keys before the chunk and R (i + 1) / G tokens of it (R = 2 T;
  // row tiles stay below 2^15)
  const unsigned before = max(sp.kv - sp.q_len, 0);
  return static_cast<int64_t>(rt) * (before / T + 1 + p.start_cost) + rt * (rt + 1u) / p.G;
}

// The line's length and where a block's share of it starts: equal shares to one tile.
struct Line {
  int64_t total, share;
  int32_t longer;  // the first blocks have one tile more
  __device__ __forceinline__ int64_t start(int b) const { return min(total, share * b + min(b, longer)); }
};

// Called by one whole warp (lanes = sequences).
template <int R, int T>
__device__ __forceinline__ Line line_of(const ChunkParams& p) {
  const int lane = threadIdx.x & 31;
  int64_t sum = 0;
#pragma unroll 1
  for (int s = lane; s < p.B; s += 32) {
    const SeqSpan sp = seq_span<R>(p, s);
    sum += line_before<R, T>(p, sp, sp.rts) * p.Hkv;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  Line ln;
  ln.total = sum;
  // total / slots in 32 bits (for lines past 2^32, coarser)
  const unsigned hi = static_cast<unsigned>(sum >> 32), slots = p.slots;
  if (hi) {
    ln.share = (static_cast<int64_t>(static_cast<unsigned>(sum >> 16) / slots) + 1) << 16;
    ln.longer = 0;
  } else {
    const unsigned q = static_cast<unsigned>(sum) / slots;
    ln.share = q;
    ln.longer = static_cast<unsigned>(sum) - q * slots;
  }
  if (ln.share < p.min_share) {
    ln.share = p.min_share;
    ln.longer = 0;
  }
  return ln;
}

// A place on the line: offset x of w in unit (s, hk, rt).
struct Walk {
  SeqSpan sp;
  int32_t s, hk, rt;
  int64_t x, w;
  template <int R, int T>
  __device__ __forceinline__ void set_unit(const ChunkParams& p) {
    w = line_before<R, T>(p, sp, rt + 1) - line_before<R, T>(p, sp, rt);
    x = 0;
  }
  // the next unit; false at the end of the batch
  template <int R, int T>
  __device__ __forceinline__ bool next(const ChunkParams& p) {
    if (++rt == sp.rts) {
      rt = 0;
      if (++hk == p.Hkv) {
        hk = 0;
        do {
          if (++s >= p.B) return false;
          sp = seq_span<R>(p, s);
        } while (sp.rts == 0);
      }
    }
    set_unit<R, T>(p);
    return true;
  }
};

// The unit at `pos` (below the line's length).  Called by one whole warp.
template <int R, int T>
__device__ __forceinline__ Walk walk_to(const ChunkParams& p, int64_t pos) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  Walk k;
  k.s = 0;
#pragma unroll 1
  for (int base = 0;; base += 32) {
    int64_t len = 0;
    if (base + lane < p.B) {
      const SeqSpan sp = seq_span<R>(p, base + lane);
      len = line_before<R, T>(p, sp, sp.rts) * p.Hkv;
    }
    int64_t end = len;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(kAll, end, d);
      if (lane >= d) end += x;
    }
    const unsigned past = __ballot_sync(kAll, pos < end);
    if (past || base + 32 >= p.B) {  // the second only guards against lengths that change under the call
      const int at = past ? __ffs(past) - 1 : min(31, p.B - 1 - base);
      k.s = base + at;
      pos -= __shfl_sync(kAll, end - len, at);
      break;
    }
    pos -= __shfl_sync(kAll, end, 31);
  }
  k.sp = seq_span<R>(p, k.s);
  const int64_t head = line_before<R, T>(p, k.sp, k.sp.rts);
  k.hk = 0;
  while (k.hk + 1 < p.Hkv && pos >= head) {
    pos -= head;
    ++k.hk;
  }
  int a = 0, b = max(k.sp.rts, 1);  // the last row tile in [a, b) with line_before <= pos
#pragma unroll 1
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (line_before<R, T>(p, k.sp, mid) <= pos) a = mid;
    else b = mid;
  }
  k.rt = a;
  const int64_t before = line_before<R, T>(p, k.sp, a);
  k.template set_unit<R, T>(p);
  k.x = min(pos - before, k.w - 1);
  return k;
}

// The cut in front of block b, whose share starts at k (`have`: it has one).
__device__ __forceinline__ void note_cut(const ChunkParams& p, const Walk& k, const Line& ln, int b, bool have) {
  Cut c = {};
  if (have && k.x > 0) {
    // cuts of the unit before this one, and behind it
    const int64_t first = ln.start(b) - k.x;
    int before = b - 1, behind = b + 1;
    while (before > 0 && ln.start(before) > first) --before;
    while (behind < p.slots && ln.start(behind) < first + k.w) ++behind;
    c.index = b - 1 - before;
    c.pieces = c.index + (behind - b) + 1;
    c.hk = k.hk;
    c.rt = k.rt;
    c.q0 = k.sp.q0;
    c.rows = k.sp.q_len * p.G;
  }
  static_cast<Cut*>(p.ws_cuts)[BFA_IDX(b, p.slots, p.err)] = c;
}

// Part [k.x, x1) of the unit at k as a piece of block b.
template <int R, int T>
__device__ __forceinline__ Piece piece_of(const ChunkParams& p, const Walk& k, int64_t x1, int b) {
  Piece pc;
  pc.sp = k.sp;
  pc.s = k.s;
  pc.hk = k.hk;
  pc.rt = k.rt;
  const int rows = k.sp.q_len * p.G, row0 = k.rt * R, first = k.sp.kv - k.sp.q_len;
  const int pos_a = first + row0 / p.G, pos_b = first + (min(row0 + R, rows) - 1) / p.G;
  pc.lo = p.window >= 0 ? max(0, pos_a - p.window + 1) : 0;
  pc.hi = min(k.sp.kv, pos_b + 1);
  const int t_lo = pc.lo / T, n = pc.hi > pc.lo ? (pc.hi + T - 1) / T - t_lo : 0;
  pc.whole = k.x == 0 && x1 == k.w;
  pc.place = 2 * b + (k.x == 0 ? 1 : 0);
  // n x / w: lengths stay far below 2^24, so a float quotient and its truncation are the same for
  // every block that asks for the same x
  const float step = static_cast<float>(n) / static_cast<float>(k.w);
  pc.t0 = t_lo + (k.x == 0 ? 0 : min(n, static_cast<int>(static_cast<float>(k.x) * step)));
  pc.t1 = t_lo + (x1 == k.w ? n : min(n, static_cast<int>(static_cast<float>(x1) * step)));
  // a unit of the batch, its keys inside the table, its place inside the workspace
  BFA_CHECK(pc.s >= 0 && pc.s < p.B && pc.hk >= 0 && pc.hk < p.Hkv && pc.rt >= 0 && row0 < rows, p.err);
  BFA_CHECK(pc.t0 <= pc.t1 && (n == 0 || static_cast<int64_t>(pc.hi) <= static_cast<int64_t>(p.pages_per_seq) * p.page_size),
            p.err);
  BFA_CHECK(pc.whole || (pc.place >= 0 && pc.place < 2 * p.slots), p.err);
  return pc;
}

}  // namespace bfa
