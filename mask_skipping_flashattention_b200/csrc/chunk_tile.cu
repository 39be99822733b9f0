// Attention of the newest tokens over a paged cache (chunk.cu) for sequences with
// many query rows a kv head: pieces of a prompt.
//
// Bound by the tensor core and the exponentials, as the planned forward is, and
// built as it is (fwd.cu: two 128-row slots a CTA that share every key tile,
// S = Q K^T and O += P V as tcgen05 products with S, P and O in tensor memory, one
// query row a softmax thread).  What differs:
//   - a unit is 256 rows (tokens x the G heads of a kv head) of one sequence with
//     the key tiles that its rows see, and one CTA a SM stays resident and works off an
//     equal share of all units' tiles (chunk_split.cuh), at most its first and last
//     unit in part; both slots walk all tiles, since their rows are at most 256 / G
//     tokens apart.  The barriers' phases run on from piece to piece;
//   - Q rows go from global memory into the swizzled tile by the softmax threads,
//     one row each: any G, any strides, rows past the end as zeros;
//   - the producer warp loads a tile page by page, one page a lane, with the page
//     ids of the next tile already in registers; pages that do not exist are
//     loaded from past the cache's end, which reads as zeros;
//   - value rows outside the unit's keys (the rest of the last page, the keys before a
//     window) are zeroed in shared memory before the product reads them, since a
//     weight of 0 does not cancel a NaN there; scores of such keys are masked.
// P is rounded to bf16 for P V, as V is given in it (at most 2^-8 of each weight; the
// sum of the weights is taken before); statistics, sums and the parts of cut units stay in fp32.
// Measured: 2048 new tokens behind 14336, 32 / 8 heads, D 128, 421 to 425 us with the join in a
// burst of ten calls = 1.21 to 1.23 PFLOP/s (0.73 of the measured burst peak; tensor pipe 61 %
// active, exponentials 61 %), 487 us in a row of calls, which the power cap slows; a step of two
// slots takes 2 us, a piece 2 us to its first scores and 4 to 7 us to end.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "chunk_params.cuh"
#include "chunk_split.cuh"
#include "device_once.cuh"
#include "fwd_tiles.cuh"
#include "plan_types.cuh"
#include "ptx.cuh"
#include "score.cuh"

namespace bfa {

using namespace ptx;

namespace {

constexpr int kUnitRows = kChunkTileRows;
static_assert(kUnitRows == 2 * kTile, "two slots");

struct TileWork {
  Piece pc;
  int32_t have;         // 0: no more pieces
  int32_t rows, row0;   // rows of the sequence's chunk (a kv head), first row of the unit
  int32_t n;            // key tiles of this piece
  int32_t two;          // slot 1 has rows
};

}  // namespace

template <int D, int kScore>
__global__ void __launch_bounds__(kThreads, 1)
    k_chunk_tiles(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const ChunkParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sQ0 = smem;
  uint8_t* const sQ1 = smem + C::kTileBytes;
  uint8_t* const sK0 = smem + 2 * C::kTileBytes;
  uint8_t* const sV0 = smem + (2 + kStages) * C::kTileBytes;

  // BQ: Q rows written (8 softmax warps) and the first K.  BF[2]: V(j) and K(j + 1).
  // BE[2]: stages free.  BS[2] / BP[2]: S ready / P ready per slot.  BY: the MMA
  // thread is at an edge tile whose values have landed; BZ: their rows outside the
  // unit's keys are zeroed (one edge tile at a time).  BO: all products done.
  enum { BQ = 0, BF = 1, BE = 3, BS = 5, BP = 7, BY = 9, BZ = 10, BO = 11, BDONE = 12, NBAR = 13 };
  __shared__ __align__(8) uint64_t bars[NBAR];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ TileWork wk_s[2];  // this piece and the next one

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto sK = [&](int st) { return sK0 + st * C::kTileBytes; };
  auto sV = [&](int st) { return sV0 + st * C::kTileBytes; };
  // the block between two pieces: nothing of the last one is in flight, the next one is known
  auto meet = [&]() {
    tc_fence_before();
    named_bar_sync(0, kThreads);
    tc_fence_after();
  };

  grid_trigger();  // the row kernel, or the join, may take the place of blocks that are done
  // warp 3 walks this block's share of the line, a piece ahead of the others
  Walk walk, first_at;
  Line first_line;
  int64_t left = 0;
  bool more = false;
  auto post_piece = [&](TileWork& w) {
    if (more) {
      const int64_t x1 = min(walk.w, walk.x + left);
      const Piece pc = piece_of<kUnitRows, kTile>(p, walk, x1, blockIdx.x);
      left -= x1 - walk.x;
      if (lane == 0) {
        w.pc = pc;
        w.rows = pc.sp.q_len * p.G;
        w.row0 = pc.rt * kUnitRows;
        w.n = pc.t1 - pc.t0;
        w.two = pc.rt * kUnitRows + kTile < pc.sp.q_len * p.G;
      }
    }
    if (lane == 0) w.have = more;
    more = more && left > 0 && walk.template next<kUnitRows, kTile>(p);
  };
  if (warp == 3) {
    const Line ln = line_of<kUnitRows, kTile>(p);
    const int64_t pos = ln.start(blockIdx.x);
    left = ln.start(blockIdx.x + 1) - pos;
    more = left > 0;
    if (more) walk = walk_to<kUnitRows, kTile>(p, pos);
    first_at = walk;
    first_line = ln;
    post_piece(wk_s[0]);
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < NBAR; ++i) mbar_init(bar(i), i == BQ ? 9 : ((i == BP || i == BP + 1) ? 4 : 1));
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  meet();
  if (warp == 3 && lane == 0) note_cut(p, first_at, first_line, blockIdx.x, wk_s[0].have);
  const uint32_t tmem = tmem_slot;
  const uint64_t cap = p.wait_ns;
  // what the barriers have seen before this piece: pieces with tiles, tiles (F), commits of E,
  // tiles of each slot, edge tiles.  Every role counts for itself, all alike.
  int c_piece = 0, c_f = 0, c_e = 0, c_s1 = 0, c_z = 0;
  int cur = 0;  // this piece's half of wk_s
  auto count_piece = [&](int n, int two) {
    if (n > 0) {
      ++c_piece;
      c_f += n;
      c_e += n + 1;
      c_s1 += two ? n : 0;
    }
    cur ^= 1;
  };

  // a tile with value rows that no row of the unit may read
  auto edge = [&](const TileWork& wk, int j) {
    const int k0 = (wk.pc.t0 + j) * kTile;
    return k0 < wk.pc.lo || k0 + kTile > wk.pc.hi;
  };

  if (warp < 4) {
    // ============================================================ warpgroup 0
    regs_dec<kRegsWG0>();
    while (wk_s[cur].have) {
      const TileWork& wk = wk_s[cur];
      const int n = wk.n, two_slots = wk.two;
      if (warp == 3) post_piece(wk_s[cur ^ 1]);
      if (warp == 0 && n > 0) {
        // -------------------------------------------------------- producer
        // K of the first tile on BQ; at step j, V of tile j and K of tile j + 1 on the
        // stage of j once commit j - 1 has freed both.  Lane l loads page l of a tile (one
        // lane for pages of 128 tokens and more).
        if (lane == 0) {
          prefetch_tmap(&tmK);
          prefetch_tmap(&tmV);
        }
        const int box = min(p.page_size, kTile);
        const int boxes = kTile / box;
        const int32_t* bt = p.block_table + static_cast<int64_t>(wk.pc.s) * p.pages_per_seq;
        const int past = static_cast<int>(p.num_pages * p.page_size);  // a row outside the cache reads as zeros
        // row of the cache of this lane's box of tile j
        auto place = [&](int j) -> int {
          const int key = (wk.pc.t0 + j) * kTile + lane * box;
          if (lane >= boxes || j >= n || key >= wk.pc.hi || key + box <= wk.pc.lo) return past;
          const int pi = key / p.page_size;
          const int page = __ldg(bt + BFA_IDX(pi, p.pages_per_seq, p.err));
          return (page < 0 || page >= p.num_pages) ? past : page * p.page_size + (key - pi * p.page_size);
        };
        auto load = [&](const CUtensorMap* map, uint8_t* dst, uint32_t b, int row) {
          if (lane < boxes) {
#pragma unroll
            for (int pn = 0; pn < C::kPanels; ++pn)
              tma_load_4d(smem_u32(dst + pn * 16384 + lane * box * 128), map, b, pn * 64, wk.pc.hk, row, 0);
          }
        };
        int row = place(0);
        if (lane == 0) mbar_expect_tx(bar(BQ), C::kTileBytes);
        __syncwarp();
        load(&tmK, sK(c_f & 1), bar(BQ), row);
        int row_n = place(1);
        int last = -1;
        for (int j = 0; j < n; ++j) {
          const int row_nn = place(j + 2);
          const int f = c_f + j, e = c_e + j - 1;
          bool ok = true;
          if (lane == 0 && j >= 1) ok = mbar_wait_fast(bar(BE + (e & 1)), (e >> 1) & 1, cap, &abort_flag);
          if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
          const uint32_t fb = bar(BF + (f & 1));
          const bool have_next = j + 1 < n;
          if (lane == 0) mbar_expect_tx(fb, (have_next ? 2 : 1) * C::kTileBytes);
          __syncwarp();
          load(&tmV, sV(f & 1), fb, row);
          if (have_next) load(&tmK, sK((f + 1) & 1), fb, row_n);
          last = f;
          row = row_n;
          row_n = row_nn;
        }
        // every copy of this piece must land before the block goes on or exits
        if (lane == 0) {
          mbar_drain(bar(BQ), c_piece & 1, &abort_flag);
          if (last > c_f) mbar_drain(bar(BF + ((last - 1) & 1)), ((last - 1) >> 1) & 1, &abort_flag);
          if (last >= 0) mbar_drain(bar(BF + (last & 1)), (last >> 1) & 1, &abort_flag);
        }
        __syncwarp();
      } else if (warp == 1 && lane == 0 && n > 0) {
        // -------------------------------------------------------- MMA issuer (fwd.cu's order)
        const uint32_t tS0 = tmem + C::kColS0, tS1 = tmem + C::kColS1;
        const uint32_t tO0 = tmem + C::kColO0, tO1 = tmem + C::kColO1;
        const bool two = wk.two != 0;
        int z = c_z;
        bool ok = mbar_wait_fast(bar(BQ), c_piece & 1, cap, &abort_flag);
        if (ok) {
          tc_fence_after();
          issue_s<D>(tS0, sQ0, sK(c_f & 1));
          umma_commit(bar(BS + 0));
          if (two) {
            issue_s<D>(tS1, sQ1, sK(c_f & 1));
            umma_commit(bar(BS + 1));
          }
          umma_commit(bar(BE + (c_e & 1)));
        }
        for (int u = 0; ok && u < n; ++u) {
          const int f = c_f + u, st = f & 1, st1 = st ^ 1;
          const bool have_next = u + 1 < n;
          if (!mbar_wait_fast(bar(BF + st), (f >> 1) & 1, cap, &abort_flag)) { ok = false; break; }
          if (edge(wk, u)) {
            mbar_arrive(bar(BY));
            if (!mbar_wait_fast(bar(BZ), z & 1, cap, &abort_flag)) { ok = false; break; }
            ++z;
          }
          if (!mbar_wait_fast(bar(BP + 0), f & 1, cap, &abort_flag)) { ok = false; break; }
          tc_fence_after();
          issue_pv<D>(tO0, tS0, sV(st), u > 0);
          if (have_next) {
            issue_s<D>(tS0, sQ0, sK(st1));
            umma_commit(bar(BS + 0));
          }
          if (two) {
            if (!mbar_wait_fast(bar(BP + 1), (c_s1 + u) & 1, cap, &abort_flag)) { ok = false; break; }
            tc_fence_after();
            issue_pv<D>(tO1, tS1, sV(st), u > 0);
            if (have_next) {
              issue_s<D>(tS1, sQ1, sK(st1));
              umma_commit(bar(BS + 1));
            }
          }
          umma_commit(bar(BE + ((c_e + u + 1) & 1)));
        }
        if (ok) umma_commit(bar(BO));
        // every MMA issued must be finished before the tiles or TMEM are used again (bounded)
        umma_commit(bar(BDONE));
        mbar_drain(bar(BDONE), c_piece & 1, &abort_flag);
        c_z = z;
      } else if (warp == 2 && n > 0) {
        // -------------------------------------------------------- value rows outside the unit's keys
        for (int j = 0; j < n; ++j) {
          if (!edge(wk, j)) continue;
          // the MMA thread waits at this tile, so its stage's phase cannot move on
          const int f = c_f + j;
          bool got = mbar_wait(bar(BY), c_z & 1, cap, &abort_flag);
          got = got && mbar_wait(bar(BF + (f & 1)), (f >> 1) & 1, cap, &abort_flag);
          if (__any_sync(0xffffffffu, !got)) break;
          ++c_z;
          const int k0 = (wk.pc.t0 + j) * kTile;
          for (int i = lane; i < kTile * 8; i += 32) {  // 16-byte chunk i % 8 of row i / 8 of each panel
            const int key = k0 + (i >> 3);
            if (key >= wk.pc.lo && key < wk.pc.hi) continue;
#pragma unroll
            for (int pn = 0; pn < C::kPanels; ++pn)
              st_shared_v4(smem_u32(sV(f & 1)) + pn * 16384 + i * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BZ));
        }
      }
      __syncwarp();
      count_piece(n, two_slots);
      meet();
      if (*static_cast<volatile int*>(&abort_flag)) break;  // waits are over: the same for every thread
      meet();
    }
  } else {
    // ============================================================ softmax warpgroups
    regs_inc<kRegsSoftmax>();
    const int slot = (warp >> 2) - 1;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t tS = tmem_addr(tmem + (slot ? C::kColS1 : C::kColS0), quarter * 32, 0);
    const uint32_t tO = tmem_addr(tmem + (slot ? C::kColO1 : C::kColO0), quarter * 32, 0);
    const uint32_t barS = bar(BS + slot), barP = bar(BP + slot);
    while (wk_s[cur].have) {
      const TileWork& wk = wk_s[cur];
      const int n = wk.n, two_slots = wk.two;
      const int r = wk.row0 + slot * kTile + row;  // row of the chunk: token r / G, head r % G
      const bool valid = r < wk.rows;
      const int q_len = wk.pc.sp.q_len, kv = wk.pc.sp.kv;
      const int tok = valid ? r / p.G : 0;
      const int h = wk.pc.hk * p.G + (valid ? r - tok * p.G : 0);
      const int pos = kv - q_len + tok;
      // keys [lo, hi) of this row; rows past the end see everything (their Q is 0, nothing of them is kept)
      const int hi = valid ? min(kv, pos + 1) : 0x7fffffff;
      const int lo = valid && p.window >= 0 ? max(0, pos - p.window + 1) : 0;
      if (n > 0) {
        // The warp's 32 rows of Q into the swizzled tile (K-major operand of S), whole rows
        // at a time: a row a thread would touch 32 lines an instruction.
        constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte chunks of a row, rows an instruction
        const uint32_t tile = smem_u32(slot ? sQ1 : sQ0);
        const int c16 = lane % kChunks;
        const __nv_bfloat16* src = p.q + BFA_IDX(static_cast<int64_t>(wk.pc.sp.q0) + tok, p.total_q, p.err) * p.q_ss + static_cast<int64_t>(h) * p.q_sh;
        const uint64_t at = valid ? reinterpret_cast<uint64_t>(src) : 0;  // of this lane's row
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 v[16 / kPer];
#pragma unroll
          for (int i = 0; i < 16 / kPer; ++i) {
            const uint64_t row_at = __shfl_sync(0xffffffffu, at, half * 16 + i * kPer + lane / kChunks);
            v[i] = row_at ? *(reinterpret_cast<const uint4*>(row_at) + c16) : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < 16 / kPer; ++i) {
            const int tr = quarter * 32 + half * 16 + i * kPer + lane / kChunks;
            st_shared_v4(tile + (c16 >> 3) * 16384 + tr * 128 + (((c16 & 7) ^ (tr & 7)) << 4), v[i].x, v[i].y, v[i].z,
                         v[i].w);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BQ));
      }
      if (slot == 0 || wk.two) {
        const float c = kScore ? 1.f : p.scale_log2;
        float slope = 0.f;
        if constexpr ((kScore & kScoreSlopes) != 0) slope = __ldg(p.score.slopes + h) * kLog2e;
        // keys that every row of the warp sees: tiles inside need no mask
        const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
        const int c_s = slot ? c_s1 : c_f;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int t = 0; t < n; ++t) {
          const int k0 = (wk.pc.t0 + t) * kTile;
          const bool got = mbar_wait(barS, (c_s + t) & 1, cap, &abort_flag);
          if (__any_sync(0xffffffffu, !got)) { ok = false; break; }  // warp-uniform exit
          tc_fence_after();
          uint32_t sr[128];
          tmem_ld_32x32b_x32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_ld_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tmem_ld_32x32b_x32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
          tmem_ld_32x32b_x32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
          tmem_wait_ld();
          reg_fence(sr);
          float* s = reinterpret_cast<float*>(sr);
          if constexpr (kScore != 0) shape_row<kScore>(s, p.score, p.scale_log2, slope, pos - k0, true);
          if (k0 < all_lo || k0 + kTile > all_hi) {
            // keys [lo, hi) of the row as attend-bits, 32 to a word
            uint32_t am[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int a = lo - k0 - 32 * w, z = hi - k0 - 32 * w;
              const uint32_t from = a <= 0 ? 0xffffffffu : (a > 31 ? 0u : ~((1u << a) - 1u));
              const uint32_t to = z >= 32 ? 0xffffffffu : (z <= 0 ? 0u : ((1u << z) - 1u));
              am[w] = from & to;
            }
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (!((am[j >> 5] >> (j & 31)) & 1u)) s[j] = -INFINITY;
          }
          float mx8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mx8[i] = s[i];
#pragma unroll
          for (int j = 8; j < 128; j += 2) mx8[(j >> 1) & 7] = fmax3(mx8[(j >> 1) & 7], s[j], s[j + 1]);
          const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                 fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
          const float mnew = fmaxf(m, mx * c);
          // lazy rescale of O, decided by the whole warp (fwd.cu)
          if (__any_sync(0xffffffffu, mnew > m + kRescaleThreshold)) {
            const float alpha = (mnew == m) ? 1.f : ex2_approx(m - mnew);  // 0 when m = -inf
            l *= alpha;
            if (t > 0) {
#pragma unroll 1
              for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(tO + cc * 32, o);
                tmem_wait_ld();
                reg_fence(o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                tmem_st_32x32b_x32(tO + cc * 32, o);
              }
            }
            m = mnew;
          }
          const float mref = (m == -INFINITY) ? 0.f : m;
          uint64_t rs2[4] = {0, 0, 0, 0};
          const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-mref, -mref);
          uint32_t pk[64];
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            const uint64_t x2 = f2_fma(f2_pack(s[2 * j], s[2 * j + 1]), c2, nm2);
            float x0, x1;
            f2_unpack(x2, x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            rs2[j & 3] = f2_add(rs2[j & 3], f2_pack(p0, p1));
            pk[j] = pack_bf16x2(p0, p1);
          }
          float rr[8];
          f2_unpack(f2_add(rs2[0], rs2[1]), rr[0], rr[1]);
          f2_unpack(f2_add(rs2[2], rs2[3]), rr[2], rr[3]);
          l += (rr[0] + rr[2]) + (rr[1] + rr[3]);
          tmem_st_32x32b_x32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
          tmem_st_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(barP);
        }
        // -------------------------------------------------------- epilogue
        if (ok && n > 0) {
          const bool got = mbar_wait(bar(BO), c_piece & 1, cap, &abort_flag);
          ok = !__any_sync(0xffffffffu, !got);
        }
        tc_fence_after();
        if (ok) {
          // The rows leave through shared memory (every product is done, so all of it but the
          // other warps' parts is free), 16-byte chunks swizzled by the row so that neither
          // side meets in a bank.  Direct stores, a row a thread, took 5 us.
          const bool whole = wk.pc.whole != 0;
          const float inv = l > 0.f ? 1.f / l : 0.f;
          const int64_t gtok = BFA_IDX(static_cast<int64_t>(wk.pc.sp.q0) + tok, p.total_q, p.err);
          const int64_t wr = BFA_IDX(static_cast<int64_t>(wk.pc.place) * kUnitRows + slot * kTile + row,
                                     2LL * p.slots * kUnitRows, p.err);
          BFA_CHECK(h >= 0 && h < p.H, p.err);
          // this warp's 32 rows: bf16 in the slot's Q tile, fp32 in a K or V stage pair
          constexpr int kWide = D / 4;  // 16-byte chunks of an fp32 row
          const uint32_t stg = whole ? smem_u32(slot ? sQ1 : sQ0) + quarter * 32 * D * 2
                                     : smem_u32(sK0) + (slot * kTile + quarter * 32) * D * 4;
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            if (n > 0) {
              tmem_ld_32x32b_x32(tO + cc * 32, o);
              tmem_wait_ld();
              reg_fence(o);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = 0u;
            }
            if (whole) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = pack_bf16x2(__uint_as_float(o[8 * j + 2 * e]) * inv, __uint_as_float(o[8 * j + 2 * e + 1]) * inv);
                st_shared_v4(stg + lane * D * 2 + (((cc * 4 + j) ^ (lane & (D / 8 - 1))) << 4), w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                st_shared_v4(stg + lane * D * 4 + (((cc * 8 + j) ^ (lane & (kWide - 1))) << 4), o[4 * j], o[4 * j + 1],
                             o[4 * j + 2], o[4 * j + 3]);
            }
          }
          if (whole) {
            __syncwarp();
            constexpr int kChunks = D / 8, kPer = 32 / kChunks;
            const int c16 = lane % kChunks;
            const uint64_t at = valid ? reinterpret_cast<uint64_t>(p.out + gtok * p.o_ss + static_cast<int64_t>(h) * p.o_sh) : 0;
#pragma unroll 8
            for (int i = 0; i < 32 / kPer; ++i) {
              const int wrow = i * kPer + lane / kChunks;
              const uint64_t row_at = __shfl_sync(0xffffffffu, at, wrow);
              const float4 v = ld_shared_f4(stg + wrow * D * 2 + ((c16 ^ (wrow & (kChunks - 1))) << 4));
              if (row_at) *(reinterpret_cast<float4*>(row_at) + c16) = v;
            }
            if (valid && p.lse) p.lse[static_cast<int64_t>(h) * p.total_q + gtok] = lse_of(m, l);
          } else {
            // the swizzled rows go to the workspace as they are (the join undoes it)
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              bulk_store(p.ws_o + (wr - row + quarter * 32) * D, stg, 32 * D * 4);
              bulk_commit_group();
            }
            p.ws_ml[wr] = make_float2(m, l);
            if (lane == 0) bulk_wait_group_read0();  // the stages are the next piece's
            __syncwarp();
          }
        }
      }
      count_piece(n, two_slots);
      meet();
      if (*static_cast<volatile int*>(&abort_flag)) break;
      meet();
    }
  }

  // ------------------------------------------------------------ teardown
  bulk_wait_group0();  // the workspace is written before the join may read it
  tc_fence_before();
  __syncthreads();
  if (abort_flag && threadIdx.x == 0) atomicOr(p.err, DEVERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ----------------------------------------------------------------------------
// launcher (host)
// ----------------------------------------------------------------------------
template <int D, int kScore>
static cudaError_t launch_tiles_one(const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& p, cudaStream_t s) {
  static DeviceOnce once;
  const cudaError_t ready = once.run([] {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, k_chunk_tiles<D, kScore>);
    if (e != cudaSuccess) return e;
    // the setmaxnreg split is only safe with exactly this many registers a thread
    if (a.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;
    return cudaFuncSetAttribute(k_chunk_tiles<D, kScore>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<D>::kSmemBytes);
  });
  if (ready != cudaSuccess) return ready;
  k_chunk_tiles<D, kScore><<<p.slots, kThreads, Cfg<D>::kSmemBytes, s>>>(tk, tv, p);
  return cudaGetLastError();
}

cudaError_t launch_chunk_tiles(const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& p, cudaStream_t s) {
  return for_score_mode(p.score.mode(), [&](auto mode) {
    constexpr int kMode = decltype(mode)::value;
    return p.D == 64 ? launch_tiles_one<64, kMode>(tk, tv, p, s) : launch_tiles_one<128, kMode>(tk, tv, p, s);
  });
}

}  // namespace bfa
