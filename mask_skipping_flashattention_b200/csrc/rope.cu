// Rotary positions, and the paged cache's writer.
//
// A pair (a, b) of a head at position n turns by the angle n * f_i:
//   a' = amp (a cos - b sin),  b' = amp (a sin + b cos)
// (the inverse rotation, which is also the gradient, has -sin).  The angle is
// reduced in double: n f_i / (2 pi) minus its nearest integer is exact to about
// 1e-11 turns at position 10^6, where a product in fp32 would be off by 0.06
// radians.
//
// Bound by HBM: two bytes in and two out a value.  A block takes a few whole tokens:
// their positions, then the cos and sin of every pair once into shared memory, then
// all heads.  A thread owns one chunk pair of a head (two 16-byte chunks, 8 pairs) or
// one chunk that is copied, in every kHeadLanes-th head: neighbouring threads cover
// kHeadLanes whole heads (1 KB at D 128), and a batch of heads is loaded before the first is
// stored.  Measured: 268 MB (4 x 4096 x 32 x 128) 44.8 us, 0.91 of the measured copy rate (54 us
// with a thread's heads side by side and the angles computed by every thread).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "plan_types.cuh"
#include "ptx.cuh"
#include "rope_params.cuh"

namespace bfa {

using namespace ptx;

namespace {

constexpr int kRopeThreads = 256;
constexpr int kHeadLanes = 4;
constexpr int kRopeTokens = 32;                 // most tokens of a block (8 threads a token at least)
constexpr int kRopePairs = kRopeThreads / kHeadLanes * 8;  // most pairs of a block's tokens: 8 a chunk pair

__device__ __forceinline__ float2 bf2_to_f2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// sequence of token t: the last s with cu[s] <= t (empty sequences are passed over)
__device__ __forceinline__ int seq_of_token(const int32_t* cu, int n_seq, int64_t t) {
  int lo = 0, hi = n_seq;  // first s in (0, n_seq] with cu[s] > t, minus one
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

}  // namespace

// kRagged: positions and places from a ragged batch's lengths, keys and values into a cache.
// kBatch heads are in flight a thread: the ragged form, which waits longer for its start,
// holds fewer so that more blocks are resident.
template <bool kRagged, int kBatch>
__global__ void __launch_bounds__(kRopeThreads, kRagged ? 4 : 3) k_rope(const RopeParams p) {
  __shared__ int64_t pos_s[kRopeTokens], row_s[kRopeTokens];
  __shared__ __align__(16) float2 turn_s[kRopePairs];     // (cos, sin) of a token's pairs, token-major
  const unsigned pairs = p.rotary / 16;                   // chunk pairs of a head that turn
  const unsigned chunks = pairs + (p.D - p.rotary) / 8;   // and chunks that are copied
  const unsigned lanes = chunks * kHeadLanes;             // threads of a token
  const unsigned per = p.tokens_per_block;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * per;

  // position of each token, and its place in the cache: an element offset, -1 none, -2 not a token
  if (threadIdx.x < per) {
    const int64_t tok = tok0 + threadIdx.x;
    int64_t pos = 0, row = -2;
    if (tok < p.tokens) {
      if constexpr (!kRagged) {
        const int64_t b = tok / p.S, i = b * p.pos_sb + (tok - b * p.S);
        pos = p.positions64 ? static_cast<const int64_t*>(p.positions)[i]
                            : static_cast<int64_t>(static_cast<const int32_t*>(p.positions)[i]);
        row = -1;
      } else {
        const int s = seq_of_token(p.cu_seqlens, p.n_seq, tok);
        if (s < p.n_seq) {  // else a row behind the last sequence
          const int first = __ldg(p.cu_seqlens + s), end = __ldg(p.cu_seqlens + s + 1);
          if (tok >= first) {
            row = -1;
            pos = static_cast<int64_t>(__ldg(p.seqused_k + s)) - (end - first) + (tok - first);
            if (pos >= 0 && pos < static_cast<int64_t>(p.pages_per_seq) * p.page_size) {
              const int pi = static_cast<int>(pos) / p.page_size;
              const int64_t page = __ldg(p.block_table + static_cast<int64_t>(s) * p.pages_per_seq +
                                         BFA_IDX(pi, p.pages_per_seq, p.err));
              if (page >= 0 && page < p.num_pages)
                row = page * p.c_sp + (static_cast<int>(pos) - pi * p.page_size) * p.c_st;
            }
          }
        }
      }
    }
    pos_s[threadIdx.x] = pos;
    row_s[threadIdx.x] = row;
  }
  __syncthreads();
  const unsigned half = p.rotary / 2;
  for (unsigned i = threadIdx.x; i < per * half; i += kRopeThreads) {
    const unsigned t = i / half;
    // turns, minus the nearest integer: in [-1/2, 1/2]
    const double x = static_cast<double>(pos_s[t]) * __ldg(p.inv_freq + (i - t * half)) * 0.15915494309189533577;
    float sn, cs;
    sincospif(2.f * static_cast<float>(x - rint(x)), &sn, &cs);
    turn_s[BFA_IDX(i, kRopePairs, p.err)] = make_float2(cs * p.amplitude, sn * p.amplitude * p.sign);
  }
  __syncthreads();
  const unsigned t = threadIdx.x / lanes, in_tok = threadIdx.x - t * lanes;
  const unsigned c = in_tok % chunks;
  if (t >= per || row_s[t] == -2) return;
  const int64_t tok = tok0 + t, row = row_s[t];
  BFA_CHECK(tok >= 0 && tok < p.tokens && per <= kRopeTokens, p.err);
  BFA_CHECK(row < p.num_pages * p.c_sp, p.err);
  const int64_t b = kRagged ? 0 : tok / p.S, st = tok - b * p.S;

  const bool turn = c < pairs;
  // element offsets of the thread's one or two chunks inside a head
  int ca, cb;
  if (!turn) ca = cb = p.rotary + (c - pairs) * 8;
  else if (p.interleaved) { ca = c * 16; cb = ca + 8; }
  else { ca = c * 8; cb = ca + p.rotary / 2; }
  BFA_CHECK(ca >= 0 && ca + 8 <= p.D && cb >= 0 && cb + 8 <= p.D, p.err);
  float co[8], si[8];
  if (turn) {
    const float4* v = reinterpret_cast<const float4*>(turn_s + t * half + c * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = v[i];
      co[2 * i] = x.x;
      si[2 * i] = x.y;
      co[2 * i + 1] = x.z;
      si[2 * i + 1] = x.w;
    }
  }

  auto rotate = [&](uint4& A, uint4& B) {
    const uint32_t a[4] = {A.x, A.y, A.z, A.w}, bb[4] = {B.x, B.y, B.z, B.w};
    uint32_t ra[4], rb[4];
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = bf2_to_f2(a[i]), y = bf2_to_f2(bb[i]);
        ra[i] = pack_bf16x2(x.x * co[i] - x.y * si[i], x.x * si[i] + x.y * co[i]);
        rb[i] = pack_bf16x2(y.x * co[4 + i] - y.y * si[4 + i], y.x * si[4 + i] + y.y * co[4 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = bf2_to_f2(a[i]), y = bf2_to_f2(bb[i]);
        ra[i] = pack_bf16x2(x.x * co[2 * i] - y.x * si[2 * i], x.y * co[2 * i + 1] - y.y * si[2 * i + 1]);
        rb[i] = pack_bf16x2(x.x * si[2 * i] + y.x * co[2 * i], x.y * si[2 * i + 1] + y.y * co[2 * i + 1]);
      }
    }
    A = make_uint4(ra[0], ra[1], ra[2], ra[3]);
    B = make_uint4(rb[0], rb[1], rb[2], rb[3]);
  };

  // heads of q, then k, then v
  const int heads = kRagged ? p.H + 2 * p.Hkv : p.H;
  const __nv_bfloat16* const q = p.q + b * p.q_sb + st * p.q_ss;
  __nv_bfloat16* const qo = p.q_out + b * p.qo_sb + st * p.qo_ss;
  const int h1 = min(heads, static_cast<int>(blockIdx.y + 1) * p.heads_per_block);
  for (int h0 = blockIdx.y * p.heads_per_block + in_tok / chunks; h0 < h1; h0 += kHeadLanes * kBatch) {
    uint4 A[kBatch], B[kBatch];
    __nv_bfloat16* dst[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * kHeadLanes;
      const __nv_bfloat16* src;
      dst[i] = nullptr;  // past the heads, or no place for this token
      if (h >= h1) continue;
      if (!kRagged || h < p.H) {
        src = q + static_cast<int64_t>(h) * p.q_sh;
        dst[i] = qo + static_cast<int64_t>(h) * p.qo_sh;
      } else {
        if (row < 0) continue;
        const bool is_v = h >= p.H + p.Hkv;
        const int64_t hk = h - p.H - (is_v ? p.Hkv : 0);
        src = is_v ? p.v + tok * p.v_ss + hk * p.v_sh : p.k + tok * p.k_ss + hk * p.k_sh;
        dst[i] = (is_v ? p.v_cache : p.k_cache) + row + hk * p.c_sh;
      }
      A[i] = *reinterpret_cast<const uint4*>(src + ca);
      if (turn) B[i] = *reinterpret_cast<const uint4*>(src + cb);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!dst[i]) continue;
      if (turn) {
        if (!kRagged || h0 + i * kHeadLanes < p.H + p.Hkv) rotate(A[i], B[i]);  // values are copied
        *reinterpret_cast<uint4*>(dst[i] + cb) = B[i];
      }
      *reinterpret_cast<uint4*>(dst[i] + ca) = A[i];
    }
  }
}

cudaError_t launch_rope(const RopeParams& p0, int sms, cudaStream_t s) {
  RopeParams p = p0;
  const bool ragged = p.positions == nullptr;
  const int heads = p.H + 2 * p.Hkv;
  if (p.tokens <= 0 || heads <= 0) return cudaSuccess;
  const int lanes = kHeadLanes * (p.rotary / 16 + (p.D - p.rotary) / 8);  // 16 .. 64
  p.tokens_per_block = kRopeThreads / lanes;
  const int64_t blocks = (p.tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // a block's share of the heads: all of them while that still gives every SM 4 blocks
  const int rounds = (heads + kHeadLanes - 1) / kHeadLanes;
  int64_t groups = (static_cast<int64_t>(sms) * 4 + blocks - 1) / blocks;
  groups = groups < 1 ? 1 : (groups > rounds ? rounds : groups);
  p.heads_per_block = static_cast<int>((rounds + groups - 1) / groups) * kHeadLanes;
  const unsigned gy = static_cast<unsigned>((heads + p.heads_per_block - 1) / p.heads_per_block);
  if (gy > 65535u) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks), gy);
  if (ragged) k_rope<true, 2><<<grid, kRopeThreads, 0, s>>>(p);
  else k_rope<false, 4><<<grid, kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace bfa
