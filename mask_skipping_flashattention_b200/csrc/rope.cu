// Rotary positions, and the paged cache's writer.
//
// A pair (a, b) of a head at position n turns by the angle n * f_i:
//   a' = amp (a cos - b sin),  b' = amp (a sin + b cos)
// (the inverse rotation, which is also the gradient, has -sin).  The angle is
// reduced in double: n f_i / (2 pi) minus its nearest integer is exact to about
// 1e-11 turns at position 10^6, where a product in fp32 would be off by 0.06
// radians.
//
// Bound by HBM: two bytes in and two out a value.  A thread owns one 16-byte
// chunk pair of a token (8 pairs: one cos / sin evaluation each) and walks the
// heads with it, so the trigonometry is paid once for `heads_per_thread` heads.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "rope_params.cuh"

namespace bfa {

using namespace ptx;

namespace {

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

__global__ void __launch_bounds__(256) k_rope(const RopeParams p) {
  const int pairs = p.rotary / 16;               // chunk pairs of a head that turn
  const int chunks = pairs + (p.D - p.rotary) / 8;  // and chunks that are copied
  const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t tok = id / chunks;
  const int c = static_cast<int>(id - tok * chunks);
  if (tok >= p.tokens) return;
  const int64_t b = tok / p.S, st = tok - b * p.S;

  // position of the token, and its place in the cache
  int64_t pos;
  int64_t row = -1;  // element offset of the token's cache row, or -1
  if (p.positions) {
    const int64_t i = b * p.pos_sb + st;
    pos = p.positions64 ? static_cast<const int64_t*>(p.positions)[i]
                        : static_cast<int64_t>(static_cast<const int32_t*>(p.positions)[i]);
  } else {
    const int s = seq_of_token(p.cu_seqlens, p.n_seq, tok);
    if (s >= p.n_seq) return;  // a row behind the last sequence
    const int first = __ldg(p.cu_seqlens + s), end = __ldg(p.cu_seqlens + s + 1);
    if (tok < first) return;
    pos = static_cast<int64_t>(__ldg(p.seqused_k + s)) - (end - first) + (tok - first);
    const int64_t pi = pos / p.page_size;
    if (pos >= 0 && pi < p.pages_per_seq) {
      const int64_t page = __ldg(p.block_table + static_cast<int64_t>(s) * p.pages_per_seq + pi);
      if (page >= 0 && page < p.num_pages) row = page * p.c_sp + (pos - pi * p.page_size) * p.c_st;
    }
  }

  const bool turn = c < pairs;
  // element offsets of the thread's one or two chunks inside a head
  int ca, cb;
  if (!turn) ca = cb = p.rotary + (c - pairs) * 8;
  else if (p.interleaved) { ca = c * 16; cb = ca + 8; }
  else { ca = c * 8; cb = ca + p.rotary / 2; }
  float co[8], si[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // turns, minus the nearest integer: in [-1/2, 1/2]
      const double t = static_cast<double>(pos) * p.inv_freq[c * 8 + i] * 0.15915494309189533577;
      float sn, cs;
      sincospif(2.f * static_cast<float>(t - rint(t)), &sn, &cs);
      co[i] = cs * p.amplitude;
      si[i] = sn * p.amplitude * p.sign;
    }
  }

  auto rotate = [&](const uint4& A, const uint4& B, uint4& oa, uint4& ob) {
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
    oa = make_uint4(ra[0], ra[1], ra[2], ra[3]);
    ob = make_uint4(rb[0], rb[1], rb[2], rb[3]);
  };

  const int heads = p.H + 2 * p.Hkv;  // q, then k, then v
  const int h0 = blockIdx.y * p.heads_per_thread, h1 = min(heads, h0 + p.heads_per_thread);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    bool plain = !turn;
    if (h < p.H) {
      src = p.q + b * p.q_sb + st * p.q_ss + static_cast<int64_t>(h) * p.q_sh;
      dst = p.q_out + b * p.qo_sb + st * p.qo_ss + static_cast<int64_t>(h) * p.qo_sh;
    } else if (h < p.H + p.Hkv) {
      src = p.k + tok * p.k_ss + static_cast<int64_t>(h - p.H) * p.k_sh;
      dst = row < 0 ? nullptr : p.k_cache + row + static_cast<int64_t>(h - p.H) * p.c_sh;
    } else {
      src = p.v + tok * p.v_ss + static_cast<int64_t>(h - p.H - p.Hkv) * p.v_sh;
      dst = row < 0 ? nullptr : p.v_cache + row + static_cast<int64_t>(h - p.H - p.Hkv) * p.c_sh;
      plain = true;
    }
    if (dst == nullptr) continue;  // no page for this token
    uint4 A = *reinterpret_cast<const uint4*>(src + ca), B = A;
    if (turn) {
      B = *reinterpret_cast<const uint4*>(src + cb);
      if (!plain) {
        const uint4 A0 = A, B0 = B;
        rotate(A0, B0, A, B);
      }
      *reinterpret_cast<uint4*>(dst + cb) = B;
    }
    *reinterpret_cast<uint4*>(dst + ca) = A;
  }
}

cudaError_t launch_rope(const RopeParams& p0, int sms, cudaStream_t s) {
  RopeParams p = p0;
  const int heads = p.H + 2 * p.Hkv;
  if (p.tokens <= 0 || heads <= 0) return cudaSuccess;
  const int64_t threads = p.tokens * (p.rotary / 16 + (p.D - p.rotary) / 8);
  // heads a thread walks: all of them while that still gives every SM 2048 threads
  int64_t groups = (static_cast<int64_t>(sms) * 2048 + threads - 1) / threads;
  groups = groups < 1 ? 1 : (groups > heads ? heads : groups);
  p.heads_per_thread = static_cast<int>((heads + groups - 1) / groups);
  const int64_t blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned gy = static_cast<unsigned>((heads + p.heads_per_thread - 1) / p.heads_per_thread);
  if (gy > 65535u) return cudaErrorInvalidConfiguration;
  k_rope<<<dim3(static_cast<unsigned>(blocks), gy), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace bfa
