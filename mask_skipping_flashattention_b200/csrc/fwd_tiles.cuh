// Tile shapes, register split and product issue shared by the forward kernels
// (fwd.cu over a plan, chunk_tile.cu over a paged cache).
#pragma once

#include <cstdint>

#include "plan_types.cuh"
#include "ptx.cuh"

namespace bfa {

using namespace ptx;

// 128 * kRegsWG0 + 256 * kRegsSoftmax must equal kThreads * kRegsLaunch: the
// increase draws only on the registers the block was launched with.  The
// compiled kernel's launch count is checked before every first launch.
constexpr int kThreads = 384;
constexpr int kRegsLaunch = 168;
constexpr uint32_t kRegsWG0 = 72;
constexpr uint32_t kRegsSoftmax = 216;
static_assert(128 * kRegsWG0 + 256 * kRegsSoftmax == kThreads * kRegsLaunch, "register split");
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled only when the max grows by > 2^8
constexpr int kStages = 2;

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSmemBytes = (2 + 2 * kStages) * kTileBytes + 1024;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS0 = 0, kColS1 = 128;
  static constexpr uint32_t kColO0 = 256, kColO1 = 256 + D;
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 1);
};

// The base descriptors pass through an empty asm so that the compiler builds
// them at the point of use (one add per step) instead of hoisting every step's
// descriptor out of the tile loop, where they would stay live in the MMA
// thread's registers.  A step's descriptor is the base plus its byte offset / 16
// (the start-address field; shared-memory offsets stay inside the field).
__device__ __forceinline__ uint64_t opaque_u64(uint64_t x) {
  asm volatile("" : "+l"(x));
  return x;
}

template <int D>
__device__ __forceinline__ void issue_s(uint32_t tS, uint8_t* sQ, uint8_t* sK) {
  const uint64_t dq = opaque_u64(smem_desc(smem_u32(sQ), 16, 1024));
  const uint64_t dk = opaque_u64(smem_desc(smem_u32(sK), 16, 1024));
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off16 = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
    umma_ss(tS, dq + off16, dk + off16, Cfg<D>::kIdescQK, kk > 0);
  }
}

template <int D>
__device__ __forceinline__ void issue_pv(uint32_t tO, uint32_t tP, uint8_t* sV, bool acc) {
  const uint64_t dv = opaque_u64(smem_desc(smem_u32(sV), 16384, 1024));
#pragma unroll
  for (int kk = 0; kk < kTile / 16; ++kk)
    umma_ts(tO, tP + kk * 8, dv + kk * (2048 >> 4), Cfg<D>::kIdescPV, (acc || kk > 0) ? 1u : 0u);
}

}  // namespace bfa
