// decode_common.cuh -- what the split-KV decode kernels on mma.sync share: the
// layout of a K/V stage, the online-softmax update of a row, and per-device values
// that their launchers look up once.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace {

template <int D>
struct DecodeLayout {
  static constexpr int kBox = D >= 64 ? 64 : D;            // elements per TMA box row
  static constexpr int kSpan = kBox * 2;                    // swizzle span (bytes)
  static constexpr int kChunksPerRow = kBox / 8;            // 16-byte chunks per box row
  static constexpr int kBlocks = D / kBox;                  // boxes per tile row
  static constexpr int kBlockBytes = kDecodeTile * kSpan;         // one box of a tile
  static constexpr int kTileBytes = kBlocks * kBlockBytes;  // K (or V) tile
  static constexpr int kStageBytes = 2 * kTileBytes;        // K + V
  // Shared-memory byte offset of (token row, 16-byte chunk along d) in a tile.
  __device__ static __forceinline__ uint32_t offset(int row, int chunk) {
    const int blk = chunk / kChunksPerRow;
    const int cc = chunk % kChunksPerRow;
    return blk * kBlockBytes + swizzle<kSpan>(row * kSpan + cc * 16);
  }
};

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Online-softmax update of one query row held by a quad of lanes: x are this
// lane's 4 scores of the row in base-2 units (masked ones are -inf).  Returns
// the rescale factor for the row's O accumulators and writes exp2(x - m) to p.
__device__ __forceinline__ float online_update(float (&x)[4], float& m, float& l, float (&p)[4]) {
  const float mx = quad_max(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
  const float m_new = fmaxf(m, mx);
  const float ref = (m_new == -INFINITY) ? 0.f : m_new;  // no (-inf) - (-inf)
  const float alpha = ex2_approx(m - ref);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = ex2_approx(x[i] - ref);
  l = l * alpha + ((p[0] + p[1]) + (p[2] + p[3]));
  m = m_new;
  return alpha;
}

// Raises the dynamic shared-memory limit of `kern` once per device.
inline cudaError_t set_smem_attr_once(const void* kern, int smem, unsigned char* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;  // benign race: idempotent
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = 1;
  return e;
}

// CTAs of `kern` (`threads` threads, `smem` bytes) the current device holds at
// once, looked up once per device.
inline cudaError_t resident_ctas(const void* kern, int threads, int smem, int* cache, int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && cache[dev] > 0) {
    *out = cache[dev];
    return cudaSuccess;
  }
  int per_sm = 0, sms = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  *out = per_sm * sms;
  if (dev >= 0 && dev < 64) cache[dev] = *out;  // benign race: idempotent
  return cudaSuccess;
}

// SMs of the current device, looked up once per device.
inline cudaError_t sm_count(int* out) {
  static int cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && cache[dev] > 0) {
    *out = cache[dev];
    return cudaSuccess;
  }
  e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev >= 0 && dev < 64) cache[dev] = *out;  // benign race: idempotent
  return e;
}

}  // namespace
}  // namespace gqa
