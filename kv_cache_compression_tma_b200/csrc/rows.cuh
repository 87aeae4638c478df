// rows.cuh -- one head's row of a [tokens, heads, head_dim] tensor spread over a group of lanes, 16
// bytes (8 bf16 or 4 fp32 elements) per lane; shared by the CUDA-core kernels that stream key rows.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace ispa {

template <typename T, int HD>
struct Row {
  static constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // elements per lane
  static constexpr int kLanes = HD / kVec;                       // lanes per row
  static constexpr int kPerWarp = 32 / kLanes;                   // rows per warp-wide load
  static_assert(kLanes >= 2 && kLanes <= 32, "a row spans 2 to 32 lanes");
};

// The lane's 16 bytes as raw words; kAligned: one 16-byte load (base and row stride 16-byte aligned),
// else one load per element.
template <typename T, bool kAligned>
__device__ __forceinline__ uint4 load_raw(const T* p) {
  if constexpr (kAligned) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    uint4 w;
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
    if constexpr (sizeof(T) == 2) {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = static_cast<uint32_t>(__ldg(h + 2 * i)) | (static_cast<uint32_t>(__ldg(h + 2 * i + 1)) << 16);
    } else {
      const uint32_t* f = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __ldg(f + i);
    }
    return w;
  }
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float* v) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
  }
}

// Sum over the `kLanes` lanes of a row (every lane gets it).
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace ispa
