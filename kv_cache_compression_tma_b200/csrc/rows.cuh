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

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16.  Lane l = 4 g + c holds rows g and g + 8 of A (a0, a2 and
// a1, a3), column g of B, and D[g][2c, 2c+1] (d0, d1), D[g + 8][2c, 2c+1] (d2, d3).  The order of the 16
// products is free as long as A and B agree, so a lane may feed any four elements of its row per step.
__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scores of 16 bf16 key rows against up to 8 query rows, operands straight from memory: piece j of a
// lane is the 16 bytes (4 j + c) of its row, so four lanes cover 64 contiguous bytes.
template <int HD>
struct Mma16 {
  static constexpr int kPieces = HD / 32;
  uint4 lo[kPieces], hi[kPieces];  // key rows g and g + 8
  // row_lo, row_hi: the lane's two rows, offset by 8 c elements
  __device__ __forceinline__ void load(const __nv_bfloat16* row_lo, const __nv_bfloat16* row_hi) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) lo[j] = __ldg(reinterpret_cast<const uint4*>(row_lo + 32 * j));
#pragma unroll
    for (int j = 0; j < kPieces; ++j) hi[j] = __ldg(reinterpret_cast<const uint4*>(row_hi + 32 * j));
  }
  // In kChains chains of products, summed here.  The tensor core truncates as it adds, and short chains keep
  // what it adds to small: with four of them a weight exp(logit - L) is off by 5e-7, with two by 1e-6.
  template <int kChains>
  __device__ __forceinline__ void scores(const uint4* q, float* d) const {
    constexpr int kUsed = kChains < 2 * kPieces ? kChains : 2 * kPieces;
    float e[kUsed][4] = {};
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      mma_bf16(e[2 * j % kUsed], lo[j].x, hi[j].x, lo[j].y, hi[j].y, q[j].x, q[j].y);
      mma_bf16(e[(2 * j + 1) % kUsed], lo[j].z, hi[j].z, lo[j].w, hi[j].w, q[j].z, q[j].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i] = e[0][i] + e[1][i];
      if constexpr (kUsed == 4) d[i] += e[2][i] + e[3][i];
    }
  }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace ispa
