// mass_rows.cu -- accumulated attention weight per cached key on CUDA cores (fp32 arithmetic).
//
//   mass_out[h, j] = decay * mass[h, j] + sum_i exp(scale q_i.k_j + b_j - L_i),
//   L_i = log(exp(lse_loc_i) + exp(lse_hist_i)),
// for few queries (single-token steps, bf16) and for every fp32 call.  A row of K sits in registers
// across kLanes lanes (16 bytes each), kRows rows per lane group; the queries pass by in shared-memory
// tiles as fp32 with their L_i, so K is read once whatever n_q is.  One query: bound by the read of K.
#include <math.h>

#include "internal.h"
#include "mass.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace ispa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;    // keys per lane group and step: 4 independent 16-byte loads per lane
constexpr int kSteps = 4;   // steps per CTA
constexpr int kQTile = 16;  // queries staged at a time

template <typename T, int HD, bool kAligned>
__global__ void __launch_bounds__(kThreads) mass_rows_kernel(const MassLaunch a) {
  using R = Row<T, HD>;
  constexpr int kGroups = kThreads / R::kLanes;
  constexpr int kKeys = kGroups * kRows;  // keys per step of a CTA
  __shared__ float sq[kQTile][HD];
  __shared__ float sl[kQTile];
  const int head = blockIdx.y;
  const int group = threadIdx.x / R::kLanes, lane = threadIdx.x % R::kLanes;
  const T* K = static_cast<const T*>(a.k) + static_cast<int64_t>(head) * HD + lane * R::kVec;
  const T* Q = static_cast<const T*>(a.q) + static_cast<int64_t>(head) * HD;
  for (int step = 0; step < kSteps; ++step) {
    const int64_t j0 = (static_cast<int64_t>(blockIdx.x) * kSteps + step) * kKeys + group * kRows;
    if (j0 - group * kRows >= a.n_k) break;  // uniform over the CTA
    uint4 kw[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t j = j0 + r < a.n_k ? j0 + r : a.n_k - 1;  // rows past the end repeat the last key
      kw[r] = load_raw<T, kAligned>(K + j * a.ld_k);
    }
    float sum[kRows] = {};
    for (int64_t i0 = 0; i0 < a.n_q; i0 += kQTile) {
      const int nq = static_cast<int>(a.n_q - i0 < kQTile ? a.n_q - i0 : kQTile);
      if (i0 > 0 || step == 0 || a.n_q > kQTile) {  // one tile of queries stays staged over the steps
        __syncthreads();
        for (int x = threadIdx.x; x < nq * HD; x += kThreads)
          sq[x / HD][x % HD] = static_cast<float>(Q[(i0 + x / HD) * a.ld_q + x % HD]) * a.scale;
        if (threadIdx.x < nq) {
          const int64_t o = static_cast<int64_t>(head) * a.n_q + i0 + threadIdx.x;
          sl[threadIdx.x] = mass_row_lse(a.lse_loc[o], a.lse_hist ? a.lse_hist[o] : -INFINITY);
        }
        __syncthreads();
      }
      for (int i = 0; i < nq; ++i) {
        float qv[R::kVec];
#pragma unroll
        for (int e = 0; e < R::kVec; e += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&sq[i][lane * R::kVec + e]);
          qv[e] = w.x, qv[e + 1] = w.y, qv[e + 2] = w.z, qv[e + 3] = w.w;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float kv[R::kVec], s = 0.f;
          unpack<T>(kw[r], kv);
#pragma unroll
          for (int e = 0; e < R::kVec; ++e) s = fmaf(qv[e], kv[e], s);
          s = row_sum<R::kLanes>(s);
          sum[r] += expf(s - sl[i]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t j = j0 + r;
      if (lane != r % R::kLanes || j >= a.n_k) continue;
      const int64_t o = static_cast<int64_t>(head) * a.ld_mass + j;
      float w = sum[r];
      if (a.bias) w = mass_apply_bias(w, a.bias[static_cast<int64_t>(head) * a.ld_bias + j]);
      a.mass_out[o] = a.decay != 0.f ? fmaf(a.decay, a.mass[o], w) : w;
    }
  }
}

template <typename T, int HD>
cudaError_t launch_hd(const MassLaunch& a, cudaStream_t s, int* n) {
  constexpr int kKeys = kThreads / Row<T, HD>::kLanes * kRows * kSteps;
  const dim3 grid(static_cast<unsigned>((a.n_k + kKeys - 1) / kKeys), static_cast<unsigned>(a.n_heads));
  if (aligned16(a.k) && (a.ld_k * static_cast<int64_t>(sizeof(T))) % 16 == 0)
    mass_rows_kernel<T, HD, true><<<grid, kThreads, 0, s>>>(a);
  else
    mass_rows_kernel<T, HD, false><<<grid, kThreads, 0, s>>>(a);
  *n += 1;
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const MassLaunch& a, cudaStream_t s, int* n) {
  switch (a.head_dim) {
    case 16:
      return launch_hd<T, 16>(a, s, n);
    case 32:
      return launch_hd<T, 32>(a, s, n);
    case 64:
      return launch_hd<T, 64>(a, s, n);
    default:
      return launch_hd<T, 128>(a, s, n);
  }
}

}  // namespace

cudaError_t launch_mass_rows(const MassLaunch& a, cudaStream_t s, int* n_launched) {
  return a.dtype == 1 ? launch_t<float>(a, s, n_launched) : launch_t<__nv_bfloat16>(a, s, n_launched);
}

}  // namespace ispa
