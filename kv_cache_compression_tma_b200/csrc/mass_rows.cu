// mass_rows.cu -- accumulated attention weight per cached key for few bf16 queries (mma.sync) and on CUDA
// cores (fp32 multiply-adds).
//
//   mass_out[h, j] = decay * mass[h, j] + sum_i exp(scale q_i.k_j + b_j - L_i),
//   L_i = log(exp(lse_loc_i) + exp(lse_hist_i)),
// for few queries (single-token steps, bf16) and for every fp32, unaligned or ISPA_ATTN_CUDA_CORES call.  K is
// read once whatever n_q is.
//
// Up to 32 bf16 queries: a warp takes 16 keys at a time, their rows go from memory straight into the
// fragments of mma.m16n8k16 (8 query columns cost the same as one), and the next 16 keys are loaded
// while the present ones are worked on.  Bound by the read of K: the same sums by multiply-adds and
// shuffles took 53 instructions a key and issue, not memory, set the pace.
// Otherwise (fp32, unaligned rows, more queries than that on CUDA cores): a key row sits in registers
// across kLanes lanes (16 bytes each), kRows rows per lane group; the queries pass by in shared-memory
// tiles as fp32 with their L_i.  Few queries: every warp has keys of its own.  Many: the CTA's eight
// warps share one warp's keys and take an eighth of the queries each, their sums joined in a fixed
// order, so that a small cache still spreads over the SMs; bound by the arithmetic.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "mass.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace ispa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;    // keys per lane group and step: 4 independent 16-byte loads per lane
constexpr int kSteps = 4;   // steps per CTA (few queries)
constexpr int kQTile = 32;  // queries staged at a time

// ---------------------------------------------------------------- up to 32 bf16 queries
// kCols: groups of 8 queries (1, 2 or 4); one group's fragments stay in registers, more in shared memory.
template <int HD, int kCols>
__global__ void __launch_bounds__(kThreads, 2) mass_few_kernel(const MassLaunch a, int ctas_per_head) {
  using M = Mma16<HD>;
  __shared__ uint4 sq[kCols > 1 ? kCols * M::kPieces : 1][32];  // [group, piece][lane]
  const int head = static_cast<int>(blockIdx.x % a.n_heads);  // heads first: CTAs that run together share rows
  const int cta = static_cast<int>(blockIdx.x / a.n_heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const auto* K = static_cast<const __nv_bfloat16*>(a.k) + static_cast<int64_t>(head) * HD + 8 * c;
  const auto* Q = static_cast<const __nv_bfloat16*>(a.q) + static_cast<int64_t>(head) * HD + 8 * c;
  const int64_t units = (a.n_k + 15) / 16, stride = static_cast<int64_t>(ctas_per_head) * kWarps;
  int64_t u = static_cast<int64_t>(cta) * kWarps + warp;
  auto load = [&](int64_t unit, M& m) {  // rows past the end repeat the last key
    m.load(K + min(unit * 16 + g, a.n_k - 1) * a.ld_k, K + min(unit * 16 + g + 8, a.n_k - 1) * a.ld_k);
  };
  M cur, next;
  if (u < units) load(u, cur);
  auto piece = [&](int col, int j) {
    const int i = col * 8 + g;
    return i < a.n_q ? load_raw<__nv_bfloat16, false>(Q + i * a.ld_q + 32 * j) : make_uint4(0, 0, 0, 0);
  };
  uint4 q[M::kPieces];
  if constexpr (kCols == 1) {
#pragma unroll
    for (int j = 0; j < M::kPieces; ++j) q[j] = piece(0, j);
  } else {
    for (int x = warp; x < kCols * M::kPieces; x += kWarps) sq[x][lane] = piece(x / M::kPieces, x % M::kPieces);
    __syncthreads();
  }
  // this lane's two query columns of each group; a column without a query, or a row without keys, adds 0
  constexpr double kLog2e = 1.4426950408889634;
  const double sl2_64 = static_cast<double>(a.scale) * kLog2e;
  const float sl2 = static_cast<float>(sl2_64), sl2_lo = static_cast<float>(sl2_64 - sl2);
  float nl[kCols][2], nl_lo[kCols][2];  // -L log2(e) and what its rounding left
#pragma unroll
  for (int col = 0; col < kCols; ++col)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = col * 8 + 2 * c + x;
      const int64_t o = static_cast<int64_t>(head) * a.n_q + i;
      const double l = i < a.n_q ? -kLog2e * mass_row_lse64(a.lse_loc[o], a.lse_hist ? a.lse_hist[o] : -INFINITY) : -INFINITY;
      nl[col][x] = static_cast<float>(l);
      nl_lo[col][x] = l > -INFINITY ? static_cast<float>(l - nl[col][x]) : 0.f;
    }
  for (; u < units; u += stride) {
    if (u + stride < units) load(u + stride, next);
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int col = 0; col < kCols; ++col) {
      if constexpr (kCols > 1) {
#pragma unroll
        for (int j = 0; j < M::kPieces; ++j) q[j] = sq[col * M::kPieces + j][lane];
      }
      float d[4];
      cur.template scores<4>(q, d);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool live = nl[col][x] > -INFINITY || nl[col][x] != nl[col][x];  // a NaN stays one
        lo += live ? fast_exp2(fmaf(d[x], sl2, nl[col][x]) + fmaf(d[x], sl2_lo, nl_lo[col][x])) : 0.f;
        hi += live ? fast_exp2(fmaf(d[2 + x], sl2, nl[col][x]) + fmaf(d[2 + x], sl2_lo, nl_lo[col][x])) : 0.f;
      }
    }
    lo = row_sum<4>(lo);
    hi = row_sum<4>(hi);
    const int64_t j = u * 16 + g + 8 * c;
    if (c < 2 && j < a.n_k) {
      float w = c ? hi : lo;
      const int64_t o = static_cast<int64_t>(head) * a.ld_mass + j;
      if (a.bias) w = mass_apply_bias(w, a.bias[static_cast<int64_t>(head) * a.ld_bias + j]);
      a.mass_out[o] = a.decay != 0.f ? fmaf(a.decay, a.mass[o], w) : w;
    }
    cur = next;
  }
}

template <int HD>
cudaError_t launch_few(const MassLaunch& a, cudaStream_t s, int* n) {
  // all CTAs at once (two per SM), none with less than one unit per warp
  const int64_t units = (a.n_k + 15) / 16;
  const int64_t per_head = 296 / a.n_heads > 0 ? 296 / a.n_heads : 1;
  const int ctas = static_cast<int>(std::min(per_head, (units + kWarps - 1) / kWarps));
  const unsigned grid = static_cast<unsigned>(ctas) * static_cast<unsigned>(a.n_heads);
  if (a.n_q <= 8)
    mass_few_kernel<HD, 1><<<grid, kThreads, 0, s>>>(a, ctas);
  else if (a.n_q <= 16)
    mass_few_kernel<HD, 2><<<grid, kThreads, 0, s>>>(a, ctas);
  else
    mass_few_kernel<HD, 4><<<grid, kThreads, 0, s>>>(a, ctas);
  *n += 1;
  return cudaGetLastError();
}

// ---------------------------------------------------------------- any case
// kSplit: the warps split the queries (one step per CTA); else they split the keys.
template <typename T, int HD, bool kAligned, bool kSplit>
__global__ void __launch_bounds__(kThreads) mass_rows_kernel(const MassLaunch a) {
  using R = Row<T, HD>;
  constexpr int kWarpKeys = R::kPerWarp * kRows;
  constexpr int kKeys = kSplit ? kWarpKeys : kWarps * kWarpKeys;  // keys per step of a CTA
  __shared__ __align__(16) float sq[kQTile][HD];  // read four at a time
  __shared__ float sl[kQTile], sl_lo[kQTile];  // L and what its rounding left
  __shared__ float part[kSplit ? kWarps : 1][kWarpKeys];
  const int head = static_cast<int>(blockIdx.x % a.n_heads);  // heads first: CTAs that run together share rows
  const int64_t chunk = blockIdx.x / a.n_heads;
  const int warp = threadIdx.x >> 5;
  const int group = (threadIdx.x & 31) / R::kLanes, lane = (threadIdx.x & 31) % R::kLanes;
  const T* K = static_cast<const T*>(a.k) + static_cast<int64_t>(head) * HD + lane * R::kVec;
  const T* Q = static_cast<const T*>(a.q) + static_cast<int64_t>(head) * HD;
  const int64_t first = chunk * (kSplit ? 1 : kSteps) * kKeys;
  const int steps = kSplit ? 1 : static_cast<int>(min(static_cast<int64_t>(kSteps), (a.n_k - first + kKeys - 1) / kKeys));
  auto key_of = [&](int step, int r) {
    return first + step * kKeys + (kSplit ? 0 : warp * kWarpKeys) + r * R::kPerWarp + group;
  };
  auto load = [&](int step, uint4* kw) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t j = min(key_of(step, r), a.n_k - 1);  // rows past the end repeat the last key
      kw[r] = load_raw<T, kAligned>(K + j * a.ld_k);
    }
  };
  uint4 next[kRows];
  load(0, next);
  for (int step = 0; step < steps; ++step) {
    uint4 kw[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) kw[r] = next[r];
    if (step + 1 < steps) load(step + 1, next);
    float sum[kRows] = {};
    for (int64_t i0 = 0; i0 < a.n_q; i0 += kQTile) {
      const int nq = static_cast<int>(a.n_q - i0 < kQTile ? a.n_q - i0 : kQTile);
      if (step == 0) {  // several steps have a lone tile of queries, which stays staged
        if (i0 > 0) __syncthreads();
        for (int x = threadIdx.x; x < nq * HD; x += kThreads)
          sq[x / HD][x % HD] = static_cast<float>(Q[(i0 + x / HD) * a.ld_q + x % HD]) * a.scale;
        if (threadIdx.x < nq) {
          const int64_t o = static_cast<int64_t>(head) * a.n_q + i0 + threadIdx.x;
          const double l = mass_row_lse64(a.lse_loc[o], a.lse_hist ? a.lse_hist[o] : -INFINITY);
          sl[threadIdx.x] = static_cast<float>(l);
          sl_lo[threadIdx.x] = l < INFINITY ? static_cast<float>(l - sl[threadIdx.x]) : 0.f;
        }
        __syncthreads();
      }
      for (int i = kSplit ? warp : 0; i < nq; i += kSplit ? kWarps : 1) {
        float qv[R::kVec];
#pragma unroll
        for (int e = 0; e < R::kVec; e += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&sq[i][lane * R::kVec + e]);
          qv[e] = w.x, qv[e + 1] = w.y, qv[e + 2] = w.z, qv[e + 3] = w.w;
        }
        const float li = sl[i], li_lo = sl_lo[i];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float kv[R::kVec], s = 0.f;
          unpack<T>(kw[r], kv);
#pragma unroll
          for (int e = 0; e < R::kVec; ++e) s = fmaf(qv[e], kv[e], s);
          s = row_sum<R::kLanes>(s);
          const float w = expf((s - li) - li_lo);
          sum[r] += li == INFINITY ? 0.f : w;  // a row without keys adds nothing, whatever its scores are
        }
      }
    }
    if constexpr (kSplit) {
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (lane == 0) part[warp][r * R::kPerWarp + group] = sum[r];
      __syncthreads();
    }
    // a lane group's r-th key belongs to its lane r (in the split form to the first warp's threads)
    auto put = [&](int64_t j, float w) {
      if (j >= a.n_k) return;
      const int64_t o = static_cast<int64_t>(head) * a.ld_mass + j;
      if (a.bias) w = mass_apply_bias(w, a.bias[static_cast<int64_t>(head) * a.ld_bias + j]);
      a.mass_out[o] = a.decay != 0.f ? fmaf(a.decay, a.mass[o], w) : w;
    };
    if constexpr (kSplit) {
      for (int x = threadIdx.x; x < kWarpKeys; x += kThreads) {
        float w = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) w += part[v][x];
        put(first + x, w);
      }
    } else {
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (lane == r % R::kLanes) put(key_of(step, r), sum[r]);
    }
  }
}

template <typename T, int HD, bool kSplit>
cudaError_t launch_split(const MassLaunch& a, cudaStream_t s, int* n) {
  constexpr int kKeys = Row<T, HD>::kPerWarp * kRows * (kSplit ? 1 : kWarps * kSteps);
  const int64_t blocks = (a.n_k + kKeys - 1) / kKeys * a.n_heads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (aligned16(a.k) && (a.ld_k * static_cast<int64_t>(sizeof(T))) % 16 == 0)
    mass_rows_kernel<T, HD, true, kSplit><<<grid, kThreads, 0, s>>>(a);
  else
    mass_rows_kernel<T, HD, false, kSplit><<<grid, kThreads, 0, s>>>(a);
  *n += 1;
  return cudaGetLastError();
}

template <typename T, int HD>
cudaError_t launch_hd(const MassLaunch& a, cudaStream_t s, int* n) {
  return a.n_q > kWarps ? launch_split<T, HD, true>(a, s, n) : launch_split<T, HD, false>(a, s, n);
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

cudaError_t launch_mass_rows(const MassLaunch& a, bool cuda_cores, cudaStream_t s, int* n_launched) {
  if (!cuda_cores && a.dtype == 0 && a.n_q >= 1 && a.n_q <= kMassFewQueries && (a.head_dim == 64 || a.head_dim == 128) && aligned16(a.k) && a.ld_k % 8 == 0)
    return a.head_dim == 128 ? launch_few<128>(a, s, n_launched) : launch_few<64>(a, s, n_launched);
  return a.dtype == 1 ? launch_t<float>(a, s, n_launched) : launch_t<__nv_bfloat16>(a, s, n_launched);
}

}  // namespace ispa
