// blocks.cu -- mean keys of history blocks and the selection of blocks by (mean query) . (mean key).
//
// block_means: means[b, h, :] = mean of the keys of block b, summed in 64 bits (bf16 keys: exactly) and
// rounded to fp32 once, so that a block's mean does not depend on how the sum was split.  One read of
// the keys; the CTA's row groups are joined in shared memory in a fixed order.
//
// block_select: per head and group of q_block query rows, score_b = mean(q rows) . means[b] and the
// n_sel blocks of highest score.  Scores are formed in 64 bits: they only rank blocks, and with sums of
// 128 terms fp32 would let the order of summation decide between blocks whose scores are close; the
// work is one dot product per (group, block), small next to the attention it prunes.
// A cluster of C CTAs serves C groups of one head: CTA r pools group r's queries and hands the mean to
// all, each CTA scores 1/C of the blocks for all groups (the means are read once per cluster), sends
// each score to the CTA that owns the group, and that CTA selects (radix select on 64-bit order keys,
// ties to the lowest block) and writes the picks in ascending order.
#include <cooperative_groups.h>
#include <math.h>

#include "internal.h"
#include "rows.cuh"

namespace cg = cooperative_groups;

namespace ispa {
namespace {

// ------------------------------------------------------------------------------------------ means
constexpr int kMeanCols = 16;   // 16-byte column pieces per CTA
constexpr int kMeanRows = 16;   // row groups per CTA
constexpr int kMeanThreads = kMeanCols * kMeanRows;

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kMeanThreads) block_means_kernel(const BlockMeansLaunch a) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  __shared__ double part[kMeanRows][kMeanCols * kVec];
  const int tc = threadIdx.x % kMeanCols, tr = threadIdx.x / kMeanCols;
  const int col = (blockIdx.y * kMeanCols + tc) * kVec;
  const int64_t b = a.first + blockIdx.x;
  const int64_t row0 = b * a.block;
  const int rows = static_cast<int>(a.n_k - row0 < a.block ? a.n_k - row0 : a.block);
  double s[kVec] = {};
  if (col < a.cols) {
    const T* K = static_cast<const T*>(a.k) + row0 * a.ld_k + col;
#pragma unroll 4
    for (int r = tr; r < rows; r += kMeanRows) {
      float v[kVec];
      unpack<T>(load_raw<T, kAligned>(K + r * a.ld_k), v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[e] += static_cast<double>(v[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < kVec; ++e) part[tr][tc * kVec + e] = s[e];
  __syncthreads();
  for (int x = threadIdx.x; x < kMeanCols * kVec; x += kMeanThreads) {
    const int c = blockIdx.y * kMeanCols * kVec + x;
    if (c >= a.cols) break;
    double t = 0.0;
#pragma unroll
    for (int r = 0; r < kMeanRows; ++r) t += part[r][x];
    a.means[b * a.ld_means + c] = static_cast<float>(t / rows);
  }
}

// ------------------------------------------------------------------------------------------ select
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCluster = 8;
constexpr int kTileBlocks = 32;
constexpr int kMaxBlocks = 16384;  // one 64-bit order key per block in the owner's shared memory

__device__ __forceinline__ uint64_t order_key64(double s) {
  if (isnan(s)) s = -INFINITY;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(s + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// grid: (clusters of C CTAs per head) * C, heads.  kCluster groups per cluster.
template <typename T, int HD>
__global__ void __launch_bounds__(kSelThreads) block_select_kernel(const BlockSelectLaunch a) {
  extern __shared__ uint64_t keys[];  // [n_blocks] of the group this CTA owns
  __shared__ double qm[kSelCluster][HD];
  __shared__ double kt[kTileBlocks][HD + 2];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sum[kSelWarps];
  __shared__ uint32_t found[3];  // digit, keys below it, keys in it
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int head = blockIdx.y;
  const int64_t g0 = static_cast<int64_t>(blockIdx.x / C) * C;
  const int n_groups = static_cast<int>(a.groups - g0 < C ? a.groups - g0 : C);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nb = a.n_blocks;
  cluster.sync();  // every CTA of the cluster runs before its shared memory is written from another

  if (rank < n_groups) {  // the group's mean query, in 64 bits
    const int64_t r0 = (g0 + rank) * a.q_block;
    const int rows = static_cast<int>(a.n_q - r0 < a.q_block ? a.n_q - r0 : a.q_block);
    const T* Q = static_cast<const T*>(a.q) + r0 * a.ld_q + static_cast<int64_t>(head) * HD;
    constexpr int kParts = kSelThreads / HD;
    double (*part)[HD + 2] = kt;
    const int e = tid % HD;
    double s = 0.0;
#pragma unroll 8
    for (int r = tid / HD; r < rows; r += kParts) s += static_cast<double>(static_cast<float>(Q[r * a.ld_q + e]));
    part[tid / HD][e] = s;
    __syncthreads();
    if (tid < HD) {
      double t = 0.0;
#pragma unroll
      for (int p = 0; p < kParts; ++p) t += part[p][tid];
      t /= rows;
      for (int r = 0; r < C; ++r) cluster.map_shared_rank(&qm[0][0], r)[rank * HD + tid] = t;
    }
  }
  cluster.sync();

  // scores of this CTA's share of the blocks: lane = block of a tile, warp = group
  const int per = (nb + C - 1) / C;
  const int b0 = min(nb, rank * per), b1 = min(nb, b0 + per);
  for (int t0 = b0; t0 < b1; t0 += kTileBlocks) {
    __syncthreads();
    for (int x = tid; x < kTileBlocks * (HD / 4); x += kSelThreads) {
      const int j = x / (HD / 4), c = (x % (HD / 4)) * 4;
      if (t0 + j < b1) {
        const float* m = a.means + static_cast<int64_t>(t0 + j) * a.ld_means + static_cast<int64_t>(head) * HD + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) kt[j][c + i] = static_cast<double>(__ldg(m + i));
      }
    }
    __syncthreads();
    if (warp < n_groups && t0 + lane < b1) {
      double s0 = 0.0, s1 = 0.0;
#pragma unroll 8
      for (int e = 0; e < HD; e += 2) {
        const double2 q = *reinterpret_cast<const double2*>(&qm[warp][e]);
        const double2 k = *reinterpret_cast<const double2*>(&kt[lane][e]);
        s0 = fma(q.x, k.x, s0);
        s1 = fma(q.y, k.y, s1);
      }
      cluster.map_shared_rank(keys, warp)[t0 + lane] = order_key64(s0 + s1);
    }
  }
  cluster.sync();
  if (rank >= n_groups) return;  // nobody reads this CTA's shared memory any more

  int32_t* out = a.idx + (static_cast<int64_t>(head) * a.groups + g0 + rank) * a.n_sel;
  const uint32_t take = static_cast<uint32_t>(min(nb, a.n_sel));
  uint64_t threshold = 0;
  uint32_t stay_equal = 0xffffffffu;  // how many keys equal to the threshold are picked (the first ones)
  if (static_cast<int>(take) < nb) {
    uint32_t left = static_cast<uint32_t>(nb) - take;  // how many keys that share the prefix are not picked
    for (int shift = 56; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      __syncthreads();
      for (int i = tid; i < nb; i += kSelThreads) {
        const uint64_t k = keys[i];
        if (shift == 56 || (k >> (shift + 8)) == (threshold >> (shift + 8)))
          atomicAdd(&hist[static_cast<uint32_t>(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      const uint32_t c = hist[tid];
      uint32_t inc = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += v;
      }
      if (lane == 31) sum[warp] = inc;
      __syncthreads();
      for (int w = 0; w < warp; ++w) inc += sum[w];
      if (inc - c < left && left <= inc) {
        found[0] = static_cast<uint32_t>(tid);
        found[1] = inc - c;
        found[2] = c;
      }
      __syncthreads();
      threshold |= static_cast<uint64_t>(found[0]) << shift;
      left -= found[1];
      stay_equal = found[2] - left;
      if (left == found[2] && shift > 0) {  // none of the digit's keys is picked: the threshold is the next digit's start
        threshold += 1ull << shift;
        stay_equal = 0xffffffffu;
        break;
      }
      __syncthreads();
    }
  }
  // picks in ascending order: each warp a contiguous piece of the blocks
  const int piece = (nb + kSelWarps - 1) / kSelWarps;
  const int a0 = min(nb, warp * piece), a1 = min(nb, a0 + piece);
  uint32_t more = 0, same = 0;
  for (int i = a0 + lane; i < a1; i += 32) {
    more += keys[i] > threshold;
    same += keys[i] == threshold;
  }
  more = __reduce_add_sync(0xffffffffu, more);
  same = __reduce_add_sync(0xffffffffu, same);
  __syncthreads();
  if (lane == 0) {
    hist[warp] = more;
    hist[32 + warp] = same;
  }
  __syncthreads();
  uint32_t at = 0, eq = 0;
  for (int w = 0; w < warp; ++w) {
    const uint32_t n = hist[32 + w];
    at += hist[w] + (eq < stay_equal ? min(n, stay_equal - eq) : 0u);
    eq += n;
  }
  const uint32_t lt = (1u << lane) - 1u;
  for (int i = a0; i < a1; i += 32) {
    const bool in = i + lane < a1;
    const uint64_t k = in ? keys[i + lane] : 0ull;
    const uint32_t em = __ballot_sync(0xffffffffu, in && k == threshold);
    const bool pick = in && (k > threshold || (k == threshold && eq + __popc(em & lt) < stay_equal));
    const uint32_t pm = __ballot_sync(0xffffffffu, pick);
    if (pick) out[at + __popc(pm & lt)] = i + lane;
    at += __popc(pm);
    eq += __popc(em);
  }
  for (int i = static_cast<int>(take) + tid; i < a.n_sel; i += kSelThreads) out[i] = -1;
}

template <typename T, int HD>
cudaError_t select_hd(const BlockSelectLaunch& a, cudaStream_t s, int* n) {
  const int C = (a.groups > 1 || a.n_blocks > 128) ? kSelCluster : 1;
  const size_t smem = sizeof(uint64_t) * static_cast<size_t>(a.n_blocks > 0 ? a.n_blocks : 1);
  auto kernel = block_select_kernel<T, HD>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(uint64_t) * kMaxBlocks));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.groups + C - 1) / C * C), static_cast<unsigned>(a.n_heads));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  *n += 1;
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t select_t(const BlockSelectLaunch& a, cudaStream_t s, int* n) {
  switch (a.head_dim) {
    case 16:
      return select_hd<T, 16>(a, s, n);
    case 32:
      return select_hd<T, 32>(a, s, n);
    case 64:
      return select_hd<T, 64>(a, s, n);
    default:
      return select_hd<T, 128>(a, s, n);
  }
}

}  // namespace

cudaError_t launch_block_means(const BlockMeansLaunch& a, cudaStream_t s, int* n_launched) {
  const int es = a.dtype == 1 ? 4 : 2;
  const int64_t blocks = (a.n_k + a.block - 1) / a.block - a.first;
  if (blocks <= 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((a.cols * es + kMeanCols * 16 - 1) / (kMeanCols * 16)));
  const bool al = aligned16(a.k) && a.ld_k * es % 16 == 0;
  if (a.dtype == 1) {
    if (al)
      block_means_kernel<float, true><<<grid, kMeanThreads, 0, s>>>(a);
    else
      block_means_kernel<float, false><<<grid, kMeanThreads, 0, s>>>(a);
  } else {
    if (al)
      block_means_kernel<__nv_bfloat16, true><<<grid, kMeanThreads, 0, s>>>(a);
    else
      block_means_kernel<__nv_bfloat16, false><<<grid, kMeanThreads, 0, s>>>(a);
  }
  *n_launched += 1;
  return cudaGetLastError();
}

bool block_select_supported(int64_t n_blocks) { return n_blocks <= kMaxBlocks; }

cudaError_t launch_block_select(const BlockSelectLaunch& a, cudaStream_t s, int* n_launched) {
  return a.dtype == 1 ? select_t<float>(a, s, n_launched) : select_t<__nv_bfloat16>(a, s, n_launched);
}

}  // namespace ispa
