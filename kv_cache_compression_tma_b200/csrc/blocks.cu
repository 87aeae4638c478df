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
// A cluster of 8 CTAs serves 8 groups of one head: CTA r pools group r's queries and hands the mean to
// all, each CTA scores 1/8 of the blocks for all groups (so the means are read once per cluster), sends
// each score to the CTA that owns the group, and that CTA selects (radix select on 64-bit order keys,
// ties to the lowest block) and writes the picks in ascending order.  The scores are 8 groups x 8
// blocks x 4 products per mma.m8n8k4 in fp64.  The means go straight from memory into its fragments: a
// lane's products may be any quarter of the head_dim, so the four lanes of a row take alternate
// 16-byte pieces and a load covers whole 64-byte runs.  The mean queries stay in shared memory, which
// leaves registers for four CTAs per SM: a chunk's clusters then all run at once.  A lone group (a
// single token) is pooled by every CTA for itself and takes fused multiply-adds, an eighth of the work.
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
constexpr int kSelCluster = 8;  // CTAs, and groups, per cluster
constexpr int kMaxBlocks = 16384;  // one 64-bit order key per block in the owner's shared memory

__device__ __forceinline__ uint64_t order_key64(double s) {
  if (isnan(s)) s = -INFINITY;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(s + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// D (8 x 8) += A (8 x 4) B (4 x 8) in fp64: lane l holds A[l / 4][l % 4], B[l % 4][l / 4] and
// D[l / 4][2 (l % 4) + {0, 1}].
__device__ __forceinline__ void mma_f64(double& d0, double& d1, double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
               : "+d"(d0), "+d"(d1)
               : "d"(a), "d"(b));
}

// grid: (clusters per head) * 8, heads
template <typename T, int HD, bool kAligned>
__global__ void __launch_bounds__(kSelThreads, 4) block_select_kernel(const BlockSelectLaunch a) {
  constexpr int kQuarter = HD / 4;               // products of a lane per score
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  constexpr int kColThreads = HD / kVec;
  constexpr int kRowGroups = kSelThreads / kColThreads;
  extern __shared__ __align__(16) uint64_t keys[];  // [n_blocks] of the group this CTA owns
  __shared__ __align__(16) double qm[kSelCluster][HD + 2];  // a row's four lanes read two rows' 128 bytes at a time
  __shared__ double part[kRowGroups][HD];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sum[kSelWarps];
  __shared__ uint32_t found[3];                  // digit, keys below it, keys in it
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int head = blockIdx.y;
  const int64_t g0 = static_cast<int64_t>(blockIdx.x / kSelCluster) * kSelCluster;
  const int n_groups = static_cast<int>(a.groups - g0 < kSelCluster ? a.groups - g0 : kSelCluster);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nb = a.n_blocks;

  const int g_own = n_groups > 1 ? rank : 0;
  double mean = 0.0;
  if (g_own < n_groups) {  // the group's mean query, in 64 bits, summed in a fixed order
    const int64_t r0 = (g0 + g_own) * a.q_block;
    const int rows = static_cast<int>(a.n_q - r0 < a.q_block ? a.n_q - r0 : a.q_block);
    const int col = (tid % kColThreads) * kVec, tr = tid / kColThreads;
    const T* Q = static_cast<const T*>(a.q) + r0 * a.ld_q + static_cast<int64_t>(head) * HD + col;
    double s[kVec] = {};
#pragma unroll 4
    for (int r = tr; r < rows; r += kRowGroups) {
      float v[kVec];
      unpack<T>(load_raw<T, kAligned>(Q + r * a.ld_q), v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[e] += static_cast<double>(v[e]);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) part[tr][col + e] = s[e];
    __syncthreads();
    if (tid < HD) {
      const int used = rows < kRowGroups ? rows : kRowGroups;
      double t = 0.0;
      for (int p = 0; p < used; ++p) t += part[p][tid];
      mean = t / rows;
    }
  }
  cluster.sync();  // every CTA of the cluster runs before its shared memory is written from another
  if (tid < HD) {
    if (n_groups == 1)
      qm[0][tid] = mean;
    else
#pragma unroll
      for (int r = 0; r < kSelCluster; ++r) cluster.map_shared_rank(&qm[rank][0], r)[tid] = mean;  // 0 where no group is
  }
  if (n_groups == 1)
    __syncthreads();
  else
    cluster.sync();

  // Scores of this CTA's share of the blocks, eight at a time per warp.  Lane l: groups and blocks l / 4,
  // elements 16 i + 4 (l % 4) + {0..3}.
  const int sub = lane >> 2, c0 = (lane & 3) * 4;
  const int per = ((nb + kSelCluster - 1) / kSelCluster + 7) / 8 * 8;
  const int b0 = min(nb, rank * per), b1 = min(nb, b0 + per);
  uint64_t* owner = cluster.map_shared_rank(keys, n_groups > 1 ? sub : 0);
  for (int t = b0 + warp * 8; t < b1; t += kSelWarps * 8) {
    const int64_t b = min(t + sub, b1 - 1);
    const float* m = a.means + b * a.ld_means + static_cast<int64_t>(head) * HD + c0;
    uint4 w[kQuarter / 4];
#pragma unroll
    for (int i = 0; i < kQuarter / 4; ++i) w[i] = a.means_aligned ? load_raw<float, true>(m + 16 * i) : load_raw<float, false>(m + 16 * i);
    double d[2][2] = {};
    if (n_groups > 1) {
#pragma unroll
      for (int i = 0; i < kQuarter / 4; ++i) {
        float v[4];
        unpack<float>(w[i], v);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const double2 q = *reinterpret_cast<const double2*>(&qm[sub][16 * i + c0 + e]);
          mma_f64(d[0][0], d[0][1], q.x, static_cast<double>(v[e]));
          mma_f64(d[1][0], d[1][1], q.y, static_cast<double>(v[e + 1]));
        }
      }
      const int bo = t + 2 * (lane & 3);
      if (sub < n_groups) {
        const ulonglong2 k2 = make_ulonglong2(order_key64(d[0][0] + d[1][0]), order_key64(d[0][1] + d[1][1]));
        if (bo + 1 < b1)
          *reinterpret_cast<ulonglong2*>(owner + bo) = k2;  // bo is even
        else if (bo < b1)
          owner[bo] = k2.x;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kQuarter / 4; ++i) {
        float v[4];
        unpack<float>(w[i], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e >> 1][e & 1] = fma(qm[0][16 * i + c0 + e], static_cast<double>(v[e]), d[e >> 1][e & 1]);
      }
      double s = (d[0][0] + d[0][1]) + (d[1][0] + d[1][1]);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if ((lane & 3) == 0 && t + sub < b1) owner[t + sub] = order_key64(s);
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
  const size_t smem = sizeof(uint64_t) * static_cast<size_t>(a.n_blocks > 0 ? a.n_blocks : 1);
  const bool al = aligned16(a.q) && a.ld_q * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  auto kernel = al ? block_select_kernel<T, HD, true> : block_select_kernel<T, HD, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(uint64_t) * kMaxBlocks));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.groups + kSelCluster - 1) / kSelCluster * kSelCluster),
                     static_cast<unsigned>(a.n_heads));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSelCluster;
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

cudaError_t launch_block_select(const BlockSelectLaunch& in, cudaStream_t s, int* n_launched) {
  BlockSelectLaunch a = in;
  a.means_aligned = aligned16(a.means) && a.ld_means % 4 == 0;
  return a.dtype == 1 ? select_t<float>(a, s, n_launched) : select_t<__nv_bfloat16>(a, s, n_launched);
}

}  // namespace ispa
