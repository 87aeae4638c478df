// attn_blocks_rows.cu -- dual-stream attention over sink, local and selected history blocks, one
// query row and head per cluster (CUDA cores, fp32 arithmetic): the single-token form (bf16, each
// query with its own picks) and the kernel of every fp32 call.
//
// The row's keys are cut into units of 8 warp-wide loads inside one segment or one picked block, and
// the units go round-robin to the warps of the cluster, so a single token's keys are read by many SMs
// at once.  A key row spans kLanes lanes (16 bytes each): a warp loads 8 x 32/kLanes keys and as many
// value rows before it uses them.  Every lane group keeps its own online-softmax state (max, sum,
// accumulator) per branch; the states are joined by log-sum-exp in a fixed order: lane groups by
// shuffles, warps in shared memory, CTAs through distributed shared memory.
// Bound: the read of the keys and values, each once.
#include <cooperative_groups.h>
#include <math.h>

#include "internal.h"
#include "rows.cuh"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace ispa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 8;  // key rows per lane group and unit
constexpr int kMaxCluster = 8;

template <int HD>
struct State {  // one branch's state of a CTA
  float m, l;
  float acc[HD];
};

template <typename T, int HD, bool kAligned>
__global__ void __launch_bounds__(kThreads, 2) attn_blocks_rows_kernel(const AttnLaunch a, const BlockList b) {
  using R = Row<T, HD>;
  constexpr int kUnit = kLoads * R::kPerWarp;  // keys per unit
  __shared__ float sm[2][kWarps], sl[2][kWarps];
  __shared__ float sacc[2][kWarps][HD];
  __shared__ State<HD> cta[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int64_t row = blockIdx.x / C;
  const int head = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane / R::kLanes, gl = lane % R::kLanes;
  const int64_t col = static_cast<int64_t>(head) * HD + gl * R::kVec;

  float q[R::kVec];
  unpack<T>(load_raw<T, false>(static_cast<const T*>(a.q) + row * a.ld_q + col), q);
  const float scale = a.scale * 1.4426950408889634f;  // scores in base 2
#pragma unroll
  for (int e = 0; e < R::kVec; ++e) q[e] *= scale;

  const int32_t* list = b.idx + (static_cast<int64_t>(head) * b.groups + row / b.q_block) * b.n_sel;
  const int64_t units0 = (a.n_kv[0] + kUnit - 1) / kUnit, units1 = (a.n_kv[1] + kUnit - 1) / kUnit;
  const int per_block = (b.block + kUnit - 1) / kUnit;
  const int64_t units = units0 + units1 + static_cast<int64_t>(b.n_sel) * per_block;

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[2][R::kVec] = {};
  auto unit_range = [&](int64_t u, int& seg, int64_t& key0, int& n) {
    if (u < units0) {
      seg = 0;
      key0 = u * kUnit;
      n = static_cast<int>(min(static_cast<int64_t>(kUnit), a.n_kv[0] - key0));
    } else if (u < units0 + units1) {
      seg = 1;
      key0 = (u - units0) * kUnit;
      n = static_cast<int>(min(static_cast<int64_t>(kUnit), a.n_kv[1] - key0));
    } else {
      seg = 2;
      const int64_t w = u - units0 - units1;
      const int32_t pick = list[w / per_block];
      const int off = static_cast<int>(w % per_block) * kUnit;
      n = 0;
      key0 = 0;
      if (pick >= 0 && pick < b.n_blocks) {  // any other entry names no block
        key0 = static_cast<int64_t>(pick) * b.block + off;
        n = static_cast<int>(min(static_cast<int64_t>(min(kUnit, b.block - off)), a.n_kv[2] - key0));
        n = max(n, 0);
      }
    }
  };
  auto work = [&](int seg, int64_t key0, int n, float& mb, float& lb, float* ab) {
    const T* K = static_cast<const T*>(a.k[seg]) + col;
    const T* V = static_cast<const T*>(a.v[seg]) + col;
    uint4 kw[kLoads], vw[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = i * R::kPerWarp + grp;
      kw[i] = vw[i] = make_uint4(0, 0, 0, 0);
      if (j < n) kw[i] = load_raw<T, kAligned>(K + (key0 + j) * a.ld_k[seg]);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = i * R::kPerWarp + grp;
      if (j < n) vw[i] = load_raw<T, kAligned>(V + (key0 + j) * a.ld_v[seg]);
    }
    float s[kLoads], mx = mb;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      float kv[R::kVec], d = 0.f;
      unpack<T>(kw[i], kv);
#pragma unroll
      for (int e = 0; e < R::kVec; ++e) d = fmaf(q[e], kv[e], d);
      d = row_sum<R::kLanes>(d);
      s[i] = i * R::kPerWarp + grp < n ? d : -INFINITY;
      mx = fmaxf(mx, s[i]);
    }
    if (grp >= n && mb == -INFINITY) return;  // this lane group has met no key yet (no shuffles below)
    const float alpha = exp2f(mb - mx);
    mb = mx;
    lb *= alpha;
#pragma unroll
    for (int e = 0; e < R::kVec; ++e) ab[e] *= alpha;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      float vv[R::kVec];
      const float p = exp2f(s[i] - mx);
      unpack<T>(vw[i], vv);
      lb += p;
#pragma unroll
      for (int e = 0; e < R::kVec; ++e) ab[e] = fmaf(p, vv[e], ab[e]);
    }
  };
  for (int64_t u = static_cast<int64_t>(rank) * kWarps + warp; u < units; u += static_cast<int64_t>(C) * kWarps) {
    int seg, n;
    int64_t key0;
    unit_range(u, seg, key0, n);
    if (n == 0) continue;  // uniform over the warp
    if (seg < 2)
      work(seg, key0, n, m[0], l[0], acc[0]);
    else
      work(2, key0, n, m[1], l[1], acc[1]);
  }

  // lane groups of the warp, then the warps of the CTA
#pragma unroll
  for (int br = 0; br < 2; ++br) {
#pragma unroll
    for (int off = R::kLanes; off < 32; off <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[br], off), lo = __shfl_xor_sync(0xffffffffu, l[br], off);
      const float mx = fmaxf(m[br], mo);
      const float wa = mx == -INFINITY ? 0.f : exp2f(m[br] - mx), wb = mx == -INFINITY ? 0.f : exp2f(mo - mx);
      l[br] = l[br] * wa + lo * wb;
#pragma unroll
      for (int e = 0; e < R::kVec; ++e) acc[br][e] = acc[br][e] * wa + __shfl_xor_sync(0xffffffffu, acc[br][e], off) * wb;
      m[br] = mx;
    }
    if (lane < R::kLanes) {
#pragma unroll
      for (int e = 0; e < R::kVec; ++e) sacc[br][warp][gl * R::kVec + e] = acc[br][e];
    }
    if (lane == 0) {
      sm[br][warp] = m[br];
      sl[br][warp] = l[br];
    }
  }
  __syncthreads();
  for (int x = tid; x < 2 * HD; x += kThreads) {
    const int br = x / HD, e = x % HD;
    float mx = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[br][w]);
    float sum = 0.f, o = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = mx == -INFINITY ? 0.f : exp2f(sm[br][w] - mx);
      sum = fmaf(sl[br][w], f, sum);
      o = fmaf(sacc[br][w][e], f, o);
    }
    cta[br].acc[e] = o;
    if (e == 0) {
      cta[br].m = mx;
      cta[br].l = sum;
    }
  }
  cluster.sync();
  if (rank == 0 && tid < HD) {
    float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, o[2] = {0.f, 0.f};
    for (int br = 0; br < 2; ++br) {
      for (int r = 0; r < C; ++r) mx[br] = fmaxf(mx[br], cluster.map_shared_rank(&cta[br], r)->m);
      for (int r = 0; r < C; ++r) {
        const State<HD>* st = cluster.map_shared_rank(&cta[br], r);
        const float f = mx[br] == -INFINITY ? 0.f : exp2f(st->m - mx[br]);
        sum[br] = fmaf(st->l, f, sum[br]);
        o[br] = fmaf(st->acc[tid], f, o[br]);
      }
    }
    const float ln2 = 0.69314718055994531f;
    const bool has_hist = !(sum[1] == 0.f);  // a NaN in the branch stays one
    const float lse_l = mx[0] + log2f(sum[0]);
    const float lse_h = has_hist ? mx[1] + log2f(sum[1]) : -INFINITY;
    const float vl = o[0] / sum[0];
    float vf = vl;
    if (has_hist) {
      const float top = fmaxf(lse_l, lse_h);
      const float wl = exp2f(lse_l - top), wh = exp2f(lse_h - top);
      vf = (wl * vl + wh * (o[1] / sum[1])) / (wl + wh);
    }
    const int64_t at = row * a.ld_o + static_cast<int64_t>(head) * HD + tid;
    auto put = [&](void* base, float v) {
      if constexpr (sizeof(T) == 2)
        static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(v);
      else
        static_cast<float*>(base)[at] = v;
    };
    put(a.o_loc, vl);
    put(a.o_full, vf);
    if (a.d_out) put(a.d_out, vf - vl);
    if (tid == 0) {
      a.lse_loc[static_cast<int64_t>(head) * a.n_q + row] = lse_l * ln2;
      a.lse_hist[static_cast<int64_t>(head) * a.n_q + row] = has_hist ? lse_h * ln2 : -INFINITY;
    }
  }
  cluster.sync();  // the states stay readable until rank 0 has joined them
}

template <typename T, int HD>
cudaError_t launch_hd(const AttnLaunch& a, const BlockList& b, cudaStream_t s, int* n) {
  bool al = true;
  for (int i = 0; i < 3; ++i)
    if (a.n_kv[i] > 0)
      al = al && aligned16(a.k[i]) && aligned16(a.v[i]) && a.ld_k[i] * static_cast<int64_t>(sizeof(T)) % 16 == 0 &&
           a.ld_v[i] * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  // Cluster size: split a row's keys while the rows alone leave SMs idle and a CTA keeps at least two
  // units per warp.
  constexpr int kUnit = kLoads * Row<T, HD>::kPerWarp;
  const int64_t keys = a.n_kv[0] + a.n_kv[1] + static_cast<int64_t>(b.n_sel) * b.block;
  int C = 1;
  while (C < kMaxCluster && a.n_q * a.n_heads * C < 2 * 148 && keys > static_cast<int64_t>(2) * C * kWarps * kUnit) C *= 2;
  auto kernel = al ? attn_blocks_rows_kernel<T, HD, true> : attn_blocks_rows_kernel<T, HD, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_q * C), static_cast<unsigned>(a.n_heads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, b);
  *n += 1;
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const AttnLaunch& a, const BlockList& b, cudaStream_t s, int* n) {
  switch (a.head_dim) {
    case 16:
      return launch_hd<T, 16>(a, b, s, n);
    case 32:
      return launch_hd<T, 32>(a, b, s, n);
    case 64:
      return launch_hd<T, 64>(a, b, s, n);
    default:
      return launch_hd<T, 128>(a, b, s, n);
  }
}

}  // namespace

cudaError_t launch_attn_blocks_rows(const AttnLaunch& a, const BlockList& b, cudaStream_t s, int* n_launched) {
  return a.dtype == 1 ? launch_t<float>(a, b, s, n_launched) : launch_t<__nv_bfloat16>(a, b, s, n_launched);
}

}  // namespace ispa
