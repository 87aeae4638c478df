// attn_blocks_rows.cu -- dual-stream attention over sink, local and selected history blocks, one
// query row and head per cluster, statistics and sums in fp32: the single-token form (bf16, each query with
// its own picks), the form of few rows, and the kernel of every fp32 call.
//
// The row's keys are cut into units inside one segment or one picked block, and the units go round-robin
// to the warps of the cluster, so a single token's keys are read by many SMs at once.  Each warp keeps
// an online-softmax state (max, sum, accumulator) per branch; the states are joined by log-sum-exp in a
// fixed order: lanes by shuffles, warps in shared memory, CTAs through distributed shared memory.
//   bf16, head_dim 64 or 128, 16-byte aligned rows: units of 16 keys, both products by mma.m16n8k16.
//   S = K q^T has the query as one of eight columns; O^T = V^T p^T has the weights as three, p rounded to
//   bf16 and twice what the rounding left (so p keeps its 24 bits, at no further product).  Each warp copies
//   its units ahead (cp.async) into its own ring of kStages units in shared memory.  (By multiply-adds
//   and shuffles a unit took over 400 instructions, and their latency, not memory, set the pace.)
//   Other cases (and bf16 with ISPA_ATTN_CUDA_CORES): a key row spans kLanes lanes (16 bytes each), units of 8 warp-wide loads, dot products
//   by multiply-adds and shuffles, a state per lane group.
// Bound: the read of the keys and values, each once.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "rows.cuh"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace ispa {
namespace {

constexpr int kLoads = 8;   // key rows per lane group and unit (multiply-add form)
constexpr int kStages = 2;  // units in flight per warp (mma form)
constexpr int kMaxCluster = 8;

template <int HD>
struct State {  // one branch's state of a CTA
  float m, l;
  float acc[HD];
};

// kMma: both products by mma.sync (bf16, head_dim 64 or 128, aligned rows), else by multiply-adds.
template <typename T, int HD, bool kAligned, bool kMma_>
struct Kind {
  static constexpr bool kMma = kMma_;
  static_assert(!kMma || (sizeof(T) == 2 && kAligned && HD >= 64), "fragments of aligned bf16 rows");
  static constexpr int kUnit = kMma ? 16 : kLoads * Row<T, HD>::kPerWarp;  // keys per unit
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = kMma ? 1 : 2;  // per SM
  static constexpr int kPieces = HD / 8;  // 16-byte pieces of a lane per unit: a quarter each of two key rows, and its value rows
  static constexpr int kSmem = kMma ? kWarps * kStages * kPieces * 512 : 0;
};

__device__ __forceinline__ void cp_async16(uint32_t smem_dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(src) : "memory");
}
// The same, zeros where `real` is false (src is not read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem_dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

template <typename T, int HD, bool kAligned, bool kMma>
__global__ void __launch_bounds__(Kind<T, HD, kAligned, kMma>::kThreads, Kind<T, HD, kAligned, kMma>::kCtas)
    attn_blocks_rows_kernel(const AttnLaunch a, const BlockList b) {
  using R = Row<T, HD>;
  using X = Kind<T, HD, kAligned, kMma>;
  constexpr int kUnit = X::kUnit, kWarps = X::kWarps, kThreads = X::kThreads;
  extern __shared__ __align__(16) uint4 ring[];  // [warp][stage][piece][lane]
  __shared__ float sm[2][kWarps], sl[2][kWarps];
  __shared__ float sacc[2][kWarps][HD];
  __shared__ State<HD> cta[kMaxCluster][2];  // in CTA 0: every CTA's states
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  cluster.barrier_arrive();  // completes once every CTA of the cluster runs
  const int64_t row = blockIdx.x / C;
  const int head = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane / R::kLanes, gl = lane % R::kLanes;
  const int64_t col = static_cast<int64_t>(head) * HD + gl * R::kVec;

  const float scale = a.scale * 1.4426950408889634f;  // scores in base 2
  const int mg = lane >> 2, mc = lane & 3;            // fragment row and column group of an mma
  float q[kMma ? 1 : R::kVec];
  uint4 qf[kMma ? HD / 32 : 2];
  if constexpr (kMma) {  // the query is column 0 of the eight
#pragma unroll
    for (int j = 0; j < HD / 32; ++j)
      qf[j] = mg == 0 ? load_raw<T, false>(static_cast<const T*>(a.q) + row * a.ld_q + static_cast<int64_t>(head) * HD + 8 * mc + 32 * j)
                      : make_uint4(0, 0, 0, 0);
  } else {
    unpack<T>(load_raw<T, false>(static_cast<const T*>(a.q) + row * a.ld_q + col), q);
#pragma unroll
    for (int e = 0; e < R::kVec; ++e) q[e] *= scale;
  }

  // The units of this warp, every `step`-th: sink, local, then the picked blocks.  Positions in the list
  // advance without divisions, and a pick is loaded one unit before it is needed.
  const int32_t* list = b.idx + (static_cast<int64_t>(head) * b.groups + row / b.q_block) * b.n_sel;
  const int n_sink = static_cast<int>(a.n_kv[0]), n_loc = static_cast<int>(a.n_kv[1]), n_hist = static_cast<int>(a.n_kv[2]);
  const int units0 = (n_sink + kUnit - 1) / kUnit, units01 = units0 + (n_loc + kUnit - 1) / kUnit;
  const int per_block = (b.block + kUnit - 1) / kUnit;
  const int units = units01 + b.n_sel * per_block;
  const int step = C * kWarps, d_entry = step / per_block, d_sub = step % per_block;
  int u = rank * kWarps + warp, entry = 0, sub = 0, pick = -1;
  auto enter_history = [&]() {  // u is the warp's first unit there
    entry = (u - units01) / per_block;
    sub = (u - units01) % per_block;
    if (u < units) pick = __ldg(list + entry);
  };
  if (u >= units01) enter_history();

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[2][R::kVec] = {};              // multiply-add form
  float dacc[2][kMma ? HD / 16 : 1][4] = {};  // mma form: rows of O^T, columns 0 and 1
  // The warp's next unit: its segment, first key and number of keys (0: none; the list may name no block).
  auto next_unit = [&](int& seg, int& key0, int& n) {
    seg = 0;
    key0 = n = 0;
    if (u < units01) {
      seg = u >= units0;
      key0 = (u - (seg ? units0 : 0)) * kUnit;
      n = min(kUnit, (seg ? n_loc : n_sink) - key0);
      u += step;
      if (u >= units01) enter_history();
    } else if (u < units) {
      seg = 2;
      if (pick >= 0 && pick < b.n_blocks) {  // any other entry names no block
        key0 = pick * b.block + sub * kUnit;
        n = max(0, min(min(kUnit, b.block - sub * kUnit), n_hist - key0));
      }
      u += step;
      entry += d_entry;
      sub += d_sub;
      if (sub >= per_block) {
        sub -= per_block;
        ++entry;
      }
      if (u < units) pick = __ldg(list + entry);
    }
  };
  // bf16 unit.  Stage layout: the lane's own pieces of the key rows mg and mg + 8 ([piece][lane]), then the
  // 16 value rows, 16-byte chunk q of row r at q ^ (r & 7).
  constexpr int kPK = HD / 32;  // pieces of a lane per key row
  constexpr int kChunks = HD / 8;
  auto stage_of = [&](int st) { return ring + (warp * kStages + st) * X::kPieces * 32; };
  auto fetch = [&](int st, int seg, int key0, int n) {  // past the end: the last key again, values of 0
    const int64_t ld_k = a.ld_k[seg], ld_v = a.ld_v[seg];
    const T* k_lo = static_cast<const T*>(a.k[seg]) + static_cast<int64_t>(head) * HD + 8 * mc + (key0 + min(mg, n - 1)) * ld_k;
    const T* k_hi = k_lo + (min(mg + 8, n - 1) - min(mg, n - 1)) * ld_k;
    const T* V = static_cast<const T*>(a.v[seg]) + col + (key0 + min(grp, n - 1)) * ld_v;
    const uint32_t dst = smem_u32(stage_of(st));
#pragma unroll
    for (int j = 0; j < kPK; ++j) {
      cp_async16(dst + (j * 32 + lane) * 16, k_lo + 32 * j);
      cp_async16(dst + ((kPK + j) * 32 + lane) * 16, k_hi + 32 * j);
    }
#pragma unroll
    for (int i = 0; i < 16 / R::kPerWarp; ++i) {
      const int r = i * R::kPerWarp + grp;
      // a weight of 0 times the last value again would be NaN where that is infinite
      cp_async16_or_zero(dst + (2 * kPK * 32 + r * kChunks + (gl ^ (r & 7))) * 16, V, r < n);
      if (r + R::kPerWarp < n) V += R::kPerWarp * ld_v;  // else V stays in bounds
    }
  };
  auto work_mma = [&](int st, int n, float& mb, float& lb, float (*ab)[4]) {
    const uint4* buf = stage_of(st);
    Mma16<kMma ? HD : 64> keys;
#pragma unroll
    for (int j = 0; j < kPK; ++j) {
      keys.lo[j] = buf[j * 32 + lane];
      keys.hi[j] = buf[(kPK + j) * 32 + lane];
    }
    float d[4];
    keys.template scores<2>(qf, d);
    // column 0 lies in the lanes with mc == 0: d[0] for key mg, d[2] for key mg + 8
    float s0 = mg < n ? d[0] * scale : -INFINITY, s1 = mg + 8 < n ? d[2] * scale : -INFINITY;
    float mx = mc == 0 ? fmaxf(s0, s1) : -INFINITY;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    mx = fmaxf(mx, mb);
    if (mx != mb) {  // uniform over the warp
      const float alpha = fast_exp2(mb - mx);
      mb = mx;
      lb *= alpha;
#pragma unroll
      for (int t = 0; t < HD / 16; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) ab[t][e] *= alpha;
    }
    const float ref = mx == -INFINITY ? 0.f : mx;  // keys that score -inf weigh 0, the first ones too
    const float p0 = fast_exp2(s0 - ref), p1 = fast_exp2(s1 - ref);
    lb += p0 + p1;  // of the lanes with mc == 0
    // weights as the second operand: column mg, keys 2 mc + {0, 1} and 8 more; column 0 the rounded
    // weights, columns 1 and 2 what the rounding before left, the others zero
    uint32_t w[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float a0 = __shfl_sync(0xffffffffu, x ? p1 : p0, 8 * mc), a1 = __shfl_sync(0xffffffffu, x ? p1 : p0, 8 * mc + 4);
      const uint32_t hi = pack_bf16x2(a0, a1);
      const float r0 = a0 - __uint_as_float(hi << 16), r1 = a1 - __uint_as_float(hi & 0xFFFF0000u);
      const uint32_t mid = pack_bf16x2(r0, r1);
      const uint32_t lo = pack_bf16x2(r0 - __uint_as_float(mid << 16), r1 - __uint_as_float(mid & 0xFFFF0000u));
      w[x] = mg == 0 ? hi : (mg == 1 ? mid : (mg == 2 ? lo : 0u));
    }
    // first operand: rows 16 t + {0..15} of V^T, the four 8 x 8 parts by one transposing load
    const int r = ((lane >> 4) & 1) * 8 + (lane & 7);
    const uint32_t vrow = smem_u32(buf) + (2 * kPK * 32 + r * kChunks) * 16;
#pragma unroll
    for (int t = 0; t < HD / 16; ++t) {
      uint32_t v[4];
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                   : "r"(vrow + (((2 * t + ((lane >> 3) & 1)) ^ (r & 7)) << 4)));
      mma_bf16(ab[t], v[0], v[1], v[2], v[3], w[0], w[1]);
    }
  };
  auto work = [&](int seg, int key0, int n, float& mb, float& lb, float* ab) {
    const T* K = static_cast<const T*>(a.k[seg]) + col;
    const T* V = static_cast<const T*>(a.v[seg]) + col;
    uint4 kw[kLoads], vw[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = i * R::kPerWarp + grp;
      kw[i] = vw[i] = make_uint4(0, 0, 0, 0);
      if (j < n) kw[i] = load_raw<T, kAligned>(K + static_cast<int64_t>(key0 + j) * a.ld_k[seg]);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = i * R::kPerWarp + grp;
      if (j < n) vw[i] = load_raw<T, kAligned>(V + static_cast<int64_t>(key0 + j) * a.ld_v[seg]);
    }
    float s[kLoads], mx = mb;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      float kv[R::kVec], d = 0.f;
      unpack<T>(kw[i], kv);
#pragma unroll
      for (int e = 0; e < R::kVec; ++e) d = fmaf(q[kMma ? 0 : e], kv[e], d);
      d = row_sum<R::kLanes>(d);
      s[i] = i * R::kPerWarp + grp < n ? d : -INFINITY;
      mx = fmaxf(mx, s[i]);
    }
    const float ref = mx == -INFINITY ? 0.f : mx;  // no key yet, or keys that score -inf: weight 0
    const float alpha = exp2f(mb - ref);
    mb = mx;
    lb *= alpha;
#pragma unroll
    for (int e = 0; e < R::kVec; ++e) ab[e] *= alpha;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      float vv[R::kVec];
      const float p = exp2f(s[i] - ref);
      unpack<T>(vw[i], vv);
      lb += p;
#pragma unroll
      for (int e = 0; e < R::kVec; ++e) ab[e] = fmaf(p, vv[e], ab[e]);
    }
  };
  bool in_hist = false;
  if constexpr (kMma) {
    int segs[kStages], ns[kStages];  // of the units in flight, oldest first
    auto start = [&](int st, int& seg, int& n) {
      int key0;
      next_unit(seg, key0, n);
      if (n > 0) fetch(st, seg, key0, n);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int mine = u < units ? (units - u + step - 1) / step : 0;  // the warp's units
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) start(i, segs[i], ns[i]);
    for (int st = 0; mine > 0; --mine) {
      start(st == 0 ? kStages - 1 : st - 1, segs[kStages - 1], ns[kStages - 1]);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();  // a warp's lanes read each other's copies of the values
      if (ns[0] > 0) {  // uniform over the warp
        if (segs[0] == 2 && !in_hist) {  // the local branch is complete: set its state aside
          in_hist = true;
          m[1] = m[0], l[1] = l[0];
          m[0] = -INFINITY, l[0] = 0.f;
#pragma unroll
          for (int t = 0; t < HD / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              dacc[kMma ? 1 : 0][kMma ? t : 0][e] = dacc[0][kMma ? t : 0][e];
              dacc[0][kMma ? t : 0][e] = 0.f;
            }
        }
        work_mma(st, ns[0], m[0], l[0], dacc[0]);
      }
      __syncwarp();  // ... before the stage is filled again
      st = st == kStages - 1 ? 0 : st + 1;
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) {
        segs[i] = segs[i + 1];
        ns[i] = ns[i + 1];
      }
    }
  } else {
    while (u < units) {
      int seg, key0, n;
      next_unit(seg, key0, n);
      if (n == 0) continue;  // uniform over the warp
      if (seg == 2)
        work(2, key0, n, m[1], l[1], acc[1]);
      else
        work(seg, key0, n, m[0], l[0], acc[0]);
    }
  }

  // the warp's states, then the warps of the CTA
  if constexpr (kMma) {
#pragma unroll
    for (int br = 0; br < 2; ++br) {
      const int from = in_hist ? 1 - br : br;  // the state set aside is the local one
      float lw = mc == 0 ? (from ? l[1] : l[0]) : 0.f;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, off);
      if (lane == 0) {
        sm[br][warp] = from ? m[1] : m[0];
        sl[br][warp] = lw;
      }
#pragma unroll
      for (int t = 0; t < HD / 16; ++t) {
        const float* o = from ? dacc[1][kMma ? t : 0] : dacc[0][kMma ? t : 0];
        const float lo0 = __shfl_down_sync(0xffffffffu, o[0], 1), lo2 = __shfl_down_sync(0xffffffffu, o[2], 1);  // column 2
        if (mc == 0) {
          // an infinite value times a remainder of zero or of the other sign is no part of the sum
          sacc[br][warp][16 * t + mg] = o[0] + (isfinite(o[0]) ? o[1] + lo0 : 0.f);
          sacc[br][warp][16 * t + 8 + mg] = o[2] + (isfinite(o[2]) ? o[3] + lo2 : 0.f);
        }
      }
    }
  } else {
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
  }
  __syncthreads();
  cluster.barrier_wait();
  State<HD>* dst = cluster.map_shared_rank(cta[rank], 0);
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
    dst[br].acc[e] = o;
    if (e == 0) {
      dst[br].m = mx;
      dst[br].l = sum;
    }
  }
  cluster.barrier_arrive();
  if (rank != 0) return;  // nobody reads this CTA's shared memory
  cluster.barrier_wait();
  if (tid < HD) {  // HD <= kThreads
    float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, o[2] = {0.f, 0.f};
    for (int br = 0; br < 2; ++br) {
      for (int r = 0; r < C; ++r) mx[br] = fmaxf(mx[br], cta[r][br].m);
      for (int r = 0; r < C; ++r) {
        const State<HD>& st = cta[r][br];
        const float f = mx[br] == -INFINITY ? 0.f : exp2f(st.m - mx[br]);
        sum[br] = fmaf(st.l, f, sum[br]);
        o[br] = fmaf(st.acc[tid], f, o[br]);
      }
    }
    const float ln2 = 0.69314718055994531f;
    const bool has_hist = !(sum[1] == 0.f);  // a NaN in the branch stays one
    const float lse_l = mx[0] + log2f(sum[0]);
    const float lse_h = has_hist ? mx[1] + log2f(sum[1]) : -INFINITY;
    const float vl = o[0] / sum[0];
    float vf = vl, vd = vl - vl;
    if (has_hist) {
      const float top = fmaxf(lse_l, lse_h);
      const float wl = exp2f(lse_l - top), wh = exp2f(lse_h - top), vh = o[1] / sum[1];
      vf = (wl * vl + wh * vh) / (wl + wh);
      vd = wh / (wl + wh) * (vh - vl);  // vf - vl would lose a share below the rounding of vf
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
    if (a.d_out) put(a.d_out, vd);
    if (tid == 0) {
      a.lse_loc[static_cast<int64_t>(head) * a.n_q + row] = lse_l * ln2;
      a.lse_hist[static_cast<int64_t>(head) * a.n_q + row] = has_hist ? lse_h * ln2 : -INFINITY;
    }
  }
}

template <typename T, int HD, bool kAligned, bool kMma>
cudaError_t launch_kind(const AttnLaunch& a, const BlockList& b, cudaStream_t s, int* n) {
  using X = Kind<T, HD, kAligned, kMma>;
  // Cluster size: split a row's keys while all CTAs still run at once and a warp keeps at least two units.
  const int64_t keys = a.n_kv[0] + a.n_kv[1] + static_cast<int64_t>(b.n_sel) * b.block;
  const int64_t most = std::min(X::kCtas * 148 / (a.n_q * a.n_heads), keys / (static_cast<int64_t>(2) * X::kWarps * X::kUnit));
  const int C = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxCluster, most)));
  auto kernel = attn_blocks_rows_kernel<T, HD, kAligned, kMma>;
  if (X::kSmem > 0) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, X::kSmem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_q * C), static_cast<unsigned>(a.n_heads));
  cfg.blockDim = dim3(X::kThreads);
  cfg.dynamicSmemBytes = X::kSmem;
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

template <typename T, int HD>
cudaError_t launch_hd(const AttnLaunch& a, const BlockList& b, bool cuda_cores, cudaStream_t s, int* n) {
  bool al = true;
  for (int i = 0; i < 3; ++i)
    if (a.n_kv[i] > 0)
      al = al && aligned16(a.k[i]) && aligned16(a.v[i]) && a.ld_k[i] * static_cast<int64_t>(sizeof(T)) % 16 == 0 &&
           a.ld_v[i] * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  if constexpr (sizeof(T) == 2 && HD >= 64) {
    if (al && !cuda_cores) return launch_kind<T, HD, true, true>(a, b, s, n);
  }
  return al ? launch_kind<T, HD, true, false>(a, b, s, n) : launch_kind<T, HD, false, false>(a, b, s, n);
}

template <typename T>
cudaError_t launch_t(const AttnLaunch& a, const BlockList& b, bool cuda_cores, cudaStream_t s, int* n) {
  switch (a.head_dim) {
    case 16:
      return launch_hd<T, 16>(a, b, cuda_cores, s, n);
    case 32:
      return launch_hd<T, 32>(a, b, cuda_cores, s, n);
    case 64:
      return launch_hd<T, 64>(a, b, cuda_cores, s, n);
    default:
      return launch_hd<T, 128>(a, b, cuda_cores, s, n);
  }
}

}  // namespace

cudaError_t launch_attn_blocks_rows(const AttnLaunch& a, const BlockList& b, bool cuda_cores, cudaStream_t s, int* n_launched) {
  return a.dtype == 1 ? launch_t<float>(a, b, cuda_cores, s, n_launched) : launch_t<__nv_bfloat16>(a, b, cuda_cores, s, n_launched);
}

}  // namespace ispa
