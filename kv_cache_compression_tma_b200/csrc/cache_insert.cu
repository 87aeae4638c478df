// cache_insert.cu -- insertion of new tokens into a per-head cache of fixed capacity, evicting the
// entries of least accumulated attention weight.
//
// Per head the candidates are the n held entries (slots 0..n-1) followed by the n_new new tokens.  The
// `total` = min(capacity, n + n_new) candidates of highest rank stay; rank is the mass (NaN as -inf,
// a protected position as +inf), ties go to the lower candidate.  Held entries that stay keep their
// slot; the surviving new tokens take, in token order, the evicted slots in ascending order and then
// the slots from n on.  So only the survivors' K/V rows move, each read once from the new tokens and
// written once, and no row of the cache is read.
//
// One cluster of up to 16 CTAs per head, each with a contiguous slice of the held entries and of the
// new tokens; their 32-bit order keys stay in shared memory (beyond kMaxCached keys per CTA they are
// formed again from global memory at each use).  The lowest key that stays is found by a radix
// select, 8 bits a pass over a cluster-wide histogram (integer counts: no order dependence); counts
// per warp then give every evicted slot and every survivor its rank, and the CTA that owns the
// survivors of a rank range receives their slots in its shared memory.
#include <cooperative_groups.h>
#include <math.h>

#include "internal.h"
#include "rows.cuh"

namespace cg = cooperative_groups;

namespace ispa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxCached = 32768;   // order keys per CTA held in shared memory (128 KB)
constexpr int kMaxNewSlice = 4096;  // new tokens per CTA: their list of slots and of sources (32 KB)
constexpr int kUnroll = 4;          // state words in flight per thread while the keys are formed

struct Shared {
  // Digit counts of one pass, one column per lane: keys of a cache share few leading digits, and lanes
  // of a warp that add to one address would take turns.
  uint32_t hist[256][32];
  uint32_t total[4][256];       // ... summed, one array per pass, so one cluster barrier per pass is enough
  uint32_t sum[kWarps];         // scan scratch
  uint32_t digit, below, same;  // the pass's digit, the candidates below it, the candidates in it
  uint32_t counts[4];           // this CTA's {less, equal} of the held slice, then of the new slice
  uint32_t warp_counts[kWarps][4];
  uint32_t base[4];             // ranks before this CTA: held equal, new equal, holes, survivors
  uint32_t holes;               // evicted held entries of the head
  uint32_t first_survivor[kMaxCluster + 1];
};

// Order-preserving image of a rank: larger float, larger unsigned.
__device__ __forceinline__ uint32_t order_key(float mass, int32_t pos, int32_t keep_below, int32_t keep_from) {
  if (isnan(mass)) mass = -INFINITY;
  if (pos < keep_below || pos >= keep_from) mass = INFINITY;
  const uint32_t u = __float_as_uint(mass + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kThreads) cache_insert_kernel(const InsertLaunch a, int cached, int unit) {
  extern __shared__ uint32_t dyn[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int head = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // this CTA's slices of the held entries and of the new tokens
  const int old_per = (a.n + C - 1) / C, new_per = (a.n_new + C - 1) / C;
  const int old0 = min(a.n, rank * old_per), old_n = min(a.n, old0 + old_per) - old0;
  const int new0 = min(a.n_new, rank * new_per), new_n = min(a.n_new, new0 + new_per) - new0;
  const int all = old_n + new_n;
  const float* mass = a.mass + static_cast<int64_t>(head) * a.ld_state;
  const int32_t* pos = a.pos + static_cast<int64_t>(head) * a.ld_state;
  const float* mass_new = a.mass_new ? a.mass_new + static_cast<int64_t>(head) * a.ld_new_state : nullptr;
  float* mass_out = a.mass_out + static_cast<int64_t>(head) * a.ld_out;
  int32_t* pos_out = a.pos_out + static_cast<int64_t>(head) * a.ld_out;
  uint32_t* keys = dyn;                              // [old_n + new_n] when cached
  int32_t* slot_of = reinterpret_cast<int32_t*>(dyn + (cached ? old_per + new_per : 0));  // [new_per] by survivor rank
  int32_t* source_of = slot_of + new_per;            // [new_per] new token of each survivor

  auto make_key = [&](int i) -> uint32_t {
    if (i < old_n) return order_key(mass[old0 + i], pos[old0 + i], a.keep_below, a.keep_from);
    const int t = new0 + i - old_n;
    return order_key(mass_new ? mass_new[t] : 0.f, a.pos_new + t, a.keep_below, a.keep_from);
  };
  auto key_at = [&](int i) -> uint32_t { return cached ? keys[i] : make_key(i); };

  const int total = min(a.capacity, a.n + a.n_new);
  const uint32_t drop = static_cast<uint32_t>(a.n + a.n_new - total);
  uint32_t threshold = 0;   // candidates below it leave; of those equal to it
  uint32_t stay_equal = 0;  // the first `stay_equal` stay

  // Order keys; a state that goes to other arrays is copied on the way (slots of entries that leave are
  // overwritten by the survivors further below).
  const bool copy_mass = a.mass_out != a.mass, copy_pos = a.pos_out != a.pos;
  if ((drop > 0 && cached) || copy_mass || copy_pos) {
    for (int i0 = tid; i0 < old_n; i0 += kUnroll * kThreads) {
      float m[kUnroll];
      int32_t q[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kThreads;
        m[u] = i < old_n ? mass[old0 + i] : 0.f;
        q[u] = i < old_n ? pos[old0 + i] : 0;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kThreads;
        if (i >= old_n) break;
        if (cached) keys[i] = order_key(m[u], q[u], a.keep_below, a.keep_from);
        if (copy_mass) mass_out[old0 + i] = m[u];
        if (copy_pos) pos_out[old0 + i] = q[u];
      }
    }
  }
  if (drop > 0) {
    if (cached)
      for (int i = old_n + tid; i < all; i += kThreads) keys[i] = make_key(i);
    uint32_t prefix = 0, left = drop;  // left: how many of the candidates that share the prefix leave
    uint32_t same = 0;                 // candidates that share the prefix after the last pass
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int i = tid; i < 256 * 32; i += kThreads) (&sh.hist[0][0])[i] = 0;
      __syncthreads();
      for (int i = tid; i < all; i += kThreads) {
        const uint32_t k = key_at(i);
        if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&sh.hist[(k >> shift) & 255][lane], 1u);
      }
      __syncthreads();
#pragma unroll
      for (int d = 0; d < 256 / kWarps; ++d) {
        const uint32_t c = __reduce_add_sync(0xffffffffu, sh.hist[warp * (256 / kWarps) + d][lane]);
        if (lane == 0) sh.total[pass][warp * (256 / kWarps) + d] = c;
      }
      cluster.sync();
      // every CTA forms the same cluster-wide counts: thread d < 256 holds digit d
      uint32_t c = 0;
      if (tid < 256) {
#pragma unroll 4
        for (int r = 0; r < C; ++r) c += cluster.map_shared_rank(&sh.total[pass][0], r)[tid];
      }
      uint32_t inc = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += v;
      }
      if (lane == 31) sh.sum[warp] = inc;
      __syncthreads();
      if (tid < 256) {
        for (int w = 0; w < warp; ++w) inc += sh.sum[w];
        // the digit in which the last leaving candidate lies: below < left <= below + c
        if (inc - c < left && left <= inc) {
          sh.digit = static_cast<uint32_t>(tid);
          sh.below = inc - c;
          sh.same = c;
        }
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      left -= sh.below;
      same = sh.same;
    }
    threshold = prefix;
    stay_equal = same - left;
  }

  // Counts of candidates below and at the threshold: per warp over contiguous pieces, so that ranks
  // follow the candidate order.
  const int old_w = (old_n + kWarps - 1) / kWarps, new_w = (new_n + kWarps - 1) / kWarps;
  const int oa = min(old_n, warp * old_w), ob = min(old_n, oa + old_w);
  const int na = old_n + min(new_n, warp * new_w), nb = min(all, na + new_w);
  if (drop > 0) {
    uint32_t c[4] = {};
    for (int i = oa + lane; i < ob; i += 32) {
      const uint32_t k = key_at(i);
      c[0] += k < threshold;
      c[1] += k == threshold;
    }
    for (int i = na + lane; i < nb; i += 32) {
      const uint32_t k = key_at(i);
      c[2] += k < threshold;
      c[3] += k == threshold;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      c[x] = __reduce_add_sync(0xffffffffu, c[x]);
      if (lane == 0) sh.warp_counts[warp][x] = c[x];
    }
  } else if (lane < 4) {
    sh.warp_counts[warp][lane] = 0;
  }
  __syncthreads();
  if (tid < 4) {
    uint32_t c = 0;
    for (int w = 0; w < kWarps; ++w) c += sh.warp_counts[w][tid];
    sh.counts[tid] = c;
  }
  cluster.sync();
  // Ranks before this CTA (lane r of warp 0: CTA r).  Equal candidates count in candidate order: all
  // held slices, then all new ones.
  auto leaving = [&](uint32_t first, uint32_t n) {  // of n equal candidates from equal-rank `first` on
    const uint32_t end = first + n;
    return end > stay_equal ? end - max(first, stay_equal) : 0u;
  };
  if (warp == 0) {
    uint32_t cc[4] = {};
    if (lane < C)
#pragma unroll
      for (int x = 0; x < 4; ++x) cc[x] = cluster.map_shared_rank(&sh.counts[0], lane)[x];
    auto before = [&](uint32_t v) {  // sum over the CTAs before lane's
      uint32_t inc = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t w = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += w;
      }
      return inc - v;
    };
    const uint32_t eq = before(cc[1]);
    const uint32_t neq = before(cc[3]) + __reduce_add_sync(0xffffffffu, cc[1]);
    const int rn = lane < C ? max(0, min(a.n_new, (lane + 1) * new_per) - min(a.n_new, lane * new_per)) : 0;
    const uint32_t h = cc[0] + leaving(eq, cc[1]);
    const uint32_t v = static_cast<uint32_t>(rn) - cc[2] - leaving(neq, cc[3]);
    const uint32_t hole = before(h), surv = before(v);
    if (lane == rank) {
      sh.base[0] = eq;
      sh.base[1] = neq;
      sh.base[2] = hole;
      sh.base[3] = surv;
    }
    if (lane <= C) sh.first_survivor[lane] = surv;  // lane C: all of them
    const uint32_t all_holes = __reduce_add_sync(0xffffffffu, h);
    if (lane == 0) sh.holes = all_holes;
  }
  __syncthreads();
  const uint32_t n_holes = sh.holes;

  // Ranks before this warp.
  uint32_t eq_o = sh.base[0], eq_n = sh.base[1], hole = sh.base[2], surv = 0;
  for (int w = 0; w < warp; ++w) {
    hole += sh.warp_counts[w][0] + leaving(eq_o, sh.warp_counts[w][1]);
    eq_o += sh.warp_counts[w][1];
    const int wn = max(0, min(new_n, (w + 1) * new_w) - min(new_n, w * new_w));
    surv += static_cast<uint32_t>(wn) - sh.warp_counts[w][2] - leaving(eq_n, sh.warp_counts[w][3]);
    eq_n += sh.warp_counts[w][3];
  }
  const uint32_t lt = (1u << lane) - 1u;
  if (drop > 0) {
    // evicted held entries: slot of hole rank r goes to the CTA that owns survivor r
    for (int i = oa; i < ob; i += 32) {
      const bool in = i + lane < ob;
      const uint32_t k = in ? key_at(i + lane) : 0xffffffffu;
      const uint32_t eq_mask = __ballot_sync(0xffffffffu, in && k == threshold);
      const bool out = in && (k < threshold || (k == threshold && eq_o + __popc(eq_mask & lt) >= stay_equal));
      const uint32_t out_mask = __ballot_sync(0xffffffffu, out);
      if (out) {
        const uint32_t r = hole + __popc(out_mask & lt);
        int owner = 0;
        while (r >= sh.first_survivor[owner + 1]) ++owner;  // r < survivors of the head: one leaves per hole
        cluster.map_shared_rank(slot_of, owner)[r - sh.first_survivor[owner]] = old0 + i + lane;
      }
      hole += __popc(out_mask);
      eq_o += __popc(eq_mask);
    }
  }
  // surviving new tokens of this CTA, by rank; ranks past the holes take the unused slots from n on
  for (int i = na; i < nb; i += 32) {
    const bool in = i + lane < nb;
    const uint32_t k = in && drop > 0 ? key_at(i + lane) : 0xffffffffu;
    const uint32_t eq_mask = __ballot_sync(0xffffffffu, in && drop > 0 && k == threshold);
    const bool stay = in && (drop == 0 || k > threshold || (k == threshold && eq_n + __popc(eq_mask & lt) < stay_equal));
    const uint32_t stay_mask = __ballot_sync(0xffffffffu, stay);
    if (stay) {
      const uint32_t local = surv + __popc(stay_mask & lt);
      source_of[local] = new0 + i - old_n + lane;
      const uint32_t r = sh.base[3] + local;
      if (r >= n_holes) slot_of[local] = a.n + static_cast<int32_t>(r - n_holes);
    }
    surv += __popc(stay_mask);
    eq_n += __popc(eq_mask);
  }
  cluster.sync();  // every slot list is complete, every read of mass and pos above done, the copies made

  const int mine = static_cast<int>(sh.first_survivor[rank + 1] - sh.first_survivor[rank]);
  for (int i = tid; i < mine; i += kThreads) {
    const int t = source_of[i], slot = slot_of[i];
    mass_out[slot] = mass_new ? mass_new[t] : 0.f;
    pos_out[slot] = a.pos_new + t;
  }
  // K by the lower half of each warp, V by the upper half, kRows tokens in flight
  constexpr int kRows = 4;
  const int half = lane >> 4, hl = lane & 15;
  const int64_t col = static_cast<int64_t>(head) * a.row_bytes;
  const uint8_t* src = static_cast<const uint8_t*>(half ? a.v_new : a.k_new) + col;
  uint8_t* dst = static_cast<uint8_t*>(half ? a.v : a.k) + col;
  for (int i = warp * kRows; i < mine; i += kWarps * kRows) {
    if (unit == 16) {
      for (int b = hl * 16; b < a.row_bytes; b += 256) {
        uint4 w[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (i + r < mine) w[r] = __ldg(reinterpret_cast<const uint4*>(src + source_of[i + r] * a.ld_new_bytes + b));
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (i + r < mine) *reinterpret_cast<uint4*>(dst + slot_of[i + r] * a.ld_cache_bytes + b) = w[r];
      }
    } else {
      for (int r = 0; r < kRows && i + r < mine; ++r)
        for (int b = hl * 2; b < a.row_bytes; b += 32)
          *reinterpret_cast<uint16_t*>(dst + slot_of[i + r] * a.ld_cache_bytes + b) =
              __ldg(reinterpret_cast<const uint16_t*>(src + source_of[i + r] * a.ld_new_bytes + b));
    }
  }
}

}  // namespace

bool cache_insert_supported(int64_t n, int64_t n_new) {
  return n_new <= static_cast<int64_t>(kMaxCluster) * kMaxNewSlice && n + n_new < (1ll << 30);
}

cudaError_t launch_cache_insert(const InsertLaunch& a, cudaStream_t s, int* n_launched) {
  // Cluster size: one CTA forms and searches about 16 thousand order keys as fast as a cluster barrier
  // per pass costs, so a head is split only beyond that.
  const int64_t cand = static_cast<int64_t>(a.n) + a.n_new;
  int C = 1;
  while (C < kMaxCluster && (cand > 16384ll * C || (a.n_new + C - 1) / C > kMaxNewSlice)) C *= 2;
  const int old_per = (a.n + C - 1) / C, new_per = (a.n_new + C - 1) / C;
  const int cached = old_per + new_per <= kMaxCached;
  const size_t smem = 4ull * ((cached ? old_per + new_per : 0) + 2ll * new_per);
  const bool al = aligned16(a.k) && aligned16(a.v) && aligned16(a.k_new) && aligned16(a.v_new) &&
                  a.ld_cache_bytes % 16 == 0 && a.ld_new_bytes % 16 == 0 && a.row_bytes % 16 == 0;
  cudaError_t e = cudaFuncSetAttribute(cache_insert_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cache_insert_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * (kMaxCached + 2 * kMaxNewSlice));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(C) * static_cast<unsigned>(a.n_heads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, cache_insert_kernel, a, cached, al ? 16 : 2);
  *n_launched += 1;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ispa
