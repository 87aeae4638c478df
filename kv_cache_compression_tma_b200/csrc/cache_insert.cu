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
constexpr int kUnroll = 16;         // state words in flight per thread while the keys are formed
constexpr int kRun = 8;             // consecutive candidates of a lane where ranks are counted
constexpr int kShort = 2048;        // candidates sharing the first digit that are listed apart

struct Shared {
  // Counts of the first digit, one column per lane: the keys of a cache share few leading digits, and
  // lanes of a warp that add to one address would take turns.
  uint32_t hist[256][32];
  uint32_t total[4][256];             // the CTA's counts, one array per pass: one cluster barrier per pass
  alignas(16) uint32_t cluster_total[256];
  uint32_t shortlist[kShort];         // candidates that share the first digit, when they fit
  uint32_t n_short, digit, below;
  alignas(16) uint32_t counts[4];     // the CTA's {less, equal} of the held slice, then of the new slice
  alignas(16) uint32_t all_counts[kMaxCluster][4];  // every CTA's
  uint32_t warp_counts[kWarps][4];    // the same per warp, then the sum over the warps before
  uint32_t first_survivor[kMaxCluster + 1];
};

// Order-preserving image of a rank: larger float, larger unsigned.
__device__ __forceinline__ uint32_t order_key(float mass, int32_t pos, int32_t keep_below, int32_t keep_from) {
  if (isnan(mass)) mass = -INFINITY;
  if (pos < keep_below || pos >= keep_from) mass = INFINITY;
  const uint32_t u = __float_as_uint(mass + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of v over the lanes before this one.
__device__ __forceinline__ uint32_t warp_before(uint32_t v, int lane) {
  uint32_t inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t w = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += w;
  }
  return inc - v;
}

__global__ void __launch_bounds__(kThreads) cache_insert_kernel(const InsertLaunch a, int cached, int unit) {
  extern __shared__ __align__(16) uint32_t dyn[];
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
  uint32_t* keys = dyn;                              // [old_n + new_n] when cached (16-byte aligned)
  int32_t* slot_of = reinterpret_cast<int32_t*>(dyn + (cached ? old_per + new_per : 0));  // [new_per] by survivor rank
  int32_t* source_of = slot_of + new_per;            // [new_per] new token of each survivor

  auto make_key = [&](int i) -> uint32_t {
    if (i < old_n) return order_key(mass[old0 + i], pos[old0 + i], a.keep_below, a.keep_from);
    const int t = new0 + i - old_n;
    return order_key(mass_new ? mass_new[t] : 0.f, a.pos_new + t, a.keep_below, a.keep_from);
  };
  auto key_at = [&](int i) -> uint32_t { return cached ? keys[i] : make_key(i); };
  // kRun consecutive candidates of the held slice from i (a multiple of kRun) on, all ones past the slice (no
  // key is: NaN ranks as -inf).
  auto key_run = [&](int i, uint32_t* k) {
    if (cached && i + kRun <= old_n) {
#pragma unroll
      for (int x = 0; x < kRun; x += 4) *reinterpret_cast<uint4*>(k + x) = *reinterpret_cast<const uint4*>(keys + i + x);
    } else {
#pragma unroll
      for (int x = 0; x < kRun; ++x) k[x] = i + x < old_n ? key_at(i + x) : 0xffffffffu;
    }
  };

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
    for (int i = tid; i < 256 * 32; i += kThreads) (&sh.hist[0][0])[i] = 0;
    if (tid < 256) sh.total[1][tid] = sh.total[2][tid] = sh.total[3][tid] = 0;
    if (tid == 0) sh.n_short = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < all; i += kThreads) atomicAdd(&sh.hist[key_at(i) >> 24][lane], 1u);
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 256 / kWarps; ++d) {
      const uint32_t c = __reduce_add_sync(0xffffffffu, sh.hist[warp * (256 / kWarps) + d][lane]);
      if (lane == 0) sh.total[0][warp * (256 / kWarps) + d] = c;
    }
    uint32_t left = drop;  // how many of the candidates that share the digits so far leave
    bool listed = false;
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      if (pass > 0) {
        const int n = listed ? static_cast<int>(sh.n_short) : all;
        for (int i = tid; i < n; i += kThreads) {
          const uint32_t k = listed ? sh.shortlist[i] : key_at(i);
          if ((k >> (shift + 8)) == (threshold >> (shift + 8))) atomicAdd(&sh.total[pass][(k >> shift) & 255], 1u);
        }
      }
      const uint32_t* counts = sh.total[pass];
      if (C > 1) {  // every CTA forms the same cluster-wide counts
        cluster.sync();
        if (tid < 256) {
          uint32_t c = 0;
#pragma unroll 4
          for (int r = 0; r < C; ++r) c += cluster.map_shared_rank(&sh.total[pass][0], r)[tid];
          sh.cluster_total[tid] = c;
        }
        counts = sh.cluster_total;
      }
      __syncthreads();
      if (warp == 0) {  // the digit of the last leaving candidate: below < left <= below + count; eight a lane
        const uint4 lo = *reinterpret_cast<const uint4*>(counts + lane * 8), hi = *reinterpret_cast<const uint4*>(counts + lane * 8 + 4);
        const uint32_t c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        uint32_t sum = 0;
#pragma unroll
        for (int d = 0; d < 8; ++d) sum += c[d];
        uint32_t below = warp_before(sum, lane);
        if (below < left && left <= below + sum) {  // one lane
          int d = 0;
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (d == e && left > below + c[e]) {
              below += c[e];
              ++d;
            }
          sh.digit = static_cast<uint32_t>(lane * 8 + d);
          sh.below = below;
        }
      }
      __syncthreads();
      const uint32_t digit = sh.digit, same = counts[digit];
      threshold |= digit << shift;
      left -= sh.below;
      stay_equal = same - left;
      if (left == same) {  // all of the digit leaves: the threshold is the next digit's start (some candidate stays, so there is one)
        threshold += 1u << shift;
        stay_equal = 0xffffffffu;
        break;
      }
      if (pass == 0) {
        listed = sh.total[0][digit] <= kShort;  // this CTA's own count
        if (listed) {
#pragma unroll 4
          for (int i = tid; i < all; i += kThreads) {
            const uint32_t k = key_at(i);
            if ((k >> 24) == digit) sh.shortlist[atomicAdd(&sh.n_short, 1u)] = k;
          }
        }
      }
      __syncthreads();
    }
  }

  // Counts of candidates below and at the threshold: per warp over contiguous pieces, so that ranks
  // follow the candidate order.
  const int old_w = (old_n + 32 * kRun * kWarps - 1) / (32 * kRun * kWarps) * 32 * kRun, new_w = (new_n + kWarps - 1) / kWarps;
  const int oa = min(old_n, warp * old_w), ob = min(old_n, oa + old_w);
  const int na = old_n + min(new_n, warp * new_w), nb = min(all, na + new_w);
  if (drop > 0) {
    uint32_t c[4] = {};
    for (int i = oa + kRun * lane; i < ob; i += 32 * kRun) {
      uint32_t k[kRun];
      key_run(i, k);
#pragma unroll
      for (int x = 0; x < kRun; ++x) {
        c[0] += k[x] < threshold;
        c[1] += k[x] == threshold;
      }
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
  if (warp == 0) {  // sums over the warps before, and over all of them (kWarps == 32: lane = warp)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t v = sh.warp_counts[lane][x], before = warp_before(v, lane);
      sh.warp_counts[lane][x] = before;
      if (lane == 31) sh.counts[x] = before + v;
    }
  }
  cluster.sync();
  if (tid < C)
    *reinterpret_cast<uint4*>(sh.all_counts[tid]) = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&sh.counts[0], tid));
  __syncthreads();
  // Ranks before this warp.  Equal candidates count in candidate order: all held slices, then all new
  // ones.  Lane r looks at CTA r.
  auto leaving = [&](uint32_t n) { return n > stay_equal ? n - stay_equal : 0u; };  // of the first n equal ones
  uint32_t eq_o, eq_n, hole, surv, first, n_holes;
  {
    uint32_t cc[4] = {};
    if (lane < C)
#pragma unroll
      for (int x = 0; x < 4; ++x) cc[x] = sh.all_counts[lane][x];
    const uint32_t rn = lane < C ? static_cast<uint32_t>(min(a.n_new, (lane + 1) * new_per) - min(a.n_new, lane * new_per)) : 0u;
    const uint32_t old_eq = __reduce_add_sync(0xffffffffu, cc[1]);
    const uint32_t eq = warp_before(cc[1], lane), neq = old_eq + warp_before(cc[3], lane);
    const uint32_t less = warp_before(cc[0], lane), stayed = warp_before(rn - cc[2], lane);
    // holes before CTA `lane`, survivors before it (lane C: all)
    const uint32_t h = less + leaving(eq), v = stayed - (leaving(neq) - leaving(old_eq));
    if (warp == 0 && lane <= C) sh.first_survivor[lane] = v;
    n_holes = __reduce_add_sync(0xffffffffu, cc[0]) + leaving(old_eq);
    const uint32_t* wc = sh.warp_counts[warp];
    eq_o = __shfl_sync(0xffffffffu, eq, rank) + wc[1];
    eq_n = __shfl_sync(0xffffffffu, neq, rank) + wc[3];
    hole = __shfl_sync(0xffffffffu, less, rank) + wc[0] + leaving(eq_o);
    first = __shfl_sync(0xffffffffu, v, rank);  // the CTA's first survivor
    surv = static_cast<uint32_t>(na - old_n) - wc[2] - (leaving(eq_n) - leaving(eq_n - wc[3]));
  }
  __syncthreads();
  const uint32_t lt = (1u << lane) - 1u;
  if (drop > 0) {
    // evicted held entries: slot of hole rank r goes to the CTA that owns survivor r
    for (int i = oa; i < ob; i += 32 * kRun) {
      uint32_t k[kRun];
      key_run(i + kRun * lane, k);
      uint32_t out = 0, eq = 0;  // bit x: candidate x leaves, equals the threshold
#pragma unroll
      for (int x = 0; x < kRun; ++x) {
        out |= (k[x] < threshold ? 1u : 0u) << x;
        eq |= (k[x] == threshold ? 1u : 0u) << x;
      }
      if (!__any_sync(0xffffffffu, out | eq)) continue;
      if (__any_sync(0xffffffffu, eq)) {
        const uint32_t n_eq = __popc(eq);
        uint32_t e = eq_o + warp_before(n_eq, lane);
        for (uint32_t w = eq; w; w &= w - 1)
          if (e++ >= stay_equal) out |= w & -w;
        eq_o += __reduce_add_sync(0xffffffffu, n_eq);
      }
      const uint32_t n_out = __popc(out);
      uint32_t r = hole + warp_before(n_out, lane);
      int owner = 0;
      for (; out; out &= out - 1, ++r) {
        while (r >= sh.first_survivor[owner + 1]) ++owner;  // r < survivors of the head: one leaves per hole
        cluster.map_shared_rank(slot_of, owner)[r - sh.first_survivor[owner]] = old0 + i + kRun * lane + __ffs(out) - 1;
      }
      hole += __reduce_add_sync(0xffffffffu, n_out);
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
      const uint32_t r = first + local;
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

// One new token (a decoding step): at most one candidate leaves, the one of lowest rank (the last of
// equals), so one CTA per head takes a minimum over its candidates instead of a radix select: 17 -> 6 us
// for 40 heads of 14040 entries.
__global__ void __launch_bounds__(kThreads) cache_insert_one_kernel(const InsertLaunch a, int unit) {
  __shared__ unsigned long long lowest[kWarps];
  const int head = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const float* mass = a.mass + static_cast<int64_t>(head) * a.ld_state;
  const int32_t* pos = a.pos + static_cast<int64_t>(head) * a.ld_state;
  float* mass_out = a.mass_out + static_cast<int64_t>(head) * a.ld_out;
  int32_t* pos_out = a.pos_out + static_cast<int64_t>(head) * a.ld_out;
  const float m_new = a.mass_new ? a.mass_new[static_cast<int64_t>(head) * a.ld_new_state] : 0.f;
  const bool full = a.n == a.capacity;
  const bool copy_mass = a.mass_out != a.mass, copy_pos = a.pos_out != a.pos;
  // (order key, candidate counted from the end): the least pair leaves
  auto pair = [&](float m, int32_t p, int i) {
    return static_cast<unsigned long long>(order_key(m, p, a.keep_below, a.keep_from)) << 32 | static_cast<uint32_t>(a.n - i);
  };
  unsigned long long least = pair(m_new, a.pos_new, a.n);
  if (full || copy_mass || copy_pos) {
    for (int i0 = tid; i0 < a.n; i0 += kUnroll * kThreads) {
      float m[kUnroll];
      int32_t q[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = min(i0 + u * kThreads, a.n - 1);
        m[u] = mass[i];
        q[u] = pos[i];
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kThreads;
        if (i >= a.n) break;
        least = min(least, pair(m[u], q[u], i));
        if (copy_mass) mass_out[i] = m[u];
        if (copy_pos) pos_out[i] = q[u];
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, off));
  if (lane == 0) lowest[tid >> 5] = least;
  __syncthreads();  // also: every read of the state is done before its slot is written
  if (tid >= 32) return;
  least = lowest[lane];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, off));
  const int slot = full ? a.n - static_cast<int>(static_cast<uint32_t>(least)) : a.n;
  if (slot == a.capacity) return;  // the token itself leaves
  if (lane == 0) {
    mass_out[slot] = m_new;
    pos_out[slot] = a.pos_new;
  }
  const int64_t col = static_cast<int64_t>(head) * a.row_bytes;
  const uint8_t* src = static_cast<const uint8_t*>(lane < 16 ? a.k_new : a.v_new) + col;
  uint8_t* dst = static_cast<uint8_t*>(lane < 16 ? a.k : a.v) + slot * a.ld_cache_bytes + col;
  if (unit == 16) {
    for (int b = (lane & 15) * 16; b < a.row_bytes; b += 256)
      *reinterpret_cast<uint4*>(dst + b) = __ldg(reinterpret_cast<const uint4*>(src + b));
  } else {
    for (int b = (lane & 15) * 2; b < a.row_bytes; b += 32)
      *reinterpret_cast<uint16_t*>(dst + b) = __ldg(reinterpret_cast<const uint16_t*>(src + b));
  }
}

}  // namespace

bool cache_insert_supported(int64_t n, int64_t n_new) {
  return n_new <= static_cast<int64_t>(kMaxCluster) * kMaxNewSlice && n + n_new < (1ll << 30);
}

cudaError_t launch_cache_insert(const InsertLaunch& a, cudaStream_t s, int* n_launched) {
  const bool al = aligned16(a.k) && aligned16(a.v) && aligned16(a.k_new) && aligned16(a.v_new) &&
                  a.ld_cache_bytes % 16 == 0 && a.ld_new_bytes % 16 == 0 && a.row_bytes % 16 == 0;
  const int unit = al ? 16 : 2;
  if (a.n_new == 1) {
    cache_insert_one_kernel<<<static_cast<unsigned>(a.n_heads), kThreads, 0, s>>>(a, unit);
    *n_launched += 1;
    return cudaGetLastError();
  }
  // Cluster size: a CTA (one per SM: 1024 threads) forms and searches about 16 thousand order keys in the
  // time of the cluster barriers, so a head is split only beyond that, and only while all clusters
  // can run at once (clusters of 16 fit 8 times on the GPU's 8 GPCs of 16 to 20 SMs, of 8 twice as often).
  const int64_t cand = static_cast<int64_t>(a.n) + a.n_new;
  int C = 1;
  while (C < kMaxCluster && cand > 16384ll * C && static_cast<int64_t>(a.n_heads) * 2 * C <= 128) C *= 2;
  while (C < kMaxCluster && (cand > static_cast<int64_t>(kMaxCached) * C || (a.n_new + C - 1) / C > kMaxNewSlice)) C *= 2;
  const int old_per = (a.n + C - 1) / C, new_per = (a.n_new + C - 1) / C;
  const int cached = old_per + new_per <= kMaxCached;
  const size_t smem = 4ull * ((cached ? old_per + new_per : 0) + 2ll * new_per);
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
  e = cudaLaunchKernelEx(&cfg, cache_insert_kernel, a, cached, unit);
  *n_launched += 1;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ispa
