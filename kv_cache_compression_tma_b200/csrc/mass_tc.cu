// mass_tc.cu -- accumulated attention weight per cached key on tcgen05 tensor cores:
//   mass_out[h, j] = decay * mass[h, j] + exp(b_j) sum_i exp(scale q_i.k_j - L_i).
//
// The sum runs over queries, so keys are the rows (M) of the product S^T = K Q^T: a key is one TMEM
// lane, i.e. one thread, which adds up its row of weights in registers -- no reduction between
// threads and no atomics.
//
// Persistent CTAs, one per SM, each with a contiguous range of 128-key tiles.  A CTA takes two tiles of
// a head at a time (each query tile then serves two products) or, where one is left, a single tile.
// The key tiles come by TMA into a staging buffer while the previous ones are worked on, and go into
// TMEM as the first operand, so the products read only the queries from shared memory.  Products of
// 128 keys x 128 queries rotate through three TMEM accumulators (the rest of TMEM holds the keys),
// drained by two pairs of warpgroups in turn (with two key tiles a pair always has the same one), 64
// columns per warpgroup: a thread takes its columns into registers and frees the accumulator before
// it computes.  Sixteen warps, because the work per element is a chain (scale, exponential, add) whose
// latency eight do not cover.
//
// Bound: the hand-over of accumulators between the MMAs and the drain warps, then the exponentials, then the power
// cap.  12 heads x 4680 queries x 14040 keys: 0.205 ms in a short burst (202 GFLOP, 0.124 ms at the
// measured bf16 peak; 0.171 ms if the special-function unit did every exponential at 1965 MHz), 0.240 ms
// back to back at 990 W and 1.65 GHz, with 72 % of that unit, 66 % of the issue slots and 47 % of the
// tensor pipe busy.  Measured
// beside it: 0.246 ms with 8 warps and 0.234 with 16 while a lone lane issued the MMAs (the warp-uniform
// form has fewer instructions to squeeze in between the sixteen busy warps; 0.243 -> 0.226 on one
// variant), 0.226 without the polynomial exponential, 0.205 with products 192 or 256 queries wide on two
// accumulators, 0.235 with 96 on four (more hand-offs).  A burst without any exponential runs at 0.16 ms.
//
// Warp roles (608 threads): warp 0 TMA producer, warp 1 TMEM and the MMAs, warp 2 idle, warps 3..18 the
// four warpgroups.  TMEM columns: [0,384) three accumulators, [384,512) two key tiles (bf16 pairs).
// Every barrier wait is bounded (sm100.cuh); one that runs out records ISPA_ERR_TIMEOUT and unwinds.
#include <math.h>
#include <string.h>

#include "internal.h"
#include "mass.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace ispa {
namespace {

constexpr int kTile = 128;       // keys per tile
constexpr int kSub = 128;        // queries per product
constexpr int kAcc = 3;          // accumulators
constexpr int kCols = kSub / 2;  // accumulator columns of a thread
constexpr int kQTile = 2 * kSub;  // queries per load
constexpr int kStages = 2;       // query tiles in flight
constexpr int kChunk = 6144;     // queries whose -L sits in shared memory at a time
constexpr int kFirstEpiWarp = 3;
constexpr int kEpiThreads = 512;
constexpr int kThreads = 32 * kFirstEpiWarp + kEpiThreads;
// Of eight pairs of queries, those whose exponentials run on the multiply-add pipes, the others on the
// special-function unit: it alone takes 16 a clock, less than the products deliver.  They have sums of their own,
// which are infinite once one of them passes 2^127.5 (the polynomial's end; clamping each at 128 instead cost 3 %).
constexpr int kPolyPairs = 0b10001000;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  int n_q, n_k, tiles_per_head, n_tiles;
  float scale_log2, decay;
  const float* lse_loc;
  const float* lse_hist;
  const float* bias;
  int64_t ld_bias;
  const float* mass;
  float* mass_out;
  int64_t ld_mass;
  unsigned* status;
};

template <int HD>
struct Cfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kBoxK = kTile * 128, kBoxQ = kQTile * 128;  // 64 columns of a tile
  static constexpr int kBytesK = kTile * HD * 2, kBytesQ = kQTile * HD * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kStages * kBytesQ;
  static constexpr int kOffL = kOffK + 2 * kBytesK;         // [kChunk] -L * log2(e)
  static constexpr int kOffBar = kOffL + kChunk * 4;
  // q_full[kStages], q_empty[kStages], acc_full[kAcc], acc_empty[kAcc], k_full, k_free, k_ready, final
  static constexpr int kNumBars = 2 * kStages + 2 * kAcc + 4;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8 + 8;
  static constexpr int kOffEmpty = kOffMisc + 16;                // [kChunk / 32] a bit per query: without keys, or past the last
  static constexpr int kOffSums = kOffEmpty + kChunk / 32 * 4;  // the warpgroups' sums of an item, by its parity
  static constexpr int kSmemBytes = kOffSums + 2 * 3 * kTile * 4;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// The CTA's tiles [first, last) one or two at a time: two only within a head.
__device__ __forceinline__ int tiles_at(const Params& p, int t, int last) {
  return (t + 1 < last && (t + 1) % p.tiles_per_head != 0) ? 2 : 1;
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k, const Params p) {
  using C = Cfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023) != 0) {  // the swizzled TMA / UMMA layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicOr(p.status, kStatusInternal);
    return;
  }
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_empty = q_full + kStages;
  uint64_t* acc_full = q_empty + kStages;
  uint64_t* acc_empty = acc_full + kAcc;
  uint64_t* k_full = acc_empty + kAcc;  // the staging buffer holds the item's key tiles
  uint64_t* k_free = k_full + 1;     // ... and they are in TMEM: the buffer may be filled again,
  uint64_t* k_ready = k_free + 1;    // and the products may start
  uint64_t* final_bar = k_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* never = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  uint32_t* empty = reinterpret_cast<uint32_t*>(smem + C::kOffEmpty);
  float* other = reinterpret_cast<float*>(smem + C::kOffSums);
  float* neg_l = reinterpret_cast<float*>(smem + C::kOffL);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp-uniform
  const int first = static_cast<int>(static_cast<int64_t>(p.n_tiles) * blockIdx.x / gridDim.x);
  const int last = static_cast<int>(static_cast<int64_t>(p.n_tiles) * (blockIdx.x + 1) / gridDim.x);
  const int n_sub = (p.n_q + kSub - 1) / kSub;  // products per key tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 8);
    }
    mbar_init(k_full, 1);
    mbar_init(k_free, 16);
    mbar_init(k_ready, 16);
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    *never = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      bool ok = true;
      int item = 0, n_issued = 0, k_issued = 0;
      for (int t = first; ok && t < last; ++item) {
        const int count = tiles_at(p, t, last), head = t / p.tiles_per_head, key0 = (t % p.tiles_per_head) * kTile;
        if (item > 0 && !mbar_wait(k_free, (item - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(k_full, count * C::kBytesK);
        for (int i = 0; i < count; ++i)
#pragma unroll
          for (int b = 0; b < C::kBoxes; ++b)
            tma_load_2d(smem + C::kOffK + i * C::kBytesK + b * C::kBoxK, &map_k, k_full, head * HD + 64 * b, key0 + i * kTile);
        ++k_issued;
        for (int n = 0; n < n_sub; n += kQTile / kSub) {
          const int s = n_issued % kStages;
          if (n_issued >= kStages && !mbar_wait(q_empty + s, (n_issued / kStages - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(q_full + s, C::kBytesQ);
#pragma unroll
          for (int b = 0; b < C::kBoxes; ++b)
            tma_load_2d(smem + C::kOffQ + s * C::kBytesQ + b * C::kBoxQ, &map_q, q_full + s, head * HD + 64 * b, n * kSub);
          ++n_issued;
        }
        t += count;
      }
      if (!ok) {
        atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
      // Never leave the CTA with bulk copies in flight: wait for the last load of every stage.
      if (*abort_flag) {
        for (int n = n_issued - 1; n >= 0 && n >= n_issued - kStages; --n)
          mbar_wait(q_full + n % kStages, (n / kStages) & 1, never);
        if (k_issued > 0) mbar_wait(k_full, (k_issued - 1) & 1, never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    {
      const uint32_t leader = elect_leader();
      bool ok = true;
      int item = 0, n_done = 0, seq = 0;
      for (int t = first; ok && t < last; ++item) {
        const int count = tiles_at(p, t, last);
        ok = mbar_wait_warp(k_ready, item & 1, abort_flag);
        for (int n = 0; ok && n < n_sub; ++n) {
          const int s = n_done % kStages, part = n % (kQTile / kSub);
          if (part == 0) ok = mbar_wait_warp(q_full + s, (n_done / kStages) & 1, abort_flag);
          const uint32_t qb = smem_u32(smem + C::kOffQ + s * C::kBytesQ + part * kSub * 128);
          const int width = min(kSub, (p.n_q - n * kSub + 15) / 16 * 16);  // the last one may be narrower
          const uint32_t idesc = idesc_bf16_f32(kTile, width, false, false);
          for (int i = 0; ok && i < count; ++i, ++seq) {
            const int a = seq % kAcc;
            if (seq >= kAcc && !mbar_wait_warp(acc_empty + a, (seq / kAcc - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              umma_ts_warp(tmem + a * kSub, tmem + kAcc * kSub + i * 64 + kk * 8,
                           sw128_desc(qb + (kk >> 2) * C::kBoxQ + (kk & 3) * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u, leader);
            umma_commit_warp(acc_full + a, leader);
          }
          if (ok && (part == kQTile / kSub - 1 || n + 1 == n_sub)) {
            umma_commit_warp(q_empty + s, leader);
            ++n_done;
          }
        }
        t += count;
      }
      if (!ok) {
        if (leader) atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
      umma_commit_warp(final_bar, leader);
      mbar_wait_warp(final_bar, 0, never);  // every MMA this thread issued has completed before TMEM is released
    }
  } else if (warp >= kFirstEpiWarp) {
    // ------------------------------------------------------------------ sums
    const int quarter = warp & 3;  // TMEM lane quarter this warp may access
    const int wg = (warp - kFirstEpiWarp) >> 2;
    const int sel = wg & 1, half = wg >> 1;  // which accumulator, which 64 of its columns
    const int row = quarter * 32 + lane;     // key within the tile == TMEM lane
    const int tid = wg * 128 + row;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint64_t sl2x2 = pack_f2(p.scale_log2, p.scale_log2);
    bool alive = true;  // warp-uniform; a warp whose wait ran out only keeps meeting the barriers
    int item = 0, seq0 = 0, staged_head = -1;
    for (int t = first; t < last; ++item) {
      const int count = tiles_at(p, t, last), head = t / p.tiles_per_head, key0 = (t % p.tiles_per_head) * kTile;
      // Every product of the item before is complete: the barrier at its end follows the last drains.
      if (alive) alive = mbar_wait_warp(k_full, item & 1, abort_flag);
      if (alive && sel < count) {
        tc_fence_after();
        const uint8_t* src = smem + C::kOffK + sel * C::kBytesK + row * 128;
        for (int b = half; b < C::kBoxes; b += 2) {  // this key's 64 elements of a box: 16-byte chunk c sits at c ^ (row & 7)
          uint32_t r[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + b * C::kBoxK + ((c ^ (row & 7)) << 4));
            r[4 * c] = w.x;
            r[4 * c + 1] = w.y;
            r[4 * c + 2] = w.z;
            r[4 * c + 3] = w.w;
          }
          tmem_st32(tmem + lane_addr + kAcc * kSub + sel * 64 + b * 32, r);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(k_free);
        mbar_arrive(k_ready);
      }
      float total = 0.f;
      for (int c0 = 0; c0 < p.n_q; c0 += kChunk) {
        const int c1 = min(p.n_q, c0 + kChunk);
        // -L of the chunk's queries; padding rows get weight 0.  One fp32 number each: its rounding, 2^-24 of |L|, goes
        // one way in one query and the other in the next, and a second number would take a fused add per weight.
        if (head != staged_head || p.n_q > kChunk) {
          asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory");
          for (int i = tid; i < (c1 - c0 + kQTile - 1) / kQTile * kQTile; i += kEpiThreads) {
            const int64_t o = static_cast<int64_t>(head) * p.n_q + c0 + i;
            neg_l[i] = c0 + i < p.n_q ? -kLog2e * mass_row_lse(p.lse_loc[o], p.lse_hist ? p.lse_hist[o] : -INFINITY) : -INFINITY;
            const uint32_t bits = __ballot_sync(0xffffffffu, neg_l[i] == -INFINITY);  // the loop's bounds are whole warps
            if (lane == 0) empty[i / 32] = bits;
          }
          asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory");
          staged_head = head;
        }
        for (int n = c0 / kSub; alive && n * kSub < c1; ++n) {
          for (int i = 0; i < count; ++i) {
            const int seq = seq0 + n * count + i, a = seq % kAcc;
            if ((seq & 1) != sel) continue;
            alive = mbar_wait_warp(acc_full + a, (seq / kAcc) & 1, abort_flag);
            if (!alive) break;
            tc_fence_after();
            const float* nl = neg_l + n * kSub - c0 + half * kCols;
            uint32_t r[kCols];
            const uint32_t src = tmem + lane_addr + a * kSub + half * kCols;
#pragma unroll
            for (int x = 0; x < kCols / 32; ++x) tmem_ld32(src + 32 * x, r + 32 * x);
            tmem_wait_ld();
            tc_fence_before();  // in registers: free the accumulator for the MMAs before any arithmetic
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + a);
            // Columns past the last query hold what an earlier product left, and the scores of a row without keys
            // may be anything: 0 there, so that the -inf beside it decides.
#pragma unroll
            for (int h = 0; h < kCols / 32; ++h) {
              const uint32_t bits = empty[(n * kSub - c0 + half * kCols) / 32 + h];
              if (bits != 0) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if ((bits >> j) & 1) r[32 * h + j] = 0u;
              }
            }
            uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};  // [3]: the polynomials'
            float most = -INFINITY;                      // their largest exponent
#pragma unroll
            for (int j = 0; j < kCols; j += 4) {
              const float4 l4 = *reinterpret_cast<const float4*>(nl + j);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int pair = j >> 1 | h;
                const uint64_t y = fma_f2(pack_f2(__uint_as_float(r[j + 2 * h]), __uint_as_float(r[j + 2 * h + 1])), sl2x2,
                                          h ? pack_f2(l4.z, l4.w) : pack_f2(l4.x, l4.y));
                float y0, y1;
                unpack_f2(y, y0, y1);
                if ((kPolyPairs >> (pair & 7)) & 1) {
                  uint64_t pv, scale;
                  exp2_poly2(y, pv, scale);
                  acc[3] = fma_f2(pv, scale, acc[3]);
                  most = max3f_nan(most, y0, y1);
                } else {
                  static_assert((kPolyPairs & 0x77) == 0, "the fourth sum is the polynomials'");
                  acc[pair & 3] = add_f2(acc[pair & 3], pack_f2(fast_exp2(y0), fast_exp2(y1)));
                }
              }
            }
            float a0, a1, a2, a3, a4, a5, a6, a7;
            unpack_f2(acc[0], a0, a1);
            unpack_f2(acc[1], a2, a3);
            unpack_f2(acc[2], a4, a5);
            unpack_f2(acc[3], a6, a7);
            if (most > 127.5f) a6 = a7 = INFINITY;
            total += ((a0 + a1) + (a2 + a3)) + ((a4 + a5) + (a6 + a7));
          }
        }
      }
      // With two tiles a warpgroup had the tile of its parity; with one, all four worked on it.  The sums
      // are joined in a fixed order; the next item's may be written while these are read.
      const int mine = count == 2 ? sel ^ (seq0 & 1) : 0;
      seq0 += n_sub * count;
      float* sums = other + (item & 1) * 3 * kTile + row;
      if (wg > 0) sums[(wg - 1) * kTile] = total;
      asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory");
      const bool owner = half == 0 && (count == 2 || sel == 0);
      if (owner) {
        total += sums[(wg + 1) * kTile];
        if (count == 1) total += sums[0] + sums[2 * kTile];
      }
      const int j = key0 + mine * kTile + row;
      if (alive && owner && j < p.n_k) {
        if (p.bias) total = mass_apply_bias(total, p.bias[static_cast<int64_t>(head) * p.ld_bias + j]);
        const int64_t o = static_cast<int64_t>(head) * p.ld_mass + j;
        p.mass_out[o] = p.decay != 0.f ? fmaf(p.decay, p.mass[o], total) : total;
      }
      t += count;
    }
    if (!alive) {
      atomicOr(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD>
cudaError_t launch_hd(const MassLaunch& a, cudaStream_t s, int* n_launched) {
  using C = Cfg<HD>;
  CUtensorMap map_q, map_k;
  const uint64_t d = static_cast<uint64_t>(a.n_heads) * HD;
  if (!make_map_bf16_2d(&map_q, a.q, a.n_q, d, a.ld_q, 64, kQTile) || !make_map_bf16_2d(&map_k, a.k, a.n_k, d, a.ld_k, 64, kTile))
    return cudaErrorInvalidValue;
  Params p;
  p.n_q = static_cast<int>(a.n_q);
  p.n_k = static_cast<int>(a.n_k);
  p.tiles_per_head = (p.n_k + kTile - 1) / kTile;
  p.n_tiles = p.tiles_per_head * a.n_heads;
  p.scale_log2 = a.scale * kLog2e;
  p.decay = a.decay;
  p.lse_loc = a.lse_loc;
  p.lse_hist = a.lse_hist;
  p.bias = a.bias;
  p.ld_bias = a.ld_bias;
  p.mass = a.mass;
  p.mass_out = a.mass_out;
  p.ld_mass = a.ld_mass;
  p.status = a.status;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(mass_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  mass_tc_kernel<HD><<<p.n_tiles < sms ? p.n_tiles : sms, kThreads, C::kSmemBytes, s>>>(map_q, map_k, p);
  *n_launched += 1;
  return cudaGetLastError();
}

}  // namespace

bool mass_tc_supported(const MassLaunch& a) {
  return a.dtype == 0 && (a.head_dim == 64 || a.head_dim == 128) && aligned16(a.q) && aligned16(a.k) && a.ld_q % 8 == 0 &&
         a.ld_k % 8 == 0 && (a.n_k + kTile - 1) / kTile * a.n_heads < (1ll << 30);
}

cudaError_t launch_mass_tc(const MassLaunch& a, cudaStream_t s, int* n_launched) {
  return a.head_dim == 128 ? launch_hd<128>(a, s, n_launched) : launch_hd<64>(a, s, n_launched);
}

}  // namespace ispa
