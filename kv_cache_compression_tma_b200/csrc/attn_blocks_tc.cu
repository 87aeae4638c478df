// attn_blocks_tc.cu -- dual-stream attention over sink, local and selected history blocks on tcgen05
// tensor cores: one CTA per (128 query rows, head), whose rows share one list of history blocks.
//
// Keys are walked once in tiles of 128, local branch first, with an online softmax (m, l, fp32
// accumulator in TMEM) per branch, and
//   O_loc = O_A / l_loc,  O_full = w_loc O_loc + w_hist O_B / l_hist,  D = w_hist (O_B / l_hist - O_loc).
// The CTA first turns its list into halves of 64 keys (a block is one or two of them; entries that name
// no block, and empty halves of the history's last block, are dropped), and a history tile is any two
// consecutive halves: two 64-row TMA boxes per 64 columns instead of one 128-row box.  So both block
// sizes fill whole MMA tiles, and a ragged block may lie anywhere in the list.
//
// Two groups of four softmax warps, a query row per thread, take the tiles by turns, so that one forms
// its maximum or waits while the other keeps the exponentials going.  Both scale by one running maximum per
// row, which a group reads after the other's last tile and hands on (m_ready); each keeps a partial
// sum of its own.  S runs two tiles ahead of P V in three TMEM buffers.  That leaves one accumulator: at
// the branch switch O_loc goes to its place in memory, rounded, and the bits that the rounding took go to
// O_full's place, where the same thread finds them again for the epilogue (together the 32 bits of O_loc).
// P is rounded to bf16 for its product, as in the dense kernel: the tensor cores take no wider operand
// beside bf16 values, and a second product for what the rounding left would cost half as much again.
//
// Bound: the loop of three tiles (softmax of one, P V and the S that waits for its buffer) at about 1430
// clocks per tile (1024 of MMA), and power.  12 heads x 4680 queries over 6240 local keys and 64 blocks of
// 128 (415 GFLOP, 0.254 ms at the measured bf16 peak): 0.40 ms alone, tensor pipe 62 % busy, 0.47 ms back
// to back at 990 W.  The softmax warps are capped at 168 registers (eleven warps are allocated as twelve)
// and spill 68 bytes, about 7 loads from L1 per warp and tile.  Measured beside it: two threads per row and
// one group on two S buffers, a second accumulator (2090 clocks, 0.49 ms); two groups with accumulators of
// their own on two S buffers (the same); two threads per row here (0.467 against 0.452); S read a second
// time instead of held in registers (0.50); the two products issued by two warps (their operands
// alternate: 10 % slower); three V stages and polynomial exponentials (nothing, and slower).
//
// Warp roles (352 threads): warp 0 Q and the K ring, warp 2 the V ring, warp 1 TMEM and the MMAs, warps
// 3..10 softmax and epilogue.  Commits: s_full[t%3] (also frees K_t), o_done[t%2] (also frees V_t).
// TMEM columns: [0,384) three S/P buffers (P_t over the first half of S_t), [384,384+HD) O.
// Every barrier wait is bounded (sm100.cuh); one that runs out records ISPA_ERR_TIMEOUT and unwinds.
#include <math.h>
#include <string.h>

#include "internal.h"
#include "rows.cuh"
#include "sm100.cuh"

namespace ispa {
namespace {

constexpr int kBM = 128;    // query rows per CTA
constexpr int kBN = 128;    // keys per tile
constexpr int kHalf = 64;   // keys per half
constexpr int kSBufs = 3;   // S/P buffers
constexpr int kTmemO = kSBufs * kBN;
constexpr int kFirstSoftmaxWarp = 3;
constexpr int kSoftmaxThreads = 256;
constexpr int kThreads = 32 * kFirstSoftmaxWarp + kSoftmaxThreads;
constexpr int kMaxSel = 4096;             // list entries per row group
constexpr float kRescaleThreshold = 8.0f;  // log2 units

struct Maps {
  CUtensorMap q;
  CUtensorMap k[3];    // sink, local: {64 cols, 128 rows}; history: {64 cols, 64 rows}
  CUtensorMap v[3];
  CUtensorMap out[2];  // O_full, D
};

struct Params {
  int n_q, n_kv[3];
  int tiles[2];  // sink, local
  float scale_log2;
  bool want_d;
  __nv_bfloat16* o_loc;
  __nv_bfloat16* o_full;
  int64_t ld_o;
  float* lse_loc;
  float* lse_hist;
  unsigned* status;
  const int32_t* idx;  // [n_heads, groups, n_sel]
  int n_sel, block, groups, rows_per_group, n_blocks;
};

template <int HD>
struct Cfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kBoxBytes = 128 * 128;  // 64 columns of 128 rows
  static constexpr int kTileBytes = 128 * HD * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kTileBytes;
  static constexpr int kOffV = kOffK + 2 * kTileBytes;
  static constexpr int kOffBar = kOffV + 2 * kTileBytes;
  // q_full, k_full[2], v_full[2], s_full[3], p_ready[3], o_done[2], m_ready[2], o_local, o_final, final
  static constexpr int kNumBars = 18;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8 + 8;
  static constexpr int kOffSum = kOffMisc + 32;             // [group][128 rows] sums of a branch
  static constexpr int kOffRun = kOffSum + 2 * kBM * 4;     // [tile % 2][128 rows] running maxima
  static constexpr int kOffList = kOffRun + 2 * kBM * 4;    // first key of each half
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(kBM, kBN, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, HD, false, true);
  static_assert(kOffList + 2 * kMaxSel * 4 <= 232448, "shared memory budget");
};

__device__ __forceinline__ void store_tile_2d(const CUtensorMap* map, const void* smem_src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(smem_src)), "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// O_loc, kCols columns of a thread's row from TMEM: rounded, to its place; with a history, the lower 16 bits of the
// fp32 value wait in O_full's.  Read as a signed number they are what the rounding left, so adding them below the
// rounded value's bits gives the fp32 value again; only a value halfway between two bf16 ones (read as -32768
// either way) cannot be told from its neighbour and moves to the even one's side first, by one unit of fp32.
// Not inlined: the softmax loop around its call keeps its registers (410 -> 405 us on the case above).
template <int kCols>
__device__ __noinline__ void set_aside(uint32_t src, float inv_l, __nv_bfloat16* o_loc, __nv_bfloat16* o_full,
                                       bool has_hist, bool live) {
#pragma unroll 1
  for (int c = 0; c < kCols / 16; ++c) {
    uint32_t o0[16];
    float o[16];
    tmem_ld16(src + c * 16, o0);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = __uint_as_float(o0[j]) * inv_l;
    if (live) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (has_hist) {
          uint32_t lo[4];
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            uint32_t b[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              b[x] = __float_as_uint(o[8 * i + j + x]);
              if ((b[x] & 0xFFFFu) == 0x8000u) b[x] += (b[x] & 0x10000u) ? 1u : 0xFFFFFFFFu;
              o[8 * i + j + x] = __uint_as_float(b[x]);
            }
            lo[j / 2] = __byte_perm(b[0], b[1], 0x5410);
          }
          *reinterpret_cast<uint4*>(o_full + c * 16 + 8 * i) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        *reinterpret_cast<uint4*>(o_loc + c * 16 + 8 * i) = pack8(o + 8 * i);
      }
    }
    __syncwarp();  // the next columns' load takes the whole warp
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) attn_blocks_tc_kernel(const __grid_constant__ Maps maps, const Params p) {
  using C = Cfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023) != 0) {  // the swizzled TMA / UMMA layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicOr(p.status, kStatusInternal);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* v_full = bars + 3;
  uint64_t* s_full = bars + 5;
  uint64_t* p_ready = bars + 8;
  uint64_t* o_done = bars + 11;
  uint64_t* m_ready = bars + 13;
  uint64_t* o_local = bars + 15;  // every tile of the local branch is in O
  uint64_t* o_final = bars + 16;
  uint64_t* final_bar = bars + 17;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* never = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);  // stays 0: drain waits
  int* n_halves_slot = reinterpret_cast<int*>(smem + C::kOffMisc + 12);
  int* list = reinterpret_cast<int*>(smem + C::kOffList);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // warp-uniform
  const int lane = threadIdx.x & 31;
  const int head = blockIdx.y;
  const int q0 = blockIdx.x * kBM;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(v_full + i, 1);
      mbar_init(o_done + i, 1);
      mbar_init(m_ready + i, 4);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_ready + i, kSoftmaxThreads / 64);
    }
    mbar_init(o_local, 1);
    mbar_init(o_final, 1);
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    *never = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 2) {  // the list of halves, in list order
    const int32_t* row = p.idx + (static_cast<int64_t>(head) * p.groups + q0 / p.rows_per_group) * p.n_sel;
    const int per = p.block / kHalf;
    int n = 0;
    for (int i = 0; i < p.n_sel; i += 32) {
      const int pick = i + lane < p.n_sel ? row[i + lane] : -1;
      int c = 0, key0 = 0;
      if (pick >= 0 && pick < p.n_blocks) {
        key0 = pick * p.block;
        c = min(per, (p.n_kv[2] - key0 + kHalf - 1) / kHalf);
      }
      int inc = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += v;
      }
      for (int j = 0; j < c; ++j) list[n + inc - c + j] = key0 + j * kHalf;
      n += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      *n_halves_slot = n;
      list[n] = p.n_kv[2];  // the missing half of an odd list: past the end, so TMA fills zeros
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_halves = *n_halves_slot;
  const int T1 = p.tiles[0] + p.tiles[1];
  const int T = T1 + (n_halves + 1) / 2;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------------ TMA producers (K: warp 0, V: warp 2)
    if (lane == 0) {
      const bool is_k = warp == 0;
      uint64_t* full = is_k ? k_full : v_full;
      if (is_k) {
        mbar_arrive_expect_tx(q_full, C::kTileBytes);
#pragma unroll
        for (int b = 0; b < C::kBoxes; ++b)
          tma_load_2d(smem + C::kOffQ + b * C::kBoxBytes, &maps.q, q_full, head * HD + 64 * b, q0);
      }
      int issued = 0;
      for (int t = 0; t < T; ++t) {
        const int s = t & 1;
        // stage t % 2 frees with the MMA of tile t - 2
        if (t >= 2 && !(is_k ? mbar_wait(s_full + (t - 2) % kSBufs, ((t - 2) / kSBufs) & 1, abort_flag)
                             : mbar_wait(o_done + s, ((t >> 1) - 1) & 1, abort_flag))) {
          atomicOr(p.status, kStatusTimeout);
          *abort_flag = 1;
          break;
        }
        mbar_arrive_expect_tx(full + s, C::kTileBytes);
        uint8_t* dst = smem + (is_k ? C::kOffK : C::kOffV) + s * C::kTileBytes;
        if (t < T1) {
          const int seg = t < p.tiles[0] ? 0 : 1;
          const int key0 = (t - (seg ? p.tiles[0] : 0)) * kBN;
          const CUtensorMap* map = is_k ? &maps.k[seg] : &maps.v[seg];
#pragma unroll
          for (int b = 0; b < C::kBoxes; ++b) tma_load_2d(dst + b * C::kBoxBytes, map, full + s, head * HD + 64 * b, key0);
        } else {
          const CUtensorMap* map = is_k ? &maps.k[2] : &maps.v[2];
          const int key0 = list[2 * (t - T1)], key1 = list[2 * (t - T1) + 1];
#pragma unroll
          for (int b = 0; b < C::kBoxes; ++b) {
            tma_load_2d(dst + b * C::kBoxBytes, map, full + s, head * HD + 64 * b, key0);
            tma_load_2d(dst + b * C::kBoxBytes + kHalf * 128, map, full + s, head * HD + 64 * b, key1);
          }
        }
        issued = t + 1;
      }
      // Never leave the CTA with bulk copies in flight: wait for the last load of every stage.
      if (*abort_flag) {
        for (int t = issued - 1; t >= 0 && t >= issued - 2; --t) mbar_wait(full + (t & 1), (t >> 1) & 1, never);
        if (is_k) mbar_wait(q_full, 0, never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    {
      const uint32_t leader = elect_leader();
      bool ok = mbar_wait_warp(q_full, 0, abort_flag);
      tc_fence_after();
      const uint32_t q_base = smem_u32(smem + C::kOffQ);
      auto issue_qk = [&](int t) -> bool {
        const int s = t & 1, buf = t % kSBufs;  // the buffer is free: PV_{t-3} was issued before
        if (!mbar_wait_warp(k_full + s, (t >> 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t k_base = smem_u32(smem + C::kOffK + s * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kBoxBytes + (kk & 3) * 32;
          umma_ss_warp(tmem + buf * kBN, sw128_desc(q_base + off, 16, 1024), sw128_desc(k_base + off, 16, 1024), C::kIdescQK,
                       kk > 0 ? 1u : 0u, leader);
        }
        umma_commit_warp(s_full + buf, leader);
        return true;
      };
      auto issue_pv = [&](int t) -> bool {
        const int s = t & 1, buf = t % kSBufs;
        if (!mbar_wait_warp(v_full + s, (t >> 1) & 1, abort_flag)) return false;
        if (!mbar_wait_warp(p_ready + buf, (t / kSBufs) & 1, abort_flag)) return false;
        tc_fence_after();
        const bool first = t == 0 || t == T1;
        const uint32_t v_base = smem_u32(smem + C::kOffV + s * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          umma_ts_warp(tmem + kTmemO, tmem + buf * kBN + kk * 8,
                       sw128_desc(v_base + kk * 16 * 128, C::kBoxBytes, 1024), C::kIdescPV, (!first || kk > 0) ? 1u : 0u, leader);
        umma_commit_warp(o_done + s, leader);
        if (t == T1 - 1) umma_commit_warp(o_local, leader);
        return true;
      };
      if (ok && T > 0) ok = issue_qk(0);
      if (ok && T > 1) ok = issue_qk(1);
      for (int t = 0; ok && t < T; ++t) {
        if (t + 2 < T) ok = issue_qk(t + 2);
        ok = ok && issue_pv(t);
      }
      if (!ok) {
        if (leader) atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
      umma_commit_warp(o_final, leader);
      umma_commit_warp(final_bar, leader);
      mbar_wait_warp(final_bar, 0, never);  // every MMA this thread issued has completed before TMEM is released
    }
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    const int quarter = warp & 3;                             // TMEM lane quarter this warp may access
    const int group = (warp - kFirstSoftmaxWarp) >> 2;        // takes the tiles t % 2 == group
    const int row = quarter * 32 + lane;                      // query row within the tile == TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const float sl2 = p.scale_log2;
    constexpr int kOCols = HD / 2;  // output columns per thread
    float* sums = reinterpret_cast<float*>(smem + C::kOffSum);
    float* running = reinterpret_cast<float*>(smem + C::kOffRun);
    // m: the reference of this thread's partial sum l, the row's running maximum after the group's last tile
    float m = -INFINITY, l = 0.f;
    const bool has_hist = n_halves > 0;
    // A warp whose bounded wait ran out stops working but keeps meeting the barriers.
    bool alive = true;

    // The end of a branch whose last tile is `last`: every thread gets the row's (m, l), and O is complete.
    float m_row, l_row;
    auto join = [&](int last, uint64_t* done) {
      if (alive) alive = mbar_wait_warp(done, 0, abort_flag);
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");  // every tile's maxima are read
      m_row = running[(last & 1) * kBM + row];
      sums[group * kBM + row] = m == m_row ? l : l * exp2f(m - m_row);
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
      l_row = sums[row] + sums[kBM + row];
      tc_fence_after();
    };
    // 16 columns from c * 16 of this thread's part of the branch's output
    const int o_col = group * kOCols;
    auto output = [&](int c, float inv_l, float* o) {
      uint32_t o0[16];
      tmem_ld16(tmem + lane_addr + kTmemO + o_col + c * 16, o0);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __uint_as_float(o0[j]) * inv_l;
    };
    const bool live_row = q0 + row < p.n_q;
    const int64_t o_at = static_cast<int64_t>(q0 + row) * p.ld_o + head * HD + o_col;
    auto store_local = [&]() {
      set_aside<kOCols>(tmem + lane_addr + kTmemO + o_col, 1.f / l_row, p.o_loc + o_at, p.o_full + o_at, has_hist, live_row);
    };
    // the eight values of O_loc set aside at `at`
    auto load_local = [&](int64_t at, float* v) {
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      const uint4 hi4 = live_row ? *reinterpret_cast<const uint4*>(p.o_loc + at) : zero;
      const uint4 lo4 = live_row ? *reinterpret_cast<const uint4*>(p.o_full + at) : zero;
      const uint32_t hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w}, lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float((hi[j] << 16) + static_cast<uint32_t>(static_cast<int32_t>(lo[j] << 16) >> 16));
        v[2 * j + 1] = __uint_as_float((hi[j] & 0xFFFF0000u) + static_cast<uint32_t>(static_cast<int32_t>(lo[j]) >> 16));
      }
    };

    float lse_loc2 = 0.f;  // in log2 units
    bool in_hist = false;
    for (int t = group;; t += 2) {
      if (has_hist && !in_hist && t >= T1) {  // branch switch: set the local branch aside, both groups together
        in_hist = true;
        join(T1 - 1, o_local);
        if (alive) {
          lse_loc2 = m_row + __log2f(l_row);
          store_local();
          tc_fence_before();
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");  // O may be overwritten
        m = -INFINITY;
        l = 0.f;
      }
      if (t >= T) break;
      const uint32_t s_addr = tmem + lane_addr + t % kSBufs * kBN;
      int lim[2];  // how many of each half's columns hold real keys
      if (t < T1) {
        const int seg = t < p.tiles[0] ? 0 : 1;
        lim[0] = p.n_kv[seg] - (t - (seg ? p.tiles[0] : 0)) * kBN;
        lim[1] = lim[0] - kHalf;
      } else {
        lim[0] = p.n_kv[2] - list[2 * (t - T1)];
        lim[1] = p.n_kv[2] - list[2 * (t - T1) + 1];
      }
      if (alive) alive = mbar_wait_warp(s_full + t % kSBufs, (t / kSBufs) & 1, abort_flag);
      if (!alive) continue;
      tc_fence_after();
      uint32_t r[kBN];
#pragma unroll
      for (int c = 0; c < kBN / 32; ++c) tmem_ld32(s_addr + c * 32, r + c * 32);
      tmem_wait_ld();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lim[h] < kHalf) {
#pragma unroll
          for (int j = 0; j < kHalf; ++j)
            if (j >= lim[h]) r[h * kHalf + j] = __float_as_uint(-INFINITY);
        }
      float m16[kBN / 8];
#pragma unroll
      for (int i = 0; i < kBN / 8; ++i) {
        const float* v = reinterpret_cast<const float*>(r + 8 * i);
        m16[i] = max3f(max3f(v[0], v[1], v[2]), max3f(v[3], v[4], v[5]), fmaxf(v[6], v[7]));
      }
#pragma unroll
      for (int i = 0; i < 5; ++i) m16[i] = max3f(m16[i], m16[i + 5], m16[i + 10]);
      const float top = fmaxf(max3f(m16[0], m16[1], m16[2]), max3f(m16[3], m16[4], m16[15])) * sl2;
      // the running maximum after the other group's last tile
      float m_prev = -INFINITY;
      if (t != 0 && t != T1) {
        alive = mbar_wait_warp(m_ready + ((t - 1) & 1), ((t - 1) >> 1) & 1, abort_flag);
        m_prev = running[((t - 1) & 1) * kBM + row];
      }
      const float m_new = m_prev == -INFINITY || top > m_prev + kRescaleThreshold ? top : m_prev;
      running[(t & 1) * kBM + row] = m_new;
      __syncwarp();
      if (lane == 0) mbar_arrive(m_ready + (t & 1));
      if (!alive) continue;
      const bool rescale = m_new != m_prev && m_prev != -INFINITY;
      if (m != m_new) {  // m = -inf: nothing to scale yet
        l *= fast_exp2(m - m_new);
        m = m_new;
      }
      const float neg_m = m == -INFINITY ? 0.f : -m;  // a row whose keys so far all score -inf: weights 0
      const uint64_t sl2x2 = pack_f2(sl2, sl2), negm2 = pack_f2(neg_m, neg_m);
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[kHalf / 2];
#pragma unroll
        for (int j = 0; j < kHalf; j += 2) {
          const int x = h * kHalf + j;
          const uint64_t y = fma_f2(pack_f2(__uint_as_float(r[x]), __uint_as_float(r[x + 1])), sl2x2, negm2);
          float y0, y1;
          unpack_f2(y, y0, y1);
          const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
          acc[(j >> 1) & 3] = add_f2(acc[(j >> 1) & 3], pack_f2(p0, p1));
          pk[j >> 1] = pack_bf16x2(p0, p1);
        }
        tmem_st32(s_addr + h * (kHalf / 2), pk);  // over S, read by now
      }
      float a0, a1, a2, a3, a4, a5, a6, a7;
      unpack_f2(acc[0], a0, a1);
      unpack_f2(acc[1], a2, a3);
      unpack_f2(acc[2], a4, a5);
      unpack_f2(acc[3], a6, a7);
      l += ((a0 + a1) + (a2 + a3)) + ((a4 + a5) + (a6 + a7));
      // The warp rescales together if any of its rows needs it; only then must PV_{t-1} be complete.
      // S_t complete implies PV_{t-3} complete, so the parity wait on o_done cannot alias.
      const bool any = __any_sync(0xffffffffu, rescale);
      if (any) alive = mbar_wait_warp(o_done + ((t - 1) & 1), ((t - 1) >> 1) & 1, abort_flag);
      if (!alive) continue;
      if (any) {
        tc_fence_after();
        const float alpha = rescale ? fast_exp2(m_prev - m_new) : 1.f;
        const uint32_t o_addr = tmem + lane_addr + kTmemO;
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_addr + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
          tmem_st32(o_addr + c * 32, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready + t % kSBufs);
    }
    join(T - 1, o_final);
    // staging tile of output w (0 O_full, 1 D) in the idle V ring: o_final has seen every MMA complete, and
    // every load the MMAs waited for
    auto stage = [&](int w) -> uint8_t* { return smem + C::kOffV + w * C::kTileBytes; };
    if (!alive) {
      atomicOr(p.status, kStatusTimeout);
      *abort_flag = 1;
    } else {
      const float lse2 = m_row + __log2f(l_row);
      float w_loc = 1.f, w_hist = 0.f;
      if (has_hist) {
        const float mm = fmaxf(lse_loc2, lse2);
        const float a = exp2f(lse_loc2 - mm), bb = exp2f(lse2 - mm);
        w_loc = a / (a + bb);
        w_hist = bb / (a + bb);
      } else {
        lse_loc2 = lse2;
        store_local();
      }
      const float inv_l = l_row != 0.f ? 1.f / l_row : 0.f;
      auto put = [&](int which, int col, const float* v8) {  // 8 values at tile column col, 128-byte swizzle
        *reinterpret_cast<uint4*>(stage(which) + (col >> 6) * C::kBoxBytes + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4)) =
            pack8(v8);
      };
#pragma unroll 1
      for (int c = 0; c < kOCols / 16; ++c) {
        float o[16];
        output(c, has_hist ? inv_l : 1.f / l_row, o);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float vf[8], vd[8];
          if (has_hist) {
            float vl[8];
            load_local(o_at + c * 16 + 8 * i, vl);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              vf[j] = fmaf(w_loc, vl[j], w_hist * o[8 * i + j]);
              vd[j] = w_hist * (o[8 * i + j] - vl[j]);  // vf - vl would lose a share below the rounding of vf
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              vf[j] = o[8 * i + j];
              vd[j] = vf[j] - vf[j];
            }
          }
          const int col = o_col + c * 16 + 8 * i;
          put(0, col, vf);
          if (p.want_d) put(1, col, vd);
        }
      }
      if (live_row && group == 0) {
        const float ln2 = 0.69314718055994531f;
        const int64_t at = static_cast<int64_t>(head) * p.n_q + q0 + row;
        p.lse_loc[at] = lse_loc2 * ln2;
        p.lse_hist[at] = has_hist ? lse2 * ln2 : -INFINITY;
      }
      asm volatile("fence.proxy.async;" ::: "memory");  // of the staging tiles, and of O_full's place in memory
    }
    // every softmax thread has staged its part (or the CTA gave up); one thread stores the tiles
    asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
    if (warp == kFirstSoftmaxWarp && lane == 0 && !*abort_flag) {
      for (int w = 0; w < (p.want_d ? 2 : 1); ++w)
        for (int b = 0; b < C::kBoxes; ++b) store_tile_2d(&maps.out[w], stage(w) + b * C::kBoxBytes, head * HD + 64 * b, q0);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
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
cudaError_t launch_hd(const AttnLaunch& a, const BlockList& b, cudaStream_t stream, int* n_launched) {
  using C = Cfg<HD>;
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  const uint64_t d = static_cast<uint64_t>(a.n_heads) * HD;
  bool ok = make_map_bf16_2d(&maps.q, a.q, a.n_q, d, a.ld_q, 64, kBM);
  Params p;
  memset(&p, 0, sizeof(p));
  for (int s = 0; s < 3; ++s) {
    p.n_kv[s] = static_cast<int>(a.n_kv[s]);
    if (a.n_kv[s] == 0) continue;
    if (s < 2) p.tiles[s] = (p.n_kv[s] + kBN - 1) / kBN;
    const uint32_t box = s == 2 ? kHalf : kBN;
    ok = ok && make_map_bf16_2d(&maps.k[s], a.k[s], a.n_kv[s], d, a.ld_k[s], 64, box) &&
         make_map_bf16_2d(&maps.v[s], a.v[s], a.n_kv[s], d, a.ld_v[s], 64, box);
  }
  ok = ok && make_map_bf16_2d(&maps.out[0], a.o_full, a.n_q, d, a.ld_o, 64, kBM) &&
       (!a.d_out || make_map_bf16_2d(&maps.out[1], a.d_out, a.n_q, d, a.ld_o, 64, kBM));
  if (!ok) return cudaErrorInvalidValue;
  p.n_q = static_cast<int>(a.n_q);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.want_d = a.d_out != nullptr;
  p.o_loc = static_cast<__nv_bfloat16*>(a.o_loc);
  p.o_full = static_cast<__nv_bfloat16*>(a.o_full);
  p.ld_o = a.ld_o;
  p.lse_loc = a.lse_loc;
  p.lse_hist = a.lse_hist;
  p.status = a.status;
  p.idx = b.idx;
  p.n_sel = a.n_kv[2] > 0 ? b.n_sel : 0;
  p.block = b.block;
  p.groups = static_cast<int>(b.groups);
  p.rows_per_group = b.q_block;
  p.n_blocks = b.n_blocks;
  cudaError_t e = cudaFuncSetAttribute(attn_blocks_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kOffList + 2 * kMaxSel * 4 + 16);
  if (e != cudaSuccess) return e;
  // the list holds one or two halves per entry, and one entry past an odd count
  const int smem = C::kOffList + (p.n_sel * (b.block / kHalf) + 1) * 4;
  dim3 grid(static_cast<unsigned>((a.n_q + kBM - 1) / kBM), static_cast<unsigned>(a.n_heads));
  attn_blocks_tc_kernel<HD><<<grid, kThreads, smem, stream>>>(maps, p);
  *n_launched += 1;
  return cudaGetLastError();
}

}  // namespace

bool attn_blocks_tc_supported(const AttnLaunch& a, const BlockList& b) {
  return attn_tc_supported(a) && (b.block == 64 || b.block == 128) && b.q_block % kBM == 0 && b.n_sel <= kMaxSel;
}

cudaError_t launch_attn_blocks_tc(const AttnLaunch& a, const BlockList& b, cudaStream_t s, int* n_launched) {
  return a.head_dim == 128 ? launch_hd<128>(a, b, s, n_launched) : launch_hd<64>(a, b, s, n_launched);
}

}  // namespace ispa
