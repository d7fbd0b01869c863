// Routed product of a mixture-of-experts layer for batches that give an
// expert few rows (decoding): row r of C is the codes of A's row src[r] / k
// (or r) against the weight of the expert whose range offs[e] .. offs[e+1]
// holds r, in the method of the 1x128 x 128x128 GEMM ("Mask a_s/b_s scale
// loads in blockwise FP8 training GEMM kernels"):
//   C[r,n] = sum over 128-wide K-blocks kb of a_s[row,kb] b_s[n/128,kb] P_kb,
// P_kb the e4m3 x e4m3 partial product, promoted per K-block into fp32.
//
// Each reached expert's weight is read once from memory, which is what bounds
// the product; so the operands swap places in the MMA, as in the dense GEMM
// for few rows: 128 rows of W are the instruction's A, streamed by TMA through
// a ring that holds most of an SM's shared memory, and R = 16, 32 or 64 tokens
// its B, gathered by TMA from the tokens' codes (four rows a gather; gathers past
// the expert's last row are left out).  A persistent CTA per SM goes through a contiguous
// run of (128-row tile, R tokens) walks over all reached experts without
// draining the ring in between; a tile is walked again for the next R rows of
// its expert, from L2.  Where the batch is so small that the tiles leave SMs idle
// (and its rows are few enough for one walk), each tile's K-blocks are split over
// a cluster instead and the partial sums added in rank order through distributed
// shared memory.
// 64 experts of 2048 x 4096, eight a token: 64 tokens (every expert reached, 537 MB
// of weights) 87.4 us, 6.1 TB/s, 0.91 of the copy rate; 512 tokens 120; one token
// with the weights in memory 15.2 us, in L2 12.1.  (The codes straight into the
// registers of an 8-bit mma.sync: 116 us for 32 tokens, against 86.)
//
//   warps 0, 8..  producers: warp 0 W's tile, each of them 16 tokens
//   warps 1, 3    MMA issuers (M = 128, N = R) on alternate K-blocks
//   warp 2        a_s of the tokens and b_s of the tile, per K-block
//   warps 4-7     promotion (lane n: column n of the tile, its R tokens), stores
// Every mbarrier wait is bounded; a role that gives up sets the abort flag, the
// others leave their loops, and copies and MMAs in flight finish before the
// CTA exits.
#include <cudaTypedefs.h>
#include <string.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

static __device__ uint32_t g_routed_error;

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRpTile = 128;  // rows of W a tile

template <int R>
struct RpCfg {
  static_assert(R == 16 || R == 32 || R == 64, "tokens of one walk");
  // one producer warp for each 16 tokens: a warp issues a gather of four every 84
  // cycles or so, and a K-block's weights arrive every 700
  static constexpr int kProducers = R / 16;
  static constexpr int kThreads = 256 + 32 * (kProducers - 1);
  static constexpr int kStages = R == 16 ? 11 : R == 32 ? 10 : 8;
  static constexpr int kBufs = R == 64 ? 4 : 8;             // R-column partial products in tensor memory
  static constexpr int kTmemCols = kBufs * R;               // 128 or 256
  static constexpr int kWBytes = kRpTile * kBlock;          // 16 KiB
  static constexpr int kXBytes = R * kBlock;
  static constexpr int kSlotBytes = (4 * R + 16 + 127) / 128 * 128;  // a_s[R], then b_s at byte 4R
  static constexpr int kOffX = kStages * kWBytes;
  static constexpr int kOffSlot = kOffX + kStages * kXBytes;
  static constexpr int kOffExpert = kOffSlot + kStages * kSlotBytes;
  static constexpr int kOffWalk = kOffExpert + kMaxGroups * 4;      // walks before each reached expert
  static constexpr int kOffBar = kOffWalk + (kMaxGroups + 4) * 4;
  // full[S] empty[S] sfull[S] sempty[S] tfull[T] tempty[T] drain
  static constexpr int kNumBars = 4 * kStages + 2 * kBufs + 1;
  static constexpr int kOffMisc = kOffBar + (kNumBars + 1) / 2 * 16;  // tensor memory's address, abort flag, a zero
  static constexpr int kOffCount = kOffMisc + 16;
  static constexpr int kSmemBytes = kOffCount + 2 * 4 * (kThreads / 32) + 1024;
  static_assert(kRpTile * R * 4 <= kStages * kWBytes, "the partial sums of a split tile fit in the W stages");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// Four rows y0 .. y3 x 128 bytes from byte x on, one after the other at dst; rows past the tensor's are zeros.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y0,
                                            int32_t y1, int32_t y2, int32_t y3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float lds32_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// The A row that is gathered for sorted row m of an expert whose rows end at r1: its
// slot's token, or m itself; a.T (past A, read as zeros) where there is none.
__device__ __forceinline__ int token_of(const GemmRoutedArgs& a, int64_t m, int64_t r1) {
  if (m >= r1) return (int)a.T;
  int64_t t = m;
  if (a.src) {
    const int slot = __ldg(a.src + m);
    t = slot >= 0 ? (int64_t)((uint32_t)slot / (uint32_t)a.k) : a.T;
  }
  return (int)(t < a.T ? t : a.T);
}

}  // namespace

template <int R>
__global__ void __launch_bounds__(RpCfg<R>::kThreads, 1)
    gemm_routed_kernel(const __grid_constant__ CUtensorMap tma_w, const __grid_constant__ CUtensorMap tma_x,
                       const GemmRoutedArgs a, const int splits) {
  using Cfg = RpCfg<R>;
  constexpr int ST = Cfg::kStages, NT = Cfg::kBufs, kWarps = Cfg::kThreads / 32;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem), sX = sbase + Cfg::kOffX, sSlot = sbase + Cfg::kOffSlot;
  const uint32_t full0 = sbase + Cfg::kOffBar, empty0 = full0 + 8 * ST, sfull0 = empty0 + 8 * ST,
                 sempty0 = sfull0 + 8 * ST, tfull0 = sempty0 + 8 * ST, tempty0 = tfull0 + 8 * NT,
                 drain = tempty0 + 8 * NT;
  int* s_expert = reinterpret_cast<int*>(smem + Cfg::kOffExpert);
  int* s_walk = reinterpret_cast<int*>(smem + Cfg::kOffWalk);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  volatile int* never = abort_flag + 1;
  int* s_count = reinterpret_cast<int*>(smem + Cfg::kOffCount);
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = __shfl_sync(kAll, tid >> 5, 0);
  const int E = (int)a.E;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full0 + 8 * i, Cfg::kProducers);
      mbar_init(empty0 + 8 * i, 1);
      mbar_init(sfull0 + 8 * i, 32);  // one cp.async arrival per loader lane
      mbar_init(sempty0 + 8 * i, 4);  // the promotion warps
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(tfull0 + 8 * i, 1);
      mbar_init(tempty0 + 8 * i, 4);
    }
    mbar_init(drain, 2);  // one commit per issuer
    *abort_flag = 0;
    *never = 0;
    fence_barrier_init();
    fence_proxy_async_shared();
    if (a.K > 0) {
      tma_prefetch_desc(&tma_w);
      tma_prefetch_desc(&tma_x);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), Cfg::kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  // the experts that hold rows, in order, and the walks (of R rows) before each
  int reached = 0, walks = 0;
  constexpr int kFell = 1 << 16;  // added to the count for a warp whose experts' offsets decrease
  for (int e0 = 0; e0 < E; e0 += Cfg::kThreads) {
    const int e = e0 + tid;
    int64_t rows = 0;
    bool falls = false;
    if (e < E) {
      const int o0 = __ldg(a.offs + e), o1 = __ldg(a.offs + e + 1);
      rows = min((int64_t)o1, a.R) - max(o0, 0);
      falls = o1 < o0;
    }
    const int mine = rows > 0 ? (int)((rows + R - 1) / R) : 0;
    const uint32_t vote = __ballot_sync(kAll, mine > 0);
    const int fell = __any_sync(kAll, falls) ? kFell : 0;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) {
      s_count[warp] = __popc(vote) + fell;
      s_count[kWarps + warp] = inc;
    }
    __syncthreads();
    int at = reached, before = walks;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += s_count[w], before += s_count[kWarps + w];
      reached += s_count[w];
      walks += s_count[kWarps + w];
    }
    if (mine > 0) {
      at = (at & (kFell - 1)) + __popc(vote & ((1u << lane) - 1u));
      s_expert[at] = e;
      s_walk[at] = before + inc - mine;
    }
    __syncthreads();
  }
  if (reached >= kFell) {
    // decreasing offsets are no plan's: experts may overlap, and their walks pass the launcher's bound
    reached = walks = 0;
    if (blockIdx.x == 0 && tid == 0) atomicOr(&g_routed_error, kRoutedOffsets);
  }
  if (tid == 0) s_walk[reached] = walks;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  const int Kb = (int)cdiv(a.K, kBlock), blocks = (int)cdiv(a.N, kRpTile);
  // Work: walks, each R rows of an expert against a 128-row tile of its weight;
  // expert by expert, tile by tile, the walks of one tile side by side (they
  // share it through L2).  Walk x of the launch belongs to the last reached
  // expert i with s_walk[i] * blocks <= x.  This CTA takes a contiguous run of
  // them, and its share of each one's K-blocks (split = the rank in the cluster);
  // every role goes through the same walks in the same order.
  // (The launcher keeps the number of walks below 2^31.)
  const int all = walks * blocks;
  const int group = (int)blockIdx.x / splits, groups = (int)gridDim.x / splits, split = (int)blockIdx.x % splits;
  const int first = (int)((int64_t)all * group / groups), last = (int)((int64_t)all * (group + 1) / groups);
  const int kb0 = smallm_kb_lo(split, splits, Kb), kbn = smallm_kb_lo(split + 1, splits, Kb) - kb0;
  struct Walk {
    int x;
    int i, e, block;  // reached expert, expert, tile
    int64_t m0, r1;   // first row, end of the expert's rows
  };
  auto enter = [&](Walk& w) {
    while (w.i + 1 < reached && s_walk[w.i + 1] * blocks <= w.x) ++w.i;
    const int in = w.x - s_walk[w.i] * blocks, per = s_walk[w.i + 1] - s_walk[w.i];
    w.e = s_expert[w.i];
    w.block = per == 1 ? in : in / per;
    w.m0 = max(__ldg(a.offs + w.e), 0) + (int64_t)(in - w.block * per) * R;
    w.r1 = min((int64_t)__ldg(a.offs + w.e + 1), a.R);
  };
  auto next = [&](Walk& w) {
    if (++w.x < last) enter(w);
  };
  auto fail = [&](uint32_t code) {
    if (!*abort_flag) atomicOr(&g_routed_error, code);
    *abort_flag = 1;
  };
  Walk w{first, 0, 0, 0, 0, 0};
  if (first < last) {
    int hi = reached;  // s_walk[w.i] * blocks <= first < s_walk[hi] * blocks
    while (hi - w.i > 1) {
      const int mid = (w.i + hi) >> 1;
      if (s_walk[mid] * blocks <= first) w.i = mid;
      else hi = mid;
    }
    enter(w);
  }
  const Walk w_first = w;
  bool ok = true;

  if (warp == 0 || warp >= 8) {
    // ------------------------------------------------------------ producers: tokens 16 q .. 16 q + 15, q = 0 also W
    const int q = warp == 0 ? 0 : warp - 7;
    constexpr uint32_t kPart = 16 * kBlock;  // bytes of a producer's tokens
    // Gathers of four rows that hold a row of the walk; the others are left out:
    // what their rows of the stage hold feeds columns that are not stored.
    auto gathers = [&]() { return (int)((min(max(w.r1 - w.m0 - 16 * q, (int64_t)0), (int64_t)16) + 3) / 4); };
    int n = 0;                               // K-blocks issued
    int at_e = -1;
    int64_t at_m = -1;
    int tok[4] = {};
    auto issue_w = [&](int j, int st, int row) {  // lane 0 of producer 0
      mbar_arrive_expect_tx(full0 + 8 * st, (uint32_t)(Cfg::kWBytes + 512 * gathers()));
      tma_load_2d(sbase + (uint32_t)(st * Cfg::kWBytes), &tma_w, full0 + 8 * st, (kb0 + j) * kBlock, row);
    };
    // the first stages' weights go out before the tokens are known
    const int ahead = w.x < last ? min(ST, kbn) : 0;
    if (q == 0 && lane == 0)
      for (int j = 0; j < ahead; ++j) issue_w(j, j, w.e * (int)a.N + w.block * kRpTile);
    for (; w.x < last && ok; next(w)) {
      if (w.e != at_e || w.m0 != at_m) {
        at_e = w.e, at_m = w.m0;
        if (lane < 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) tok[i] = token_of(a, w.m0 + 16 * q + 4 * lane + i, w.r1);
        }
      }
      const int row = w.e * (int)a.N + w.block * kRpTile, live = gathers();
      for (int j = 0; j < kbn; ++j, ++n) {
        const int st = n % ST;
        if (n >= ahead) {
          ok = mbar_wait_bounded(empty0 + 8 * st, (uint32_t)((n / ST) & 1) ^ 1u, kWaitLimitNs, abort_flag);
          if (!__all_sync(kAll, ok)) {
            if (lane == 0) fail(1u);
            ok = false;
            break;
          }
          if (q == 0 && lane == 0) issue_w(j, st, row);
        }
        if (q > 0 && lane == 0) mbar_arrive_expect_tx(full0 + 8 * st, (uint32_t)(512 * live));
        __syncwarp();
        if (lane < live)
          tma_gather4(sX + (uint32_t)(st * Cfg::kXBytes) + q * kPart + lane * 512, &tma_x, full0 + 8 * st,
                      (kb0 + j) * kBlock, tok[0], tok[1], tok[2], tok[3]);
      }
    }
    if (!ok && lane == 0)  // copies already issued land before this CTA's shared memory goes away
      for (int i = n > ST ? n - ST : 0; i < max(n, ahead); ++i)
        mbar_wait_bounded(full0 + 8 * (i % ST), (uint32_t)((i / ST) & 1), kWaitLimitNs, never);
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issuers (alternate K-blocks)
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kRpTile, R);
      int n = 0;
      for (; w.x < last && ok; next(w)) {
        for (int j = 0; j < kbn && ok; ++j, ++n) {
          if ((n & 1) != (warp == 1 ? 0 : 1)) continue;
          const int st = n % ST, buf = n % NT;
          ok = mbar_spin_bounded(tempty0 + 8 * buf, (uint32_t)((n / NT) & 1) ^ 1u, kWaitLimitNs, abort_flag) &&
               mbar_spin_bounded(full0 + 8 * st, (uint32_t)((n / ST) & 1), kWaitLimitNs, abort_flag);
          if (!ok) {
            fail(2u);
            break;
          }
          tc_fence_after();
          const uint64_t da = desc_kmajor_sw128(sbase + (uint32_t)(st * Cfg::kWBytes));
          const uint64_t db = desc_kmajor_sw128(sX + (uint32_t)(st * Cfg::kXBytes));
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k)
            mma_e4m3(tmem_base + (uint32_t)(buf * R), da + (uint64_t)(2 * k), db + (uint64_t)(2 * k), idesc,
                     k > 0 ? 1u : 0u);
          mma_commit(empty0 + 8 * st);
          mma_commit(tfull0 + 8 * buf);
        }
      }
      // every MMA issued completes before tensor memory is released
      mma_commit(drain);
      if (!mbar_wait_bounded(drain, 0, kWaitLimitNs, never)) fail(4u);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ scale loader
    const int Nb = (int)cdiv(a.N, kBlock);
    constexpr int kPer = (R + 31) / 32;
    int n = 0, at_e = -1;
    int64_t at_m = -1;
    int tok[kPer] = {};
    for (; w.x < last && ok; next(w)) {
      if (w.e != at_e || w.m0 != at_m) {
        at_e = w.e, at_m = w.m0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) tok[i] = lane + 32 * i < R ? token_of(a, w.m0 + lane + 32 * i, w.r1) : (int)a.T;
      }
      const float* sb = a.sb + ((int64_t)w.e * Nb + w.block) * a.ldsb;
      for (int j = 0; j < kbn; ++j, ++n) {
        const int st = n % ST, kb = kb0 + j;
        ok = mbar_wait_bounded(sempty0 + 8 * st, (uint32_t)((n / ST) & 1) ^ 1u, kWaitLimitNs, abort_flag);
        if (!__all_sync(kAll, ok)) {
          if (lane == 0) fail(8u);
          ok = false;
          break;
        }
        const uint32_t slot = sSlot + (uint32_t)(st * Cfg::kSlotBytes);
        const float* sa = a.sa + (int64_t)kb * a.ldsa;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const bool in = (int64_t)tok[i] < a.T;  // zeros for no token
          if (lane + 32 * i < R) cp_async_4(slot + 4u * (uint32_t)(lane + 32 * i), in ? sa + tok[i] : sb, in ? 4u : 0u);
        }
        if (lane == 0) cp_async_4(slot + 4u * R, sb + kb, 4u);
        cp_async_mbar_arrive(sfull0 + 8 * st);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------------------ promotion
    const int nl = 32 * (warp - 4) + lane;  // tensor-memory lane = column nl of the tile
    const uint32_t lane_base = (uint32_t)(32 * (warp - 4)) << 16;
    int n = 0;
    for (; w.x < last && ok; next(w)) {
      float acc[R];
#pragma unroll
      for (int m = 0; m < R; ++m) acc[m] = 0.0f;
      for (int j = 0; j < kbn; ++j, ++n) {
        const int st = n % ST, buf = n % NT;
        ok = mbar_wait_bounded(sfull0 + 8 * st, (uint32_t)((n / ST) & 1), kWaitLimitNs, abort_flag) &&
             mbar_wait_bounded(tfull0 + 8 * buf, (uint32_t)((n / NT) & 1), kWaitLimitNs, abort_flag);
        if (!__all_sync(kAll, ok)) {
          if (lane == 0) fail(16u);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t slot = sSlot + (uint32_t)(st * Cfg::kSlotBytes);
        float bsc;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(bsc) : "r"(slot + 4u * R));
        const uint64_t b2 = f2_pack(bsc, bsc);
        constexpr int CH = R < 32 ? R : 32;  // columns per tensor-memory load
#pragma unroll
        for (int c = 0; c < R / CH; ++c) {
          uint32_t r[CH];
          const uint32_t taddr = tmem_base + lane_base + (uint32_t)(buf * R + c * CH);
          if constexpr (CH == 32) tmem_ld_32x32b_x32(taddr, r);
          else tmem_ld_32x32b_x16(taddr, r);
          tmem_ld_wait();
          tmem_regs_after_wait(r);
          // acc[m] += (a_s[m] * b_s) * P[m], two tokens per fp32x2 operation
#pragma unroll
          for (int q = 0; q < CH / 4; ++q) {
            float4 a4;
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(a4.x), "=f"(a4.y), "=f"(a4.z), "=f"(a4.w)
                         : "r"(slot + 4u * (uint32_t)(c * CH + 4 * q)));
            const int m = c * CH + 4 * q;
            const uint64_t s01 = f2_mul(f2_pack(a4.x, a4.y), b2), s23 = f2_mul(f2_pack(a4.z, a4.w), b2);
            f2_unpack(f2_fma(s01, f2_pack(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1])),
                             f2_pack(acc[m], acc[m + 1])),
                      acc[m], acc[m + 1]);
            f2_unpack(f2_fma(s23, f2_pack(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3])),
                             f2_pack(acc[m + 2], acc[m + 3])),
                      acc[m + 2], acc[m + 3]);
          }
        }
        // the partial and the scales have been read: release the buffer and the slot
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(tempty0 + 8 * buf);
          mbar_arrive(sempty0 + 8 * st);
        }
      }
      if (!ok) break;
      const int64_t col = (int64_t)w.block * kRpTile + nl;
      if (splits == 1) {
        if (col < a.N) {
          uint16_t* c = a.c + w.m0 * a.ldc + col;
          const int rows = (int)min(w.r1 - w.m0, (int64_t)R);
#pragma unroll
          for (int m = 0; m < R; ++m)
            if (m < rows) c[(int64_t)m * a.ldc] = (uint16_t)(pack_bf16x2(acc[m], 0.0f) & 0xFFFFu);
        }
      } else {
        // the CTA's only walk (every MMA has completed, every copy has landed): the sums go into the W stages
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int m = 0; m < R; ++m) part[m * kRpTile + nl] = acc[m];
      }
    }
  }
  __syncwarp();
  if (splits > 1) {
    // Every thread of every CTA of the cluster reaches both barriers (every
    // wait before them is bounded): the first makes the partial sums visible,
    // the second keeps each CTA resident until no peer reads them any more.
    cluster_sync_all();
    if (warp >= 4 && warp < 8 && first < last) {
      const Walk& f = w_first;
      // Row m of the walk's rows is rank m % splits' to join; the loads of four
      // rows are in flight at once (one after another, a pair of CTAs took 3 us
      // for 16 rows).
      const int nl = 32 * (warp - 4) + lane, live = (int)min(f.r1 - f.m0, (int64_t)R);
      const int64_t col = (int64_t)f.block * kRpTile + nl;
      for (int m0 = split; m0 < live; m0 += 4 * splits) {
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if (m0 + i * splits < live && s < splits)
              v[i][s] = lds32_cluster(mapa_shared(sbase + 4u * (uint32_t)((m0 + i * splits) * kRpTile + nl), (uint32_t)s));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = m0 + i * splits;
          float sum = 0.0f;
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if (m < live && s < splits) sum += v[i][s];
          if (m < live && col < a.N) a.c[(f.m0 + m) * a.ldc + col] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
        }
      }
    }
    __syncwarp();
    cluster_sync_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

static PFN_cuTensorMapEncodeTiled_v12000 rp_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Row-major [rows, inner] bytes with row stride ld: boxes of 128 bytes x box_rows rows, 128-byte swizzled, zeros
// outside.
static bool rp_map(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int64_t ld, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {kBlock, (cuuint32_t)box_rows};
  cuuint32_t elem[2] = {1, 1};
  return rp_encode_fn() != nullptr &&
         rp_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, elem,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs a tile's K-blocks are split over: 8, 4 or 2, the most for which `tiles`
// clusters are resident at once, from 8 K-blocks on.  The hand-over of the sums
// takes about 1 us, a K-block 0.2.  Measured with a split / with one CTA a tile,
// in us, tokens in brackets:
//   4 K-blocks, 16 experts of 512 columns [1]: over 4 CTAs 5.7 / 5.3;
//   6, 256 columns [1]: over 4, 5.8 / 5.6;   8, 8 experts of 128 [1]: over 8, 5.5 / 6.2;
//   8, 512 columns [1]: over 4, 5.9 / 6.2;   8, 8 experts of 1024 [1 / 4]: over 2, 6.4 / 6.2, 6.9 / 6.5;
//   16, 8 experts of 1000 [8]: over 2, 8.2 / 9.3;   16, 256 experts of 512 [1]: over 4, 6.8 / 8.3;
//   32, 16 experts of 256 [1 / 4]: over 8, 6.2 / 11.7, over 4, 7.4 / 11.7.
template <int R>
static int rp_splits(int64_t tiles, int Kb, int num_sms) {
  static std::once_flag once;
  static int max_clusters[9] = {};
  std::call_once(once, [] {
    for (int s = 2; s <= 8; s *= 2) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(s * 16));
      cfg.blockDim = dim3(RpCfg<R>::kThreads);
      cfg.dynamicSmemBytes = RpCfg<R>::kSmemBytes;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)s;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, gemm_routed_kernel<R>, &cfg) == cudaSuccess) max_clusters[s] = n;
    }
    (void)cudaGetLastError();  // a size the device refuses leaves no error behind
  });
  for (int s = 8; s >= 2; s /= 2)
    if (Kb >= 8 && tiles * s <= num_sms && tiles <= max_clusters[s]) return s;
  return 1;
}

template <int R>
static cudaError_t run_routed(const CUtensorMap& mw, const CUtensorMap& mx, const GemmRoutedArgs& a, int num_sms,
                              cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(gemm_routed_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    RpCfg<R>::kSmemBytes);
  });
  if (attr_err != cudaSuccess) return attr_err;
  const int64_t reach = a.E < a.R ? a.E : a.R;  // experts that can hold rows
  const int64_t tiles = reach * cdiv(a.N, kRpTile);
  // a split tile has one walk: only where every row fits in it
  const int splits = a.R <= R ? rp_splits<R>(tiles, (int)cdiv(a.K, kBlock), num_sms) : 1;
  const int64_t walks = (reach + a.R / R) * cdiv(a.N, kRpTile);  // at most
  const int64_t groups = splits > 1 ? tiles : walks < num_sms ? walks : num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * splits));
  cfg.blockDim = dim3(RpCfg<R>::kThreads);
  cfg.dynamicSmemBytes = RpCfg<R>::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemm_routed_kernel<R>, mw, mx, a, splits);
}

cudaError_t launch_gemm_routed(const GemmRoutedArgs& a, int num_sms, cudaStream_t st, const char** msg) {
  CUtensorMap mw, mx;
  memset(&mw, 0, sizeof(mw));
  memset(&mx, 0, sizeof(mx));
  if (a.K > 0 && a.T > 0 && (!rp_map(&mw, a.qb, a.K, a.E * a.N, a.ldb, kRpTile) || !rp_map(&mx, a.qa, a.K, a.T, a.lda, 1))) {
    *msg = "cuTensorMapEncodeTiled failed for an operand (alignment, stride or size out of range)";
    return cudaErrorInvalidValue;
  }
  // R, by the rows of an expert were they spread evenly: room for twice that, as
  // a walk less is a pass less over the tile.  Measured with R = 16 / 32 / 64, in us, at
  //   64 experts of 2048 x 4096:  1 row 58.8 / 58.5 / 60.5 (8 rows in all 12.4 / 13.0 / 14.5),
  //     8 rows 88.8 / 87.9 / 88.6, 16 rows 99.9 / 88.9 / 90.6, 32 rows 168 / 107 / 91.4, 64 rows 301 / 183 / 120;
  //   256 experts of 512 x 2048:  1 row (one token) 7.7 / 8.9 / 11.3, 16 rows 54.2 / 48.1 / 49.9.
  // Where walks of 64 are fewer than half the SMs, more of 32 share the work better:
  //   8 experts of 1000 x 2000:   38 rows (64 walks) 15.0 / 10.8 / 11.4, 100 rows (128 walks) 20.3 / 16.7 / 12.0.
  const int64_t reach = a.E < a.R ? a.E : a.R, rows = cdiv(a.R, a.E), tiles = reach * cdiv(a.N, kRpTile);
  if ((reach + a.R / 16) * cdiv(a.N, kRpTile) >= (int64_t)1 << 31) {
    *msg = "too many rows and columns: (experts + R/16) * ceil(N/128) must stay below 2^31";
    return cudaErrorInvalidValue;
  }
  if (rows <= 8) return run_routed<16>(mw, mx, a, num_sms, st);
  if (rows <= 16 || tiles * cdiv(rows, 64) < num_sms / 2) return run_routed<32>(mw, mx, a, num_sms, st);
  return run_routed<64>(mw, mx, a, num_sms, st);
}

cudaError_t routed_read_errors(uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_routed_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_routed_error, &zero, sizeof(uint32_t));
}

}  // namespace bfp8
