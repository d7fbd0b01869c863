// A whole layer of gated experts for a few tokens, after its router's launch, in
// one persistent kernel.  With the token's choices (idx, w) of bfp8_moe_route,
//   a_tj = silu(G_e q(x_t)) * (U_e q(x_t)),   y_t = sum over j of w_tj D_e q(a_tj),
// e = idx[t,j]; q quantises in 1x128 groups, G, U (one [2I, K] weight an expert,
// gate rows first) and D [N, I] are codes with 128x128 tile scales, and every
// product is promoted per 128-wide K-block into fp32 ("Mask a_s/b_s scale loads
// in blockwise FP8 training GEMM kernels": the 1x128 x 128x128 GEMM).
//
// The reached experts' codes are read once, which is what bounds the layer; so
// the kernel is one stream of them, that no part of the work interrupts:
//   - one CTA an SM, whose producers bring 16 KB stages by TMA through a ring
//     that holds most of shared memory, first its share of the gate and up rows,
//     then of the down rows;
//   - the exchange of the activations between the two (every CTA needs all of
//     them) is two barriers over the grid that only the warps behind the ring wait
//     for: the down weights do not depend on them and fill the ring meanwhile.  The
//     activations pass in fp32; each CTA codes its share behind the first barrier,
//     and takes everyone's codes behind the second, by cp.async straight into the
//     operand's place (each CTA coding all of them for itself, with one barrier: one
//     token 43.5 us against 43.8, but 16 tokens of 64 experts 248 against 213, whose
//     coding took a CTA as long as reading its weights; codes by way of registers:
//     16 tokens of 128 narrow experts 76 us against 64).
//
// First part: a unit is 16 gate rows and the 16 up rows of the same features; the
// units of all reached experts are shared evenly.  Second part: CTA c takes the
// rows [c R, c R + R) of D of every reached expert, R = N over the CTAs, so y's
// sums over experts never leave its registers.  Tiles of 128 rows of W, the usual
// operand of tcgen05.mma, would give some CTAs two and some one (one token's eight
// experts of 2 x 2048 rows are 256 of them for 152 SMs).  So the instruction's 128
// rows are 32 rows of W (or 16, 64, 128: the power of two that holds R) of four
// K-blocks, one below the other, and its columns the tokens' codes of the same
// four K-blocks side by side.  Of the product only the blocks where the two
// K-blocks are the same are read; the others cost tensor-core time that nothing
// else wants (128 x 32 x 128 a stage: a tenth of the time that its bytes take).
// (mma.sync on 16 rows instead, which needs no such blocks: 59 us for one token,
// 399 for 16, as its 8-bit form takes 250 issued instructions a warp and stage.)
//
//   warps 0, 14, 15  producers: each a third of a stage's boxes (one warp takes longer to
//                  issue a box than memory to bring it where it is small: narrow experts'
//                  13 rows of a K-block are 1.7 KB)
//   warps 1, 3     MMA issuers, on alternate stages
//   warp 2         the weights' scales, into slots ahead of the products (loaded where
//                  they are used they cost a trip to L2 a stage)
//   warps 4-7      promotion: lane l of warp w is row 32 w + l of the 128
//   warps 8-13     the activations' codes: this CTA's share of their coding, then each
//                  expert's into its buffer, ahead of the products: one, two or all
//                  six warps an expert, no more experts at once than buffers
// Producers and issuers are whole warps that stay together, of which an elected lane
// issues: a lane that left the others took 326 cycles for the four MMAs and two commits
// of a stage, an elected one 252.
//
// Measured (with the router's launch; the floor is the reached experts' codes at the
// rate of a plain copy): 64 experts of 3 x 2048 x 4096, 8 a token: one token 44 us
// (floor 30), 4 tokens 109 (99), 16 tokens 213 (212); 128 of 3 x 704 x 1920, 6 a
// token, 5 tokens 34 (16.5).  What is left at few tokens does not grow with the
// weights: the router's launch, the plan, the tokens' codes and the exchange of the
// activations.
//
// Waits are bounded; a role that gives up sets the abort flag, the others leave
// their loops, and copies and MMAs in flight finish before the CTA exits.
#include <cudaTypedefs.h>
#include <string.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

static __device__ uint32_t g_mlp_error;

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kMlpThreads = 512;
constexpr int kProducers = 3;       // warps 0, 14, 15
constexpr int kIssuers = 2;         // warps 1, 3
constexpr int kCoders = 6;          // warps 8-13
// Warps that wait for a buffer of activations, all of which have seen its codes before it is coded again: promotion's, and
// both issuers, also where an expert is one stage and so one issuer's alone (the other could find the barrier two phases
// on, whose parity is that of codes that are not there yet, and wait for good).
constexpr int kBufferReaders = 4 + kIssuers;
constexpr int kStageBytes = 128 * kBlock;
constexpr int kPairs = 16;          // gate (and up) rows of a unit
constexpr int kUnitRows = 2 * kPairs, kUnitBlocks = 128 / kUnitRows;  // K-blocks of a stage of the first part
constexpr int kMlpMaxStages = 12;
constexpr int kAtom = 1024;         // 8 rows x 128 B, 128-byte swizzled
constexpr int kTmemCols = 512, kMaxBufs = 8;
constexpr int kSlots = 8;  // slots of the scales of a few stages: 32 of them

// Shared memory after the ring, the codes and their scales (offsets from MlpArgs::off_misc).
constexpr int kOffRed = 0;                                           // two sets of [128 rows][8 NT tokens] sums
constexpr int kRedBytes = 2 * 128 * kMlpMaxTokens * 4;
constexpr int kOffMask = kOffRed + kRedBytes;                        // [E] the tokens of an expert, and the first of its slots
constexpr int kOffExpert = kOffMask + kMaxGroups * 4;                // [reached] expert | mask << 16
constexpr int kOffStart = kOffExpert + kMlpMaxSlots * 4;             // [reached] first of its slots
constexpr int kOffSlot = kOffStart + kMlpMaxSlots * 4;               // slots by expert, in token order: slot | token << 16
constexpr int kOffWeight = kOffSlot + kMlpMaxSlots * 4;              // routing weights, by slot
constexpr int kOffWsc = kOffWeight + kMlpMaxSlots * 4;               // [8 slots][stages][K-blocks][gate, up; or the two tiles of a CTA's rows]
constexpr int kOffBars = kOffWsc + kSlots * 32 * 4;
// full[12] empty[12] tfull[8] tempty[8] hfull[8] hempty[8] sfull[8] sempty[8], x ready, drain
constexpr int kOffFlag = kOffBars + 8 * (2 * kMlpMaxStages + 2 * kMaxBufs + 2 * kMlpMaxBuffers + 2 * kSlots + 2);
constexpr int kMiscBytes = kOffFlag + 16 + 4 * 16;                   // abort flag, a zero, tensor memory's address; scan[16]

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// max(amax, 1e-12) / 448 as one product with 1/448: within an ulp of group_scale's quotient.
__device__ __forceinline__ float scale_near(float amax) { return __fmul_rn(fmaxf(amax, kAmaxFloor), 1.0f / kE4m3Max); }
// Place n of a ring of `size`, by steps of at most its size, and the parity of its turn.
struct Ring {
  int at;
  uint32_t parity;
  __device__ __forceinline__ void step(int by, int size) {
    at += by;
    if (at >= size) at -= size, parity ^= 1u;
  }
};

// Eight values of a group of 16 lanes: their codes and the group's scale.
__device__ __forceinline__ float code8(const float4& p, const float4& q, uint32_t& lo, uint32_t& hi) {
  float m = fmaxf(fmaxf(fmaxf(fabsf(p.x), fabsf(p.y)), fmaxf(fabsf(p.z), fabsf(p.w))),
                  fmaxf(fmaxf(fabsf(q.x), fabsf(q.y)), fmaxf(fabsf(q.z), fabsf(q.w))));
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  const float s = scale_near(m), y = recip_rn(s);
  // (quotients, not products with y: those take the other code of a tie for one in nine of the values next to it)
  lo = cvt_e4m3x2(quotient(p.x, s, y), quotient(p.y, s, y)) | cvt_e4m3x2(quotient(p.z, s, y), quotient(p.w, s, y)) << 16;
  hi = cvt_e4m3x2(quotient(q.x, s, y), quotient(q.y, s, y)) | cvt_e4m3x2(quotient(q.z, s, y), quotient(q.w, s, y)) << 16;
  return s;
}
// C consecutive 32-bit columns of this warp's 32 lanes of tensor memory.
template <int C>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, uint32_t (&r)[C]) {
  if constexpr (C == 8) tmem_ld_32x32b_x8(taddr, r);
  else if constexpr (C == 16) tmem_ld_32x32b_x16(taddr, r);
  else tmem_ld_32x32b_x32(taddr, r);
  tmem_ld_wait();
  tmem_regs_after_wait(r);
}
// acc[t] += (xs[t] b) P[t]; `mask`: the tokens that take part (the others' columns hold anything).
template <int NC, bool MASKED>
__device__ __forceinline__ void promote(float (&acc)[NC], const uint32_t (&p)[NC], const float* xs, float b, uint32_t mask) {
#pragma unroll
  for (int t = 0; t < NC; t += 4) {
    const float4 s = *reinterpret_cast<const float4*>(xs + t);
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!MASKED || (mask >> (t + i) & 1u)) acc[t + i] = fmaf(v[i] * b, __uint_as_float(p[t + i]), acc[t + i]);
  }
}

}  // namespace

template <int NT>
__global__ void __launch_bounds__(kMlpThreads, 1)
    moe_mlp_kernel(const __grid_constant__ CUtensorMap map_gu, const __grid_constant__ CUtensorMap map_d, const MlpArgs a) {
  constexpr int NC = 8 * NT;  // token columns
  // partial products in tensor memory: at most eight K-blocks side by side
  constexpr int kBufCols = 8 * NC, kBufs = kTmemCols / kBufCols;
  static_assert(kBufs <= kMaxBufs, "their barriers");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t ring = smem_u32(smem);
  const uint32_t area = ring + (uint32_t)a.stages * kStageBytes;
  uint8_t* misc = smem + a.off_misc;
  const uint32_t full0 = smem_u32(misc + kOffBars), empty0 = full0 + 8 * kMlpMaxStages, tfull0 = empty0 + 8 * kMlpMaxStages,
                 tempty0 = tfull0 + 8 * kMaxBufs, hfull0 = tempty0 + 8 * kMaxBufs, hempty0 = hfull0 + 8 * kMlpMaxBuffers,
                 sfull0 = hempty0 + 8 * kMlpMaxBuffers, sempty0 = sfull0 + 8 * kSlots, xready = sempty0 + 8 * kSlots,
                 drain = xready + 8;
  // scales of the codes, [block][NC]; in the second part each buffer's
  float* s_scale = reinterpret_cast<float*>(smem + a.off_scale);
  float* s_wsc = reinterpret_cast<float*>(misc + kOffWsc);
  float* s_red = reinterpret_cast<float*>(misc + kOffRed);
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(misc + kOffMask);
  uint32_t* s_expert = reinterpret_cast<uint32_t*>(misc + kOffExpert);
  int* s_start = reinterpret_cast<int*>(misc + kOffStart);
  int* s_slot = reinterpret_cast<int*>(misc + kOffSlot);
  float* s_weight = reinterpret_cast<float*>(misc + kOffWeight);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + kOffFlag);
  volatile int* never = abort_flag + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + kOffFlag + 8);
  int* s_scan = reinterpret_cast<int*>(misc + kOffFlag + 16);
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = __shfl_sync(kAll, tid >> 5, 0);
  const int ST = a.stages, slots = a.T * a.k;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full0 + 8 * i, kProducers);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(tfull0 + 8 * i, 1);
      mbar_init(tempty0 + 8 * i, 4);
    }
    for (int i = 0; i < kMlpMaxBuffers; ++i) {
      mbar_init(hfull0 + 8 * i, 32 * kCoders);
      mbar_init(hempty0 + 8 * i, kBufferReaders);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(sfull0 + 8 * i, 32);  // one cp.async arrival a lane
      mbar_init(sempty0 + 8 * i, 4);
    }
    mbar_init(xready, kMlpThreads / 32 - kProducers - kIssuers);
    mbar_init(drain, kIssuers);
    *abort_flag = 0;
    *never = 0;
    fence_barrier_init();
    fence_proxy_async_shared();
    tma_prefetch_desc(&map_gu);
    tma_prefetch_desc(&map_d);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), kTmemCols);
    tmem_relinquish();
  }
  for (int e = tid; e < a.E; e += kMlpThreads) s_mask[e] = 0;
  pdl_wait();
  // The first of the tokens' values are on their way while the plan is made (half h of warps 2, 4, 5, .. takes the groups h,
  // h + kHalves, ..; later they would wait behind the weights).
  const int Kb = (int)cdiv(a.K, kBlock), Ib = (int)cdiv(a.I, kBlock);
  const int l16 = lane & 15, half = 2 * (warp == 2 ? 0 : warp - 3) + (lane >> 4), groups = a.T * Kb;
  constexpr int kHalves = 2 * (kMlpThreads / 32 - kProducers - kIssuers), kBatch = 6;
  uint4 xv[kBatch];
  int x_t = half / Kb, x_kb = half - x_t * Kb;  // token and K-block of the half's next group
  auto load_tokens = [&](int g0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (g0 + i * kHalves >= groups) break;
      const int k = x_kb * kBlock + 8 * l16;
      xv[i] = make_uint4(0, 0, 0, 0);
      if (x_t < a.T && k < a.K) {
        const uint16_t* p = a.x + (int64_t)x_t * a.ldx + k;
        if (a.vec) {
          xv[i] = __ldg(reinterpret_cast<const uint4*>(p));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = (k + 2 * q < a.K ? (uint32_t)__ldg(p + 2 * q) : 0u) |
                   (k + 2 * q + 1 < a.K ? (uint32_t)__ldg(p + 2 * q + 1) : 0u) << 16;
          xv[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      for (x_kb += kHalves; x_kb >= Kb; x_kb -= Kb) ++x_t;
    }
  };
  if (warp == 2 || (warp >= 4 && warp < 14)) load_tokens(0);
  __syncthreads();
  // ------------------------------------------------------------ plan: the reached experts in order, their slots by token
  for (int s = tid; s < slots; s += kMlpThreads) {
    const int e = __ldg(a.idx + s);
    if (e >= 0 && e < a.E) atomicOr(s_mask + e, 1u << (s / a.k));
    s_weight[s] = __ldg(a.w + s);
  }
  __syncthreads();
  int reached;
  {
    // thread i takes the experts 4i .. 4i + 3; counts of experts (high half) and of slots (low half), scanned together
    uint32_t m[4];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = 4 * tid + i < a.E ? s_mask[4 * tid + i] : 0u;
      mine += (m[i] ? 1 << 16 : 0) + __popc(m[i]);
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    int before = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kMlpThreads / 32; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    reached = total >> 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (m[i]) {
        const int at = before >> 16;
        s_expert[at] = (uint32_t)(4 * tid + i) | m[i] << 16;
        s_start[at] = before & 0xFFFF;
        s_mask[4 * tid + i] = (uint32_t)(before & 0xFFFF) << 16 | m[i];
        before += (1 << 16) + __popc(m[i]);
      }
    __syncthreads();
    for (int s = tid; s < slots; s += kMlpThreads) {
      const int e = __ldg(a.idx + s);
      if (e < 0 || e >= a.E) continue;
      const uint32_t v = s_mask[e];
      const int t = s / a.k;
      s_slot[(v >> 16) + __popc(v & ((1u << t) - 1u))] = s | t << 16;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem_base = *tmem_holder;

  const int grid = (int)gridDim.x, cta = (int)blockIdx.x;
  const int items1 = (int)cdiv(Kb, kUnitBlocks);                            // stages of a unit
  const int per_expert = a.I / kPairs, units = reached * per_expert;
  const int u0 = (int)((int64_t)units * cta / grid), u1 = (int)((int64_t)units * (cta + 1) / grid);
  const int n0 = cta * a.rows;                                              // second part: rows of D, in groups of
  const int group = a.group, blocks2 = 128 / group;                         // `group` rows of `blocks2` K-blocks a stage
  const int items2 = (int)cdiv(Ib, blocks2);
  const int experts2 = n0 < a.N ? reached : 0;
  auto fail = [&](uint32_t code) {
    if (!*abort_flag) atomicOr(&g_mlp_error, code);
    *abort_flag = 1;
  };

  if (warp == 0 || warp >= 14) {
    // ------------------------------------------------------------ producers (one elected lane of a warp that stays together)
    {
      const int me = warp == 0 ? 0 : warp - 13;
      const bool lead = elect_one();
      Ring at{0, 0};
      int issued = 0;
      bool ok = true;
      // the next stage, free, of `blocks` boxes of `bytes`; this producer's: me, me + kProducers, ..
      auto stage = [&](int blocks, int bytes, auto&& box) {
        const int st = at.at;
        ok = __all_sync(kAll, mbar_wait_bounded(empty0 + 8 * st, at.parity ^ 1u, kWaitLimitNs, abort_flag));
        if (!ok) {
          if (lane == 0) fail(1u);
          return;
        }
        if (lead) {
          mbar_arrive_expect_tx(full0 + 8 * st, (uint32_t)((blocks + kProducers - 1 - me) / kProducers * bytes));
          for (int b = me; b < blocks; b += kProducers) box(ring + st * kStageBytes, full0 + 8 * st, b);
        }
        __syncwarp();
        at.step(1, ST);
        ++issued;
      };
      for (int u = u0; u < u1 && ok; ++u) {
        const int r = u / per_expert, i0 = (u - r * per_expert) * kPairs, e = (int)(s_expert[r] & 0xFFFFu);
        for (int kb0 = 0; kb0 < Kb && ok; kb0 += kUnitBlocks)
          stage(min(kUnitBlocks, Kb - kb0), kUnitRows * kBlock, [&](uint32_t to, uint32_t bar, int b) {
            tma_load_4d(to + b * kUnitRows * kBlock, &map_gu, bar, (kb0 + b) * kBlock, i0, 0, e);
          });
      }
      for (int r = 0; r < experts2 && ok; ++r) {
        const int e = (int)(s_expert[r] & 0xFFFFu);
        for (int kb0 = 0; kb0 < Ib && ok; kb0 += blocks2)
          stage(min(blocks2, Ib - kb0), a.rows * kBlock, [&](uint32_t to, uint32_t bar, int b) {
            tma_load_3d(to + b * group * kBlock, &map_d, bar, (kb0 + b) * kBlock, n0, e);
          });
      }
      if (!ok && lead) {  // copies already issued land before this CTA's shared memory goes away
        for (int i = issued > ST ? issued - ST : 0; i < issued; ++i)
          mbar_wait_bounded(full0 + 8 * (i % ST), (uint32_t)((i / ST) & 1), kWaitLimitNs, never);
      }
      __syncwarp();
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issuers
    // (The whole warp goes through the loop and one elected lane issues: a lane by itself takes 326 cycles a stage, this way 252.)
    {
      const int me = warp >> 1;
      const bool lead = elect_one();
      Ring at{me, 0}, buf{me, 0};  // (both rings have a place an issuer at least)
      int n = 0;                   // stages of all issuers
      bool ok = true;
      auto issue = [&](uint32_t codes, uint32_t idesc) {
        ok = mbar_spin_bounded(tempty0 + 8 * buf.at, buf.parity ^ 1u, kWaitLimitNs, abort_flag) &&
             mbar_spin_bounded(full0 + 8 * at.at, at.parity, kWaitLimitNs, abort_flag);
        ok = __all_sync(kAll, ok);
        if (!ok) {
          if (lane == 0) fail(2u);
          return;
        }
        tc_fence_after();
        const uint64_t da = desc_kmajor_sw128(ring + (uint32_t)(at.at * kStageBytes)), db = desc_kmajor_sw128(codes);
        const uint32_t d = tmem_base + (uint32_t)(buf.at * kBufCols);
        if (lead) {
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k) mma_e4m3(d, da + (uint64_t)(2 * k), db + (uint64_t)(2 * k), idesc, k > 0 ? 1u : 0u);
          mma_commit(empty0 + 8 * at.at);
          mma_commit(tfull0 + 8 * buf.at);
        }
        __syncwarp();
        at.step(kIssuers, ST);
        buf.step(kIssuers, kBufs);
      };
      ok = __all_sync(kAll, mbar_wait_bounded(xready, 0, kWaitLimitNs, abort_flag));
      if (!ok && lane == 0) fail(2u);
      constexpr uint32_t idesc1 = idesc_e4m3_f32(128, kUnitBlocks * NC);
      for (int u = u0; u < u1 && ok; ++u)
        for (int j = 0; j < items1 && ok; ++j, ++n)
          if (n % kIssuers == me) issue(area + (uint32_t)(j * kUnitBlocks * NT * kAtom), idesc1);
      const uint32_t idesc2 = idesc_e4m3_f32(128, max(blocks2 * NC, 16));
      Ring h{0, 0};
      for (int r = 0; r < experts2 && ok; ++r) {
        ok = __all_sync(kAll, mbar_wait_bounded(hfull0 + 8 * h.at, h.parity, 2 * kWaitLimitNs, abort_flag));
        if (!ok && lane == 0) fail(4u);
        fence_proxy_async_shared();  // (codes that cp.async brought: no thread waited for them but by the barrier)
        if (ok && lead) mbar_arrive(hempty0 + 8 * h.at);  // seen (promotion's arrivals wait for the products)
        for (int j = 0; j < items2 && ok; ++j, ++n)
          if (n % kIssuers == me) issue(area + (uint32_t)((h.at * Ib + j * blocks2) * NT * kAtom), idesc2);
        h.step(1, a.buffers);
      }
      // every MMA issued completes before tensor memory is released
      if (lead) {
        mma_commit(drain);
        if (!mbar_wait_bounded(drain, 0, kWaitLimitNs, never)) fail(32u);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ the tokens' codes, by all of these warps
    int t = half / Kb, kb = half - t * Kb;
    for (int g0 = 0; g0 < groups; g0 += kBatch * kHalves) {
      uint4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) v[i] = xv[i];
      if (g0 + kBatch * kHalves < groups) load_tokens(g0 + kBatch * kHalves);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (g0 + i * kHalves >= groups) break;
        uint32_t m = amax2(amax2(v[i].x, v[i].y), amax2(v[i].z, v[i].w));
        m = amax2(m, __byte_perm(m, 0, 0x1032));
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = amax2(m, __shfl_xor_sync(kAll, m, o));
        // (neg_codes2 gives the codes of the IEEE quotient for this scale too: checked exhaustively on the CPU)
        const float s = scale_near(__uint_as_float(m & 0x7FFF0000u)), ny = neg_rcp(s);
        const uint64_t s2 = f2_pack(s, s), ny2 = f2_pack(ny, ny);
        const uint32_t lo = (neg_codes2(v[i].x, s2, ny2) | neg_codes2(v[i].y, s2, ny2) << 16) ^ 0x80808080u;
        const uint32_t hi = (neg_codes2(v[i].z, s2, ny2) | neg_codes2(v[i].w, s2, ny2) << 16) ^ 0x80808080u;
        if (t < a.T) {
          const uint32_t at = area + (uint32_t)((kb * NT + (t >> 3)) * kAtom + (t & 7) * 128 +
                                                (((l16 >> 1) ^ (t & 7)) << 4) + 8 * (l16 & 1));
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(lo), "r"(hi) : "memory");
          if (l16 == 0) s_scale[kb * NC + t] = s;
        }
        for (kb += kHalves; kb >= Kb; kb -= Kb) ++t;
      }
    }
    fence_proxy_async_shared();  // the MMA reads the codes
    __syncwarp();
    if (lane == 0) mbar_arrive(xready);

    if (warp == 2) {
      // ------------------------------------------------------------ the weights' scales
      Ring slot{0, 0};
      const int Nb1 = 2 * a.I / kBlock, Nb2 = (int)cdiv(a.N, kBlock);
      bool ok = true;
      // `stages` stages of `per` scales, lane l of a slot the scale l % per of its stage l / per: at(stage, scale), null
      // where there is none
      auto run = [&](int stages, int per, auto&& address) {
        for (int before = 0; before < stages && ok; before += 32 / per) {
          const bool free = mbar_wait_bounded(sempty0 + 8 * slot.at, slot.parity ^ 1u, kWaitLimitNs, abort_flag);
          if (!(ok = __all_sync(kAll, free))) {
            if (lane == 0) fail(64u);
            break;
          }
          const int n = before + lane / per;
          const float* from = n < stages ? address(n, lane % per) : nullptr;
          if (from) cp_async_4(smem_u32(s_wsc + slot.at * 32 + lane), from, 4u);
          cp_async_mbar_arrive(sfull0 + 8 * slot.at);
          slot.step(1, kSlots);
        }
      };
      run((u1 - u0) * items1, 2 * kUnitBlocks, [&](int n, int i) -> const float* {
        const int u = u0 + n / items1, r = u / per_expert, kb = (n % items1) * kUnitBlocks + (i >> 1);
        const int row = (u - r * per_expert) * kPairs + (i & 1) * a.I;
        return kb < Kb ? a.sgu + ((int64_t)(s_expert[r] & 0xFFFFu) * Nb1 + row / kBlock) * a.ldsgu + kb : nullptr;
      });
      run(experts2 * items2, 2 * blocks2, [&](int n, int i) -> const float* {
        const int r = n / items2, kb = (n % items2) * blocks2 + (i >> 1), tile = n0 / kBlock + (i & 1);
        return kb < Ib && tile < Nb2 ? a.sd + ((int64_t)(s_expert[r] & 0xFFFFu) * Nb2 + tile) * a.ldsd + kb : nullptr;
      });
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4 && warp < 8) {
      // ------------------------------------------------------------ promotion
      const int w = warp - 4, ct = tid - 128;
      const uint32_t lane_base = (uint32_t)(32 * w) << 16;
      Ring at{0, 0}, slot{0, 0};
      int in_slot = 0;
      bool ok = mbar_wait_bounded(xready, 0, kWaitLimitNs, abort_flag);
      ok = __all_sync(kAll, ok);
      auto wait_product = [&]() {
        const bool in = mbar_wait_bounded(tfull0 + 8 * at.at, at.parity, kWaitLimitNs, abort_flag);
        if (__all_sync(kAll, in)) {
          tc_fence_after();
          return true;
        }
        if (lane == 0) fail(8u);
        return false;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8 * at.at);
        at.step(1, kBufs);
      };
      // this thread's scale in the stage, of `per` in the stage, slot by slot
      auto next_scale = [&](int per, int which, float& b) {
        if (in_slot == 0) {
          const bool there = mbar_wait_bounded(sfull0 + 8 * slot.at, slot.parity, kWaitLimitNs, abort_flag);
          if (!__all_sync(kAll, there)) {
            if (lane == 0) fail(64u);
            return false;
          }
        }
        b = s_wsc[slot.at * 32 + in_slot + which];
        in_slot += per;
        return true;
      };
      auto leave_slot = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty0 + 8 * slot.at);
        slot.step(1, kSlots);
        in_slot = 0;
      };
      float acc[NC];
      auto write_sums = [&](float* red) {  // this thread's row of the 128
#pragma unroll
        for (int t = 0; t < NC; t += 4)
          *reinterpret_cast<float4*>(red + ct * NC + ((t + 4 * (ct >> 1)) & (NC - 1))) =
              make_float4(acc[t], acc[t + 1], acc[t + 2], acc[t + 3]);
      };
      auto sum_at = [&](const float* red, int row, int t) {  // (rows' tokens are rotated: fewer bank conflicts)
        return red[row * NC + (((t & ~3) + 4 * (row >> 1)) & (NC - 1)) + (t & 3)];
      };
      // First part: lane's row is half (lane / 16: gate, up) of pair lane % 16, K-block w of the stage.
      int turn = 0;
      // (a warp whose wait gave up goes on through the units without their stages, so that the barriers between them match)
      for (int u = u0; u < u1; ++u) {
#pragma unroll
        for (int t = 0; t < NC; ++t) acc[t] = 0.0f;
        for (int j = 0; j < items1 && ok; ++j) {
          float b;
          if (!(ok = next_scale(2 * kUnitBlocks, 2 * w + (lane >> 4), b) && wait_product())) break;
          if (in_slot == 32) leave_slot();
          const int kb = j * kUnitBlocks + w;
          if (kb < Kb) {
            uint32_t p[NC];
            tmem_cols<NC>(tmem_base + lane_base + (uint32_t)(at.at * kBufCols + w * NC), p);
            promote<NC, false>(acc, p, s_scale + kb * NC, b, 0u);
          }
          release();
        }
        float* red = s_red + turn * (128 * NC);
        turn ^= 1;
        write_sums(red);
        named_sync(2, 128);
        const int r = u / per_expert, i0 = (u - r * per_expert) * kPairs;
        const uint32_t mask = s_expert[r] >> 16;
        for (int o = ct; o < kPairs * NC; o += 128) {
          const int t = o / kPairs, i = o % kPairs;
          if (mask >> t & 1u) {
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int b = 0; b < kUnitBlocks; ++b) {
              gate += sum_at(red, b * kUnitRows + i, t);
              up += sum_at(red, b * kUnitRows + kPairs + i, t);
            }
            const int slot = s_slot[s_start[r] + __popc(mask & ((1u << t) - 1u))] & 0xFFFF;
            a.act[(int64_t)slot * a.I + i0 + i] = gate / (1.0f + expf(-gate)) * up;
          }
        }
      }
      // The activations of this CTA are written: one arrival a CTA.  (Where a wait gave up there is none; the others'
      // waits for it then give up too.)
      named_sync(2, 128);
      if (ct == 0 && ok) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.arrived) : "memory");

      // Second part: row 32 w + lane is K-block (32 w + lane) / group of the stage, row (32 w + lane) % group of the CTA's.
      if (n0 < a.N) {
        const int block = ct / group, row = ct & (group - 1);
        const int tile = (n0 % kBlock + row) / kBlock & 1;  // of the two that the CTA's rows may touch
#pragma unroll
        for (int t = 0; t < NC; ++t) acc[t] = 0.0f;
        if (in_slot > 0) leave_slot();  // (the second part begins with a slot of its own)
        Ring h{0, 0};
        for (int r = 0; r < experts2 && ok; ++r, h.step(1, a.buffers)) {
          const int buf = h.at;
          const float* scales = s_scale + buf * Ib * NC;
          const uint32_t mask = s_expert[r] >> 16;
          const bool there = mbar_wait_bounded(hfull0 + 8 * buf, h.parity, 2 * kWaitLimitNs, abort_flag);
          if (!(ok = __all_sync(kAll, there))) {
            if (lane == 0) fail(4u);
            break;
          }
          for (int j = 0; j < items2; ++j) {
            float b;
            if (!(ok = next_scale(2 * blocks2, 2 * block + tile, b) && wait_product())) break;
            if (in_slot == 32) leave_slot();
            const int kb = j * blocks2 + block;
            const uint32_t from = tmem_base + lane_base + (uint32_t)(at.at * kBufCols);
            uint32_t p[NC];
            if (group == 16) {  // two K-blocks in a warp
              uint32_t q[2 * NC];
              tmem_cols<2 * NC>(from + (uint32_t)(2 * w * NC), q);
#pragma unroll
              for (int t = 0; t < NC; ++t) p[t] = lane < 16 ? q[t] : q[NC + t];
            } else {
              tmem_cols<NC>(from + (uint32_t)(32 * w / group * NC), p);
            }
            if (kb < Ib) promote<NC, true>(acc, p, scales + kb * NC, b, mask);
            release();
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(hempty0 + 8 * buf);
        }
        // sums of the K-blocks; y (also where no expert was reached: zeros)
        float* red = s_red + turn * (128 * NC);
        write_sums(red);
        named_sync(2, 128);
        const int rows = min(a.rows, a.N - n0);
        if (ok)
          for (int o = ct; o < rows * a.T; o += 128) {
            const int t = o / rows, i = o - t * rows;
            float sum = 0.0f;
            for (int b = 0; b < blocks2; ++b) sum += sum_at(red, b * group + i, t);
            a.y[(int64_t)t * a.ldy + n0 + i] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
          }
      }
    } else if (reached > 0) {
      // ------------------------------------------------------------ the activations' codes
      // Teams of the six warps take an expert each, in turn: six teams or three, but no more of them than buffers (a team
      // that is a whole turn of the buffers ahead of another could not tell the phases of their barriers apart), and all
      // six warps an expert where there are two buffers or one (16 tokens of 64 experts: 213.3 us with two teams, 211.5).
      const int coder = warp - 8;
      const int teams = a.buffers <= 2 ? 1 : a.buffers < kCoders ? 3 : kCoders, size = kCoders / teams;
      bool ok = true;
      // until every CTA has arrived (one warp asks: more of them hold the arrivals up)
      auto wait_arrived = [&](const uint32_t* count) {
        const uint64_t t0 = globaltimer_ns();
        bool in = true;
        while (in && ld_acquire_gpu(count) < (uint32_t)grid) in = !*abort_flag && globaltimer_ns() - t0 < kWaitLimitNs;
        return __all_sync(kAll, in) != 0;
      };
      if (coder == 0 && !wait_arrived(a.arrived) && lane == 0) fail(16u);
      named_sync(3, 32 * kCoders);
      ok = !*abort_flag;
      // this CTA's share of the groups: every (grid x 2 kCoders)-th, half a warp each
      for (int g0 = 0; g0 < slots * Ib; g0 += grid * 2 * kCoders) {
        const int g = g0 + (2 * coder + (lane >> 4)) * grid + cta, slot = g / Ib, blk = g - slot * Ib, k = blk * kBlock + 8 * l16;
        float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f), q = p;
        const bool in = ok && g < slots * Ib;
        if (in && k < a.I) {  // (a slot without an expert: whatever was there, and not read)
          const float4* from = reinterpret_cast<const float4*>(a.act + (int64_t)slot * a.I + k);
          p = __ldcg(from);
          q = __ldcg(from + 1);
        }
        uint32_t lo, hi;
        const float s = code8(p, q, lo, hi);
        if (in) {
          *reinterpret_cast<uint2*>(a.codes + (int64_t)g * kBlock + 8 * l16) = make_uint2(lo, hi);
          if (l16 == 0) a.scales[g] = s * s_weight[slot];  // (the promotion wants the product)
        }
      }
      named_sync(3, 32 * kCoders);
      if (coder == 0) {
        if (lane == 0 && ok) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.arrived + 1) : "memory");
        if (!wait_arrived(a.arrived + 1) && lane == 0) fail(16u);
      }
      named_sync(3, 32 * kCoders);
      ok = !*abort_flag;
      Ring at{0, 0};  // expert r's buffer
      int r = coder / size;
      for (int i = 0; i < r; ++i) at.step(1, a.buffers);
      for (; r < experts2 && ok; r += teams) {
        const uint32_t mask = s_expert[r] >> 16, codes = area + (uint32_t)(at.at * Ib * NT * kAtom);
        float* scales = s_scale + at.at * Ib * NC;
        auto buffer_free = [&]() {
          const bool in = mbar_wait_bounded(hempty0 + 8 * at.at, at.parity ^ 1u, kWaitLimitNs, abort_flag);
          if (__all_sync(kAll, in)) return true;
          if (lane == 0) fail(16u);
          return false;
        };
        const int first = s_start[r], of_expert = __popc(mask) * Ib;
        // Codes as they are: 16 bytes a lane, eight lanes a group, and its scale.  They pass no registers and nobody waits
        // for them here, so a team's next expert is under way while they land.
        if (!(ok = buffer_free())) break;
        const int sub = lane & 7;
        int c = 0, blk = 4 * (coder % size) + (lane >> 3);  // of the next group: token of the expert, K-block
        for (;; blk += 4 * size) {
          while (blk >= Ib) blk -= Ib, ++c;
          if (c * Ib + blk >= of_expert) break;
          const int slot = s_slot[first + c], t = slot >> 16, g = (slot & 0xFFFF) * Ib + blk;
          cp_async_16(codes + (uint32_t)((blk * NT + (t >> 3)) * kAtom + (t & 7) * 128 + ((sub ^ (t & 7)) << 4)),
                      a.codes + (int64_t)g * kBlock + 16 * sub, 16u);
          if (sub == 0) cp_async_4(smem_u32(scales + blk * NC + t), a.scales + g, 4u);
        }
        __syncwarp();
        for (int i = 0; i < kCoders / size; ++i) cp_async_mbar_arrive(hfull0 + 8 * at.at);
        for (int i = 0; i < teams; ++i) at.step(1, a.buffers);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

static PFN_cuTensorMapEncodeTiled_v12000 mlp_encode_fn() {
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

// Bytes in `rank` dimensions, the first one contiguous, in boxes that land 128-byte swizzled; zeros outside.
static bool mlp_map(CUtensorMap* m, const void* base, int rank, const int64_t* dim, const int64_t* stride, const int* box) {
  cuuint64_t dims[5], strides[4];
  cuuint32_t boxes[5], elem[5];
  for (int i = 0; i < rank; ++i) {
    dims[i] = (cuuint64_t)dim[i];
    boxes[i] = (cuuint32_t)box[i];
    elem[i] = 1;
    if (i) strides[i - 1] = (cuuint64_t)stride[i];
  }
  return mlp_encode_fn() != nullptr &&
         mlp_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, boxes,
                         elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

MlpGeom mlp_geom(int64_t T, int64_t K, int64_t I, int64_t N, int num_sms) {
  MlpGeom g = {};
  const int64_t nt = T <= 8 ? 1 : 2, Kb = cdiv(K, kBlock), Ib = cdiv(I, kBlock);
  const int64_t most = kMlpCodeBytes, x = Kb * nt * kAtom, h = Ib * nt * kAtom;
  const int64_t rows = cdiv(N, num_sms);
  if (x > most || h > most || rows > 128) return g;  // stages 0: out of range
  g.rows = (int)rows;
  // Buffers of activations: two, or what the tokens' space (or 48 KB) holds; one where two pass the limit.  The ring gets
  // what they leave.
  int64_t room = x > 2 * h ? x : 2 * h;
  room = room < (48 << 10) ? (48 << 10) : room < most ? room : most;
  g.buffers = (int)(room / h < kMlpMaxBuffers ? room / h : kMlpMaxBuffers);
  const int64_t codes = x > g.buffers * h ? x : g.buffers * h;
  const int64_t scales = (Kb > g.buffers * Ib ? Kb : g.buffers * Ib) * 8 * nt * 4;
  g.group = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  const int64_t stages = ((int64_t)227 * 1024 - 1024 - codes - scales - kMiscBytes) / kStageBytes;
  // An even number of stages: the two issuers take alternate ones, and a place's next use must be the same issuer's, who
  // has seen the one before (the other could take a phase that is two behind for the one it waits for).
  g.stages = (int)(stages < kMlpMaxStages ? stages : kMlpMaxStages) & ~1;
  g.off_scale = (int)(g.stages * kStageBytes + codes);
  g.off_misc = (int)(g.off_scale + scales);
  g.smem = g.off_misc + kMiscBytes + 1024;
  return g;
}

template <int NT>
static cudaError_t run_mlp(const CUtensorMap& gu, const CUtensorMap& d, const MlpArgs& a, int smem, int num_sms,
                           cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(moe_mlp_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  });
  if (attr_err != cudaSuccess) return attr_err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_sms);
  cfg.blockDim = dim3(kMlpThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs wait for one another: all or none are resident
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_mlp_kernel<NT>, gu, d, a);
}

cudaError_t launch_moe_mlp(const MlpArgs& args, const uint8_t* qgu, int64_t ldgu, const uint8_t* qd, int64_t ldd,
                           int num_sms, cudaStream_t st, const char** msg) {
  MlpArgs a = args;
  const MlpGeom g = mlp_geom(a.T, a.K, a.I, a.N, num_sms);
  a.rows = g.rows, a.group = g.group, a.buffers = g.buffers, a.stages = g.stages;
  a.off_scale = g.off_scale, a.off_misc = g.off_misc;
  a.vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % 8 == 0 && a.K % 8 == 0;
  CUtensorMap gu, d;
  memset(&gu, 0, sizeof(gu));
  memset(&d, 0, sizeof(d));
  const int64_t E = a.E, I = a.I, N = a.N, K = a.K;
  // features, rows, gate / up, expert; features, rows, expert
  const int64_t dim1[4] = {K, I, 2, E}, stride1[4] = {1, ldgu, I * ldgu, 2 * I * ldgu};
  const int box1[4] = {kBlock, kPairs, 2, 1};
  const int64_t dim2[3] = {I, N, E}, stride2[3] = {1, ldd, N * ldd};
  const int box2[3] = {kBlock, g.rows, 1};
  if (!mlp_map(&gu, qgu, 4, dim1, stride1, box1) || !mlp_map(&d, qd, 3, dim2, stride2, box2)) {
    *msg = "cuTensorMapEncodeTiled failed for a weight (alignment, stride or size out of range)";
    return cudaErrorInvalidValue;
  }
  return a.T <= 8 ? run_mlp<1>(gu, d, a, g.smem, num_sms, st) : run_mlp<2>(gu, d, a, g.smem, num_sms, st);
}

cudaError_t mlp_read_errors(uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_mlp_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_mlp_error, &zero, sizeof(uint32_t));
}

}  // namespace bfp8
