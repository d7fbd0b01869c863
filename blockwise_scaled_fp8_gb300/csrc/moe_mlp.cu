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
//   - one CTA an SM, whose producer brings 16 KB stages by TMA through a ring
//     that holds most of shared memory, first its share of the gate and up rows,
//     then of the down rows;
//   - the exchange of the activations between the two (every CTA needs all of
//     them) is a barrier over the grid that only the warps behind the ring wait
//     for: the down weights do not depend on it and fill the ring meanwhile.
//
//   warp 0       producer
//   warps 1-8    products: a stage's K-blocks are split over them, their sums meet
//                in shared memory at the end of a unit
//   warps 9-12   the activations' codes, an expert ahead of the products
//
// First part: a unit is 8 gate rows and the 8 up rows of the same features; the
// units of all reached experts are shared evenly.  Second part: CTA c takes the
// rows [c R, c R + R) of D of every reached expert, so y's sums over experts
// never leave its registers.  Both give every CTA the same bytes to within a few
// percent, where tiles of 128 rows (the operand of tcgen05.mma, in the routed
// product) would give some of them two and some one: 256 tiles of one token's
// eight experts of 2 x 2048 rows over 152 SMs.  16 rows and up to 16 tokens are the
// shape of an 8-bit mma.sync, whose rate does not matter here: a CTA needs one
// in about 40 cycles to keep up with its share of the memory.
//
// Waits are bounded; a role that gives up sets the abort flag, the others leave
// their loops, and copies in flight land before the CTA exits.
#include <cudaTypedefs.h>
#include <string.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

static __device__ uint32_t g_mlp_error;

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kMmaWarps = 8, kQuantWarps = 4;
constexpr int kMlpThreads = 32 * (1 + kMmaWarps + kQuantWarps);
constexpr int kStageBytes = 16384;
constexpr int kUnit = 8;            // gate (and up) rows of a unit
constexpr int kUnitBlocks = 8;      // K-blocks of a stage of the first part: 2 x 8 rows x 128 B each
constexpr int kMlpMaxStages = 12;
constexpr int kAtom = 1024;         // 8 rows x 128 B, 128-byte swizzled
static_assert(kUnitBlocks == kMmaWarps && 2 * kUnit * kBlock * kUnitBlocks == kStageBytes, "a K-block a warp");

// Shared memory after the ring and the codes (offsets from MlpArgs::off_misc).
constexpr int kOffRed = 0;                                           // two sets of [8 warps][16 rows][8 NT tokens] sums
constexpr int kRedBytes = 2 * kMmaWarps * 16 * kMlpMaxTokens * 4;
constexpr int kOffMask = kOffRed + kRedBytes;                        // [E] tokens of an expert; [E] its rank from the plan's end on
constexpr int kOffExpert = kOffMask + kMaxGroups * 4;                // [reached] expert | mask << 16
constexpr int kOffStart = kOffExpert + kMlpMaxSlots * 4;             // [reached] first of its slots
constexpr int kOffSlot = kOffStart + kMlpMaxSlots * 4;               // slots by expert, in token order
constexpr int kOffWeight = kOffSlot + kMlpMaxSlots * 4;              // [slots] routing weights, by slot
constexpr int kOffBars = kOffWeight + kMlpMaxSlots * 4;              // full[12] empty[12] hfull[2] hempty[2]
constexpr int kOffFlag = kOffBars + 8 * (2 * kMlpMaxStages + 4);     // abort flag, a zero, scan[16]
constexpr int kMiscBytes = kOffFlag + 8 + 4 * 16;

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
          dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}
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
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// d[16 x 8] += a[16 x 32] b[32 x 8], e4m3 into fp32: thread 4g + t holds rows g, g + 8 and columns 2t, 2t + 1 of d.
__device__ __forceinline__ void mma_16x8x32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// max(amax, 1e-12) / 448 as one product with 1/448: within an ulp of group_scale's quotient.
__device__ __forceinline__ float scale_near(float amax) { return __fmul_rn(fmaxf(amax, kAmaxFloor), 1.0f / kE4m3Max); }
// The codes of two bf16 values over s (IEEE quotients).
__device__ __forceinline__ uint32_t codes2(uint32_t w, float s) {
  return cvt_e4m3x2(__fdiv_rn(bf16_lo(w), s), __fdiv_rn(bf16_hi(w), s));
}
// The 16 x 8 NT partial product of one K-block: A's 16 rows, whose first eight lie at lines a0 .. and the others at
// a1 .. of 128 bytes (swizzled by their address), against the codes of 8 NT tokens at b.
template <int NT>
__device__ __forceinline__ void block_product(float (&p)[NT][4], uint32_t stage, int a0, int a1, uint32_t b, int lane) {
  const int line = (lane & 8 ? a1 : a0) + (lane & 7);
  const uint32_t row = stage + (uint32_t)line * 128u;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) p[n][i] = 0.0f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t bv[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      ldmatrix_x4(b + (uint32_t)(n * kAtom + (lane & 7) * 128 + (((4 * half + (lane >> 3)) ^ (lane & 7)) << 4)), bv[n]);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t av[4];
      ldmatrix_x4(row + (uint32_t)(((4 * half + 2 * s + (lane >> 4)) ^ (line & 7)) << 4), av);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_16x8x32(p[n], av, bv[n][2 * s], bv[n][2 * s + 1]);
    }
  }
}

}  // namespace

template <int NT>
__global__ void __launch_bounds__(kMlpThreads, 1)
    moe_mlp_kernel(const __grid_constant__ CUtensorMap map_gu, const __grid_constant__ CUtensorMap map_gu_tail,
                   const __grid_constant__ CUtensorMap map_d, const __grid_constant__ CUtensorMap map_d_tail,
                   const MlpArgs a) {
  constexpr int NC = 8 * NT;  // token columns
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t ring = smem_u32(smem);
  const uint32_t area = ring + (uint32_t)a.stages * kStageBytes;
  uint8_t* misc = smem + a.off_misc;
  const uint32_t full0 = smem_u32(misc + kOffBars), empty0 = full0 + 8 * kMlpMaxStages, hfull0 = empty0 + 8 * kMlpMaxStages,
                 hempty0 = hfull0 + 16;
  float* s_scale = reinterpret_cast<float*>(smem + a.off_scale);  // of the codes: [block][NC], each buffer of the second part
  float* s_red = reinterpret_cast<float*>(misc + kOffRed);
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(misc + kOffMask);
  uint32_t* s_expert = reinterpret_cast<uint32_t*>(misc + kOffExpert);
  int* s_start = reinterpret_cast<int*>(misc + kOffStart);
  int* s_slot = reinterpret_cast<int*>(misc + kOffSlot);
  float* s_weight = reinterpret_cast<float*>(misc + kOffWeight);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + kOffFlag);
  volatile int* never = abort_flag + 1;
  int* s_scan = reinterpret_cast<int*>(misc + kOffFlag + 8);
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = __shfl_sync(kAll, tid >> 5, 0);
  const int ST = a.stages, slots = a.T * a.k;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, kMmaWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(hfull0 + 8 * i, kQuantWarps);
      mbar_init(hempty0 + 8 * i, kMmaWarps);
    }
    *abort_flag = 0;
    *never = 0;
    fence_barrier_init();
    fence_proxy_async_shared();
    tma_prefetch_desc(&map_gu);
    tma_prefetch_desc(&map_d);
    if (a.K % kBlock) tma_prefetch_desc(&map_gu_tail);
    if (a.I % kBlock) tma_prefetch_desc(&map_d_tail);
  }
  for (int e = tid; e < a.E; e += kMlpThreads) s_mask[e] = 0;
  pdl_wait();
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
        s_mask[4 * tid + i] = (uint32_t)(before & 0xFFFF) << 16 | m[i];  // (the slots' pass needs both)
        before += (1 << 16) + __popc(m[i]);
      }
    __syncthreads();
    for (int s = tid; s < slots; s += kMlpThreads) {
      const int e = __ldg(a.idx + s);
      if (e < 0 || e >= a.E) continue;
      const uint32_t v = s_mask[e];
      s_slot[(v >> 16) + __popc(v & ((1u << (s / a.k)) - 1u))] = s;
    }
    __syncthreads();
  }

  const int grid = (int)gridDim.x, cta = (int)blockIdx.x;
  const int Kf = a.K / kBlock, If = a.I / kBlock;                           // whole K-blocks
  const int Kb = (int)cdiv(a.K, kBlock), Ib = (int)cdiv(a.I, kBlock);
  const int items1 = (int)cdiv(Kf, kUnitBlocks) + (Kb > Kf ? 1 : 0);        // stages of a unit
  const int per_expert = a.I / kUnit, units = reached * per_expert;
  const int u0 = (int)((int64_t)units * cta / grid), u1 = (int)((int64_t)units * (cta + 1) / grid);
  const int n0 = cta * a.rows;                                              // second part: rows of D
  const int blocks2 = a.blocks;                                             // K-blocks of a stage of the second part
  const int items2 = (int)cdiv(If, blocks2) + (Ib > If ? 1 : 0);
  const bool second = n0 < a.N;
  auto fail = [&](uint32_t code) {
    if (!*abort_flag) atomicOr(&g_mlp_error, code);
    *abort_flag = 1;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int n = 0;
      bool ok = true;
      auto stage = [&](uint32_t bytes) {  // the next stage, free; its barrier expects `bytes`
        const int st = n % ST;
        ok = mbar_wait_bounded(empty0 + 8 * st, (uint32_t)((n / ST) & 1) ^ 1u, kWaitLimitNs, abort_flag);
        if (!ok) {
          fail(1u);
          return -1;
        }
        mbar_arrive_expect_tx(full0 + 8 * st, bytes);
        ++n;
        return st;
      };
      for (int u = u0; u < u1 && ok; ++u) {
        const int r = u / per_expert, i0 = (u - r * per_expert) * kUnit, e = (int)(s_expert[r] & 0xFFFFu);
        for (int j = 0; j < items1 && ok; ++j) {
          const bool tail = j * kUnitBlocks >= Kf;
          const int st = stage(tail ? 2 * kAtom : kStageBytes);
          if (st < 0) break;
          if (!tail) tma_load_5d(ring + st * kStageBytes, &map_gu, full0 + 8 * st, 0, i0, j * kUnitBlocks, 0, e);
          else tma_load_4d(ring + st * kStageBytes, &map_gu_tail, full0 + 8 * st, Kf * kBlock, i0, 0, e);
        }
      }
      for (int r = 0; second && r < reached && ok; ++r) {
        const int e = (int)(s_expert[r] & 0xFFFFu);
        for (int j = 0; j < items2 && ok; ++j) {
          const bool tail = j * blocks2 >= If;
          const int st = stage((uint32_t)((tail ? 1 : blocks2) * a.rows * kBlock));
          if (st < 0) break;
          if (!tail) tma_load_4d(ring + st * kStageBytes, &map_d, full0 + 8 * st, 0, n0, j * blocks2, e);
          else tma_load_3d(ring + st * kStageBytes, &map_d_tail, full0 + 8 * st, If * kBlock, n0, e);
        }
      }
      if (!ok)  // copies already issued land before this CTA's shared memory goes away
        for (int i = n > ST ? n - ST : 0; i < n; ++i)
          mbar_wait_bounded(full0 + 8 * (i % ST), (uint32_t)((i / ST) & 1), kWaitLimitNs, never);
    }
    return;
  }

  // ------------------------------------------------------------ the tokens' codes, by all other warps
  {
    const int half = (tid - 32) >> 4, halves = (kMlpThreads - 32) >> 4, l16 = lane & 15;
    const int groups = a.T * Kb;
    for (int g0 = 0; g0 < groups; g0 += 2 * halves) {
      uint4 v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int g = g0 + half + i * halves, t = g / Kb, k = (g - t * Kb) * kBlock + 8 * l16;
        v[i] = make_uint4(0, 0, 0, 0);
        if (g < groups && k < a.K) {
          const uint16_t* p = a.x + (int64_t)t * a.ldx + k;
          if (a.vec) {
            v[i] = __ldg(reinterpret_cast<const uint4*>(p));
          } else {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = (k + 2 * q < a.K ? (uint32_t)__ldg(p + 2 * q) : 0u) |
                     (k + 2 * q + 1 < a.K ? (uint32_t)__ldg(p + 2 * q + 1) : 0u) << 16;
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int g = g0 + half + i * halves, t = g / Kb, kb = g - t * Kb;
        uint32_t m = amax2(amax2(v[i].x, v[i].y), amax2(v[i].z, v[i].w));
        m = amax2(m, __byte_perm(m, 0, 0x1032));
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = amax2(m, __shfl_xor_sync(kAll, m, o));
        const float s = scale_near(__uint_as_float(m & 0x7FFF0000u));
        const uint32_t lo = codes2(v[i].x, s) | codes2(v[i].y, s) << 16, hi = codes2(v[i].z, s) | codes2(v[i].w, s) << 16;
        if (g < groups) {
          const uint32_t at = area + (uint32_t)((kb * NT + (t >> 3)) * kAtom + (t & 7) * 128 +
                                                (((l16 >> 1) ^ (t & 7)) << 4) + 8 * (l16 & 1));
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(lo), "r"(hi) : "memory");
          if (l16 == 0) s_scale[kb * NC + t] = s;
        }
      }
    }
  }
  named_sync(1, kMlpThreads - 32);

  if (warp <= kMmaWarps) {
    // ------------------------------------------------------------ products
    const int cw = warp - 1, ct = tid - 32, g = lane >> 2, t2 = 2 * (lane & 3);
    int n = 0, turn = 0;
    bool ok = true;
    auto wait_full = [&]() {
      const int st = n % ST;
      const bool in = mbar_wait_bounded(full0 + 8 * st, (uint32_t)((n / ST) & 1), kWaitLimitNs, abort_flag);
      if (__all_sync(kAll, in)) return true;
      if (lane == 0) fail(2u);
      return false;
    };
    auto release = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * (n % ST));
      ++n;
    };
    float acc[NT][4];
    // the scales of 32 stages of a unit, stage l's in lane l, fetched a unit ahead
    const int Nb1 = (int)cdiv(2 * a.I, kBlock);
    auto unit_scales = [&](int u, int j0, float& sg, float& su) {
      sg = su = 0.0f;
      if (u >= u1) return;
      const int r = u / per_expert, i0 = (u - r * per_expert) * kUnit, e = (int)(s_expert[r] & 0xFFFFu);
      const int j = j0 + lane, kb = j * kUnitBlocks >= Kf ? Kf : j * kUnitBlocks + cw;
      if (j < items1 && kb < Kb) {
        sg = __ldg(a.sgu + ((int64_t)e * Nb1 + i0 / kBlock) * a.ldsgu + kb);
        su = __ldg(a.sgu + ((int64_t)e * Nb1 + (a.I + i0) / kBlock) * a.ldsgu + kb);
      }
    };
    float sg, su, sg_next, su_next;
    unit_scales(u0, 0, sg_next, su_next);
    // (a warp whose wait gave up goes on through the units without their stages, so that the barriers between them match)
    for (int u = u0; u < u1; ++u) {
      sg = sg_next, su = su_next;
      unit_scales(u + 1, 0, sg_next, su_next);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][q] = 0.0f;
      for (int j = 0; j < items1 && ok; ++j) {
        if (j > 0 && (j & 31) == 0) unit_scales(u, j, sg, su);
        if (!(ok = wait_full())) break;
        const bool tail = j * kUnitBlocks >= Kf;
        const int kb = tail ? Kf : j * kUnitBlocks + cw;
        const float bg = __shfl_sync(kAll, sg, j & 31), bu = __shfl_sync(kAll, su, j & 31);
        if (tail ? cw == 0 : kb < Kf) {
          float p[NT][4];
          const int at = tail ? 0 : cw, up = tail ? 1 : kUnitBlocks;
          block_product<NT>(p, ring + (n % ST) * kStageBytes, 8 * at, 8 * (up + at), area + (uint32_t)(kb * NT * kAtom), lane);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const float2 xs = *reinterpret_cast<const float2*>(s_scale + kb * NC + 8 * i + t2);
            acc[i][0] = fmaf(xs.x * bg, p[i][0], acc[i][0]);
            acc[i][1] = fmaf(xs.y * bg, p[i][1], acc[i][1]);
            acc[i][2] = fmaf(xs.x * bu, p[i][2], acc[i][2]);
            acc[i][3] = fmaf(xs.y * bu, p[i][3], acc[i][3]);
          }
        }
        release();
      }
      float* red = s_red + turn * (kMmaWarps * 16 * NC);
      turn ^= 1;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        *reinterpret_cast<float2*>(red + (cw * 16 + g) * NC + 8 * i + t2) = make_float2(acc[i][0], acc[i][1]);
        *reinterpret_cast<float2*>(red + (cw * 16 + g + 8) * NC + 8 * i + t2) = make_float2(acc[i][2], acc[i][3]);
      }
      named_sync(2, 32 * kMmaWarps);
      if (ct < kUnit * NC) {
        const int t = ct / kUnit, i = ct % kUnit;
        const int r = u / per_expert, i0 = (u - r * per_expert) * kUnit;
        const uint32_t mask = s_expert[r] >> 16;
        if (mask >> t & 1u) {
          float gate = 0.0f, up = 0.0f;
#pragma unroll
          for (int w = 0; w < kMmaWarps; ++w) {
            gate += red[(w * 16 + i) * NC + t];
            up += red[(w * 16 + 8 + i) * NC + t];
          }
          const int slot = s_slot[s_start[r] + __popc(mask & ((1u << t) - 1u))];
          a.act[(int64_t)slot * a.I + i0 + i] = gate / (1.0f + expf(-gate)) * up;
        }
      }
    }
    // the activations of this CTA are written: one arrival a CTA (not where a wait gave up: the others' give up too)
    named_sync(2, 32 * kMmaWarps);
    if (ct == 0 && ok) {
      __threadfence();
      atomicAdd(a.arrived, 1u);
    }

    if (second) {
      const int mt = cw % a.mtiles, split = cw / a.mtiles;  // 16 rows, K-block of a stage
      const int Nb2 = (int)cdiv(a.N, kBlock);
      const int row0 = min(n0 + 16 * mt, a.N - 1) / kBlock, row1 = min(n0 + 16 * mt + 15, a.N - 1) / kBlock;
      const bool hi0 = min(n0 + 16 * mt + g, a.N - 1) / kBlock != row0, hi1 = min(n0 + 16 * mt + g + 8, a.N - 1) / kBlock != row0;
      auto expert_scales = [&](int r, int j0, float& s0, float& s1) {
        s0 = s1 = 0.0f;
        if (r >= reached) return;
        const int e = (int)(s_expert[r] & 0xFFFFu), j = j0 + lane;
        const int kb = j * blocks2 >= If ? If : j * blocks2 + split;
        if (j < items2 && kb < Ib) {
          s0 = __ldg(a.sd + ((int64_t)e * Nb2 + row0) * a.ldsd + kb);
          s1 = __ldg(a.sd + ((int64_t)e * Nb2 + row1) * a.ldsd + kb);
        }
      };
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][q] = 0.0f;
      float s0, s1, s0_next, s1_next;
      expert_scales(0, 0, s0_next, s1_next);
      for (int r = 0; r < reached && ok; ++r) {
        s0 = s0_next, s1 = s1_next;
        expert_scales(r + 1, 0, s0_next, s1_next);
        const int buf = r % a.buffers;
        const uint32_t codes = area + (uint32_t)(buf * Ib * NT * kAtom);
        const float* scales = s_scale + buf * Ib * NC;
        const uint32_t mask = s_expert[r] >> 16;
        const bool there = mbar_wait_bounded(hfull0 + 8 * buf, (uint32_t)((r / a.buffers) & 1), 2 * kWaitLimitNs, abort_flag);
        if (!(ok = __all_sync(kAll, there))) {
          if (lane == 0) fail(4u);
          break;
        }
        for (int j = 0; j < items2; ++j) {
          if (j > 0 && (j & 31) == 0) expert_scales(r, j, s0, s1);
          if (!(ok = wait_full())) break;
          const bool tail = j * blocks2 >= If;
          const int kb = tail ? If : j * blocks2 + split;
          const float b0 = __shfl_sync(kAll, s0, j & 31), b1 = __shfl_sync(kAll, s1, j & 31);
          if (tail ? split == 0 : kb < If) {
            float p[NT][4];
            const int line = (tail ? 0 : split) * a.rows + 16 * mt;
            block_product<NT>(p, ring + (n % ST) * kStageBytes, line, line + 8, codes + (uint32_t)(kb * NT * kAtom), lane);
            const float bl = hi0 ? b1 : b0, bh = hi1 ? b1 : b0;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              // (columns of tokens that are not this expert's hold whatever was in the buffer)
              const float2 hs = *reinterpret_cast<const float2*>(scales + kb * NC + 8 * i + t2);
              if (mask >> (8 * i + t2) & 1u) {
                acc[i][0] = fmaf(hs.x * bl, p[i][0], acc[i][0]);
                acc[i][2] = fmaf(hs.x * bh, p[i][2], acc[i][2]);
              }
              if (mask >> (8 * i + t2 + 1) & 1u) {
                acc[i][1] = fmaf(hs.y * bl, p[i][1], acc[i][1]);
                acc[i][3] = fmaf(hs.y * bh, p[i][3], acc[i][3]);
              }
            }
          }
          release();
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(hempty0 + 8 * buf);
      }
      // sums of the splits; y (also where no expert was reached: zeros)
      float* red = s_red + turn * (kMmaWarps * 16 * NC);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        *reinterpret_cast<float2*>(red + (cw * 16 + g) * NC + 8 * i + t2) = make_float2(acc[i][0], acc[i][1]);
        *reinterpret_cast<float2*>(red + (cw * 16 + g + 8) * NC + 8 * i + t2) = make_float2(acc[i][2], acc[i][3]);
      }
      named_sync(2, 32 * kMmaWarps);
      const int rows = min(a.rows, a.N - n0);
      if (ok)
        for (int i = ct; i < rows * a.T; i += 32 * kMmaWarps) {
          const int t = i / rows, row = i - t * rows;
          float sum = 0.0f;
          for (int s = 0; s < kMmaWarps / a.mtiles; ++s)
            sum += red[((s * a.mtiles + row / 16) * 16 + row % 16) * NC + t];
          a.y[(int64_t)t * a.ldy + n0 + row] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
        }
    }
  } else if (second && reached > 0) {
    // ------------------------------------------------------------ the activations' codes
    const int half = (tid - 32 * (1 + kMmaWarps)) >> 4, l16 = lane & 15;
    constexpr int kHalves = 2 * kQuantWarps;
    bool ok = true;
    {
      const uint64_t t0 = globaltimer_ns();
      while (ld_acquire_gpu(a.arrived) < (uint32_t)grid)
        if (*abort_flag || globaltimer_ns() - t0 > kWaitLimitNs) {
          ok = ld_acquire_gpu(a.arrived) >= (uint32_t)grid;
          break;
        }
      ok = __all_sync(kAll, ok);
      if (!ok && lane == 0) fail(8u);
    }
    for (int r = 0; r < reached && ok; ++r) {
      const int buf = r % a.buffers;
      const bool free = mbar_wait_bounded(hempty0 + 8 * buf, (uint32_t)((r / a.buffers) & 1) ^ 1u, kWaitLimitNs, abort_flag);
      if (!(ok = __all_sync(kAll, free))) {
        if (lane == 0) fail(16u);
        break;
      }
      const uint32_t mask = s_expert[r] >> 16, codes = area + (uint32_t)(buf * Ib * NT * kAtom);
      float* scales = s_scale + buf * Ib * NC;
      const int count = __popc(mask), groups = count * Ib;
      for (int g0 = 0; g0 < groups; g0 += 2 * kHalves) {
        float4 v[2][2];
        int tok[2], blk[2], slot[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int g = g0 + half + i * kHalves, c = g / Ib;
          blk[i] = g - c * Ib;
          v[i][0] = v[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          slot[i] = tok[i] = 0;
          if (g < groups) {
            slot[i] = s_slot[s_start[r] + c];
            tok[i] = slot[i] / a.k;
            const int k = blk[i] * kBlock + 8 * l16;
            if (k < a.I) {
              const float4* p = reinterpret_cast<const float4*>(a.act + (int64_t)slot[i] * a.I + k);
              v[i][0] = __ldcg(p);
              v[i][1] = __ldcg(p + 1);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 p = v[i][0], q = v[i][1];
          float m = fmaxf(fmaxf(fmaxf(fabsf(p.x), fabsf(p.y)), fmaxf(fabsf(p.z), fabsf(p.w))),
                          fmaxf(fmaxf(fabsf(q.x), fabsf(q.y)), fmaxf(fabsf(q.z), fabsf(q.w))));
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
          const float s = scale_near(m), y = recip_rn(s);
          const uint32_t lo = cvt_e4m3x2(p.x * y, p.y * y) | cvt_e4m3x2(p.z * y, p.w * y) << 16;
          const uint32_t hi = cvt_e4m3x2(q.x * y, q.y * y) | cvt_e4m3x2(q.z * y, q.w * y) << 16;
          if (g0 + half + i * kHalves < groups) {
            const int t = tok[i];
            const uint32_t at = codes + (uint32_t)((blk[i] * NT + (t >> 3)) * kAtom + (t & 7) * 128 +
                                                   (((l16 >> 1) ^ (t & 7)) << 4) + 8 * (l16 & 1));
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(lo), "r"(hi) : "memory");
            if (l16 == 0) scales[blk[i] * NC + t] = s * s_weight[slot[i]];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(hfull0 + 8 * buf);
    }
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
  g.rows = (int)cdiv(N, num_sms);
  if (x > most || h > most || g.rows > 128) return g;  // stages 0: out of range
  g.buffers = 2 * h <= most ? 2 : 1;
  const int64_t codes = x > g.buffers * h ? x : g.buffers * h;
  const int64_t scales = (Kb > g.buffers * Ib ? Kb : g.buffers * Ib) * 8 * nt * 4;
  g.mtiles = g.rows <= 16 ? 1 : g.rows <= 32 ? 2 : g.rows <= 64 ? 4 : 8;
  g.blocks = kMmaWarps / g.mtiles;
  const int64_t rest = codes + (scales + 15) / 16 * 16 + kMiscBytes;
  int64_t stages = ((int64_t)227 * 1024 - 1024 - rest) / kStageBytes;
  g.stages = (int)(stages < kMlpMaxStages ? stages : kMlpMaxStages);
  g.off_scale = (int)(g.stages * kStageBytes + codes);
  g.off_misc = (int)(g.off_scale + (scales + 15) / 16 * 16);
  g.smem = g.off_misc + kMiscBytes + 1024;
  return g;
}

template <int NT>
static cudaError_t run_mlp(const CUtensorMap (&m)[4], const MlpArgs& a, int smem, int num_sms, cudaStream_t st) {
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
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs wait for one another: all or none are resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_mlp_kernel<NT>, m[0], m[1], m[2], m[3], a);
}

cudaError_t launch_moe_mlp(const MlpArgs& args, const uint8_t* qgu, int64_t ldgu, const uint8_t* qd, int64_t ldd,
                           int num_sms, cudaStream_t st, const char** msg) {
  MlpArgs a = args;
  const MlpGeom g = mlp_geom(a.T, a.K, a.I, a.N, num_sms);
  a.rows = g.rows, a.mtiles = g.mtiles, a.blocks = g.blocks, a.buffers = g.buffers, a.stages = g.stages;
  a.off_scale = g.off_scale, a.off_misc = g.off_misc;
  a.vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % 8 == 0 && a.K % 8 == 0;
  CUtensorMap m[4];
  memset(m, 0, sizeof(m));
  const int64_t Kf = a.K / kBlock, If = a.I / kBlock, E = a.E, I = a.I, N = a.N, K = a.K;
  bool ok = true;
  // features, K-blocks, then gate / up, expert: a box is 8 K-blocks of 8 gate and 8 up rows, a K-block's 8 rows together
  if (Kf) {
    const int64_t dim[5] = {kBlock, I, Kf, 2, E}, stride[5] = {1, ldgu, kBlock, I * ldgu, 2 * I * ldgu};
    const int box[5] = {kBlock, kUnit, kUnitBlocks, 2, 1};
    ok = mlp_map(&m[0], qgu, 5, dim, stride, box);
  }
  if (ok && K % kBlock) {
    const int64_t dim[4] = {K, I, 2, E}, stride[4] = {1, ldgu, I * ldgu, 2 * I * ldgu};
    const int box[4] = {kBlock, kUnit, 2, 1};
    ok = mlp_map(&m[1], qgu, 4, dim, stride, box);
  }
  if (ok && If) {
    const int64_t dim[4] = {kBlock, N, If, E}, stride[4] = {1, ldd, kBlock, N * ldd};
    const int box[4] = {kBlock, g.rows, g.blocks, 1};
    ok = mlp_map(&m[2], qd, 4, dim, stride, box);
  }
  if (ok && I % kBlock) {
    const int64_t dim[3] = {I, N, E}, stride[3] = {1, ldd, N * ldd};
    const int box[3] = {kBlock, g.rows, 1};
    ok = mlp_map(&m[3], qd, 3, dim, stride, box);
  }
  if (!ok) {
    *msg = "cuTensorMapEncodeTiled failed for a weight (alignment, stride or size out of range)";
    return cudaErrorInvalidValue;
  }
  return a.T <= 8 ? run_mlp<1>(m, a, g.smem, num_sms, st) : run_mlp<2>(m, a, g.smem, num_sms, st);
}

cudaError_t mlp_read_errors(uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_mlp_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_mlp_error, &zero, sizeof(uint32_t));
}

}  // namespace bfp8
