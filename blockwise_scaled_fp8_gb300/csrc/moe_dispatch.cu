// Dispatch of a mixture-of-experts layer: the tokens of the sorted rows are
// gathered, scaled by their slot's weight where one is given, and quantised in
// 1x128 groups along the features and 128x1 groups along the rows ("Enable
// blockwise FP8 dense training kernels on ROCm": act_quant_lhs, act_quant_rhs;
// s = amax/448, q = RNE_e4m3(clamp(x/s, +-448))) without the gathered tensor
// ever being written: with X[r] = w[src[r]] x[src[r] / k] (zero where src[r]
// is -1), the outputs are those of quantising X both ways.
//
// Persistent CTAs (two per SM: eight quantising warps and two that gather)
// over 128 x 128 tiles:
//   1. The gathering warps bring the tile's 128 rows into one of two stages,
//      four rows of 64 columns a TMA gather, 128-byte swizzled; rows past the
//      tensor (padding) and columns past C arrive as zeros.
//   2. Quantising warp w takes the 16 columns 16w .., lane l the rows 4l ..
//      4l+3, in fp32 registers.  A column's 128 rows are one warp's, so its
//      maximum, its scale and its codes need no other warp: a halving exchange
//      leaves each lane with one column's maximum over all rows.  A row's eight
//      partial maxima meet in shared memory.
//   3. The codes go to a staging tile (row-major and transposed) and leave by
//      one TMA store per output; a stage is free for the tile after the next
//      as soon as its values are in registers.
// What bounds it: 131072 routed rows x 4096 (16384 tokens, 64 experts, 8 each)
// write 1.12 GB and read 0.18 (x nearly once) in 329 us with weights, 315
// without; a plain fill of the same bytes takes 283 us on this memory, the
// instructions of the two quantisations about 230.  Steps that led here:
// gathering by cp.async from the quantising warps 675 us; by TMA from two warps
// of their own, 16 columns a warp 349; the warps' barriers split into arrival
// and wait 318 (with one product a code of weighted rows, whose quotients take
// the other 11 us).  (cp.async from the two gathering warps: 340 and 348, since
// the copies share the quantisers' path to shared memory.)
// The tiles are walked down the rows of a column block before the next block:
// a token's rows (one per chosen expert) then read the same 256 bytes of it
// within a short time, from L2 after the first (16384 tokens x 4096, eight
// experts each: 342 us at the time; four column blocks at once 348, all 32 of them 383).
// A NaN's code is 0x7F, where the quantisation entries, which form the codes of
// -x/s and turn their signs, give 0xFF (that way here: 327 us without weights).
#include <cudaTypedefs.h>
#include <string.h>

#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

static __device__ uint32_t g_dispatch_error;

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kDsConsumers = 256;                 // 8 warps that quantise, and two that gather
constexpr int kDsProducers = 64;
constexpr int kDsThreads = kDsConsumers + kDsProducers;
constexpr int kDsCtasPerSm = 2;
constexpr int kDsBoxBytes = 128 * 128;            // 64 bf16 columns x 128 rows
constexpr int kDsStageBytes = 2 * kDsBoxBytes;
constexpr int kDsOffRow = 2 * kDsStageBytes;      // q_row tile: 128 rows x 128 B, 128-byte swizzled
constexpr int kDsOffCol = kDsOffRow + 128 * 128;  // q_col tile: 128 columns x 128 B
constexpr int kDsOffRed = kDsOffCol + 128 * 128;  // [8 warps][128 rows] bf16x2 row maxima
constexpr int kDsOffSc = kDsOffRed + 8 * 128 * 4;  // [128 rows] (hi, lo) of 1/s
constexpr int kDsOffCsc = kDsOffSc + 128 * 8;     // [8 warps][8 column pairs] (hi, hi', lo, lo') of 1/s
constexpr int kDsOffW = kDsOffCsc + 8 * 8 * 16;  // [2 stages][128 rows] weights
constexpr int kDsOffBar = kDsOffW + 2 * 128 * 4;  // full[2], empty[2], rows, scales, codes ready; the abort flag, a zero
constexpr int kDsSmemBytes = kDsOffBar + 64 + 1024;  // + alignment slack
static_assert(2 * (kDsSmemBytes + 1024) <= 228 * 1024, "two CTAs an SM");

struct DispatchParams {
  DispatchArgs a;
  int C_al, R_al;  // C & ~15, R & ~15: extents of the two store maps
  int tiles_c, tiles_t, num_tiles;
  // quotients by tiles_t and by k (see magic)
  uint32_t t_mul, k_mul;
  int t_shift, k_shift;
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int q) {
  return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w;
}

// Four e4m3 codes (RNE, saturating): bytes a.lo, a.hi, b.lo, b.hi.
__device__ __forceinline__ uint32_t cvt4(uint64_t a, uint64_t b) {
  float a0, a1, b0, b1;
  f2_unpack(a, a0, a1);
  f2_unpack(b, b0, b1);
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
  return r;
}
// Four rows y0 .. y3 x 64 columns from column x on, 128 bytes each, one after
// the other at dst; rows past the tensor's are filled with zeros.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y0,
                                            int32_t y1, int32_t y2, int32_t y3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 1/s as hi + lo with lo >= 0: hi the hardware's approximation, two ulps down
// where it is above 1/s, lo what it lacks.  RN(x hi + RN(x lo)) rounds to the
// e4m3 code of the IEEE quotient x/s for every bf16 x with |x| <= 448 s, sign
// of zero included (checked exhaustively on the CPU).  Of products x = RN(x' w)
// it is x/s to within 2^-43 before its rounding, so the quotient unless that
// lies as near to halfway between two floats (no code differs in 6e9 products
// checked on the CPU).  One product x hi would not do: with a weight that a
// whole row shares, x/s is 448 x'/max|x'| but for roundings, which are often
// within an ulp of a tie of the codes (1.3 in a thousand differ).
__device__ __forceinline__ float2 recip_hi_lo(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  if (__fmaf_rn(-s, y, 1.0f) < 0.0f) y = __uint_as_float(__float_as_uint(y) - 2u);
  return make_float2(y, __fmul_rn(__fmaf_rn(-s, y, 1.0f), y));
}

struct TilePos {
  int t, c;  // row and column block
};
__device__ __forceinline__ TilePos tile_pos(int tile, const DispatchParams& p) {
  const int c = p.tiles_t > 1 ? (int)__umulhi((uint32_t)tile, p.t_mul) >> p.t_shift : tile;  // tile / tiles_t
  return TilePos{tile - c * p.tiles_t, c};
}

}  // namespace

// Position of row r of a tile in the per-row arrays, which hold a lane's four
// rows in the order the lane reads them: 4l + ((i + rot) & 3), rot = (l >> 1) & 3
// (so that the 16-byte reads of a quarter-warp fall into eight bank groups).
__device__ __forceinline__ int row_pos(int r) { return (r & ~3) | ((r - (r >> 3)) & 3); }

template <bool COL, bool WEIGHTED, bool TMA>
__global__ void __launch_bounds__(kDsThreads, kDsCtasPerSm)
    moe_dispatch_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_qrow,
                        const __grid_constant__ CUtensorMap tmap_qcol, const DispatchParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t full0 = sbase + kDsOffBar, empty0 = full0 + 16;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kDsOffBar + 56);
  volatile int* never = abort_flag + 1;
  float* s_w = reinterpret_cast<float*>(smem + kDsOffW);
  const int tid = (int)threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
  const int C = (int)p.a.C, R = (int)p.a.R, step = (int)gridDim.x;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(full0 + 8 * s, TMA ? kDsProducers / 32 : kDsProducers);
      mbar_init(empty0 + 8 * s, kDsConsumers / 32);
    }
    for (int i = 0; i < 3; ++i) mbar_init(full0 + 32 + 8 * i, kDsConsumers / 32);  // rows, scales, codes ready
    *abort_flag = 0;
    *never = 0;
    fence_barrier_init();
    fence_proxy_async_shared();
    if (TMA) tma_prefetch_desc(&tmap_x);
    if (p.C_al > 0) tma_prefetch_desc(&tmap_qrow);
    if (COL && p.R_al > 0) tma_prefetch_desc(&tmap_qcol);
  }
  __syncthreads();
  pdl_wait();

  if (warp >= kDsConsumers / 32) {
    // ------------------------------------------------------------ producers
    // Warp w gathers the rows 64w .. 64w + 63, lane l the four rows 4 (l & 15) ..
    // of them and the 64-column half l >> 4.  Their slots are read two tiles
    // ahead, their weights one, so that no copy waits for its own address.
    const int r4 = 64 * (warp - kDsConsumers / 32) + 4 * (lane & 15), half = lane >> 4;
    int slot[4], tok[4];  // of the tile after next, of the next
    float wgt[4];
    auto read_slots = [&](int tile) {
      const int64_t at = tile < p.num_tiles ? (int64_t)tile_pos(tile, p).t * 128 + r4 : R;
#pragma unroll
      for (int i = 0; i < 4; ++i) slot[i] = at + i < R ? __ldg(p.a.src + at + i) : -1;
    };
    auto read_weights = [&]() {  // and the tokens, from the slots
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t t = p.k_mul ? __umulhi((uint32_t)slot[i], p.k_mul) >> p.k_shift : (uint32_t)slot[i];
        const bool ok = slot[i] >= 0 && (int64_t)t < p.a.T;
        tok[i] = ok ? (int)t : (int)p.a.T;  // past the tensor: zeros
        if constexpr (WEIGHTED) wgt[i] = ok ? __ldg(p.a.weight + slot[i]) : 0.0f;
      }
    };
    read_slots((int)blockIdx.x);
    read_weights();
    read_slots((int)blockIdx.x + step);
    int it = 0;
    bool ok = true;
    for (int tile = (int)blockIdx.x; tile < p.num_tiles; tile += step, ++it) {
      const int s = it & 1;
      ok = mbar_wait_bounded(empty0 + 8 * s, (uint32_t)((it >> 1) & 1) ^ 1u, kWaitLimitNs, abort_flag);
      if (!__all_sync(kAll, ok)) {
        if (lane == 0 && !*abort_flag) atomicOr(&g_dispatch_error, 1u);
        *abort_flag = 1;
        ok = false;
        break;
      }
      const uint32_t stage = sbase + (uint32_t)(s * kDsStageBytes);
      const int c0 = tile_pos(tile, p).c * 128;
      if constexpr (WEIGHTED) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (half == 0) s_w[s * 128 + row_pos(r4 + i)] = wgt[i];
      }
      if constexpr (TMA) {
        __syncwarp();  // the weights, before the arrival that publishes them
        if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * s, (uint32_t)(kDsStageBytes / (kDsProducers / 32)));
        __syncwarp();
        tma_gather4(stage + (uint32_t)(half * kDsBoxBytes + r4 * 128), &tmap_x, full0 + 8 * s, c0 + 64 * half, tok[0],
                    tok[1], tok[2], tok[3]);
      } else {
        // rows that TMA cannot read, element by element: lane l columns l, l + 32, ..
        const int r0 = 64 * (warp - kDsConsumers / 32);
        constexpr int kRows = 8;  // in flight
        for (int i0 = 0; i0 < 64; i0 += kRows) {
          uint16_t v[kRows][4];
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int t = __shfl_sync(kAll, tok[i & 3], (i0 + i) >> 2);
            const uint16_t* from = p.a.x + (int64_t)t * p.a.ldx + c0 + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = t < p.a.T && c0 + lane + 32 * j < C ? __ldg(from + 32 * j) : (uint16_t)0;
          }
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i0 + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int c = lane + 32 * j;
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage + (uint32_t)((c >> 6) * kDsBoxBytes + r * 128 +
                                                                              ((((c >> 3) & 7) ^ (r & 7)) << 4) + (c & 7) * 2)),
                           "h"(v[i][j])
                           : "memory");
            }
          }
        }
        mbar_arrive(full0 + 8 * s);
      }
      read_weights();
      read_slots(tile + 2 * step);
    }
    if (TMA && !ok && lane == 0)  // copies already issued land before this CTA's shared memory goes away
      for (int i = it > 2 ? it - 2 : 0; i < it; ++i)
        mbar_wait_bounded(full0 + 8 * (i & 1), (uint32_t)((i >> 1) & 1), kWaitLimitNs, never);
  } else {
    // ------------------------------------------------------------ quantisers
    // Warp w takes the 16 columns 16w .. of the tile, lane l the rows 4l .. 4l+3.
    // The warps meet twice a tile, by arriving early and waiting late:
    //   rows ready   the row maxima (and the stage and the staging tiles free)
    //   scales ready the row scales, while each warp forms its columns' codes
    // A warp goes on to the next tile without waiting for the others' codes;
    // thread 0 alone waits for them, to store the tile.
    const uint32_t outr = sbase + kDsOffRow, outc = sbase + kDsOffCol;
    const uint32_t rows_ready = full0 + 32, scales_ready = full0 + 40, codes_ready = full0 + 48;
    const int rot = (lane >> 1) & 3;
    uint32_t sel_e = 0, sel_o = 0;  // byte selectors of the transposed words (rows in order)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t i = (uint32_t)((k - rot) & 3);
      sel_e |= (2 * i) << (4 * k);
      sel_o |= (2 * i + 1) << (4 * k);
    }
    uint32_t* s_red = reinterpret_cast<uint32_t*>(smem + kDsOffRed);
    float* s_csc = reinterpret_cast<float*>(smem + kDsOffCsc) + 32 * warp;
    const int g = tid >> 1, gpos = row_pos(g);  // the row whose scale this thread and its neighbour form
    const bool ragged = p.C_al < C || (COL && p.R_al < R);
    auto arrive = [&](uint32_t bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto wait = [&](uint32_t bar, int phase) {
      const bool ok = mbar_wait_bounded(bar, (uint32_t)phase, kWaitLimitNs, abort_flag);
      if (__all_sync(kAll, ok)) return true;
      if (lane == 0 && !*abort_flag) atomicOr(&g_dispatch_error, 1u);
      *abort_flag = 1;
      return false;
    };
    int it = 0;
    for (int tile = (int)blockIdx.x; tile < p.num_tiles; tile += step, ++it) {
      const int s = it & 1, phase = it & 1;
      const uint32_t stage = sbase + (uint32_t)(s * kDsStageBytes);
      const TilePos pos = tile_pos(tile, p);
      const int t0 = pos.t * 128, c0 = pos.c * 128;
      if (!wait(full0 + 8 * s, (it >> 1) & 1)) break;

      // ---------------------------------------------- values (times the rows' weights) in fp32, row maxima
      uint64_t x2[4][8];  // row i, column pair q
      uint32_t rm[4];
      float w[4];
      if constexpr (WEIGHTED) {
        const float4 w4 = *reinterpret_cast<const float4*>(s_w + s * 128 + 4 * lane);
        w[0] = w4.x, w[1] = w4.y, w[2] = w4.z, w[3] = w4.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * lane + ((i + rot) & 3);
        uint4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[h] = lds128(stage + (uint32_t)((warp >> 2) * kDsBoxBytes + r * 128 + ((((2 * warp + h) & 7) ^ (r & 7)) << 4)));
        rm[i] = amax2(amax2(amax2(v[0].x, v[0].y), amax2(v[0].z, v[0].w)),
                      amax2(amax2(v[1].x, v[1].y), amax2(v[1].z, v[1].w)));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t x = word_of(v[q >> 2], q & 3);
          x2[i][q] = f2_pack(bf16_lo(x), bf16_hi(x));
          if constexpr (WEIGHTED) x2[i][q] = f2_mul(x2[i][q], f2_pack(w[i], w[i]));
        }
      }
      *reinterpret_cast<uint4*>(s_red + warp * 128 + 4 * lane) = make_uint4(rm[0], rm[1], rm[2], rm[3]);
      const float wrow = WEIGHTED ? fabsf(s_w[s * 128 + gpos]) : 1.0f;
      if (tid == 0) bulk_wait_read_all();  // the last tile's stores have read the staging tiles
      arrive(rows_ready);

      // ---------------------------------------------- column maxima and scales: the warp's own
      if constexpr (COL) {
        // Halving exchange over the lanes: each step keeps half of the columns
        // (bits 4, 3, .. of the lane choose it): lane l ends with column l >> 1.
        float m[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float lo[4], hi[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) f2_unpack(x2[i][q], lo[i], hi[i]);
          m[2 * q] = fmaxf(max3_abs(lo[0], lo[1], lo[2]), fabsf(lo[3]));
          m[2 * q + 1] = fmaxf(max3_abs(hi[0], hi[1], hi[2]), fabsf(hi[3]));
        }
#pragma unroll
        for (int h = 8; h >= 1; h >>= 1) {
          const bool up = (lane & (2 * h)) != 0;
#pragma unroll
          for (int i = 0; i < h; ++i) {
            const float give = up ? m[i] : m[i + h], keep = up ? m[i + h] : m[i];
            m[i] = fmaxf(keep, __shfl_xor_sync(kAll, give, 2 * h));
          }
        }
        const float cmax = fmaxf(m[0], __shfl_xor_sync(kAll, m[0], 1));
        if ((lane & 1) == 0) {
          const float sc = scale_of(cmax);
          const float2 y = recip_hi_lo(sc);
          const int j = lane >> 1, c = c0 + 16 * warp + j;
          float* dst = s_csc + (j >> 1) * 4 + (j & 1);
          dst[0] = y.x;
          dst[2] = y.y;
          if (c < C) p.a.s_col[(int64_t)pos.t * p.a.lds_col + c] = sc;
        }
        __syncwarp();
      }
      if (!wait(rows_ready, phase)) break;
      // the stage is in registers: the row maxima, stored before the wait above, were formed from every value read
      if (lane == 0) mbar_arrive(empty0 + 8 * s);

      // ---------------------------------------------- row scales: two threads a row
      {
        uint32_t m = amax2(amax2(s_red[(4 * (tid & 1)) * 128 + gpos], s_red[(4 * (tid & 1) + 1) * 128 + gpos]),
                           amax2(s_red[(4 * (tid & 1) + 2) * 128 + gpos], s_red[(4 * (tid & 1) + 3) * 128 + gpos]));
        m = amax2(m, __shfl_xor_sync(kAll, m, 1));
        m = amax2(m, __byte_perm(m, 0, 0x1032));
        // rounding is monotonic: the largest |x w| of the row is |w| times its largest |x|
        const float sc = scale_of(__uint_as_float(m & 0x7FFF0000u) * wrow);
        if ((tid & 1) == 0) {
          *reinterpret_cast<float2*>(smem + kDsOffSc + 8 * gpos) = recip_hi_lo(sc);
          if (t0 + g < R) p.a.s_row[(int64_t)pos.c * p.a.lds_row + t0 + g] = sc;
        }
      }
      arrive(scales_ready);
      // ---------------------------------------------- codes
      if constexpr (COL) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {  // columns 16 warp + 2q, + 1
          const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(s_csc + 4 * q);
          uint64_t cv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            cv[i] = f2_fma(x2[i][q], y.x, f2_mul(x2[i][q], y.y));
          const uint32_t dst = outc + (uint32_t)((16 * warp + 2 * q) * 128 + 4 * lane);
          const uint32_t lo = cvt4(cv[0], cv[1]), hi = cvt4(cv[2], cv[3]);
          sts32(dst, __byte_perm(lo, hi, sel_e));
          sts32(dst + 128u, __byte_perm(lo, hi, sel_o));
        }
      }
      if (!wait(scales_ready, phase)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = *reinterpret_cast<const float2*>(smem + kDsOffSc + 8 * (4 * lane + i));
        const uint64_t hi = f2_pack(y.x, y.x), lo = f2_pack(y.y, y.y);
        uint32_t rc[4];
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
          const uint64_t a = f2_fma(x2[i][q], hi, f2_mul(x2[i][q], lo));
          const uint64_t b = f2_fma(x2[i][q + 1], hi, f2_mul(x2[i][q + 1], lo));
          rc[q >> 1] = cvt4(a, b);
        }
        const int r = 4 * lane + ((i + rot) & 3);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(outr + (uint32_t)(r * 128 + ((warp ^ (r & 7)) << 4))),
                     "r"(rc[0]), "r"(rc[1]), "r"(rc[2]), "r"(rc[3])
                     : "memory");
      }
      fence_proxy_async_shared();
      arrive(codes_ready);
      if (warp == 0 || ragged) {
        if (!wait(codes_ready, phase)) break;
        if (tid == 0) {
          if (c0 < p.C_al) tma_store_2d(&tmap_qrow, outr, c0, t0);
          if (COL && t0 < p.R_al) tma_store_2d(&tmap_qcol, outc, t0, c0);
          bulk_commit();
        }
      }
      // the last C % 16 (R % 16) bytes of a row, past the maps' extents
      if (p.C_al < C && c0 + 128 > p.C_al && t0 + g < R) {
        for (int c = p.C_al + (tid & 1); c < C; c += 2)
          p.a.q_row[(int64_t)(t0 + g) * p.a.ldq_row + c] =
              smem[kDsOffRow + g * 128 + (((((c - c0) >> 4) ^ (g & 7)) << 4) | ((c - c0) & 15))];
      }
      if (COL && p.R_al < R && t0 + 128 > p.R_al && c0 + g < C) {
        for (int r = p.R_al + (tid & 1); r < R; r += 2)
          p.a.q_col[(int64_t)(c0 + g) * p.a.ldq_col + r] = smem[kDsOffCol + g * 128 + (r - t0)];
      }
    }
    if (tid == 0) bulk_wait_all();  // stores complete before the CTA exits
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

static PFN_cuTensorMapEncodeTiled_v12000 ds_encode_fn() {
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

// u8 matrix [rows, inner] with row stride ld bytes, written by 128 x 128-byte boxes.
static bool ds_store_map(CUtensorMap* m, void* base, int64_t inner, int64_t rows, int64_t ld, bool swizzle) {
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {128, 128};
  cuuint32_t elem[2] = {1, 1};
  return ds_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, elem,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// x bf16 [T, C], gathered by rows of 64 columns, 128-byte swizzled.
static bool ds_gather_map(CUtensorMap* m, const uint16_t* x, int64_t C, int64_t T, int64_t ldx) {
  cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)T};
  cuuint64_t strides[1] = {(cuuint64_t)ldx * 2};
  cuuint32_t box[2] = {64, 1};
  cuuint32_t elem[2] = {1, 1};
  return ds_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(x), dims, strides, box, elem,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// n / d = umulhi(n, mul) >> shift for 0 <= n < 2^31 and d >= 2: with 2^(shift
// + 1) >= d, mul = floor(2^(32 + shift) / d) + 1 is 2^(32 + shift) / d + e, 0 <
// e <= 1, which adds at most n e / 2^(32 + shift) < 2^-(shift + 1) <= 1/d to the
// quotient: not enough to reach the next whole number.  d = 1: mul = 0.
static void magic(uint32_t d, uint32_t* mul, int* shift) {
  int sh = 0;
  while (((uint64_t)2 << sh) < d) ++sh;
  *mul = d == 1 ? 0u : (uint32_t)((((uint64_t)1 << (32 + sh)) / d) + 1);
  *shift = sh;
}

template <bool COL, bool WEIGHTED, bool TMA>
static cudaError_t run_dispatch(const CUtensorMap& mx, const CUtensorMap& mr, const CUtensorMap& mc, const DispatchParams& p, int num_sms,
                                cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(moe_dispatch_kernel<COL, WEIGHTED, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kDsSmemBytes);
  });
  if (attr != cudaSuccess) return attr;
  const int cap = kDsCtasPerSm * num_sms;
  return launch_pdl(moe_dispatch_kernel<COL, WEIGHTED, TMA>, (unsigned)(p.num_tiles < cap ? p.num_tiles : cap),
                    kDsThreads, kDsSmemBytes, st, mx, mr, mc, p);
}

cudaError_t launch_moe_dispatch(const DispatchArgs& a, int num_sms, cudaStream_t st, const char** msg) {
  DispatchParams p;
  p.a = a;
  p.C_al = (int)(a.C & ~(int64_t)15);
  p.R_al = (int)(a.R & ~(int64_t)15);
  const int64_t tc = cdiv(a.C, 128), tt = cdiv(a.R, 128);
  if (tc * tt >= ((int64_t)1 << 30)) {
    *msg = "too many 128x128 tiles (2^30 at most)";
    return cudaErrorInvalidValue;
  }
  p.tiles_c = (int)tc;
  p.tiles_t = (int)tt;
  p.num_tiles = (int)(tc * tt);
  magic((uint32_t)tt, &p.t_mul, &p.t_shift);
  magic((uint32_t)a.k, &p.k_mul, &p.k_shift);
  CUtensorMap mx, mr, mc;
  memset(&mx, 0, sizeof(mx));
  memset(&mr, 0, sizeof(mr));
  memset(&mc, 0, sizeof(mc));
  // TMA gathers need 16-byte aligned rows; others are gathered by the elements (8192 tokens to
  // eight experts each: 2000 columns 90 us, 1999 190)
  const bool tma = a.T > 0 && (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ldx % 8 == 0;
  if (ds_encode_fn() == nullptr || (tma && !ds_gather_map(&mx, a.x, a.C, a.T, a.ldx)) ||
      (p.C_al > 0 && !ds_store_map(&mr, a.q_row, p.C_al, a.R, a.ldq_row, true)) ||
      (a.q_col && p.R_al > 0 && !ds_store_map(&mc, a.q_col, p.R_al, a.C, a.ldq_col, false))) {
    *msg = "cuTensorMapEncodeTiled failed for an operand (alignment, stride or size out of range)";
    return cudaErrorInvalidValue;
  }
  auto pick = [&](auto col, auto weighted) {
    constexpr bool kCol = decltype(col)::value, kW = decltype(weighted)::value;
    return tma ? run_dispatch<kCol, kW, true>(mx, mr, mc, p, num_sms, st)
               : run_dispatch<kCol, kW, false>(mx, mr, mc, p, num_sms, st);
  };
  using T = std::true_type;
  using F = std::false_type;
  if (a.q_col) return a.weight ? pick(T{}, T{}) : pick(T{}, F{});
  return a.weight ? pick(F{}, T{}) : pick(F{}, F{});
}

cudaError_t dispatch_read_errors(uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_dispatch_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_dispatch_error, &zero, sizeof(uint32_t));
}

}  // namespace bfp8
