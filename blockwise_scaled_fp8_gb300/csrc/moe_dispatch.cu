// Dispatch of a mixture-of-experts layer: the tokens of the sorted rows are
// gathered, scaled by their slot's weight where one is given, and quantised in
// 1x128 groups along the features and 128x1 groups along the rows ("Enable
// blockwise FP8 dense training kernels on ROCm": act_quant_lhs, act_quant_rhs;
// s = amax/448, q = RNE_e4m3(clamp(x/s, +-448))) without the gathered tensor
// ever being written: with X[r] = w[src[r]] x[src[r] / k] (zero where src[r]
// is -1), the outputs are those of quantising X both ways.
//
// Persistent CTAs (two per SM, 16 warps each) over 128 x 128 tiles:
//   1. cp.async gathers the tile's 128 rows (256 bytes each; zero-filled on
//      padding and past the last column) into one of two stages, swizzled as a
//      128-byte-swizzled TMA box would be.  The rows' slots were read one tile
//      earlier, so that no copy waits for its own address.
//   2. Warp w takes the 8-column chunk w, lane l the rows 4l .. 4l+3.  A
//      column's 128 rows are one warp's, so its maximum, its scale and its
//      codes need no CTA barrier: a halving exchange leaves each lane with one
//      column's maximum over all rows.  A row's 16 chunk maxima meet in shared
//      memory.
//   3. The codes go to a staging tile (row-major and transposed) and leave by
//      one TMA store per output; the stage is free for the tile after the next
//      as soon as its values are in registers.
// The tiles are walked in bands of kBand column blocks, all rows of a band
// before the next band: a token's rows (one per chosen expert) then read the
// same few hundred bytes of it within a short time, from L2 after the first.
#include <cudaTypedefs.h>
#include <string.h>

#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

namespace {

constexpr int kDsThreads = 512;
constexpr int kDsCtasPerSm = 2;
constexpr int kBand = 4;                          // column blocks of a band
constexpr int kDsBoxBytes = 128 * 128;            // 64 bf16 columns x 128 rows
constexpr int kDsStageBytes = 2 * kDsBoxBytes;
constexpr int kDsOffRow = 2 * kDsStageBytes;      // q_row tile: 128 rows x 128 B, 128-byte swizzled
constexpr int kDsOffCol = kDsOffRow + 128 * 128;  // q_col tile: 128 columns x 128 B
constexpr int kDsOffRed = kDsOffCol + 128 * 128;  // [16 chunks][128 rows] bf16x2 row maxima
constexpr int kDsOffSc = kDsOffRed + 16 * 128 * 4;  // [128 rows] (s, -1/s)
constexpr int kDsOffW = kDsOffSc + 128 * 8;       // [2 stages][128 rows] weights
constexpr int kDsSmemBytes = kDsOffW + 2 * 128 * 4 + 1024;  // + alignment slack
static_assert(2 * (kDsSmemBytes + 1024) <= 228 * 1024, "two CTAs an SM");

struct DispatchParams {
  DispatchArgs a;
  int64_t C_al, R_al;  // C & ~15, R & ~15: extents of the two store maps
  int tiles_c, tiles_t, num_tiles;
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int q) {
  return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w;
}

// The e4m3 codes of -(x w / s) for the bf16 pair x, w2 = (w, w): neg_codes2 with the product formed first.
__device__ __forceinline__ uint32_t neg_codes2_w(uint32_t x, uint64_t w2, uint64_t s2, uint64_t ny2) {
  const uint64_t x2 = f2_mul(f2_pack(bf16_lo(x), bf16_hi(x)), w2);
  const uint64_t q0 = f2_mul(x2, ny2);
  const uint64_t r = f2_fma(s2, q0, x2);
  const uint64_t q1 = f2_fma(r, ny2, q0);
  return cvt_e4m3x2(__uint_as_float((uint32_t)q1), __uint_as_float((uint32_t)(q1 >> 32)));
}

struct TilePos {
  int t, c;
};
__device__ __forceinline__ TilePos tile_pos(int tile, int tiles_t, int tiles_c) {
  const int band = tile / (kBand * tiles_t), c0 = band * kBand;
  const int width = min(kBand, tiles_c - c0), rem = tile - band * kBand * tiles_t;
  return TilePos{rem / width, c0 + rem % width};
}

}  // namespace

template <bool COL, bool WEIGHTED, bool VEC>
__global__ void __launch_bounds__(kDsThreads, kDsCtasPerSm)
    moe_dispatch_kernel(const __grid_constant__ CUtensorMap tmap_qrow, const __grid_constant__ CUtensorMap tmap_qcol,
                        const DispatchParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t outr = sbase + kDsOffRow, outc = sbase + kDsOffCol, red = sbase + kDsOffRed;
  float* s_w = reinterpret_cast<float*>(smem + kDsOffW);
  const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t C = p.a.C, R = p.a.R;
  pdl_launch_dependents();
  if (tid == 0) {
    if (p.C_al > 0) tma_prefetch_desc(&tmap_qrow);
    if (COL && p.R_al > 0) tma_prefetch_desc(&tmap_qcol);
  }
  pdl_wait();

  const int rot = (lane >> 1) & 3;  // the order a lane reads its rows in: 4l + ((i + rot) & 3)
  uint32_t sel_e = 0, sel_o = 0;    // byte selectors of the transposed words (rows in order)
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = (k - rot) & 3;
    sel_e |= (uint32_t)((i & 1) + 4 * (i >> 1)) << (4 * k);
    sel_o |= (uint32_t)(2 + (i & 1) + 4 * (i >> 1)) << (4 * k);
  }
  // gather role: thread tid copies 16-byte chunk tid % 16 of rows tid / 16 + 32 i
  const int gc = tid & 15, gr = tid >> 4;
  int slot[4];  // of the rows of the tile that is copied next
  auto fetch_slots = [&](int tile) {
    const int64_t t0 = tile < p.num_tiles ? (int64_t)tile_pos(tile, p.tiles_t, p.tiles_c).t * 128 : R;
#pragma unroll
    for (int i = 0; i < 4; ++i) slot[i] = t0 + gr + 32 * i < R ? __ldg(p.a.src + t0 + gr + 32 * i) : -1;
  };
  auto issue = [&](int tile, int s) {
    if (tile < p.num_tiles) {
      const int64_t c = (int64_t)tile_pos(tile, p.tiles_t, p.tiles_c).c * 128 + gc * 8;
      const int cols = C - c >= 8 ? 8 : C - c > 0 ? (int)(C - c) : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = gr + 32 * i;
        const int64_t tok = slot[i] >= 0 ? (int64_t)((uint32_t)slot[i] / (uint32_t)p.a.k) : p.a.T;
        const bool ok = tok < p.a.T;
        const uint32_t dst = sbase + (uint32_t)(s * kDsStageBytes + (gc >> 3) * kDsBoxBytes + r * 128 +
                                                (((gc & 7) ^ (r & 7)) << 4));
        const uint16_t* from = p.a.x + (ok ? tok * p.a.ldx + c : 0);
        if constexpr (VEC) {
          cp_async_16(dst, ok && cols > 0 ? from : p.a.x, ok ? 2u * cols : 0u);
        } else {
          uint32_t v[4] = {};
          if (ok)
            for (int j = 0; j < cols; ++j) v[j >> 1] |= (uint32_t)__ldg(from + j) << (16 * (j & 1));
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                       : "memory");
        }
        if (WEIGHTED && gc == 0) s_w[s * 128 + r] = ok ? __ldg(p.a.weight + slot[i]) : 0.0f;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int step = (int)gridDim.x;
  fetch_slots((int)blockIdx.x);
  issue((int)blockIdx.x, 0);
  fetch_slots((int)blockIdx.x + step);
  issue((int)blockIdx.x + step, 1);
  fetch_slots((int)blockIdx.x + 2 * step);

  int it = 0;
  for (int tile = (int)blockIdx.x; tile < p.num_tiles; tile += step, ++it) {
    const int s = it & 1;
    const uint32_t stage = sbase + (uint32_t)(s * kDsStageBytes);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();  // the tile has landed
    const TilePos pos = tile_pos(tile, p.tiles_t, p.tiles_c);
    const int64_t t0 = (int64_t)pos.t * 128, c0 = (int64_t)pos.c * 128;

    // ------------------------------------------------ values and maxima
    uint4 v[4];
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * lane + ((i + rot) & 3);
      v[i] = lds128(stage + (uint32_t)((warp >> 3) * kDsBoxBytes + r * 128 + (((warp & 7) ^ (r & 7)) << 4)));
      w[i] = WEIGHTED ? s_w[s * 128 + r] : 1.0f;
      sts32(red + 4u * (uint32_t)(warp * 128 + r), amax2(amax2(v[i].x, v[i].y), amax2(v[i].z, v[i].w)));
    }
    const float wrow = WEIGHTED ? fabsf(s_w[s * 128 + (tid >> 2)]) : 1.0f;  // of the row whose scale this thread joins
    float csc = 0.0f, cny = 0.0f;  // lane l: scale and -1/scale of column 8 warp + (l >> 2)
    if constexpr (COL) {
      float m[8];
      if constexpr (WEIGHTED) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float lo = 0.0f, hi = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo = fmaxf(lo, fabsf(bf16_lo(word_of(v[i], q)) * w[i]));
            hi = fmaxf(hi, fabsf(bf16_hi(word_of(v[i], q)) * w[i]));
          }
          m[2 * q] = lo, m[2 * q + 1] = hi;
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t c2 = amax2(amax2(word_of(v[0], q), word_of(v[1], q)), amax2(word_of(v[2], q), word_of(v[3], q)));
          m[2 * q] = __uint_as_float((c2 << 16) & 0x7FFF0000u);
          m[2 * q + 1] = __uint_as_float(c2 & 0x7FFF0000u);
        }
      }
      // halving exchange: after it lane l holds column l >> 2 (bits 4, 3, 2 of the lane choose the half kept)
#pragma unroll
      for (int h = 4; h >= 1; h >>= 1) {
        const bool up = (lane & (4 * h)) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i) {
          const float give = up ? m[i] : m[i + h], keep = up ? m[i + h] : m[i];
          m[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 4 * h));
        }
      }
      m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
      m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 2));
      csc = WEIGHTED ? group_scale(m[0]) : scale_of(m[0]);
      cny = neg_rcp(csc);
      const int64_t c = c0 + 8 * warp + (lane >> 2);
      if ((lane & 3) == 0 && c < C) p.a.s_col[(t0 / 128) * p.a.lds_col + c] = csc;
    }
    if (tid == 0) bulk_wait_read_all();  // the last tile's stores have read the staging tiles
    __syncthreads();  // row maxima visible; the stage is in registers
    // ------------------------------------------------ the copy after the next
    issue(tile + 2 * step, s);
    fetch_slots(tile + 3 * step);

    // ------------------------------------------------ row scales: four threads a row
    {
      const int g = tid >> 2, qd = tid & 3;
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t x;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(red + 4u * (uint32_t)((4 * qd + j) * 128 + g)));
        m = amax2(m, x);
      }
      m = amax2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = amax2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = amax2(m, __byte_perm(m, 0, 0x1032));
      const float amax = __uint_as_float(m & 0x7FFF0000u);
      // rounding is monotonic: the largest |x w| of the row is |w| times its largest |x|
      if (qd == 0) {
        const float sc = WEIGHTED ? group_scale(amax * wrow) : scale_of(amax);
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sbase + kDsOffSc + 8u * g), "f"(sc), "f"(neg_rcp(sc))
                     : "memory");
        if (t0 + g < R) p.a.s_row[(c0 / 128) * p.a.lds_row + t0 + g] = sc;
      }
    }
    // ------------------------------------------------ transposed codes
    if constexpr (COL) {
      const uint32_t dst = outc + (uint32_t)(8 * warp * 128 + 4 * lane);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint64_t s2 = f2_pack(__shfl_sync(0xffffffffu, csc, 8 * q), __shfl_sync(0xffffffffu, csc, 8 * q + 4));
        const uint64_t ny2 = f2_pack(__shfl_sync(0xffffffffu, cny, 8 * q), __shfl_sync(0xffffffffu, cny, 8 * q + 4));
        uint32_t cc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          cc[i] = WEIGHTED ? neg_codes2_w(word_of(v[i], q), f2_pack(w[i], w[i]), s2, ny2)
                           : neg_codes2(word_of(v[i], q), s2, ny2);
        const uint32_t X = __byte_perm(cc[0], cc[1], 0x5140), Y = __byte_perm(cc[2], cc[3], 0x5140);
        sts32(dst + (uint32_t)((2 * q) * 128), __byte_perm(X, Y, sel_e) ^ 0x80808080u);
        sts32(dst + (uint32_t)((2 * q + 1) * 128), __byte_perm(X, Y, sel_o) ^ 0x80808080u);
      }
    }
    __syncthreads();  // row scales visible
    // ------------------------------------------------ row-major codes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * lane + ((i + rot) & 3);
      float rs, rny;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(rs), "=f"(rny) : "r"(sbase + kDsOffSc + 8u * r));
      const uint64_t s2 = f2_pack(rs, rs), ny2 = f2_pack(rny, rny), w2 = f2_pack(w[i], w[i]);
      uint32_t cd[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        cd[q] = WEIGHTED ? neg_codes2_w(word_of(v[i], q), w2, s2, ny2) : neg_codes2(word_of(v[i], q), s2, ny2);
      sts64(outr + (uint32_t)(r * 128 + ((((warp >> 1) ^ (r & 7)) << 4) | ((warp & 1) << 3))),
            __byte_perm(cd[0], cd[1], 0x5410) ^ 0x80808080u, __byte_perm(cd[2], cd[3], 0x5410) ^ 0x80808080u);
    }
    fence_proxy_async_shared();
    __syncthreads();  // the output tiles are complete
    if (tid == 0) {
      if (c0 < p.C_al) tma_store_2d(&tmap_qrow, outr, (int32_t)c0, (int32_t)t0);
      if (COL && t0 < p.R_al) tma_store_2d(&tmap_qcol, outc, (int32_t)t0, (int32_t)c0);
      bulk_commit();
    }
    // the last C % 16 (R % 16) bytes of a row, past the maps' extents
    const int g = tid >> 2, b0 = 4 * (tid & 3);
    if (c0 + 128 > p.C_al && p.C_al < C && t0 + g < R) {
      for (int b = b0; b < b0 + 4; ++b)
        if (p.C_al + b < C) {
          const int cl = (int)(p.C_al + b - c0);
          p.a.q_row[(t0 + g) * p.a.ldq_row + p.C_al + b] =
              smem[kDsOffRow + g * 128 + ((((cl >> 4) ^ (g & 7)) << 4) | (cl & 15))];
        }
    }
    if (COL && t0 + 128 > p.R_al && p.R_al < R && c0 + g < C) {
      for (int b = b0; b < b0 + 4; ++b)
        if (p.R_al + b < R) p.a.q_col[(c0 + g) * p.a.ldq_col + p.R_al + b] = smem[kDsOffCol + g * 128 + (p.R_al + b - t0)];
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (tid == 0) bulk_wait_all();  // stores complete before the CTA exits
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

template <bool COL, bool WEIGHTED, bool VEC>
static cudaError_t run_dispatch(const CUtensorMap& mr, const CUtensorMap& mc, const DispatchParams& p, int num_sms,
                                cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(moe_dispatch_kernel<COL, WEIGHTED, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kDsSmemBytes);
  });
  if (attr != cudaSuccess) return attr;
  const int cap = kDsCtasPerSm * num_sms;
  return launch_pdl(moe_dispatch_kernel<COL, WEIGHTED, VEC>, (unsigned)(p.num_tiles < cap ? p.num_tiles : cap),
                    kDsThreads, kDsSmemBytes, st, mr, mc, p);
}

cudaError_t launch_moe_dispatch(const DispatchArgs& a, int num_sms, cudaStream_t st, const char** msg) {
  DispatchParams p;
  p.a = a;
  p.C_al = a.C & ~(int64_t)15;
  p.R_al = a.R & ~(int64_t)15;
  const int64_t tc = cdiv(a.C, 128), tt = cdiv(a.R, 128);
  if (tc * tt >= ((int64_t)1 << 30)) {
    *msg = "too many 128x128 tiles (2^30 at most)";
    return cudaErrorInvalidValue;
  }
  p.tiles_c = (int)tc;
  p.tiles_t = (int)tt;
  p.num_tiles = (int)(tc * tt);
  CUtensorMap mr, mc;
  memset(&mr, 0, sizeof(mr));
  memset(&mc, 0, sizeof(mc));
  if (ds_encode_fn() == nullptr ||
      (p.C_al > 0 && !ds_store_map(&mr, a.q_row, p.C_al, a.R, a.ldq_row, true)) ||
      (a.q_col && p.R_al > 0 && !ds_store_map(&mc, a.q_col, p.R_al, a.C, a.ldq_col, false))) {
    *msg = "cuTensorMapEncodeTiled failed for an output (alignment, stride or size out of range)";
    return cudaErrorInvalidValue;
  }
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ldx % 8 == 0;
  auto pick = [&](auto col, auto weighted) {
    constexpr bool kCol = decltype(col)::value, kW = decltype(weighted)::value;
    return vec ? run_dispatch<kCol, kW, true>(mr, mc, p, num_sms, st)
               : run_dispatch<kCol, kW, false>(mr, mc, p, num_sms, st);
  };
  using T = std::true_type;
  using F = std::false_type;
  if (a.q_col) return a.weight ? pick(T{}, T{}) : pick(T{}, F{});
  return a.weight ? pick(F{}, T{}) : pick(F{}, F{});
}

}  // namespace bfp8
