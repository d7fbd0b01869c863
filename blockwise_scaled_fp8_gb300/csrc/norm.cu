// Root-mean-square norm of a transformer's residual stream with the addition
// before it and quantised outputs after it, and its gradient.
//   h = bf16(x + residual)  (x itself without a residual)
//   r = 1 / sqrt(mean(h^2) + eps),   y = h r w
// y leaves as e4m3 codes in 1x128 groups along the features (the forward's
// operand), in 128x1 groups along the tokens, transposed (the weight gradient's
// operand), as bf16, or any of these; it is not rounded before its quantisation
// ("Enable blockwise FP8 dense training kernels on ROCm": act_quant_lhs,
// act_quant_rhs; s = max(amax, 1e-12) / 448, q = RNE_e4m3(clamp(y/s, +-448))).
//
// Within a row's group r is a common factor and within a column's w is, so the
// codes are formed as (h w) (r / s) and (h r) (w / s): one product a value.
//
// Gradient, with n = h r and g = dy w:
//   dx = r (g - n mean(g n)) + dh,   dw[k] = sum over t of dy n.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kVec = 8;  // features a thread takes side by side: 16 bytes of bf16, 16 threads a group of 128

struct Team {
  int size, lane, index, count;  // threads a row, this thread's place, this thread's team, teams a CTA
};
__device__ __forceinline__ Team team_of(int size) {
  const int tid = (int)threadIdx.x;
  return Team{size, tid & (size - 1), tid / size, (int)blockDim.x / size};
}

// 16 bytes that another CTA of the cluster may have written (not the read-only path).
__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_u16(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}

// Eight bf16 of a row from feature k on, zeros past its end.
template <bool VEC>
__device__ __forceinline__ uint4 load_row8(const uint16_t* row, int k, int K) {
  if constexpr (VEC) {
    return k < K ? ld_v4(row + k) : make_uint4(0, 0, 0, 0);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = k + 2 * i < K ? ld_u16(row + k + 2 * i) : 0u;
      const uint32_t hi = k + 2 * i + 1 < K ? ld_u16(row + k + 2 * i + 1) : 0u;
      w[i] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <bool VEC>
__device__ __forceinline__ void store_row8(uint16_t* row, int k, int K, const uint4& v) {
  if (VEC) {
    if (k < K) *reinterpret_cast<uint4*>(row + k) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < K) row[k + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ float weight_at(const void* w, int f32, int64_t k) {
  return f32 ? __ldg(static_cast<const float*>(w) + k)
             : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(w) + k) << 16);
}
// Eight weights from feature k on, zeros past the end.
template <bool VEC>
__device__ __forceinline__ void load_weight8(const void* w, int f32, int k, int K, float (&f)[8]) {
  if constexpr (VEC) {
    if (k >= K) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.0f;
    } else if (f32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + k);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
      unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + k)), f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = k + i < K ? weight_at(w, f32, k + i) : 0.0f;
  }
}

// The sum of v over a team's threads, the same bits in each of them.  `slots`: one of
// two sets of a float a warp, used in turn, so that one barrier a sum is enough.
__device__ __forceinline__ float team_sum(float v, const Team& t, float* slots) {
  for (int o = min(t.size, 32) >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  if (t.size <= 32) return v;
  const int warp = (int)threadIdx.x >> 5, warps = t.size >> 5;
  if ((threadIdx.x & 31) == 0) slots[warp] = v;
  __syncthreads();
  float sum = 0.0f;
  const float* mine = slots + t.index * warps;
  for (int i = 0; i < warps; ++i) sum += mine[i];
  return sum;
}

// Four e4m3 codes (RNE, saturating), the first in the lowest byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return cvt_e4m3x2(a, b) | cvt_e4m3x2(c, d) << 16;
}

}  // namespace

// One row after another by teams of threads, each thread VPT chunks of eight
// features (chunk u of a thread starts at feature 8 (u size + lane)).  With COLS
// a cluster takes 128 rows, its CTAs 128 / C of them each; then, the rows written
// and every CTA's rstd known, each CTA takes every C-th block of 128 columns and
// reads it back, from L2, to quantise it along the rows.
template <int THREADS, int VPT, bool VEC, bool COLS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : COLS || VPT > 4 ? 2 : 3)
    rms_norm_kernel(const NormArgs a) {
  __shared__ float s_slots[2][THREADS / 32];
  const Team team = team_of(a.team);
  const int K = (int)a.K, lane = team.lane;
  int64_t t0, t_end;  // rows [t0, t_end), every step-th
  int64_t step = team.count;
  const int ctas = a.cluster, rank = COLS ? (int)blockIdx.x % ctas : 0;
  const int64_t block = COLS ? (int64_t)blockIdx.x / ctas : 0;
  if (COLS) {
    const int rows = kBlock / ctas;
    t0 = block * kBlock + rank * rows;
    t_end = min(t0 + rows, a.T);
  } else {
    t0 = (int64_t)blockIdx.x * team.count;
    t_end = a.T;
    step *= gridDim.x;
  }
  pdl_launch_dependents();
  pdl_wait();
  const uint16_t* stream = a.residual ? a.h : a.x;
  const int64_t lds = a.residual ? a.ldh : a.ldx;
  int turn = 0;
  for (int64_t first = t0; first < t_end; first += step, turn ^= 1) {
    const int64_t t = first + team.index;
    const bool live = t < t_end;
    uint4 hv[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u)
      hv[u] = live ? load_row8<VEC>(a.x + t * a.ldx, kVec * (u * team.size + lane), K) : make_uint4(0, 0, 0, 0);
    if (a.residual && live) {
      uint4 rv[VPT];
#pragma unroll
      for (int u = 0; u < VPT; ++u) rv[u] = load_row8<VEC>(a.residual + t * a.ldr, kVec * (u * team.size + lane), K);
#pragma unroll
      for (int u = 0; u < VPT; ++u) {
        float x[8], r[8];
        unpack8(hv[u], x);
        unpack8(rv[u], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += r[i];
        hv[u] = pack8(x);
        store_row8<VEC>(a.h + t * a.ldh, kVec * (u * team.size + lane), K, hv[u]);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      float x[8];
      unpack8(hv[u], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
    }
    sum = team_sum(sum, team, s_slots[turn]);
    const float r = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)K) + a.eps));
    if (live && lane == 0) a.rstd[t] = r;
    if (a.q_row || a.y) {
#pragma unroll
      for (int u = 0; u < VPT; ++u) {
        const int k = kVec * (u * team.size + lane);
        float x[8], w[8];
        unpack8(hv[u], x);
        load_weight8<VEC>(a.weight, a.weight_f32, k, K, w);
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= w[i];
          amax = fmaxf(amax, fabsf(x[i]));
        }
        if (a.y && live) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i] * r;
          store_row8<VEC>(a.y + t * a.ldy, k, K, pack8(y));
        }
        if (a.q_row) {
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
          const float s = group_scale(amax * r), m = __fdiv_rn(r, s);
          if (live && k < K) {
            const uint32_t lo = codes4(x[0] * m, x[1] * m, x[2] * m, x[3] * m);
            const uint32_t hi = codes4(x[4] * m, x[5] * m, x[6] * m, x[7] * m);
            uint8_t* q = a.q_row + t * a.ldq_row + k;
            if (k + kVec <= K) {
              *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (k + i < K) q[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
            }
            if ((lane & 15) == 0) a.s_row[(int64_t)(k / kBlock) * a.lds_row + t] = s;
          }
        }
      }
    }
  }
  if constexpr (COLS) {
    static_assert(THREADS == 256, "16 rows of 16 threads");
    __shared__ float s_max[8][kBlock], s_mul[kBlock], s_r[kBlock];
    __shared__ uint32_t s_tile[kBlock][32];  // codes [column][four rows], word w of column c at w ^ 2 (c / 8 % 16)
    __syncwarp();
    cluster_sync_all();  // the rows of this block, and their rstd, are written
    const int tid = (int)threadIdx.x, warp = tid >> 5, c8 = tid & 15, g = tid >> 4;
    const int64_t b0 = block * kBlock;
    if (tid < kBlock) s_r[tid] = b0 + tid < a.T ? *(volatile float*)(a.rstd + b0 + tid) : 0.0f;
    __syncthreads();
    float rr[8];  // of this thread's rows 4g .. 4g + 3 and 64 + 4g ..
#pragma unroll
    for (int i = 0; i < 8; ++i) rr[i] = s_r[4 * g + (i & 3) + 64 * (i >> 2)];
    const int Kb = (int)cdiv(K, kBlock);
    for (int kb = rank; kb < Kb; kb += ctas) {
      const int k = kb * kBlock + kVec * c8;
      uint4 hv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t t = b0 + 4 * g + (i & 3) + 64 * (i >> 2);
        hv[i] = t < a.T ? load_row8<VEC>(stream + t * lds, k, K) : make_uint4(0, 0, 0, 0);
      }
      float m[8] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[8];
        unpack8(hv[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], fabsf(x[j] * rr[i]));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(kAll, m[j], 16));
      if ((tid & 16) == 0) {
        *reinterpret_cast<float4*>(&s_max[warp][kVec * c8]) = make_float4(m[0], m[1], m[2], m[3]);
        *reinterpret_cast<float4*>(&s_max[warp][kVec * c8 + 4]) = make_float4(m[4], m[5], m[6], m[7]);
      }
      __syncthreads();
      if (tid < kBlock) {
        float amax = s_max[0][tid];
#pragma unroll
        for (int i = 1; i < 8; ++i) amax = fmaxf(amax, s_max[i][tid]);
        const int c = kb * kBlock + tid;
        const float w = c < K ? weight_at(a.weight, a.weight_f32, c) : 0.0f;
        const float s = group_scale(amax * fabsf(w));
        s_mul[tid] = __fdiv_rn(w, s);
        if (c < K) a.s_col[block * a.lds_col + c] = s;
      }
      __syncthreads();
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {  // column pairs
        const float2 mul = *reinterpret_cast<const float2*>(&s_mul[kVec * c8 + 2 * jj]);
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t wd = jj == 0 ? hv[i].x : jj == 1 ? hv[i].y : jj == 2 ? hv[i].z : hv[i].w;
          lo[i] = bf16_lo(wd) * rr[i] * mul.x;
          hi[i] = bf16_hi(wd) * rr[i] * mul.y;
        }
        const int c = kVec * c8 + 2 * jj;
        s_tile[c][g ^ 2 * c8] = codes4(lo[0], lo[1], lo[2], lo[3]);
        s_tile[c][(16 + g) ^ 2 * c8] = codes4(lo[4], lo[5], lo[6], lo[7]);
        s_tile[c + 1][g ^ 2 * c8] = codes4(hi[0], hi[1], hi[2], hi[3]);
        s_tile[c + 1][(16 + g) ^ 2 * c8] = codes4(hi[4], hi[5], hi[6], hi[7]);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (tid >> 4) + 16 * i, pair = tid & 15;
        const int64_t t = b0 + 8 * pair;
        const uint2 v = *reinterpret_cast<const uint2*>(&s_tile[c][2 * (pair ^ (c >> 3 & 15))]);
        if (kb * kBlock + c < K && t < a.T) {
          uint8_t* q = a.q_col + (int64_t)(kb * kBlock + c) * a.ldq_col + t;
          if (t + 8 <= a.T) {
            *reinterpret_cast<uint2*>(q) = v;
          } else {
#pragma unroll
            for (int b = 0; b < 8; ++b)
              if (t + b < a.T) q[b] = (uint8_t)((b < 4 ? v.x : v.y) >> (8 * (b & 3)));
          }
        }
      }
    }
  }
}

// Gradient of a run of rows a team; the teams' sums for the weight go to partial[team of the launch][K].
template <int VPT, bool VEC>
__global__ void __launch_bounds__(256, VPT <= 2 ? 3 : VPT <= 4 ? 2 : 1) rms_norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float s_slots[2][8];
  const Team team = team_of(a.team);
  const int K = (int)a.K, lane = team.lane;
  pdl_launch_dependents();
  pdl_wait();
  float dw[VPT][8] = {};
  int turn = 0;
  const int64_t me = (int64_t)blockIdx.x * team.count + team.index, teams = (int64_t)gridDim.x * team.count;
  for (int64_t first = (int64_t)blockIdx.x * team.count; first < a.T; first += teams, turn ^= 1) {
    const int64_t t = first + team.index;
    const bool live = t < a.T;
    uint4 hv[VPT], dv[VPT], rv[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int k = kVec * (u * team.size + lane);
      hv[u] = live ? load_row8<VEC>(a.h + t * a.ldh, k, K) : make_uint4(0, 0, 0, 0);
      dv[u] = live ? load_row8<VEC>(a.dy + t * a.lddy, k, K) : make_uint4(0, 0, 0, 0);
      rv[u] = live && a.dh ? load_row8<VEC>(a.dh + t * a.lddh, k, K) : make_uint4(0, 0, 0, 0);
    }
    const float r = live ? a.rstd[t] : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      float n[8], d[8], w[8];
      unpack8(hv[u], n);
      unpack8(dv[u], d);
      load_weight8<VEC>(a.weight, a.weight_f32, kVec * (u * team.size + lane), K, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] *= r;
        dw[u][i] = fmaf(d[i], n[i], dw[u][i]);
        sum = fmaf(d[i] * w[i], n[i], sum);
      }
    }
    const float mean = team_sum(sum, team, s_slots[turn]) / (float)K;
    if (live) {
#pragma unroll
      for (int u = 0; u < VPT; ++u) {
        const int k = kVec * (u * team.size + lane);
        float n[8], d[8], w[8], e[8];
        unpack8(hv[u], n);
        unpack8(dv[u], d);
        unpack8(rv[u], e);
        load_weight8<VEC>(a.weight, a.weight_f32, k, K, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = fmaf(r, d[i] * w[i] - n[i] * r * mean, e[i]);
        store_row8<VEC>(a.dx + t * a.lddx, k, K, pack8(e));
      }
    }
  }
  float* out = a.partial + me * K;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int k = kVec * (u * team.size + lane);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) out[k + i] = dw[u][i];
  }
}

// dw[k] = the teams' sums, added in their order: 32 columns a CTA, warp w the teams w, w + 32, ...
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float* partial, int64_t teams, int K, float* dw) {
  __shared__ double s[32][33];
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5, k = (int)blockIdx.x * 32 + lane;
  pdl_launch_dependents();
  pdl_wait();
  double sum = 0.0;
  if (k < K)
    for (int64_t i = warp; i < teams; i += 32) sum += partial[i * K + k];
  s[warp][lane] = sum;
  __syncthreads();
  double v = s[lane][warp];  // column `warp` of the CTA, over its 32 sums
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  if (lane == 0 && (int)blockIdx.x * 32 + warp < K) dw[(int)blockIdx.x * 32 + warp] = (float)v;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

static bool vec_ok(const void* p, int64_t ld) { return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0); }

// Threads a row: a power of two that covers K with `vpt` chunks each, at least a group's 16.
static int team_size(int64_t K, int vpt, int most) {
  int n = 16;
  while (n < most && (int64_t)n * vpt * kVec < K) n *= 2;
  return n;
}

template <int THREADS, int VPT, bool COLS>
static cudaError_t run_norm(NormArgs a, int64_t grid, cudaStream_t st) {
  const bool vec = a.K % 8 == 0 && vec_ok(a.x, a.ldx) && vec_ok(a.residual, a.ldr) && vec_ok(a.h, a.ldh) && vec_ok(a.y, a.ldy) &&
                   vec_ok(a.weight, 0);
  auto kernel = vec ? rms_norm_kernel<THREADS, VPT, true, COLS> : rms_norm_kernel<THREADS, VPT, false, COLS>;
  if constexpr (!COLS) {
    return launch_pdl(kernel, (unsigned)grid, THREADS, 0, st, a);
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  }
}

cudaError_t launch_rms_norm(const NormArgs& args, int num_sms, cudaStream_t st) {
  NormArgs a = args;
  const int64_t K = a.K;
  if (a.q_col) {
    a.cluster = 1;
    while (a.cluster < 8 && a.cluster < cdiv(K, kBlock)) a.cluster *= 2;
    const int64_t grid = cdiv(a.T, kBlock) * a.cluster;
    auto go = [&](auto vpt) {
      a.team = team_size(K, decltype(vpt)::value, 256);
      return run_norm<256, decltype(vpt)::value, true>(a, grid, st);
    };
    if (K <= 2048) return go(std::integral_constant<int, 1>{});
    if (K <= 4096) return go(std::integral_constant<int, 2>{});
    if (K <= 8192) return go(std::integral_constant<int, 4>{});
    return go(std::integral_constant<int, 8>{});
  }
  a.cluster = 1;
  if (a.T <= num_sms && K > 2048) {  // a row a CTA, as many threads as it has chunks
    if (K <= 4096) {
      a.team = 512;
      return run_norm<512, 1, false>(a, a.T, st);
    }
    a.team = 1024;
    if (K <= 8192) return run_norm<1024, 1, false>(a, a.T, st);
    return run_norm<1024, 2, false>(a, a.T, st);
  }
  auto go = [&](auto vpt) {
    constexpr int V = decltype(vpt)::value;
    a.team = team_size(K, V, 256);
    const int64_t ctas = cdiv(a.T, 256 / a.team), most = (int64_t)num_sms * 6;
    return run_norm<256, V, false>(a, ctas < most ? ctas : most, st);
  };
  if (K <= 2048) return go(std::integral_constant<int, 1>{});
  if (K <= 4096) return go(std::integral_constant<int, 2>{});
  if (K <= 8192) return go(std::integral_constant<int, 4>{});
  return go(std::integral_constant<int, 8>{});
}

NormBwdGeom norm_bwd_geom(int64_t T, int64_t K, int num_sms) {
  NormBwdGeom g;
  g.vpt = K <= 2048 ? 1 : K <= 4096 ? 2 : K <= 8192 ? 4 : 8;
  g.team = team_size(K, g.vpt, 256);
  const int64_t per = 256 / g.team, most = (int64_t)num_sms * 3;
  const int64_t ctas = cdiv(T, per * 4);  // four rows a team at least: each writes a row of sums
  g.grid = ctas < most ? ctas : most;
  g.teams = g.grid * per;
  return g;
}

cudaError_t launch_rms_norm_bwd(const NormBwdArgs& args, int num_sms, cudaStream_t st) {
  NormBwdArgs a = args;
  const NormBwdGeom g = norm_bwd_geom(a.T, a.K, num_sms);
  a.team = g.team;
  if (a.T > 0) {
    const bool vec = a.K % 8 == 0 && vec_ok(a.dy, a.lddy) && vec_ok(a.h, a.ldh) && vec_ok(a.dh, a.lddh) &&
                     vec_ok(a.dx, a.lddx) && vec_ok(a.weight, 0);
    auto go = [&](auto vpt) {
      constexpr int V = decltype(vpt)::value;
      return launch_pdl(vec ? rms_norm_bwd_kernel<V, true> : rms_norm_bwd_kernel<V, false>, (unsigned)g.grid, 256, 0, st, a);
    };
    const cudaError_t e = g.vpt == 1   ? go(std::integral_constant<int, 1>{})
                          : g.vpt == 2 ? go(std::integral_constant<int, 2>{})
                          : g.vpt == 4 ? go(std::integral_constant<int, 4>{})
                                       : go(std::integral_constant<int, 8>{});
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(rms_norm_dw_kernel, (unsigned)cdiv(a.K, 32), 1024, 0, st, (const float*)a.partial, g.teams, (int)a.K, a.dweight);
}

}  // namespace bfp8
