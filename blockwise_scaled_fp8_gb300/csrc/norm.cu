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
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

static __device__ uint32_t g_norm_error;

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kNormWarps = 12, kNormMaxSlots = 32;
constexpr int kVec = 8;  // features a thread takes side by side: 16 bytes of bf16, 16 threads a group of 128

struct Team {
  int size, lane, index, count;  // threads a row, this thread's place, this thread's team, teams a CTA
};
__device__ __forceinline__ Team team_of(int size) {
  const int tid = (int)threadIdx.x;
  return Team{size, tid & (size - 1), tid / size, (int)blockDim.x / size};
}

// 16 bytes, not by the read-only path (a row may be written in place by the same thread).
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
// Keeps the compiler from carrying what it derived from the values (their fp32 forms, twice the registers) past here.
template <int N>
__device__ __forceinline__ void only_packed(uint4 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i].x), "+r"(v[i].y), "+r"(v[i].z), "+r"(v[i].w));
}
// Eight bf16 as four pairs of fp32.
__device__ __forceinline__ void pairs8(const uint4& v, uint64_t (&p)[4]) {
  p[0] = f2_pack(bf16_lo(v.x), bf16_hi(v.x));
  p[1] = f2_pack(bf16_lo(v.y), bf16_hi(v.y));
  p[2] = f2_pack(bf16_lo(v.z), bf16_hi(v.z));
  p[3] = f2_pack(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ float weight_at(const void* w, int f32, int64_t k) {
  return f32 ? __ldg(static_cast<const float*>(w) + k)
             : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(w) + k) << 16);
}
// Eight weights from feature k on as four pairs, zeros past the end.
template <bool VEC>
__device__ __forceinline__ void load_weight8(const void* w, int f32, int k, int K, uint64_t (&f)[4]) {
  if constexpr (VEC) {
    if (k >= K) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = 0;
    } else if (f32) {
      const ulonglong2* p = reinterpret_cast<const ulonglong2*>(static_cast<const float*>(w) + k);
      const ulonglong2 a = __ldg(p), b = __ldg(p + 1);
      f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    } else {
      pairs8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + k)), f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = f2_pack(k + 2 * i < K ? weight_at(w, f32, k + 2 * i) : 0.0f, k + 2 * i + 1 < K ? weight_at(w, f32, k + 2 * i + 1) : 0.0f);
  }
}

// Eight bf16 + eight bf16, rounded to bf16.
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
  uint64_t p[4], q[4];
  pairs8(a, p);
  pairs8(b, q);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f2_add(p[i], q[i]), lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// sum + the squares of eight bf16, even and odd ones apart.
__device__ __forceinline__ uint64_t squares8(const uint4& a, uint64_t sum) {
  uint64_t p[4];
  pairs8(a, p);
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = f2_fma(p[i], p[i], sum);
  return sum;
}
__device__ __forceinline__ float f2_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ void times8(const uint4& a, const uint64_t (&w)[4], uint64_t (&v)[4]) {
  pairs8(a, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2_mul(v[i], w[i]);
}
__device__ __forceinline__ void row_times(const uint4& a, float r, uint64_t (&v)[4]) {
  pairs8(a, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2_mul(v[i], f2_pack(r, r));
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float amax8(const uint64_t (&v)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(v[i], lo, hi);
    m = max3_abs(m, lo, hi);
  }
  return m;
}
__device__ __forceinline__ uint4 scaled_bf16(const uint64_t (&v)[4], float r) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f2_mul(v[i], f2_pack(r, r)), lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Four e4m3 codes (RNE, saturating), the first in the lowest byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return cvt_e4m3x2(a, b) | cvt_e4m3x2(c, d) << 16;
}
// The codes of v m at feature k of a row of codes.
__device__ __forceinline__ void store_codes8(uint8_t* row, int k, int K, const uint64_t (&v)[4], float m) {
  if (k >= K) return;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(f2_mul(v[i], f2_pack(m, m)), f[2 * i], f[2 * i + 1]);
  const uint32_t lo = codes4(f[0], f[1], f[2], f[3]), hi = codes4(f[4], f[5], f[6], f[7]);
  if (k + kVec <= K) {
    *reinterpret_cast<uint2*>(row + k) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (k + i < K) row[k + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
}
__device__ __forceinline__ float rstd_of(float sum, int K, float eps) {
  return __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)K) + eps));
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void lds_2x64(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
// `bytes` (a multiple of 16, both addresses 16-byte aligned) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// The sum of v over a team's threads, the same bits in each of them.  `slots`: one of
// two sets of a float a warp, used in turn, so that one barrier a sum is enough.
__device__ __forceinline__ float team_sum(float v, const Team& t, float* slots) {
  for (int o = min(t.size, 32) >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  if (t.size <= 32) return v;
  const int warp = (int)threadIdx.x >> 5, warps = t.size >> 5;
  if ((threadIdx.x & 31) == 0) slots[warp] = v;
  __syncthreads();
  const int lane = (int)threadIdx.x & 31;
  float sum = lane < warps ? slots[t.index * warps + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  return sum;
}

}  // namespace

// The row a thread's chunks make up, from its values to its outputs.
template <int VPT, bool VEC>
__device__ __forceinline__ void finish_row(const NormArgs& a, const Team& team, int64_t t, bool live, const uint4 (&hv)[VPT],
                                           float r) {
  const int K = (int)a.K;
  if (live && team.lane == 0) a.rstd[t] = r;
  if (!a.q_row && !a.y) return;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int k = kVec * (u * team.size + team.lane);
    uint64_t w2[4], v2[4];
    load_weight8<VEC>(a.weight, a.weight_f32, k, K, w2);
    times8(hv[u], w2, v2);
    if (a.y && live) store_row8<VEC>(a.y + t * a.ldy, k, K, scaled_bf16(v2, r));
    if (a.q_row) {
      float amax = amax8(v2);
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
      const float s = group_scale(amax * r);
      if (live) {
        store_codes8(a.q_row + t * a.ldq_row, k, K, v2, __fdiv_rn(r, s));
        if ((team.lane & 15) == 0 && k < K) a.s_row[(int64_t)(k / kBlock) * a.lds_row + t] = s;
      }
    }
  }
}

// One row a team of threads, each thread VPT chunks of eight features (chunk u of a
// thread starts at feature 8 (u size + lane)): few rows, and rows that are not
// 16-byte aligned.
template <int THREADS, int VPT, bool VEC>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 4 : THREADS <= 512 ? 2 : 1) rms_norm_kernel(const NormArgs a) {
  __shared__ float s_slots[THREADS / 32];
  const Team team = team_of(a.team);
  const int K = (int)a.K;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = (int64_t)blockIdx.x * team.count + team.index;
  const bool live = t < a.T;
  uint4 hv[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u)
    hv[u] = live ? load_row8<VEC>(a.x + t * a.ldx, kVec * (u * team.size + team.lane), K) : make_uint4(0, 0, 0, 0);
  if (a.residual && live) {
    uint4 rv[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u) rv[u] = load_row8<VEC>(a.residual + t * a.ldr, kVec * (u * team.size + team.lane), K);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      hv[u] = add8(hv[u], rv[u]);
      store_row8<VEC>(a.h + t * a.ldh, kVec * (u * team.size + team.lane), K, hv[u]);
    }
  }
  uint64_t sum2 = 0;
#pragma unroll
  for (int u = 0; u < VPT; ++u) sum2 = squares8(hv[u], sum2);
  finish_row<VPT, VEC>(a, team, t, live, hv, rstd_of(team_sum(f2_sum(sum2), team, s_slots), K, a.eps));
}

// Many aligned rows: one CTA an SM, a warp a row, and no barrier between warps.  Rows
// arrive by bulk copies in slots that hold all of shared memory, whatever the
// threads are waiting for; row i of a CTA is slot i % slots and warp i % warps, and
// the warp that is done with a row asks for the one that takes its slot.  A row is
// read twice from its slot (the sum of the residual goes back into it): once for its
// squares, once for its codes, four chunks of 256 features at a time, whose eight
// groups' maxima a halving exchange leaves in a lane each.
__global__ void __launch_bounds__(32 * kNormWarps, 1) rms_norm_ring_kernel(const NormArgs a) {
  extern __shared__ __align__(128) uint8_t s_ring[];  // weights, then the slots: [x, residual][K]
  __shared__ uint64_t s_full[kNormMaxSlots];
  const int K = (int)a.K, tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31, slots = a.slots;
  const int warps = slots < kNormWarps ? slots : kNormWarps;  // that have rows
  const uint32_t row_bytes = 2u * (uint32_t)K, slot_bytes = row_bytes * (a.residual ? 2u : 1u), weight_bytes = a.weight_f32 ? 2u * row_bytes : row_bytes;
  const uint32_t weights = smem_u32(s_ring), ring = weights + (weight_bytes + 127u) / 128u * 128u, full = smem_u32(s_full);
  const int64_t rows = a.T > blockIdx.x ? cdiv(a.T - blockIdx.x, (int64_t)gridDim.x) : 0;  // of this CTA: every grid-th
  const volatile int never = 0;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(full + 8 * i, 1);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  __syncthreads();
  pdl_wait();
  auto issue = [&](int64_t i, int slot) {
    const int64_t t = blockIdx.x + i * gridDim.x;
    const uint32_t to = ring + (uint32_t)slot * slot_bytes;
    mbar_arrive_expect_tx(full + 8 * slot, slot_bytes);
    bulk_load(to, a.x + t * a.ldx, row_bytes, full + 8 * slot);
    if (a.residual) bulk_load(to + row_bytes, a.residual + t * a.ldr, row_bytes, full + 8 * slot);
  };
  if (tid == 0)
    for (int i = 0; i < slots && i < rows; ++i) issue(i, i);
  for (uint32_t i = 16u * (uint32_t)tid; i < weight_bytes; i += 16u * blockDim.x) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.weight) + i));
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(weights + i), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
  }
  __syncthreads();
  if (warp >= warps) return;
  int slot = warp;  // warps <= slots
  uint32_t parity = 0;
  for (int64_t i = warp; i < rows; i += warps) {
    const int64_t t = blockIdx.x + i * gridDim.x;
    const uint32_t from = ring + (uint32_t)slot * slot_bytes;
    if (!__all_sync(kAll, mbar_wait_bounded(full + 8 * slot, parity, kWaitLimitNs, &never))) {
      if (lane == 0) atomicOr(&g_norm_error, 1u);
      break;  // (the copies have not landed after four seconds: nothing is left to wait for)
    }
    uint64_t sum2 = 0;
#pragma unroll 4
    for (int k = kVec * lane; k < K; k += 32 * kVec) {
      uint4 h = lds_v4(from + 2u * (uint32_t)k);
      if (a.residual) {
        h = add8(h, lds_v4(from + row_bytes + 2u * (uint32_t)k));
        *reinterpret_cast<uint4*>(a.h + t * a.ldh + k) = h;
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(from + 2u * (uint32_t)k), "r"(h.x), "r"(h.y), "r"(h.z),
                     "r"(h.w)
                     : "memory");
      }
      sum2 = squares8(h, sum2);
    }
    float sum = f2_sum(sum2);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    const float r = rstd_of(sum, K, a.eps);
    if (lane == 0) a.rstd[t] = r;
    if (a.q_row || a.y) {
      for (int k0 = 0; k0 < K; k0 += 4 * 32 * kVec) {
        uint64_t v[4][4];
        float am[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = k0 + kVec * (32 * u + lane);
          uint64_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[u][j] = w[j] = 0;
          if (k < K) {
            if (a.weight_f32) {
              lds_2x64(weights + 4u * (uint32_t)k, w[0], w[1]);
              lds_2x64(weights + 4u * (uint32_t)k + 16u, w[2], w[3]);
            } else {
              pairs8(lds_v4(weights + 2u * (uint32_t)k), w);
            }
            times8(lds_v4(from + 2u * (uint32_t)k), w, v[u]);
          }
          am[u] = amax8(v[u]);
        }
        if (a.y) {
#pragma unroll
          for (int u = 0; u < 4; ++u) store_row8<true>(a.y + t * a.ldy, k0 + kVec * (32 * u + lane), K, scaled_bf16(v[u], r));
        }
        if (a.q_row) {
          // lane l: chunk u = (l & 8 ? 2 : 0) + (l & 4 ? 1 : 0), group l / 16 of it
          const bool up8 = (lane & 8) != 0, up4 = (lane & 4) != 0;
          float m0 = fmaxf(up8 ? am[2] : am[0], __shfl_xor_sync(kAll, up8 ? am[0] : am[2], 8));
          float m1 = fmaxf(up8 ? am[3] : am[1], __shfl_xor_sync(kAll, up8 ? am[1] : am[3], 8));
          float m = fmaxf(up4 ? m1 : m0, __shfl_xor_sync(kAll, up4 ? m0 : m1, 4));
          m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
          m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
          const float s = group_scale(m * r), mul = __fdiv_rn(r, s);
          const int g = k0 / kBlock + (up8 ? 4 : 0) + (up4 ? 2 : 0) + (lane >> 4);
          if ((lane & 3) == 0 && g * kBlock < K) a.s_row[(int64_t)g * a.lds_row + t] = s;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float mu = __shfl_sync(kAll, mul, (lane & 16) | (u & 2 ? 8 : 0) | (u & 1 ? 4 : 0));
            store_codes8(a.q_row + t * a.ldq_row, k0 + kVec * (32 * u + lane), K, v[u], mu);
          }
        }
      }
    }
    fence_proxy_async_shared();  // this row's reads and writes of the slot, before the copy that takes it
    __syncwarp();
    if (lane == 0 && i + slots < rows) issue(i + slots, slot);
    slot += warps;
    if (slot >= slots) slot -= slots, parity ^= 1u;
  }
}

// Codes along the columns, from h and rstd: a CTA a 128 x 128 tile, a thread eight
// columns of 2 x 4 rows.  The row blocks are taken last first: what the rows' pass
// wrote last is still in L2.
template <bool VEC>
__global__ void __launch_bounds__(256, 4) rms_norm_cols_kernel(const NormArgs a) {
  __shared__ float s_max[8][kBlock], s_mul[kBlock], s_r[kBlock];
  __shared__ uint32_t s_tile[kBlock][32];  // codes [column][four rows], word w of column c at w ^ 2 (c / 8 % 16)
  const int tid = (int)threadIdx.x, warp = tid >> 5, c8 = tid & 15, g = tid >> 4, K = (int)a.K;
  const int col_blocks = (int)cdiv(K, kBlock);
  const int64_t row_blocks = cdiv(a.T, kBlock), block = row_blocks - 1 - (int64_t)blockIdx.x / col_blocks;
  const int kb = (int)((int64_t)blockIdx.x % col_blocks);
  const int64_t b0 = block * kBlock;
  const int k = kb * kBlock + kVec * c8;
  const uint16_t* stream = a.residual ? a.h : a.x;
  const int64_t ld = a.residual ? a.ldh : a.ldx;
  pdl_launch_dependents();
  pdl_wait();
  uint4 hv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t t = b0 + 4 * g + (i & 3) + 64 * (i >> 2);
    hv[i] = t < a.T ? load_row8<VEC>(stream + t * ld, k, K) : make_uint4(0, 0, 0, 0);
  }
  if (tid < kBlock) s_r[tid] = b0 + tid < a.T ? a.rstd[b0 + tid] : 0.0f;
  __syncthreads();
  float rr[8];  // of this thread's rows 4g .. 4g + 3 and 64 + 4g ..
  *reinterpret_cast<float4*>(rr) = *reinterpret_cast<const float4*>(s_r + 4 * g);
  *reinterpret_cast<float4*>(rr + 4) = *reinterpret_cast<const float4*>(s_r + 64 + 4 * g);
  float m[8] = {};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    uint64_t p[4], q[4];
    row_times(hv[i], rr[i], p);
    row_times(hv[i + 1], rr[i + 1], q);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float p0, p1, q0, q1;
      f2_unpack(p[j], p0, p1);
      f2_unpack(q[j], q0, q1);
      m[2 * j] = max3_abs(m[2 * j], p0, q0);
      m[2 * j + 1] = max3_abs(m[2 * j + 1], p1, q1);
    }
  }
  only_packed(hv);
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
  for (int j = 0; j < 4; ++j) {  // column pairs
    const uint64_t mul = *reinterpret_cast<const uint64_t*>(&s_mul[kVec * c8 + 2 * j]);
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = j == 0 ? hv[i].x : j == 1 ? hv[i].y : j == 2 ? hv[i].z : hv[i].w;
      f2_unpack(f2_mul(f2_mul(f2_pack(bf16_lo(w), bf16_hi(w)), f2_pack(rr[i], rr[i])), mul), lo[i], hi[i]);
    }
    const int c = kVec * c8 + 2 * j;
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
        for (int b = 0; b < 7; ++b)
          if (t + b < a.T) q[b] = (uint8_t)((b < 4 ? v.x : v.y) >> (8 * (b & 3)));
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
      uint64_t w2[4];
      load_weight8<VEC>(a.weight, a.weight_f32, kVec * (u * team.size + lane), K, w2);
#pragma unroll
      for (int i = 0; i < 4; ++i) f2_unpack(w2[i], w[2 * i], w[2 * i + 1]);
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
        uint64_t w2[4];
        load_weight8<VEC>(a.weight, a.weight_f32, k, K, w2);
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(w2[i], w[2 * i], w[2 * i + 1]);
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

// dw[k] = the teams' sums, added in their order: 32 columns a CTA, warp w the teams w, w + 32, ..; each warp's sum keeps
// what its additions lose (T. J. Dekker's fast two-sum needs the larger first, so D. E. Knuth's), in fp32, since this part
// adds few fp64 numbers a cycle (15 us for 456 sums of 4096 that way).
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float* partial, int64_t teams, int K, float* dw) {
  __shared__ float s[32][33];
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5, k = (int)blockIdx.x * 32 + lane;
  pdl_launch_dependents();
  pdl_wait();
  float sum = 0.0f, lost = 0.0f;
  auto add = [&](float v) {
    const float to = __fadd_rn(sum, v), back = __fsub_rn(to, sum);
    lost = __fadd_rn(lost, __fadd_rn(__fsub_rn(sum, __fsub_rn(to, back)), __fsub_rn(v, back)));
    sum = to;
  };
  if (k < K) {
    for (int64_t i = warp; i < teams; i += 8 * 32) {  // (eight loads in flight)
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = i + 32 * j < teams ? partial[(i + 32 * j) * K + k] : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) add(v[j]);
    }
  }
  s[warp][lane] = sum + lost;
  __syncthreads();
  float v = s[lane][warp];  // column `warp` of the CTA, over its 32 sums
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  if (lane == 0 && (int)blockIdx.x * 32 + warp < K) dw[(int)blockIdx.x * 32 + warp] = v;
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

static bool norm_vec(const NormArgs& a) {
  return a.K % 8 == 0 && vec_ok(a.x, a.ldx) && vec_ok(a.residual, a.ldr) && vec_ok(a.h, a.ldh) && vec_ok(a.y, a.ldy) &&
         vec_ok(a.weight, 0);
}

template <int THREADS, int VPT>
static cudaError_t run_norm(const NormArgs& a, int64_t grid, cudaStream_t st) {
  return launch_pdl(norm_vec(a) ? rms_norm_kernel<THREADS, VPT, true> : rms_norm_kernel<THREADS, VPT, false>, (unsigned)grid,
                    THREADS, 0, st, a);
}

static cudaError_t run_norm_ring(NormArgs a, int num_sms, cudaStream_t st) {
  constexpr int64_t most = 220 * 1024;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(rms_norm_ring_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  });
  if (attr_err != cudaSuccess) return attr_err;
  const int64_t weights = cdiv(a.K * (a.weight_f32 ? 4 : 2), 128) * 128, slot = a.K * 2 * (a.residual ? 2 : 1);
  const int64_t fit = (most - weights) / slot;  // (two of the largest rows)
  a.slots = (int)(fit < kNormMaxSlots ? fit : kNormMaxSlots);
  return launch_pdl(rms_norm_ring_kernel, (unsigned)(a.T < num_sms ? a.T : num_sms), 32 * kNormWarps,
                    (size_t)(weights + a.slots * slot), st, a);
}

static cudaError_t norm_rows(NormArgs a, int num_sms, cudaStream_t st) {
  const int64_t K = a.K;
  if (a.T <= num_sms && K > 2048) {  // a row a CTA, as many threads as it has chunks
    if (K <= 4096) {
      a.team = 512;
      return run_norm<512, 1>(a, a.T, st);
    }
    a.team = 1024;
    return K <= 8192 ? run_norm<1024, 1>(a, a.T, st) : run_norm<1024, 2>(a, a.T, st);
  }
  if (norm_vec(a) && K >= 512 && a.T > num_sms) return run_norm_ring(a, num_sms, st);
  auto go = [&](auto threads, auto vpt) {
    constexpr int N = decltype(threads)::value, V = decltype(vpt)::value;
    a.team = team_size(K, V, N);
    return run_norm<N, V>(a, cdiv(a.T, N / a.team), st);
  };
  if (K <= 2048) return go(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (K <= 4096) return go(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (K <= 8192) return go(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t st) {
  const cudaError_t e = norm_rows(a, num_sms, st);
  if (e != cudaSuccess || !a.q_col) return e;
  const unsigned tiles = (unsigned)(cdiv(a.T, kBlock) * cdiv(a.K, kBlock));
  const bool vec = a.K % 8 == 0 && (a.residual ? vec_ok(a.h, a.ldh) : vec_ok(a.x, a.ldx));
  return launch_pdl(vec ? rms_norm_cols_kernel<true> : rms_norm_cols_kernel<false>, tiles, 256, 0, st, a);
}

cudaError_t norm_read_errors(uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_norm_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(uint32_t));
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
