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
//
// What bounds them is memory: each input once and each output once, but for the
// codes along the columns, which need 128 rows of h after every row's rstd is known:
// a second pass reads h again (10 bytes an element for 8).  One launch instead (a
// cluster of CTAs for 128 rows, which reads them again from L2 once its sums of
// squares are joined) took 203 us for both codes of 16384 x 4096 with residual; the
// two passes take 116: the rows' codes 78 (6.0 TB/s), the columns' 38 (5.3).  The
// gradient with the sum of its partial dw takes 90 (6.0 TB/s); a plain copy of such
// sizes moves 6.2-6.7 TB/s.
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

static __device__ uint32_t g_norm_error;

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kNormWarps = 16, kNormMaxSlots = 32;
constexpr int kBwdMaxStages = 8;
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
// The four words that start `sh` (0 or 16) bits into the five.
__device__ __forceinline__ uint4 shift_words(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t sh) {
  return make_uint4(__funnelshift_r(a, b, sh), __funnelshift_r(b, c, sh), __funnelshift_r(c, d, sh), __funnelshift_r(d, e, sh));
}
// The eight bf16 that start `off` bytes (even) into the 32, zeros after the first n.
__device__ __forceinline__ uint4 shifted8(const uint4& a, const uint4& b, int off, int n) {
  const uint32_t sh = 8u * (uint32_t)(off & 2);
  uint4 out;
  switch (off >> 2) {  // (the same for a whole row)
    case 0: out = shift_words(a.x, a.y, a.z, a.w, b.x, sh); break;
    case 1: out = shift_words(a.y, a.z, a.w, b.x, b.y, sh); break;
    case 2: out = shift_words(a.z, a.w, b.x, b.y, b.z, sh); break;
    default: out = shift_words(a.w, b.x, b.y, b.z, b.w, sh);
  }
  if (n < kVec) {
    out.x = n >= 2 ? out.x : n == 1 ? out.x & 0xFFFFu : 0u;
    out.y = n >= 4 ? out.y : n == 3 ? out.y & 0xFFFFu : 0u;
    out.z = n >= 6 ? out.z : n == 5 ? out.z & 0xFFFFu : 0u;
    out.w = n == 7 ? out.w & 0xFFFFu : 0u;
  }
  return out;
}
// Eight bf16 of a row from feature k on, zeros past its end.
template <bool VEC>
__device__ __forceinline__ uint4 load_row8(const uint16_t* row, int k, int K) {
  if constexpr (VEC) {
    return k < K ? ld_v4(row + k) : make_uint4(0, 0, 0, 0);
  } else {
    // the two aligned 16 bytes that hold them, shifted (each holds one of the row's elements at least, or is not read)
    if (k >= K) return make_uint4(0, 0, 0, 0);
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
    const int off = (int)(at & 15);
    const uint4* p = reinterpret_cast<const uint4*>(at - off);
    const uint4 a = ld_v4(p);
    uint4 b = make_uint4(0, 0, 0, 0);
    if (k + (16 - off) / 2 < K) b = ld_v4(p + 1);
    return shifted8(a, b, off, K - k);
  }
}
template <bool VEC>
__device__ __forceinline__ void store_row8(uint16_t* row, int k, int K, const uint4& v) {
  if (VEC) {
    if (k < K) *reinterpret_cast<uint4*>(row + k) = v;
    return;
  }
  uint16_t* to = row + k;
  if (k + kVec <= K) {  // 32 bits at a time where they are aligned
    if ((reinterpret_cast<uintptr_t>(to) & 2) == 0) {
      uint32_t* p = reinterpret_cast<uint32_t*>(to);
      p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
    } else {
      uint32_t* p = reinterpret_cast<uint32_t*>(to + 1);
      to[0] = (uint16_t)v.x;
      p[0] = __funnelshift_r(v.x, v.y, 16), p[1] = __funnelshift_r(v.y, v.z, 16), p[2] = __funnelshift_r(v.z, v.w, 16);
      to[7] = (uint16_t)(v.w >> 16);
    }
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (k + i < K) to[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}
// A warp's eight elements a lane of N chunks of 256 side by side, chunk u's from feature k0 + 256 u on, to a row.  Where
// the row is not aligned, a lane writes the 16-byte block that its elements share with the lane's before it (a
// write of 4 bytes in each 16 of a row passes L2 four times), and only the run's two ends go element by element.
template <bool VEC, int N>
__device__ __forceinline__ void store_run(uint16_t* row, int k0, int K, const uint4 (&v)[N]) {
  const int lane = (int)threadIdx.x & 31;
  const int off = VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(row + k0) & 15), head = off >> 1;  // (the same for a warp)
  if (off == 0) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int k = k0 + kVec * (32 * u + lane);
      if (VEC || k + kVec <= K) store_row8<true>(row, k, K, v[u]);
      else store_row8<false>(row, k, K, v[u]);
    }
    return;
  }
  uint4 carry = make_uint4(0, 0, 0, 0);  // lane 0's: the last lane's elements of the chunk before
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int k = k0 + kVec * (32 * u + lane), from = (lane + 31) & 31;
    uint4 p;
    p.x = __shfl_sync(kAll, v[u].x, from);
    p.y = __shfl_sync(kAll, v[u].y, from);
    p.z = __shfl_sync(kAll, v[u].z, from);
    p.w = __shfl_sync(kAll, v[u].w, from);
    const uint4 before = lane == 0 ? carry : p;
    carry = p;
    // elements k - head .. k - head + 7, of which the run's first block holds 8 - head only
    const uint4 block = shifted8(before, v[u], 16 - off, kVec);
    const int first = u == 0 && lane == 0 ? k : k - head, last = min(k - head + kVec, K);
    if (first == k - head && last == k - head + kVec) {
      *reinterpret_cast<uint4*>(row + k - head) = block;
    } else {
      const uint32_t w[4] = {block.x, block.y, block.z, block.w};
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (k - head + i >= first && k - head + i < last) row[k - head + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  }
  if (lane == 0) {  // the last lane's last elements
    const int k = k0 + 256 * N - head;
    const uint32_t w[4] = {carry.x, carry.y, carry.z, carry.w};
#pragma unroll
    for (int i = 1; i < kVec; ++i)
      if (i >= kVec - head && k + i - (kVec - head) < K) row[k + i - (kVec - head)] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
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
template <bool WHOLE = false>
__device__ __forceinline__ void store_codes8(uint8_t* row, int k, int K, const uint64_t (&v)[4], float m) {
  if (!WHOLE && k >= K) return;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(f2_mul(v[i], f2_pack(m, m)), f[2 * i], f[2 * i + 1]);
  const uint32_t lo = codes4(f[0], f[1], f[2], f[3]), hi = codes4(f[4], f[5], f[6], f[7]);
  if (WHOLE || k + kVec <= K) {
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
// The weights in shared memory, in fp32 (zeros up to a whole chunk), and eight of them from feature k on, k below that.
__host__ __device__ __forceinline__ uint32_t staged_bytes(int K) { return ((uint32_t)K * 4u + 127u) / 128u * 128u; }
__device__ __forceinline__ void stage_weights(const void* w, int f32, int K, uint32_t to) {
  const int padded = (K + kVec - 1) / kVec * kVec;
  if (f32 && K == padded && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
    for (uint32_t i = 16u * threadIdx.x; i < (uint32_t)K * 4u; i += 16u * blockDim.x) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(w) + i));
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + i), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    }
  } else {
    for (int i = (int)threadIdx.x; i < padded; i += (int)blockDim.x)
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + 4u * (uint32_t)i), "f"(i < K ? weight_at(w, f32, i) : 0.0f) : "memory");
  }
}
__device__ __forceinline__ void staged_weight8(uint32_t from, int k, uint64_t (&w)[4]) {
  lds_2x64(from + 4u * (uint32_t)k, w[0], w[1]);
  lds_2x64(from + 4u * (uint32_t)k + 16u, w[2], w[3]);
}
// A row in shared memory as bulk copies bring it: the 16-byte blocks that hold it, its first element `off` bytes into them
// (0 where it is aligned).  Each block holds a byte of the row, so no copy leaves the tensor's own 16-byte blocks.
__host__ __device__ __forceinline__ uint32_t row_space(int K, bool aligned) {
  return aligned ? 2u * (uint32_t)K : (2u * (uint32_t)K + 15u) / 16u * 16u + 32u;
}
template <bool ALIGNED>
__device__ __forceinline__ int row_off(const uint16_t* row) {
  return ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(row) & 15);
}
template <bool ALIGNED>
__device__ __forceinline__ uint32_t row_copied(const uint16_t* row, int K) {  // bytes
  return ALIGNED ? 2u * (uint32_t)K : ((uint32_t)row_off<false>(row) + 2u * (uint32_t)K + 15u) / 16u * 16u;
}
template <bool ALIGNED>
__device__ __forceinline__ uint4 lds_row8(uint32_t from, int off, int k, int K) {
  if (k >= K) return make_uint4(0, 0, 0, 0);
  if constexpr (ALIGNED) return lds_v4(from + 2u * (uint32_t)k);
  return shifted8(lds_v4(from + 2u * (uint32_t)k), lds_v4(from + 2u * (uint32_t)k + 16u), off, K - k);
}
// `bytes` (a multiple of 16, both addresses 16-byte aligned) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
// Until the slot was asked to take its `turn`-th row: then that row's phase of its barrier is the running one or the last
// (a team ahead of the others could ask for a row whose slot still waits for the one before, and the parity of an older
// phase would answer).
__device__ __forceinline__ bool wait_asked(const volatile int* asked, int turn, const volatile int* abort) {
  if (*asked > turn) return true;
  const uint64_t t0 = globaltimer_ns();
  while (*asked <= turn)
    if (*abort || globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}
// Behind a CTA's last barrier, where a wait gave up: copies that were asked for land before its shared memory goes away.
__device__ __forceinline__ void drain(uint32_t full, const int* asked, int slots) {
  const int never = 0;
  for (int i = 0; i < slots; ++i)
    if (asked[i] > 0) mbar_wait_bounded(full + 8 * i, (uint32_t)(asked[i] - 1) & 1u, kWaitLimitNs, &never);
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
// thread starts at feature 8 (u size + lane)): no more rows than SMs, or fewer than
// 512 features.
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

// Many rows: one CTA an SM, a team of one, two or four warps a row (so that
// the rows that fit keep every warp busy), and no barrier between teams.  Rows
// arrive by bulk copies in slots that hold all of shared memory, whatever the
// threads are waiting for; row i of a CTA is slot i % slots and team i % teams, and
// the team that is done with a row asks for the one that takes its slot.  A row is
// read twice from its slot, where it is kept (with the residual, and aligned): once for its
// squares, once for its codes, four chunks of 256 features at a time, whose eight
// groups' maxima a halving exchange leaves in a lane each.
template <bool ALIGNED>
__global__ void __launch_bounds__(32 * kNormWarps, 1) rms_norm_ring_kernel(const NormArgs a) {
  extern __shared__ __align__(128) uint8_t s_ring[];  // weights, then the slots: [x, residual][K]
  __shared__ uint64_t s_full[kNormMaxSlots];
  __shared__ float s_sum[kNormWarps];
  __shared__ int s_abort, s_asked[kNormMaxSlots];  // rows that a slot was asked to take
  const int K = (int)a.K, tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31, slots = a.slots;
  const int size = a.team, teams = min(slots, kNormWarps / size), team = warp / size, sub = warp % size;
  const uint32_t space = row_space(K, ALIGNED), slot_bytes = space * (a.residual ? 2u : 1u);
  const uint32_t weights = smem_u32(s_ring), ring = weights + staged_bytes(K), full = smem_u32(s_full);
  const int64_t rows = a.T > blockIdx.x ? cdiv(a.T - blockIdx.x, (int64_t)gridDim.x) : 0;  // of this CTA: every grid-th
  volatile int* abort_flag = &s_abort;
  pdl_launch_dependents();
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < slots; ++i) mbar_init(full + 8 * i, 1), s_asked[i] = 0;
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  __syncthreads();
  pdl_wait();
  auto issue = [&](int64_t i, int slot) {
    const int64_t t = blockIdx.x + i * gridDim.x;
    const uint32_t to = ring + (uint32_t)slot * slot_bytes;
    const uint16_t *x = a.x + t * a.ldx, *r = a.residual ? a.residual + t * a.ldr : nullptr;
    const uint32_t x_bytes = row_copied<ALIGNED>(x, K), r_bytes = r ? row_copied<ALIGNED>(r, K) : 0u;
    mbar_arrive_expect_tx(full + 8 * slot, x_bytes + r_bytes);
    *(volatile int*)(s_asked + slot) = s_asked[slot] + 1;
    bulk_load(to, x - row_off<ALIGNED>(x) / 2, x_bytes, full + 8 * slot);
    if (r) bulk_load(to + space, r - row_off<ALIGNED>(r) / 2, r_bytes, full + 8 * slot);
  };
  if (tid == 0)
    for (int i = 0; i < slots && i < rows; ++i) issue(i, i);
  stage_weights(a.weight, a.weight_f32, K, weights);
  __syncthreads();
  auto team_sync = [&]() {
    if (size > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * size) : "memory");
    else __syncwarp();
  };
  int slot = team, turn = 0;  // teams <= slots
  for (int64_t i = team < teams ? team : rows; i < rows; i += teams) {
    const int64_t t = blockIdx.x + i * gridDim.x;
    const uint32_t from = ring + (uint32_t)slot * slot_bytes;
    // (a wait that gives up leaves the error word set and wrong rows from there on, without further waits or copies)
    if (!wait_asked(s_asked + slot, turn, abort_flag) ||
        !mbar_wait_bounded(full + 8 * slot, (uint32_t)turn & 1u, kWaitLimitNs, abort_flag)) {
      atomicOr(&g_norm_error, 1u);
      *abort_flag = 1;
    }
    uint64_t sum2 = 0;
    const int off_x = row_off<ALIGNED>(a.x + t * a.ldx), off_r = a.residual ? row_off<ALIGNED>(a.residual + t * a.ldr) : 0;
    auto keep = [&](int k, const uint4& h) {
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(from + 2u * (uint32_t)k), "r"(h.x), "r"(h.y), "r"(h.z),
                   "r"(h.w)
                   : "memory");
    };
    if constexpr (ALIGNED) {
      const int step = 32 * kVec * size;
      auto take = [&](int k) {
        uint4 h = lds_v4(from + 2u * (uint32_t)k);
        if (a.residual) {
          h = add8(h, lds_v4(from + space + 2u * (uint32_t)k));
          *reinterpret_cast<uint4*>(a.h + t * a.ldh + k) = h;
          keep(k, h);
        }
        sum2 = squares8(h, sum2);
      };
      int k = kVec * (32 * sub + lane);
      for (; k + 3 * step < K; k += 4 * step) {
#pragma unroll
        for (int u = 0; u < 4; ++u) take(k + u * step);
      }
      for (; k < K; k += step) take(k);
    } else {
      // 1024 features a warp and step; a step's blocks, which reach into the next step's first one, are read by the whole
      // team before they are written
      for (int k00 = 0; k00 < K; k00 += 4 * 32 * kVec * size) {
        const int k0 = k00 + 4 * 32 * kVec * sub;
        uint4 h[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = k0 + kVec * (32 * u + lane);
          h[u] = lds_row8<false>(from, off_x, k, K);
          if (a.residual) h[u] = add8(h[u], lds_row8<false>(from + space, off_r, k, K));
          sum2 = squares8(h[u], sum2);
        }
        if (a.residual && k0 < K) store_run<false>(a.h + t * a.ldh, k0, K, h);
        team_sync();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = k0 + kVec * (32 * u + lane);
          if (k < K) keep(k, h[u]);
        }
      }
    }
    float sum = f2_sum(sum2);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (size > 1) {
      if (lane == 0) s_sum[warp] = sum;
      team_sync();  // the sums, and the row's values in the slot
      sum = s_sum[team * size];
      for (int j = 1; j < size; ++j) sum += s_sum[team * size + j];
    }
    const float r = rstd_of(sum, K, a.eps);
    if (sub == 0 && lane == 0) a.rstd[t] = r;
    // Codes of the 1024 features from k0 on; `whole`: all of them are there.
    auto codes = [&](int k0, auto whole) {
      constexpr bool W = decltype(whole)::value;
      uint64_t v[4][4];
      float am[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + kVec * (32 * u + lane);
        if (W || k < K) {
          uint64_t w[4];
          staged_weight8(weights, k, w);
          times8(lds_v4(from + 2u * (uint32_t)k), w, v[u]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = 0;
        }
        am[u] = amax8(v[u]);
      }
      if (a.y) {
        uint4 y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) y[u] = scaled_bf16(v[u], r);
        store_run<ALIGNED>(a.y + t * a.ldy, k0, K, y);
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
        if ((lane & 3) == 0 && (W || g * kBlock < K)) a.s_row[(int64_t)g * a.lds_row + t] = s;
        uint8_t* q = a.q_row + t * a.ldq_row;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float mu = __shfl_sync(kAll, mul, (lane & 16) | (u & 2 ? 8 : 0) | (u & 1 ? 4 : 0));
          store_codes8<W>(q, k0 + kVec * (32 * u + lane), K, v[u], mu);
        }
      }
    };
    if (a.q_row || a.y) {
      for (int k0 = 4 * 32 * kVec * sub; k0 < K; k0 += 4 * 32 * kVec * size) {
        if (k0 + 4 * 32 * kVec <= K) codes(k0, std::true_type{});
        else codes(k0, std::false_type{});
      }
    }
    fence_proxy_async_shared();  // this row's reads and writes of the slot, before the copy that takes it
    team_sync();
    if (sub == 0 && lane == 0 && i + slots < rows && !*abort_flag) issue(i + slots, slot);
    slot += teams;
    if (slot >= slots) slot -= slots, ++turn;
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) drain(full, s_asked, slots);
}

// Codes along the columns, from h and rstd: a CTA a 128 x 128 tile, a thread eight
// columns of 2 x 4 rows.  The row blocks are taken last first: what the rows' pass
// wrote last is still in L2 (30 MB of the 134 of 16384 x 4096).
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

// Gradient of every teams-th row, by teams of threads (chunks as above); the teams'
// sums for the weight go to partial[team of the launch][K].  The rows of dy, h and dh
// arrive by bulk copies, iterations ahead (rows loaded into registers where they are
// used: a training step's norm, forward and backward, of 16384 x 4096 265 us, so 236),
// two CTAs an SM for 2048 < K <= 4096 (three spilled registers: 229 us, two 219).  A
// thread's weights stay in its registers up to 8192 features (from shared memory,
// twice a row, they took more of its bandwidth than the rows: 98 us the gradient, so
// 91); from 4096 on 512 threads a row rather than longer threads (4096 x 8192: 72 us
// with 256, 57 with 512).
constexpr int bwd_ctas(int threads, int vpt) { return threads > 256 ? 1 : vpt <= 1 ? 3 : 2; }  // that an SM holds
template <int THREADS, int VPT, bool ALIGNED>
__global__ void __launch_bounds__(THREADS, bwd_ctas(THREADS, VPT)) rms_norm_bwd_kernel(const NormBwdArgs a) {
  constexpr bool kKeep = VPT <= 2;  // a thread's weights stay in registers
  extern __shared__ __align__(128) uint8_t s_ring[];  // weights, then [stages][dy, h, dh][rows of an iteration][K]
  __shared__ float s_slots[2][THREADS / 32];
  __shared__ uint64_t s_full[kBwdMaxStages];
  __shared__ int s_abort, s_asked[kBwdMaxStages];  // iterations that a stage was asked to take
  const Team team = team_of(a.team);
  const int K = (int)a.K, lane = team.lane, tid = (int)threadIdx.x, stages = a.stages;
  const uint32_t weights = smem_u32(s_ring), ring = weights + (kKeep ? 0u : staged_bytes(K)), full = smem_u32(s_full);
  const uint32_t space = row_space(K, ALIGNED), part_bytes = (uint32_t)team.count * space, parts = a.dh ? 3 : 2;
  const int64_t iterations = cdiv(a.T, team.count);
  volatile int* abort_flag = &s_abort;
  pdl_launch_dependents();
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < stages; ++i) mbar_init(full + 8 * i, 1), s_asked[i] = 0;
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  __syncthreads();
  pdl_wait();
  auto issue = [&](int64_t it, int st) {  // by warp 0: the rows of an iteration, a lane a row
    const int64_t t = it * team.count + tid;
    const bool in = tid < team.count && t < a.T;
    const uint16_t *d = a.dy + t * a.lddy, *h = a.h + t * a.ldh, *e = a.dh ? a.dh + t * a.lddh : nullptr;
    const uint32_t nd = in ? row_copied<ALIGNED>(d, K) : 0u, nh = in ? row_copied<ALIGNED>(h, K) : 0u,
                   ne = in && e ? row_copied<ALIGNED>(e, K) : 0u;
    const uint32_t bytes = __reduce_add_sync(kAll, nd + nh + ne);
    if (tid == 0) {
      ++s_asked[st];
      mbar_arrive_expect_tx(full + 8 * st, bytes);
    }
    __syncwarp();
    if (in) {
      const uint32_t to = ring + (uint32_t)st * parts * part_bytes + (uint32_t)tid * space;
      bulk_load(to, d - row_off<ALIGNED>(d) / 2, nd, full + 8 * st);
      bulk_load(to + part_bytes, h - row_off<ALIGNED>(h) / 2, nh, full + 8 * st);
      if (e) bulk_load(to + 2 * part_bytes, e - row_off<ALIGNED>(e) / 2, ne, full + 8 * st);
    }
  };
  if (tid < 32)
    for (int i = 0; i < stages; ++i)
      if ((int64_t)blockIdx.x + (int64_t)i * gridDim.x < iterations) issue((int64_t)blockIdx.x + (int64_t)i * gridDim.x, i);
  uint64_t kept[kKeep ? VPT : 1][4];
  if constexpr (kKeep) {
#pragma unroll
    for (int u = 0; u < VPT; ++u) load_weight8<ALIGNED>(a.weight, a.weight_f32, kVec * (u * team.size + lane), K, kept[u]);
  } else {
    stage_weights(a.weight, a.weight_f32, K, weights);
    __syncthreads();
  }
  auto weights8 = [&](int u, uint64_t (&w)[4]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = kept[u][i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = 0;
      const int k = kVec * (u * team.size + lane);
      if (k < K) staged_weight8(weights, k, w);
    }
  };
  float dw[VPT][8] = {};
  int turn = 0, st = 0;
  uint32_t parity = 0;
  const int64_t me = (int64_t)blockIdx.x * team.count + team.index;
  for (int64_t it = blockIdx.x; it < iterations; it += gridDim.x, turn ^= 1) {
    const int64_t t = it * team.count + team.index;
    const bool live = t < a.T;
    const float r = live ? a.rstd[t] : 0.0f;
    uint4 hv[VPT], dv[VPT], rv[VPT];
    // (a wait that gives up leaves the error word set and wrong rows from there on, without further waits or copies)
    if (!mbar_wait_bounded(full + 8 * st, parity, kWaitLimitNs, abort_flag)) {
      atomicOr(&g_norm_error, 1u);
      *abort_flag = 1;
    }
    const uint32_t from = ring + (uint32_t)st * parts * part_bytes + (uint32_t)team.index * space;
    const int off_d = row_off<ALIGNED>(a.dy + t * a.lddy), off_h = row_off<ALIGNED>(a.h + t * a.ldh),
              off_e = row_off<ALIGNED>(a.dh + t * a.lddh);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int k = live ? kVec * (u * team.size + lane) : K;
      dv[u] = lds_row8<ALIGNED>(from, off_d, k, K);
      hv[u] = lds_row8<ALIGNED>(from + part_bytes, off_h, k, K);
      rv[u] = a.dh ? lds_row8<ALIGNED>(from + 2 * part_bytes, off_e, k, K) : make_uint4(0, 0, 0, 0);
    }
    uint64_t sum2 = 0;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      uint64_t n[4], d[4], w[4];
      row_times(hv[u], r, n);
      pairs8(dv[u], d);
      weights8(u, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2_unpack(f2_fma(d[i], n[i], f2_pack(dw[u][2 * i], dw[u][2 * i + 1])), dw[u][2 * i], dw[u][2 * i + 1]);
        sum2 = f2_fma(f2_mul(d[i], w[i]), n[i], sum2);
      }
    }
    fence_proxy_async_shared();  // these reads, before the copy that takes their place
    const float mean = __fdiv_rn(team_sum(f2_sum(sum2), team, s_slots[turn]), (float)K);
    if (team.size <= 32) __syncthreads();  // (else it is in the sum)
    const int64_t next = it + (int64_t)stages * gridDim.x;
    if (tid < 32 && next < iterations && !__any_sync(kAll, *abort_flag)) issue(next, st);
    if (++st == stages) st = 0, parity ^= 1u;
    if (live) {
      const uint64_t r2 = f2_pack(r, r), c2 = f2_pack(-r * mean, -r * mean);  // dx = r (d w) - (r mean) n + dh
#pragma unroll
      for (int u = 0; u < VPT; ++u) {
        const int k = kVec * (u * team.size + lane);
        uint64_t n[4], d[4], w[4], e[4];
        row_times(hv[u], r, n);
        pairs8(dv[u], d);
        pairs8(rv[u], e);
        weights8(u, w);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          f2_unpack(f2_add(f2_fma(c2, n[i], f2_mul(r2, f2_mul(d[i], w[i]))), e[i]), lo, hi);
          out[i] = pack_bf16x2(lo, hi);
        }
        // (element by element where it is not aligned: store_run's two ends cost a chunk of 256 more than its blocks save,
        // 36.7 us for 33.0 at 5003 x 2001)
        store_row8<ALIGNED>(a.dx + t * a.lddx, k, K, make_uint4(out[0], out[1], out[2], out[3]));
      }
    }
  }
  if (tid == 0 && *abort_flag) drain(full, s_asked, stages);  // (all of its own asking)
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
    constexpr int kLoads = 15;  // in flight: all of three CTAs an SM on 152
    for (int64_t i = warp; i < teams; i += kLoads * 32) {
      float v[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) v[j] = i + 32 * j < teams ? partial[(i + 32 * j) * K + k] : 0.0f;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) add(v[j]);
    }
  }
  // (where the sum became infinite, what was lost is a difference of infinities: NaN)
  s[warp][lane] = fabsf(sum) < INFINITY ? sum + lost : sum;
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

template <bool ALIGNED>
static cudaError_t run_norm_ring(NormArgs a, int num_sms, cudaStream_t st) {  // more rows than SMs
  constexpr int64_t most = 220 * 1024;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(rms_norm_ring_kernel<ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  });
  if (attr_err != cudaSuccess) return attr_err;
  const int64_t weights = staged_bytes((int)a.K), slot = (int64_t)row_space((int)a.K, ALIGNED) * (a.residual ? 2 : 1);
  const int64_t fit = (most - weights) / slot;  // (two of the largest rows)
  a.slots = (int)(fit < kNormMaxSlots ? fit : kNormMaxSlots);
  // A warp a row where that keeps every warp busy, else four, or two where rows are short of that by little (16384 x 4096
  // with residual, 12 slots: one warp 83.1 us, two 86.3, four 81.3; 4096 x 8192, 5 slots: two 56.7, four 46.4; without
  // residual, 11: two 30.7, four 32.3).
  a.team = a.slots >= kNormWarps ? 1 : a.slots >= kNormWarps / 2 && !a.residual ? 2 : 4;
  return launch_pdl(rms_norm_ring_kernel<ALIGNED>, (unsigned)num_sms, 32 * kNormWarps,
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
  if (K >= 512 && a.T > num_sms) return norm_vec(a) ? run_norm_ring<true>(a, num_sms, st) : run_norm_ring<false>(a, num_sms, st);
  a.team = team_size(K, 1, 256);  // several rows a CTA: K <= 2048
  return run_norm<256, 1>(a, cdiv(a.T, 256 / a.team), st);
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
  g.threads = K <= 4096 ? 256 : 512;
  g.vpt = K <= 2048 ? 1 : K <= 8192 ? 2 : 4;
  g.team = team_size(K, g.vpt, g.threads);
  const int64_t per = g.threads / g.team, most = (int64_t)num_sms * bwd_ctas(g.threads, g.vpt);
  const int64_t ctas = cdiv(T, per * 8);  // eight rows a team at least: each writes a row of sums
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
    auto run = [&](auto threads, auto vpt, auto aligned) {
      constexpr int N = decltype(threads)::value, V = decltype(vpt)::value;
      constexpr bool A = decltype(aligned)::value;
      // the ring: what the CTAs that an SM holds leave each other (one stage of the largest rows)
      constexpr int64_t most = 220 * 1024 / bwd_ctas(N, V) - 1024;
      static std::once_flag once;
      static cudaError_t attr_err = cudaSuccess;
      std::call_once(once, [] {
        attr_err = cudaFuncSetAttribute(rms_norm_bwd_kernel<N, V, A>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
      });
      if (attr_err != cudaSuccess) return attr_err;
      const int64_t weights = V <= 2 ? 0 : staged_bytes((int)a.K);  // (kept in registers, or staged)
      const int64_t stage = N / g.team * (int64_t)row_space((int)a.K, A) * (a.dh ? 3 : 2), fit = (most - weights) / stage;
      a.stages = (int)(fit < kBwdMaxStages ? fit : kBwdMaxStages);
      return launch_pdl(rms_norm_bwd_kernel<N, V, A>, (unsigned)g.grid, N, (size_t)(weights + a.stages * stage), st, a);
    };
    auto go = [&](auto threads, auto vpt) {
      return vec ? run(threads, vpt, std::true_type{}) : run(threads, vpt, std::false_type{});
    };
    constexpr std::integral_constant<int, 256> n256;
    constexpr std::integral_constant<int, 512> n512;
    const cudaError_t e = g.vpt == 1   ? go(n256, std::integral_constant<int, 1>{})
                          : g.vpt == 4 ? go(n512, std::integral_constant<int, 4>{})
                          : g.threads == 256 ? go(n256, std::integral_constant<int, 2>{})
                                       : go(n512, std::integral_constant<int, 2>{});
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(rms_norm_dw_kernel, (unsigned)cdiv(a.K, 32), 1024, 0, st, (const float*)a.partial, g.teams, (int)a.K, a.dweight);
}

}  // namespace bfp8
