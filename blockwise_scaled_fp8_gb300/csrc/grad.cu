// The norm of a model's gradients over many tensors, and their clipping:
//   norm = sqrt(sum over every tensor's elements of g^2),
//   coef = min(1, max_norm / (norm + 1e-6)),   out = coef g.
//
// Two launches: one sums, one scales, each over all tensors at once.  The
// tensors' addresses and sizes travel as kernel parameters (no table in device
// memory, so nothing to keep or to copy, and a captured graph holds them); the
// elements of all tensors are chunks in one order, and a CTA takes a contiguous
// run of them.  Partial sums are one double a CTA and are added in a fixed
// order: the same tensors give the same norm.
//
// Squares are summed in fp32 over the 32 elements that a thread takes of a chunk, in
// small models over the 256 that a warp takes, and from there on in fp64 (which this
// part is slow at: where a CTA has one chunk, fp64 sums over its lanes are a third
// of the call).  Where an fp32 sum overflowed, or lies so low that its squares may
// have lost bits below the normal range, it is formed again in fp64 (its elements
// are in L1), so the norm of any finite gradients is finite as long as it fits fp32,
// and that of tiny ones is not 0.
//
// What bounds it is memory: every element is read for the norm, and read again
// and written for the clipping, since the norm has to be known first.  The
// second pass walks each run backwards: what the first one read last is still
// in L2 (50 MB of 600 at 300M bf16 elements).  1.2e9 bf16 elements: 1.10 ms for
// 7.2 GB, 6.5 TB/s; the norm alone of 150M mixed ones 65 us, 6.1 TB/s; 2M elements
// in 40 tensors 16 us.
#include <string.h>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kGradThreads = 512, kGradWarps = kGradThreads / 32;
constexpr int kGradVec = 8;                            // elements a thread takes at once
constexpr int kGradUnroll = 4;                         // and how often in a chunk (once where there are few chunks)
constexpr float kClipFloor = 1e-6f;
// below this a sum of up to 256 squares may hold ones that lost bits below 2^-126
constexpr float kTinySum = 1e-28f;

struct GradEntry {
  const void* in;
  void* out;
  int64_t n;
  uint32_t first;  // chunk
  uint8_t in_type, out_type, lead, vec;  // lead: elements before the first 16-byte boundary; vec: whole vectors after it
};

template <int CAP>
struct GradTable {
  int count;
  uint32_t chunks;  // of all tensors
  GradEntry e[CAP];
};

struct GradParams {
  double* partial;   // one a CTA of every launch of the norm
  int partials;      // of all launches
  int at;            // this launch's first
  float max_norm;
  float* norm;       // written by the first launch of the second kind
  int write_norm, in_place;
};

__device__ __forceinline__ float f16_to_f32(uint32_t h) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"((uint16_t)h));
  return f;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Element i of a tensor as fp32.
__device__ __forceinline__ float load1(const void* p, int type, int64_t i) {
  if (type == kGradF32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return type == kGradBf16 ? __uint_as_float(h << 16) : f16_to_f32(h);
}
__device__ __forceinline__ void store1(void* p, int type, int64_t i, float v) {
  if (type == kGradF32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)(type == kGradBf16 ? pack_bf16x2(v, 0.0f) : pack_f16x2(v, 0.0f));
}

// Eight elements from element i on (16-byte aligned there): the raw words (four of a 16-bit type, eight of fp32).
struct Raw8 {
  uint4 a, b;
};
__device__ __forceinline__ Raw8 load8(const void* p, int type, int64_t i) {
  Raw8 r;
  if (type == kGradF32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.a = q[0];
    r.b = q[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    r.b = make_uint4(0, 0, 0, 0);
  }
  return r;
}
__device__ __forceinline__ void values8(const Raw8& r, int type, float (&v)[8]) {
  if (type == kGradF32) {
    v[0] = __uint_as_float(r.a.x), v[1] = __uint_as_float(r.a.y), v[2] = __uint_as_float(r.a.z), v[3] = __uint_as_float(r.a.w);
    v[4] = __uint_as_float(r.b.x), v[5] = __uint_as_float(r.b.y), v[6] = __uint_as_float(r.b.z), v[7] = __uint_as_float(r.b.w);
    return;
  }
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if (type == kGradBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = f16_to_f32(w[i] & 0xFFFFu), v[2 * i + 1] = f16_to_f32(w[i] >> 16);
  }
}
__device__ __forceinline__ void store8(void* p, int type, int64_t i, const float (&v)[8]) {
  if (type == kGradF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    __stcs(q, make_float4(v[0], v[1], v[2], v[3]));
    __stcs(q + 1, make_float4(v[4], v[5], v[6], v[7]));
    return;
  }
  uint4 w;
  if (type == kGradBf16)
    w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  else
    w = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
  __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i), w);
}

// The tensor that holds chunk c.
template <int CAP>
__device__ __forceinline__ int entry_of(const GradTable<CAP>& t, uint32_t c) {
  int lo = 0, hi = t.count;  // t.e[lo].first <= c < t.e[hi].first
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].first <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// sqrt(v) rounded to fp32 (to within an ulp), without fp64's: the root of v scaled into [1, 4), one Newton step on its
// remainder, scaled back.  Infinities, NaN and 0 are their own roots.
__device__ __forceinline__ float root_of(double v) {
  if (!(v > 0.0) || v > 1e300) return (float)v;  // (1e300: far above the square of any fp32)
  const int e = (((int)(__double_as_longlong(v) >> 52) & 0x7FF) - 1023) & ~1;
  const double m = v * __longlong_as_double((long long)(1023 - e) << 52);
  const float y = __fsqrt_rn((float)m);
  const float rest = (float)fma(-(double)y, (double)y, m);
  return ldexpf(y + rest * __fdividef(0.5f, y), e / 2);
}

}  // namespace

// Chunk c of a tensor is its vectors [c * kGradThreads * U, ..), thread by thread; its first chunk also takes the elements before the first vector and
// after the last one.  A tensor without vectors (vec 0: its output's alignment
// differs from its input's) is taken element by element instead, a warp's lanes
// side by side.
template <int CAP, int U>
__global__ void __launch_bounds__(kGradThreads, 2)
    grad_norm_kernel(const __grid_constant__ GradTable<CAP> t, const GradParams p) {
  constexpr bool kByWarp = U == 1;  // sums are a warp's, the same in its lanes (else a thread's)
  __shared__ double s_sum[kGradWarps];
  const int tid = (int)threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t c0 = (uint32_t)((uint64_t)t.chunks * blockIdx.x / gridDim.x),
                 c1 = (uint32_t)((uint64_t)t.chunks * (blockIdx.x + 1) / gridDim.x);
  double total = 0.0;
  int at = c0 < c1 ? entry_of(t, c0) : 0;
  for (uint32_t c = c0; c < c1; ++c) {
    while (at + 1 < t.count && t.e[at + 1].first <= c) ++at;
    const GradEntry e = t.e[at];
    const uint32_t local = c - e.first;
    float sum = 0.0f;
    uint32_t any = 0;  // bits of the magnitudes: 0 where every element is 0
    if (e.vec) {
      const int64_t nv = (e.n - e.lead) / kGradVec;
      const int64_t v0 = (int64_t)local * (kGradThreads * U) + tid;
      Raw8 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t v = v0 + u * kGradThreads;
        if (v < nv) r[u] = load8(e.in, e.in_type, e.lead + v * kGradVec);
        else r[u].a = r[u].b = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        values8(r[u], e.in_type, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
        any |= r[u].a.x | r[u].a.y | r[u].a.z | r[u].a.w | r[u].b.x | r[u].b.y | r[u].b.z | r[u].b.w;
      }
      int64_t edge = -1;  // an element outside the vectors
      if (local == 0) {
        const int64_t tail = e.lead + nv * kGradVec;
        if (tid < e.lead) edge = tid;
        else if (tail + tid - e.lead < e.n) edge = tail + tid - e.lead;
      }
      if (local == 0 && tid < 32) {  // (at most 14 of them: warp 0's)
        const double v = edge >= 0 ? (double)load1(e.in, e.in_type, edge) : 0.0;
        total += kByWarp ? warp_sum(v * v) : v * v;
      }
      const float part = kByWarp ? warp_sum(sum) : sum;
      if (!(part < INFINITY) || (part < kTinySum && (kByWarp ? __any_sync(kAll, any != 0) : any != 0))) {
        double again = 0.0;
        for (int u = 0; u < U; ++u) {
          const int64_t v = v0 + u * kGradThreads;
          for (int i = 0; v < nv && i < kGradVec; ++i) {
            const double x = load1(e.in, e.in_type, e.lead + v * kGradVec + i);
            again += x * x;
          }
        }
        total += kByWarp ? warp_sum(again) : again;
      } else {
        total += (double)part;
      }
    } else {
      const int64_t e0 = (int64_t)local * (kGradThreads * kGradVec * U);
#pragma unroll 8
      for (int u = 0; u < kGradVec * U; ++u) {
        const int64_t i = e0 + u * kGradThreads + tid;
        if (i < e.n) {
          const float v = load1(e.in, e.in_type, i);
          sum = fmaf(v, v, sum);
          any |= __float_as_uint(v) << 1;
        }
      }
      const float part = kByWarp ? warp_sum(sum) : sum;
      if (!(part < INFINITY) || (part < kTinySum && (kByWarp ? __any_sync(kAll, any != 0) : any != 0))) {
        double again = 0.0;
        for (int u = 0; u < kGradVec * U; ++u) {
          const int64_t i = e0 + u * kGradThreads + tid;
          if (i < e.n) {
            const double x = load1(e.in, e.in_type, i);
            again += x * x;
          }
        }
        total += kByWarp ? warp_sum(again) : again;
      } else {
        total += (double)part;
      }
    }
  }
  if (!kByWarp) total = warp_sum(total);
  if ((tid & 31) == 0) s_sum[tid >> 5] = total;
  __syncthreads();
  if (tid < 32) {
    const double v = warp_sum(tid < kGradWarps ? s_sum[tid] : 0.0);
    if (tid == 0) p.partial[p.at + blockIdx.x] = v;
  }
}

// The norm from the partial sums, by every CTA in the same order; then its run of chunks, scaled, last one first.
template <int CAP, int U>
__global__ void __launch_bounds__(kGradThreads, 2)
    grad_scale_kernel(const __grid_constant__ GradTable<CAP> t, const GradParams p) {
  __shared__ float s_norm;
  const int tid = (int)threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  if (tid < 32) {
    double total = 0.0;
    constexpr int kLoads = 10;  // in flight (two CTAs an SM on 152 SMs: all of one table's)
    for (int i0 = 0; i0 < p.partials; i0 += 32 * kLoads) {
      double v[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) v[j] = i0 + 32 * j + tid < p.partials ? p.partial[i0 + 32 * j + tid] : 0.0;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) total += v[j];
    }
    total = warp_sum(total);
    if (tid == 0) s_norm = root_of(total);
  }
  __syncthreads();
  const float norm = s_norm;
  if (p.write_norm && blockIdx.x == 0 && tid == 0) *p.norm = norm;
  const float ratio = p.max_norm / (norm + kClipFloor);
  const float coef = ratio > 1.0f ? 1.0f : ratio;  // (a NaN stays one)
  if (p.in_place && coef == 1.0f) return;          // every product would be the element itself
  const uint32_t c0 = (uint32_t)((uint64_t)t.chunks * blockIdx.x / gridDim.x),
                 c1 = (uint32_t)((uint64_t)t.chunks * (blockIdx.x + 1) / gridDim.x);
  int at = c0 < c1 ? entry_of(t, c1 - 1) : 0;
  for (uint32_t c = c1; c-- > c0;) {
    while (t.e[at].first > c) --at;
    const GradEntry e = t.e[at];
    const uint32_t local = c - e.first;
    if (e.vec) {
      const int64_t nv = (e.n - e.lead) / kGradVec;
      const int64_t v0 = (int64_t)local * (kGradThreads * U) + tid;
      Raw8 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t v = v0 + u * kGradThreads;
        if (v < nv) r[u] = load8(e.in, e.in_type, e.lead + v * kGradVec);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at_v = v0 + u * kGradThreads;
        if (at_v < nv) {
          float v[8];
          values8(r[u], e.in_type, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= coef;
          store8(e.out, e.out_type, e.lead + at_v * kGradVec, v);
        }
      }
      if (local == 0) {
        const int64_t tail = e.lead + nv * kGradVec;
        int64_t edge = -1;
        if (tid < e.lead) edge = tid;
        else if (tail + tid - e.lead < e.n) edge = tail + tid - e.lead;
        if (edge >= 0) store1(e.out, e.out_type, edge, load1(e.in, e.in_type, edge) * coef);
      }
    } else {
      const int64_t e0 = (int64_t)local * (kGradThreads * kGradVec * U) + tid;
      for (int u0 = 0; u0 < kGradVec * U; u0 += 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t i = e0 + (u0 + u) * kGradThreads;
          if (i < e.n) v[u] = load1(e.in, e.in_type, i);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t i = e0 + (u0 + u) * kGradThreads;
          if (i < e.n) store1(e.out, e.out_type, i, v[u] * coef);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

static int size_of(int type) { return type == kGradF32 ? 4 : 2; }

// Entry of tensor i, and its chunks.
static uint32_t fill_entry(const GradArgs& a, int64_t i, int unroll, GradEntry* e) {
  memset(e, 0, sizeof(*e));
  e->in = a.in[i];
  e->out = a.out ? a.out[i] : nullptr;
  e->n = a.numel[i];
  e->in_type = (uint8_t)a.in_type[i];
  e->out_type = (uint8_t)(a.out ? a.out_type[i] : a.in_type[i]);
  const uintptr_t at = reinterpret_cast<uintptr_t>(e->in);
  int64_t lead = (int64_t)((16 - (at & 15)) & 15) / size_of(e->in_type);
  if (lead > e->n) lead = e->n;
  e->lead = (uint8_t)lead;
  e->vec = !e->out || ((reinterpret_cast<uintptr_t>(e->out) + (uintptr_t)lead * size_of(e->out_type)) & 15) == 0;
  const int64_t chunk = (int64_t)kGradThreads * unroll;
  const int64_t chunks = e->vec ? cdiv((e->n - lead) / kGradVec, chunk) : cdiv(e->n, chunk * kGradVec);
  return (uint32_t)(chunks > 0 ? chunks : 1);
}

template <int CAP, int U>
static cudaError_t run_grads(const GradArgs& a, const int64_t* which, int64_t n, int num_sms, cudaStream_t st) {
  const int64_t launches = n > 0 ? cdiv(n, CAP) : 1;
  const int grid = grad_grid(num_sms);
  GradParams p = {};
  p.partial = a.partial;
  p.partials = (int)launches * grid;
  p.max_norm = a.max_norm;
  p.norm = a.norm;
  p.in_place = a.in_place;
  GradTable<CAP> t;
  for (int pass = 0; pass < 2; ++pass) {
    for (int64_t l = 0; l < launches; ++l) {
      memset(&t, 0, sizeof(t));
      for (int64_t i = l * CAP; i < n && i < (l + 1) * CAP; ++i) {
        t.e[t.count].first = 0;
        const uint32_t chunks = fill_entry(a, which[i], U, &t.e[t.count]);
        t.e[t.count++].first = t.chunks;
        t.chunks += chunks;
      }
      p.at = (int)l * grid;
      p.write_norm = l == 0;
      cudaError_t e;
      if (pass == 0) {
        e = launch_pdl(grad_norm_kernel<CAP, U>, (unsigned)grid, kGradThreads, 0, st, t, p);
      } else {
        if (!a.out) t.count = 0, t.chunks = 0;  // the norm alone: one CTA adds the partial sums
        e = launch_pdl(grad_scale_kernel<CAP, U>, a.out ? (unsigned)grid : 1u, kGradThreads, 0, st, t, p);
      }
      if (e != cudaSuccess) return e;
      if (pass == 1 && !a.out) break;
    }
  }
  return cudaSuccess;
}

int grad_grid(int num_sms) { return 2 * num_sms; }
int64_t grad_launches(int64_t n) { return n <= kGradCapSmall ? 1 : cdiv(n, kGradCap); }

// Tables of 64 and of 640 tensors: the parameters of a launch are copied by the
// driver whatever their use, 2 KB against 20.  Chunks of 4096 elements where those
// of 16384 would be fewer than the CTAs (2M elements in 40 tensors: 25 us with the
// larger ones).
cudaError_t launch_grads(const GradArgs& a, const int64_t* which, int64_t n, int num_sms, cudaStream_t st) {
  static_assert(sizeof(GradTable<kGradCap>) + sizeof(GradParams) <= 32764, "a launch's parameters");
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) total += a.numel[which[i]];
  const bool few = total < (int64_t)grad_grid(num_sms) * kGradThreads * kGradVec * kGradUnroll;
  if (n <= kGradCapSmall)
    return few ? run_grads<kGradCapSmall, 1>(a, which, n, num_sms, st) : run_grads<kGradCapSmall, kGradUnroll>(a, which, n, num_sms, st);
  return few ? run_grads<kGradCap, 1>(a, which, n, num_sms, st) : run_grads<kGradCap, kGradUnroll>(a, which, n, num_sms, st);
}

}  // namespace bfp8
