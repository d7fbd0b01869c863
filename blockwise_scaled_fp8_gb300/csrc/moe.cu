// Mixture-of-experts operators around the experts' products: the router and
// its gradient, the plan that sorts the routed slots by expert, and the
// combine of the experts' outputs with its gradient.
//
// A slot is a (token t, choice j) pair, flat index t*k + j; a row is a place
// of the sorted buffers.  row[slot] is a slot's row, src[row] a row's slot;
// -1 marks a slot that goes nowhere and a row that holds padding.
#include <float.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// A 32-bit key with the order of the floats (no NaN), equal for the two zeros; every float's key is above 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 + 0 = +0
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// The float whose key it is (+0 for both zeros).
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
constexpr uint32_t kNoKey = 0x007FFFFFu;  // the key of -inf: not eligible

__device__ __forceinline__ float load_logit(const void* p, int f32, int64_t i) {
  return f32 ? __ldg(static_cast<const float*>(p) + i)
             : bf16_to_f32(__ldg(static_cast<const uint16_t*>(p) + i));
}

// The lowest finite value of the logits' type: it, -inf and NaN mask an expert.
// Its negative is the largest, which +inf counts as.
__device__ __forceinline__ float lowest_of(int f32) { return f32 ? -FLT_MAX : __uint_as_float(0xFF7F0000u); }

}  // namespace

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------

namespace {

template <int X, int Y, int N, typename K>
__device__ __forceinline__ void order_pair(K (&v)[N]) {
  const K hi = v[X] > v[Y] ? v[X] : v[Y], lo = v[X] > v[Y] ? v[Y] : v[X];
  v[X] = hi;
  v[Y] = lo;
}

// Sorts 1 .. 6 or 8 values, largest first (networks of the fewest exchanges).
template <int N, typename K>
__device__ __forceinline__ void sort_down(K (&v)[N]) {
  static_assert(N <= 6 || N == 8, "a network for N values");
  if constexpr (N == 2) {
    order_pair<0, 1>(v);
  } else if constexpr (N == 3) {
    order_pair<1, 2>(v); order_pair<0, 2>(v); order_pair<0, 1>(v);
  } else if constexpr (N == 4) {
    order_pair<0, 1>(v); order_pair<2, 3>(v); order_pair<0, 2>(v); order_pair<1, 3>(v); order_pair<1, 2>(v);
  } else if constexpr (N == 5) {
    order_pair<0, 1>(v); order_pair<3, 4>(v); order_pair<2, 4>(v); order_pair<2, 3>(v); order_pair<1, 4>(v);
    order_pair<0, 3>(v); order_pair<0, 2>(v); order_pair<1, 3>(v); order_pair<1, 2>(v);
  } else if constexpr (N == 6) {
    order_pair<1, 2>(v); order_pair<4, 5>(v); order_pair<0, 2>(v); order_pair<3, 5>(v); order_pair<0, 1>(v);
    order_pair<3, 4>(v); order_pair<2, 5>(v); order_pair<0, 3>(v); order_pair<1, 4>(v); order_pair<2, 4>(v);
    order_pair<1, 3>(v); order_pair<2, 3>(v);
  } else if constexpr (N == 8) {
    order_pair<0, 1>(v); order_pair<2, 3>(v); order_pair<4, 5>(v); order_pair<6, 7>(v); order_pair<0, 2>(v);
    order_pair<1, 3>(v); order_pair<4, 6>(v); order_pair<5, 7>(v); order_pair<1, 2>(v); order_pair<5, 6>(v);
    order_pair<0, 4>(v); order_pair<1, 5>(v); order_pair<2, 6>(v); order_pair<3, 7>(v); order_pair<2, 4>(v);
    order_pair<3, 5>(v); order_pair<1, 2>(v); order_pair<3, 4>(v); order_pair<5, 6>(v);
  }
}

// N logits of a row from element i on as fp32, -inf past the row's end and where the expert is masked.
template <int N, bool F32>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t at, int e0, float (&l)[N]) {
  const float low = lowest_of(F32);
  if (N % 4 == 0 && a.vec && e0 + N <= (int)a.E) {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i + 3 < N; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at + e0 + i));
        l[i] = q.x, l[i + 1] = q.y, l[i + 2] = q.z, l[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i + 3 < N; i += 4) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + at + e0 + i));
        l[i] = bf16_lo(q.x), l[i + 1] = bf16_hi(q.x), l[i + 2] = bf16_lo(q.y), l[i + 3] = bf16_hi(q.y);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = e0 + i < (int)a.E ? load_logit(a.logits, F32, at + e0 + i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) l[i] = l[i] > low ? fminf(l[i], -low) : -INFINITY;  // NaN compares false
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// exp(x) of terms that are not compared.  Of bf16 logits by __expf, off by 2 ulp
// and |x| 2^-24 (at most 2^-17 where the result is a normal number):
//   - a softmax's denominator keeps it to 2^-21, since x exp(x) is at most 1 / e
//     for x < 0 (a logit's own rounding moves it by up to 2^-9 of the logit);
//   - the gradient's dense row is rounded to bf16, 2^-9.
// Of fp32 logits by expf.
template <bool F32>
__device__ __forceinline__ float dense_exp(float x) {
  return F32 ? expf(x) : __expf(x);
}

}  // namespace

// One warp a token, lane l the VPL consecutive experts from l VPL on.  Scores
// in fp32: sigmoid 1 / (1 + exp(-l)), or softmax exp(l - max) / sum over the
// eligible experts.  The choice compares c: score + bias, or for a softmax
// without bias the logit itself (the softmax keeps its order, and no rounding
// of the denominator can change a choice), as an order-preserving integer key
// (0: not eligible).  What bounds it is instructions, so:
//   - each lane sorts its keys once (VPL <= 8), each with its place in the low
//     word so that equal ones keep their order; a choice is then one redux
//     over the lanes' first keys, a ballot for the lowest lane that holds it
//     (whose experts are the lowest), and a shift of the winner's list;
//   - bf16 logits of a softmax without bias are 16-bit keys: they share a
//     32-bit word with the expert's complement, and the redux names the winner;
//   - with more experts a lane (VPL > 8) sorting costs more than k scans;
//   - scores of the chosen are formed again from their logits, by k lanes.
// 16384 tokens x 256 fp32, 8 groups, sigmoid with bias, k = 8: 18.6 us, 1002
// warp-instructions a token (the first form, k scans of every lane's keys, took
// 1737 and 32.8 us; scores by __expf and an approximate quotient 16.9, but then
// near-equal experts are not chosen as the plain fp32 form chooses); 50021 x 160
// bf16, softmax, k = 6: 17 us, 347; one token 2.0 us.
template <int VPL, bool F32, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteArgs a) {
  // per warp: E + 32 values of groups that are not whole powers of two of lanes, later the sorted lists
  extern __shared__ __align__(16) float s_route[];
  constexpr bool kByLogit = !SIGMOID && !BIAS, kPacked = kByLogit && !F32;
  constexpr int kLists = (VPL + 7) / 8, kLen = VPL / kLists;  // sorted lists a lane
  static_assert(kLists * kLen == VPL, "lists of one length");
  pdl_launch_dependents();
  pdl_wait();
  const int lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
  const int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 32) + warp;
  if (t >= a.T) return;
  const int E = (int)a.E, e0 = lane * VPL;
  float* mine_s = s_route + warp * (VPL * 64);  // (E + 32 <= 64 VPL)
  const int64_t at = t * a.ldl;
  float c[VPL];  // logit, then the choice value (-inf: not eligible)
  load_logits<VPL, F32>(a, at, e0, c);
  float top = 0.0f, sum = 1.0f;  // softmax: p = exp(l - top) / sum
  float gv[VPL];                 // what a group's score sums the largest of (softmax without bias)
  if constexpr (!SIGMOID) {
    float m = c[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, c[i]);
    top = key_value(__reduce_max_sync(kFull, order_key(m)));
    sum = 0.0f;
    if (!kByLogit || a.groups > 1) {  // the terms are compared
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        gv[i] = c[i] > -INFINITY ? expf(c[i] - top) : 0.0f;
        sum += gv[i];
      }
    } else {
      // only their sum is used; masked: exp(-inf) = 0
      top = fmaxf(top, -FLT_MAX);  // finite where all are masked
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += dense_exp<F32>(c[i] - top);
    }
    sum = fmaxf(warp_sum(sum), FLT_MIN);
  }
  if constexpr (!kByLogit) {
    float b[VPL] = {};
    if constexpr (BIAS) {
      if (VPL % 4 == 0 && a.bias_vec && e0 + VPL <= E) {
#pragma unroll
        for (int i = 0; i + 3 < VPL; i += 4) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(a.bias + e0 + i));
          b[i] = q.x, b[i + 1] = q.y, b[i + 2] = q.z, b[i + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (e0 + i < E) b[i] = __ldg(a.bias + e0 + i);
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool ok = c[i] > -INFINITY;
      float v = SIGMOID ? sigmoid(c[i]) : gv[i] / sum;
      if (BIAS) v += b[i];
      c[i] = ok && v > -INFINITY ? v : -INFINITY;
    }
  }
  uint32_t kept = 0xffffffffu;  // bit g: group g stays
  const int S = a.groups > 1 ? E / a.groups : E;
  if (a.groups > 1) {
    auto value = [&](int i) { return kByLogit ? (c[i] > -INFINITY ? gv[i] : -INFINITY) : c[i]; };
    float m1 = -INFINITY, m2 = -INFINITY;  // the two largest of this lane's share of a group
    int L = a.group_lanes, g;              // lanes a group
    if (a.group_whole) {
      // a lane's experts lie in one group, of L consecutive lanes
      g = lane / L;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float v = value(i);
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
    } else {
      // through shared memory, padded so that the groups' lanes meet different banks
      float* buf = mine_s;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e0 + i < E) buf[e0 + i + (e0 + i) / S * L] = value(i);
      __syncwarp();
      g = lane / L;
      if (g < a.groups)
        for (int i = lane % L; i < S; i += L) {
          const float v = buf[g * (S + L) + i];
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
    }
    for (int o = L >> 1; o >= 1; o >>= 1) {
      const float n1 = __shfl_xor_sync(kFull, m1, o), n2 = __shfl_xor_sync(kFull, m2, o);
      m2 = fmaxf(fmaxf(m2, n2), fminf(m1, n1));
      m1 = fmaxf(m1, n1);
    }
    const float gs = a.group_top == 2 && m2 > -INFINITY ? m1 + m2 : m1;
    uint32_t gkey = lane % L == 0 && g < a.groups && m1 > -INFINITY ? order_key(gs) : 0u;
    kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const uint32_t best = __reduce_max_sync(kFull, gkey);
      if (best == 0) break;
      const int win = __ffs(__ballot_sync(kFull, gkey == best)) - 1;  // lowest lane = lowest group
      kept |= 1u << (win / L);
      if (lane == win) gkey = 0;
    }
    if (a.group_whole) {
      if (!((kept >> min(g, 31)) & 1u)) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!((kept >> min((e0 + i) / S, 31)) & 1u)) c[i] = -INFINITY;
    }
  }
  // k choices: lane j keeps choice j.  A key is the value's order with the
  // expert's complement below it (kPacked) or the complement of its place in
  // the lane, so that of equal values the lowest expert comes first.
  using Key = std::conditional_t<kPacked, uint32_t, uint64_t>;
  Key head[kLists];
  Key* list = reinterpret_cast<Key*>(mine_s) + lane;  // the rest, [list][place][lane]: a winner fetches its next key
  int next[kLists];                                   // where a list's next key lies
  __syncwarp();  // the groups' values, which lay here, have been read
#pragma unroll
  for (int l = 0; l < kLists; ++l) {
    Key key[kLen];
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      const int at_i = l * kLen + i;
      if constexpr (kPacked) key[i] = (order_key(c[at_i]) & 0xFFFF0000u) | (uint32_t)(0xFFFF - e0 - at_i);
      else key[i] = ((uint64_t)order_key(c[at_i]) << 32) | (uint32_t)(VPL - 1 - at_i);
    }
    sort_down(key);
    head[l] = key[0];
    next[l] = 32 * l * kLen;
#pragma unroll
    for (int i = 1; i < kLen; ++i) list[32 * (l * kLen + i - 1)] = key[i];
    list[32 * (l * kLen + kLen - 1)] = 0;  // never wins: nothing is read past it
  }
  int my_e = -1;
  for (int j = 0; j < a.k; ++j) {
    Key my = head[0];
#pragma unroll
    for (int l = 1; l < kLists; ++l) my = my > head[l] ? my : head[l];
    const uint32_t hi = (uint32_t)(kPacked ? my : my >> (kPacked ? 0 : 32)), best = __reduce_max_sync(kFull, hi);
    if (best <= kNoKey) break;
    int e;
    bool mine;
    if constexpr (kPacked) {
      e = 0xFFFF - (int)(best & 0xFFFFu);
      mine = hi == best;
    } else {
      const int win = __ffs(__ballot_sync(kFull, hi == best)) - 1;  // lowest lane = lowest experts
      e = __shfl_sync(kFull, e0 + VPL - 1 - (int)(uint32_t)my, win);
      mine = lane == win;
    }
    if (lane == j) my_e = e;
    if (mine) {
#pragma unroll
      for (int l = 0; l < kLists; ++l)
        if (kLists == 1 || head[l] == my) {
          head[l] = list[next[l]];
          next[l] += 32;
        }
    }
  }
  float p = 0.0f;
  if (my_e >= 0) {
    const float l = fminf(load_logit(a.logits, F32, at + my_e), -lowest_of(F32));
    p = SIGMOID ? sigmoid(l) : expf(l - top) / sum;
  }
  const float total = a.renormalize ? fmaxf(warp_sum(p), kRouteSumFloor) : 1.0f;
  if (lane < a.k) {
    a.idx[t * a.k + lane] = my_e;
    a.w[t * a.k + lane] = a.scale * (p / total);
  }
}

// The router's gradient.  With p the scores, S the sum of the chosen p and the
// chosen j:
//   ds_j = (scale dw_j - sum_i dw_i w_i) / S   (renormalised),  scale dw_j  (not)
//   (where S is not above the floor the weights are scale p / floor, whose
//   denominator is a constant: ds_j = scale dw_j / floor)
//   sigmoid:  dl_j = ds_j p_j (1 - p_j), zero elsewhere
//   softmax:  dl_e = p_e (ds_e - sum_i ds_i p_i), ds_e = 0 where not chosen
// One warp a token; lane j < k handles choice j.  Of the dense row lane l
// takes the pairs 2l, 2l + 64, .. (one load and one store a pair where the row
// is aligned for it), over which the chosen values go last.  Bound by
// instructions as the router is: 50021 tokens x 160 bf16, softmax, 15 us, 275
// warp-instructions a token.
//
// Tokens with little work are bound by the start of CTAs, about one a
// nanosecond: twice the warps a CTA for them (32768 x 256 sigmoid 9.6 -> 8.6
// us, x 64 softmax 10.7 -> 9.7; more pairs of a softmax 14.8 -> 15.1 at 256,
// 23.7 -> 25.5 at 384 experts).
template <int PAIRS, bool SIGMOID>
constexpr int kRouteBwdThreads = SIGMOID || PAIRS == 1 ? 2 * kRouteThreads : kRouteThreads;

template <int PAIRS, bool F32, bool SIGMOID>
__global__ void __launch_bounds__(kRouteBwdThreads<PAIRS, SIGMOID>) moe_route_bwd_kernel(const RouteBwdArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = (int)(threadIdx.x & 31);
  const int64_t t = (int64_t)blockIdx.x * (kRouteBwdThreads<PAIRS, SIGMOID> / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int E = (int)a.E;
  const float low = lowest_of(F32);
  const int64_t at = t * a.ldl, out = t * a.ldd;
  int e_j = lane < a.k ? __ldg(a.idx + t * a.k + lane) : -1;
  if (e_j >= E) e_j = -1;
  const float dw = e_j >= 0 ? __ldg(a.dw + t * a.k + lane) : 0.0f, w = e_j >= 0 ? __ldg(a.w + t * a.k + lane) : 0.0f;
  float l_j = e_j >= 0 ? load_logit(a.logits, F32, at + e_j) : -INFINITY;
  l_j = l_j > low ? fminf(l_j, -low) : -INFINITY;
  float s[2 * PAIRS], p_j, dot = 0.0f;
  if constexpr (SIGMOID) {
    p_j = sigmoid(l_j);
  } else {
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const int e = 64 * i + 2 * lane;
      float l0 = -INFINITY, l1 = -INFINITY;
      if (a.vec && e + 1 < E) {
        if constexpr (F32) {
          const float2 q = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(a.logits) + at + e));
          l0 = q.x, l1 = q.y;
        } else {
          const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.logits) + at + e));
          l0 = bf16_lo(q), l1 = bf16_hi(q);
        }
      } else {
        if (e < E) l0 = load_logit(a.logits, F32, at + e);
        if (e + 1 < E) l1 = load_logit(a.logits, F32, at + e + 1);
      }
      s[2 * i] = l0 > low ? fminf(l0, -low) : -INFINITY;
      s[2 * i + 1] = l1 > low ? fminf(l1, -low) : -INFINITY;
    }
    // p = exp(l - ref) * mult: by the first choice where its weight gives its p
    // (no renormalisation, and neither p nor the weight, scale p, so small that
    // it has lost bits), else by the largest logit and the sum over the row
    float ref = __shfl_sync(kFull, l_j, 0);
    const float w_0 = __shfl_sync(kFull, w, 0);
    float mult = w_0 / a.scale;
    if (!a.renormalize && mult > 1e-20f && mult < 2.0f && fabsf(w_0) >= FLT_MIN) {
#pragma unroll
      for (int i = 0; i < 2 * PAIRS; ++i) s[i] = dense_exp<F32>(s[i] - ref) * mult;
    } else {
      ref = s[0];
#pragma unroll
      for (int i = 1; i < 2 * PAIRS; ++i) ref = fmaxf(ref, s[i]);
      ref = fmaxf(key_value(__reduce_max_sync(kFull, order_key(ref))), -FLT_MAX);  // finite where all are masked
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * PAIRS; ++i) {
        s[i] = dense_exp<F32>(s[i] - ref);
        sum += s[i];
      }
      mult = 1.0f / fmaxf(warp_sum(sum), FLT_MIN);
#pragma unroll
      for (int i = 0; i < 2 * PAIRS; ++i) s[i] *= mult;
    }
    p_j = expf(l_j - ref) * mult;  // -inf: 0
  }
  float ds = a.scale * dw;
  if (a.renormalize) {
    const float S = warp_sum(p_j), back = warp_sum(dw * w);
    ds = S > kRouteSumFloor ? (ds - back) / S : ds / kRouteSumFloor;
  }
  if (e_j < 0) ds = 0.0f;
  if constexpr (!SIGMOID) dot = warp_sum(ds * p_j);
  const float dl_j = SIGMOID ? ds * p_j * (1.0f - p_j) : p_j * (ds - dot);
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    const int e = 64 * i + 2 * lane;
    const float d0 = SIGMOID ? 0.0f : -s[2 * i] * dot, d1 = SIGMOID ? 0.0f : -s[2 * i + 1] * dot;
    if constexpr (F32) {
      float* to = static_cast<float*>(a.dlogits) + out + e;
      if (a.vec && e + 1 < E) {
        *reinterpret_cast<float2*>(to) = make_float2(d0, d1);
      } else {
        if (e < E) to[0] = d0;
        if (e + 1 < E) to[1] = d1;
      }
    } else {
      uint16_t* to = static_cast<uint16_t*>(a.dlogits) + out + e;
      if (a.vec && e + 1 < E) {
        *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(d0, d1);
      } else {
        if (e < E) to[0] = f32_to_bf16(d0);
        if (e + 1 < E) to[1] = f32_to_bf16(d1);
      }
    }
  }
  __syncwarp();  // orders the dense row before the chosen values
  if (e_j >= 0) {
    if constexpr (F32) static_cast<float*>(a.dlogits)[out + e_j] = dl_j;
    else static_cast<uint16_t*>(a.dlogits)[out + e_j] = f32_to_bf16(dl_j);
  }
}

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of the slots by expert
// ---------------------------------------------------------------------------
//
// One launch of one cluster.  Warp w of the cluster takes a contiguous run of
// slots, 32 at a time: the lanes of one expert find each other by ballots over
// the bits of its number (a match instruction is several times slower here),
// and their rank among them follows the lane, so the order within an expert is
// the slots' order and every launch gives the same plan.  A slot's rank within
// its warp's run waits in row.  Then prefix sums of the counts: over the warps
// of a CTA, over the CTAs of the cluster through distributed shared memory,
// over the experts' aligned counts; and the slots' rows follow.  131072 slots,
// 256 experts: 14.9 us, a chain of latencies, of which the scattered stores of
// src from 16 SMs are 3.6 and the padding's 0.8 (24.0 us with a cluster of 8
// CTAs, 36.0 with matches); 384 slots, one CTA: 3.6 us.
constexpr int kPlanCtas = 16;  // of the cluster, at most
template <int BITS>  // of the experts' numbers, E (nowhere) among them
__global__ void __launch_bounds__(kPlanThreads, 1) moe_plan_kernel(const PlanArgs a) {
  extern __shared__ uint32_t s_cnt[];  // [32 warps][E] counts, then first rows; [E] CTA totals
  __shared__ uint32_t s_scan[32];
  pdl_launch_dependents();
  pdl_wait();
  const int E = (int)a.E, tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = (int)gridDim.x, rank = (int)blockIdx.x;  // the grid is one cluster
  uint32_t* mine = s_cnt + warp * E;
  uint32_t* s_tot = s_cnt + 32 * E;
  const int64_t n = a.n;
  const int64_t run = cdiv(cdiv(n, (int64_t)ctas * 32), 32) * 32;  // slots a warp, a multiple of 32
  const int64_t lo = ((int64_t)rank * 32 + warp) * run, hi = lo + run < n ? lo + run : n;
  for (int i = lane; i < E; i += 32) mine[i] = 0;
  // padding everywhere; the barriers below come before the slots' own entries
  for (int64_t r = (int64_t)rank * kPlanThreads + tid; r < a.R; r += (int64_t)ctas * kPlanThreads) a.src[r] = -1;
  __syncwarp();
  // ranks of the 32 slots from i0 on, of expert e (E: none) in this lane
  auto rank_slots = [&](int64_t i0, int e) {
    uint32_t peers = kFull;
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
      const bool set = (e >> b) & 1;
      const uint32_t vote = __ballot_sync(kFull, set);
      peers &= set ? vote : ~vote;
    }
    const bool ok = e < E;
    const uint32_t base = ok ? mine[e] : 0u, lower = (uint32_t)__popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (ok && lower == 0) mine[e] = base + (uint32_t)__popc(peers);
    __syncwarp();
    if (i0 + lane < hi) a.row[i0 + lane] = (int32_t)(base + lower);
  };
  constexpr int kAhead = 4;  // groups of 32 slots whose experts are read at once
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kAhead) {
    int e[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t slot = i0 + 32 * u + lane;
      e[u] = slot < hi ? __ldg(a.idx + slot) : -1;
      if ((uint32_t)e[u] >= (uint32_t)E) e[u] = E;
    }
    if (i0 + 32 * kAhead <= hi) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) rank_slots(i0 + 32 * u, e[u]);
    } else {  // not all of them: a group takes 0.25 us (4096 slots 6.3 us with empty ones, 5.6 without)
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + 32 * u < hi) rank_slots(i0 + 32 * u, e[u]);
    }
  }
  __syncthreads();
  if (tid < E) {  // counts of the warps -> first ranks within the CTA
    uint32_t sum = 0;
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
      const uint32_t c = s_cnt[w * E + tid];
      s_cnt[w * E + tid] = sum;
      sum += c;
    }
    s_tot[tid] = sum;
  }
  uint32_t before = 0, total = 0;  // of expert tid: slots in the CTAs before this one, in all
  if (ctas > 1) {
    cluster_sync_all();
    if (tid < E) {
      uint32_t v[kPlanCtas];  // all in flight at once
#pragma unroll
      for (int c = 0; c < kPlanCtas; ++c) {
        v[c] = 0;
        if (c < ctas)
          asm volatile("ld.shared::cluster.u32 %0, [%1];"
                       : "=r"(v[c])
                       : "r"(mapa_shared(smem_u32(s_tot + tid), (uint32_t)c))
                       : "memory");
      }
#pragma unroll
      for (int c = 0; c < kPlanCtas; ++c) {
        if (c < rank) before += v[c];
        total += v[c];
      }
    }
    cluster_sync_all();  // every CTA has read the totals: they may be replaced, and a CTA may leave
  } else if (tid < E) {
    total = s_tot[tid];
  }
  // the experts' first rows: exclusive prefix of the aligned counts
  const uint32_t al = (uint32_t)a.align;
  const uint32_t rows = (total + al - 1) / al * al;
  uint32_t inc = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    uint32_t v = s_scan[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += u;
    }
    s_scan[lane] = v;
  }
  __syncthreads();
  const uint32_t first = inc - rows + (warp ? s_scan[warp - 1] : 0u);
  if (tid < E) {
    s_tot[tid] = first + before;  // row of this CTA's first slot of the expert
    if (rank == 0) {
      a.offs[tid] = (int32_t)first;
      a.counts[tid] = (int32_t)total;
      if (tid == E - 1) a.offs[E] = (int32_t)(first + rows);
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int64_t slot = lo + lane; slot < hi; slot += 32) {
    const int e = __ldg(a.idx + slot);
    const bool ok = (uint32_t)e < (uint32_t)E;
    const int r = ok ? a.row[slot] + (int)(mine[e] + s_tot[e]) : -1;
    a.row[slot] = r;
    if (ok) a.src[r] = (int32_t)slot;
  }
}

// ---------------------------------------------------------------------------
// Combine: y[t] = sum_j w[t,j] ye[row[t,j]], and its gradient
// ---------------------------------------------------------------------------

namespace {

// VEC consecutive bf16 values as fp32
template <int VEC>
struct Bf16s {
  static_assert(VEC == 8 || VEC == 4 || VEC == 2 || VEC == 1, "one access of 16, 8, 4 or 2 bytes");
  uint32_t v[VEC == 1 ? 1 : VEC / 2];
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (VEC == 8) {
      const uint4 q = ld_nc_v4(p);
      v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else if constexpr (VEC == 4) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      v[0] = q.x, v[1] = q.y;
    } else if constexpr (VEC == 2) {
      v[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      v[0] = __ldg(p);
    }
  }
  __device__ __forceinline__ void load(const uint16_t* p, uint64_t policy) {
    if constexpr (VEC == 8) {
      asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                   : "l"(p), "l"(policy));
    } else {
      load(p);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (VEC == 1 ? 1 : VEC / 2); ++i) v[i] = 0;
  }
  __device__ __forceinline__ float get(int i) const { return (i & 1) ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]); }
};

template <int VEC>
__device__ __forceinline__ void store_bf16s(uint16_t* p, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  } else if constexpr (VEC == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(f[0], f[1]);
  } else {
    *p = f32_to_bf16(f[0]);
  }
}

template <int VEC>
__device__ __forceinline__ void store_bf16s(uint16_t* p, const float (&f)[VEC], uint64_t policy) {
  if constexpr (VEC == 8) {
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1,%2,%3,%4}, %5;" ::"l"(p), "r"(pack_bf16x2(f[0], f[1])),
                 "r"(pack_bf16x2(f[2], f[3])), "r"(pack_bf16x2(f[4], f[5])), "r"(pack_bf16x2(f[6], f[7])), "l"(policy)
                 : "memory");
  } else {
    store_bf16s<VEC>(p, f);
  }
}
// L2 policy of data that is touched once: it is the first to leave.
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// CTAs an SM that the registers leave room for, by the columns an access takes:
// narrow accesses need more warps for the same bytes in flight; a few registers
// spill for it.  8192 tokens, 8 experts each, in us, at 4001 / 4002 / 4004
// columns (1 / 2 / 4): y 272 / 114 / 98 (430 / 170 / 117 with four CTAs and a
// CTA for 256 accesses), dw 190 / 100 / 90 (334 / 134 / 102 with three), dw
// with dye 467 / 216 / 193 (642 / 230 / 224 with two).
constexpr int combine_ctas_sm(int vec) { return vec == 1 ? 8 : 4; }
constexpr int combine_dw_ctas(int vec) { return vec <= 2 ? 6 : vec == 4 ? 5 : 3; }
constexpr int combine_bwd_ctas(int vec) { return vec == 1 ? 5 : vec == 2 ? 4 : vec == 4 ? 3 : 2; }
constexpr int kCombinePiece = 16;  // rows of an expert that a CTA of the gradient takes, on average

}  // namespace

// One thread VEC columns of a token, or of the tokens whose rows make eight:
// eight rows are read before the first is used (KB of each token; one token at
// a time 8192 tokens x 4096, two experts each, took 60 us, so 33).  Narrow rows
// share a CTA (32768 tokens x 256, eight experts: 39 us, so 25).  Bound by
// memory: 16384 tokens x 4096, eight experts each, 1.21 GB in 179 us, the copy
// rate.  Four CTAs an SM: with more or fewer loads in flight than theirs the
// memory is slower (three 210 us, five 198).
template <int VEC, int KB>
__global__ void __launch_bounds__(kCombineThreads, combine_ctas_sm(VEC)) moe_combine_kernel(const CombineArgs a) {
  constexpr int kTokens = kCombineBatch / KB;
  pdl_launch_dependents();
  pdl_wait();
  const CombineThread me = combine_thread(blockIdx.x, (int)threadIdx.x, a.geom, a.T, a.N, VEC, KB);
  const int64_t t0 = me.t0;
  if (!me.on) return;
  constexpr int U = VEC == 2 ? 2 : 1;  // accesses of a row at once
  const int64_t step = (int64_t)a.geom.cols * VEC;
  for (int64_t nb = me.n0; nb < a.N; nb += U * step) {
    float acc[U][VEC] = {};
    for (int j0 = 0; j0 < a.k; j0 += KB) {  // (once where KB < 8, as k is at most KB)
      Bf16s<VEC> v[U][kCombineBatch];
      float w[kCombineBatch];
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i) {
        const int64_t t = t0 + i / KB, slot = t * a.k + j0 + i % KB;
        const int r = t < a.T && j0 + i % KB < a.k ? __ldg(a.row + slot) : -1;
        const bool ok = r >= 0 && r < a.R;
        w[i] = ok ? (a.w ? __ldg(a.w + slot) : 1.0f) : 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (ok && (u == 0 || nb + u * step < a.N)) v[u][i].load(a.ye + (int64_t)r * a.ldye + nb + u * step);
          else v[u][i].zero();
        }
      }
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t n = nb + u * step;
#pragma unroll
          for (int c = 0; c < VEC; ++c)
            acc[u][c] = fmaf(w[i], v[u][i].get(c), kTokens > 1 && i % KB == 0 ? 0.0f : acc[u][c]);
          if (kTokens > 1 && i % KB == KB - 1 && t0 + i / KB < a.T && (u == 0 || n < a.N))
            store_bf16s<VEC>(a.y + (t0 + i / KB) * a.ldy + n, acc[u]);
        }
    }
    if (kTokens == 1)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u == 0 || nb + u * step < a.N) store_bf16s<VEC>(a.y + t0 * a.ldy + nb + u * step, acc[u]);
    if (VEC == 8) break;
  }
}

// The gradient comes in two forms that give the same bits: a dot product dw is
// the sum over eight column classes in order, class c the columns c 32 VEC + l
// VEC .. of every 256 VEC (lane l), each class a chain a lane and a tree over
// the lanes.
//
// dw alone: one CTA a token (or the tokens whose rows make eight, KB each),
// whose warps are the classes; dy is read once and the rows together (16384
// tokens x 4096, 8 experts: 167 us, 1.2 GB).  WARP: narrow rows, a warp for all
// classes of its tokens (rows of 1024 values 51 us against 71, 1536 73 against
// 80, 2048 95 against 91; 16384 tokens, 8 experts).
template <int VEC, int KB, bool WARP>
__global__ void __launch_bounds__(kCombineThreads, combine_dw_ctas(VEC)) moe_combine_dw_kernel(const CombineBwdArgs a) {
  constexpr int kClasses = kCombineThreads / 32, kTokens = kCombineBatch / KB;
  __shared__ float s_part[kClasses][kCombineBatch];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = (WARP ? (int64_t)blockIdx.x * kClasses + warp : (int64_t)blockIdx.x) * kTokens;
  for (int j0 = 0; j0 < a.k; j0 += KB) {
    int r[kCombineBatch];
#pragma unroll
    for (int i = 0; i < kCombineBatch; ++i) {
      const int64_t t = t0 + i / KB;
      r[i] = t < a.T && j0 + i % KB < a.k ? __ldg(a.row + t * a.k + j0 + i % KB) : -1;
      if (r[i] >= a.R) r[i] = -1;
    }
    // the dots of class c, over all lanes
    auto dots = [&](int c, float (&dot)[kCombineBatch]) {
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i) dot[i] = 0.0f;
      for (int64_t n = (int64_t)(32 * c + lane) * VEC; n < a.N; n += kCombineThreads * VEC) {
        Bf16s<VEC> d[kTokens], v[kCombineBatch];
#pragma unroll
        for (int m = 0; m < kTokens; ++m) {
          if (t0 + m < a.T) d[m].load(a.dy + (t0 + m) * a.lddy + n);
          else d[m].zero();
        }
#pragma unroll
        for (int i = 0; i < kCombineBatch; ++i) {
          if (r[i] >= 0) v[i].load(a.ye + (int64_t)r[i] * a.ldye + n);
          else v[i].zero();
        }
#pragma unroll
        for (int i = 0; i < kCombineBatch; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) dot[i] = fmaf(d[i / KB].get(e), v[i].get(e), dot[i]);
      }
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i) dot[i] = warp_sum(dot[i]);
    };
    float dot[kCombineBatch], sum = 0.0f;  // sum: of dot `lane` (WARP), of dot `tid`
    if constexpr (WARP) {
      for (int c = 0; c < kClasses && c * 32 * VEC < a.N; ++c) {
        dots(c, dot);
#pragma unroll
        for (int i = 0; i < kCombineBatch; ++i)
          if (lane == i) sum += dot[i];
      }
    } else {
      dots(warp, dot);
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i)
        if (lane == 0) s_part[warp][i] = dot[i];
      __syncthreads();
      if (tid < kCombineBatch) {
#pragma unroll
        for (int c = 0; c < kClasses; ++c) sum += s_part[c][tid];
      }
      __syncthreads();
    }
    const int i = WARP ? lane : tid;
    if (i < kCombineBatch && t0 + i / KB < a.T && j0 + i % KB < a.k) {
      const int64_t slot = (t0 + i / KB) * a.k + j0 + i % KB;
      const int row = __ldg(a.row + slot);
      a.dw[slot] = row >= 0 && row < a.R ? sum : 0.0f;  // (dy may hold an infinity, times the zeros read for no row)
    }
  }
}

// dw and dye: a warp takes sorted rows r of slots (t, j), dye[r] = w[t,j] dy[t]
// from the same read of dy.  By rows, because dye scattered over memory, row by
// row of each token, was written at half the rate of a copy (655 us for 16384
// tokens x 4096, 8 experts each).  A CTA takes one of `pieces` equal pieces of
// one expert's rows, the CTAs piece by piece over all experts: the slots of an
// expert are sorted by token, so the rows of one piece belong to neighbouring
// tokens in every expert, and a token's dy is read from memory for one of them
// and from L2 for most others (in the order of the rows it was read 7 of 8
// times: 2.1 GB in, 1.1 out, 465 us, the memory's limit).  ye and dye, touched
// once, are marked to leave L2 first.  With less to read it is a matter of
// loads in flight: 16 a lane 397 us, 8 of them 482.  Pieces of 8 / 16 / 32 rows:
// 401 / 397 / 430.  The last CTAs write the zeros of rows past the experts and
// of slots without a row.
//
// CL: column classes of a row, all eight or fewer of narrow rows, of which a
// warp then takes 8 / CL at once and a CTA as many times the rows (32768 x 256,
// 8 experts: 60 us, row by row 216; 16384 x 1024: 99 and 134).
template <int VEC, int CL>
__global__ void __launch_bounds__(kCombineThreads, combine_bwd_ctas(VEC))
    moe_combine_bwd_kernel(const CombineBwdArgs a) {
  constexpr int kClasses = kCombineThreads / 32, kRows = kClasses / CL;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
  const uint64_t once = evict_first_policy();
  const int64_t blocks = a.E * a.pieces;
  int64_t r = 0, end = 0;
  if ((int64_t)blockIdx.x < blocks) {
    const int64_t e = blockIdx.x % a.E, piece = blockIdx.x / a.E;
    const int64_t lo = max(__ldg(a.offs + e), 0), n = min((int64_t)__ldg(a.offs + e + 1), a.R) - lo;
    if (n <= 0) return;
    r = lo + n * piece / a.pieces + warp * kRows;
    end = lo + n * (piece + 1) / a.pieces;
  } else {
    const int64_t at = (blockIdx.x - blocks) * kClasses + warp, warps = (gridDim.x - blocks) * kClasses;
    for (int64_t i = at * 32 + lane; i < a.T * a.k; i += warps * 32) {
      const int row = __ldg(a.row + i);
      if (row < 0 || row >= a.R) a.dw[i] = 0.0f;
    }
    float z[VEC] = {};
    for (int64_t q = max((int64_t)__ldg(a.offs + a.E), (int64_t)0) + at; q < a.R; q += warps)
      for (int64_t n = (int64_t)lane * VEC; n < a.N; n += 32 * VEC) store_bf16s<VEC>(a.dye + q * a.lddye + n, z, once);
    return;
  }
  auto read_slot = [&](int64_t r0) { return lane < kRows && r0 + lane < end ? __ldg(a.src + r0 + lane) : -1; };
  int slot = read_slot(r);  // of lane g: row r + g's
  for (; r < end; r += kClasses * kRows) {
    const int t_of = slot >= 0 ? (int)min((int64_t)((uint32_t)slot / (uint32_t)a.k), a.T) : (int)a.T;
    const float w_of = t_of < a.T ? (a.w ? __ldg(a.w + slot) : 1.0f) : 0.0f;
    const int slot_next = read_slot(r + kClasses * kRows);
    float dot[kClasses], w[kRows];
    int t[kRows];  // a.T: padding
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      t[g] = __shfl_sync(kFull, t_of, g);
      w[g] = __shfl_sync(kFull, w_of, g);
    }
#pragma unroll
    for (int c = 0; c < kClasses; ++c) dot[c] = 0.0f;
    for (int64_t base = (int64_t)lane * VEC; base < a.N; base += kCombineThreads * VEC) {
      Bf16s<VEC> d[kClasses], v[kClasses];
#pragma unroll
      for (int i = 0; i < kClasses; ++i) {
        const int g = i / CL;
        const int64_t n = base + i % CL * 32 * VEC;
        if (t[g] < a.T && n < a.N) {
          v[i].load(a.ye + (r + g) * a.ldye + n, once);
          d[i].load(a.dy + t[g] * a.lddy + n);
        } else {
          v[i].zero();
          d[i].zero();
        }
      }
#pragma unroll
      for (int i = 0; i < kClasses; ++i) {
        const int g = i / CL;
        const int64_t n = base + i % CL * 32 * VEC;
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          dot[i] = fmaf(d[i].get(e), v[i].get(e), dot[i]);
          o[e] = w[g] * d[i].get(e);
        }
        if (n < a.N && r + g < end) store_bf16s<VEC>(a.dye + (r + g) * a.lddye + n, o, once);
      }
      if constexpr (CL < kClasses) break;  // (N is at most CL classes)
    }
    float sum = 0.0f;  // of lane g: row r + g's
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      float of_row = 0.0f;
#pragma unroll
      for (int c = 0; c < CL; ++c) of_row += warp_sum(dot[g * CL + c]);
      if (lane == g) sum = of_row;
    }
    if (lane < kRows && t_of < a.T) a.dw[slot] = sum;
    slot = slot_next;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// f with the experts a lane takes as a compile-time number, so that they stay in
// registers: E / 32 rounded up to one of these.  The nearest against the next
// one up, 32768 tokens, k 8: 64 experts 10.9 / 11.8 us, 128 12.8 / 15.5, 160
// 14.4 / 15.4, 256 17.3 / 22.7 (in groups 34.1 / 65.2), 384 24.0 / 31.6.
template <typename F>
static cudaError_t by_vpl(int64_t E, F&& f) {
  const int64_t n = cdiv(E, 32);
  if (n <= 1) return f(std::integral_constant<int, 1>{});
  if (n <= 2) return f(std::integral_constant<int, 2>{});
  if (n <= 3) return f(std::integral_constant<int, 3>{});
  if (n <= 4) return f(std::integral_constant<int, 4>{});
  if (n <= 5) return f(std::integral_constant<int, 5>{});
  if (n <= 6) return f(std::integral_constant<int, 6>{});
  if (n <= 8) return f(std::integral_constant<int, 8>{});
  if (n <= 10) return f(std::integral_constant<int, 10>{});
  if (n <= 12) return f(std::integral_constant<int, 12>{});
  if (n <= 16) return f(std::integral_constant<int, 16>{});
  if (n <= 24) return f(std::integral_constant<int, 24>{});
  return f(std::integral_constant<int, 32>{});
}

template <typename F>
static cudaError_t by_bool(bool v, F&& f) {
  return v ? f(std::true_type{}) : f(std::false_type{});
}

static bool aligned_to(const void* p, int64_t ld_bytes, int64_t n) {
  return reinterpret_cast<uintptr_t>(p) % n == 0 && ld_bytes % n == 0;
}

cudaError_t launch_moe_route(const RouteArgs& args, cudaStream_t st) {
  RouteArgs a = args;
  const int el = a.f32 ? 4 : 2;
  // four logits, four biases a load where they are aligned: 32768 x 256 17.3 us against
  // 18.0 with an odd row stride, with a bias 24.9 against 26.1
  a.vec = aligned_to(a.logits, a.ldl * el, 4 * el);
  a.bias_vec = aligned_to(a.bias, 0, 16);
  return by_vpl(a.E, [&](auto vpl) {
    constexpr int kVpl = decltype(vpl)::value;
    if (a.groups > 1) {
      // a power of two of lanes a group, whole lanes where the groups' size allows it (no
      // exchange of the values then: 32768 x 192, sigmoid, 4 groups 27.5 us; 6 groups, which
      // do not fit lanes, 40.8)
      const int64_t S = a.E / a.groups, lanes = S / kVpl;
      a.group_whole = S % kVpl == 0 && (lanes & (lanes - 1)) == 0;
      a.group_lanes = 1;
      if (a.group_whole) a.group_lanes = (int)lanes;
      else
        while (a.group_lanes * 2 * a.groups <= 32) a.group_lanes *= 2;
    }
    constexpr size_t smem = (size_t)(kRouteThreads / 32) * kVpl * 64 * 4;
    static_assert(smem <= 48 * 1024, "no opt-in needed");
    return by_bool(a.f32, [&](auto f32) {
      return by_bool(a.sigmoid, [&](auto sig) {
        return by_bool(a.bias != nullptr, [&](auto bias) {
          return launch_pdl(moe_route_kernel<kVpl, decltype(f32)::value, decltype(sig)::value, decltype(bias)::value>,
                            (unsigned)cdiv(a.T, kRouteThreads / 32), kRouteThreads, smem, st, a);
        });
      });
    });
  });
}

cudaError_t launch_moe_route_bwd(const RouteBwdArgs& args, cudaStream_t st) {
  RouteBwdArgs a = args;
  const int el = a.f32 ? 4 : 2;
  // pairs of experts a load and a store: 32768 x 256 15.5 us against 17.1 with an odd row stride
  a.vec = aligned_to(a.logits, a.ldl * el, 2 * el) && aligned_to(a.dlogits, a.ldd * el, 2 * el);
  auto go = [&](auto pairs) {
    constexpr int kPairs = decltype(pairs)::value;
    return by_bool(a.f32, [&](auto f32) {
      return by_bool(a.sigmoid, [&](auto sig) {
        constexpr int threads = kRouteBwdThreads<kPairs, decltype(sig)::value>;
        return launch_pdl(moe_route_bwd_kernel<kPairs, decltype(f32)::value, decltype(sig)::value>,
                          (unsigned)cdiv(a.T, threads / 32), threads, 0, st, a);
      });
    });
  };
  // pairs a lane, a compile-time number as in the forward; the nearest against the next one up,
  // 32768 tokens: 64 experts 10.6 / 11.6 us, 160 13.4 / 22.9 (8 pairs for 3), 256 15.5 / 22.7
  const int64_t n = cdiv(a.E, 64);
  if (n <= 1) return go(std::integral_constant<int, 1>{});
  if (n <= 2) return go(std::integral_constant<int, 2>{});
  if (n <= 3) return go(std::integral_constant<int, 3>{});
  if (n <= 4) return go(std::integral_constant<int, 4>{});
  if (n <= 8) return go(std::integral_constant<int, 8>{});
  return go(std::integral_constant<int, 16>{});
}

template <int BITS>
static cudaError_t run_plan(const PlanArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)(33 * a.E) * 4;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  static int most = 8;  // CTAs of the cluster: kPlanCtas where the device can hold one, else the portable 8
  std::call_once(once, [] {
    const int max_smem = 33 * kMaxGroups * 4;
    attr_err = cudaFuncSetAttribute(moe_plan_kernel<BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
    if (attr_err != cudaSuccess) return;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlanCtas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = max_smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPlanCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(moe_plan_kernel<BITS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, moe_plan_kernel<BITS>, &cfg) == cudaSuccess && n >= 1)
      most = kPlanCtas;
    (void)cudaGetLastError();  // a size the device refuses leaves no error behind
  });
  if (attr_err != cudaSuccess) return attr_err;
  // A CTA for every 1024 slots: fewer leave a warp more steps, more pay the cluster's barriers
  // (about 1 us).  With 512 / 1024 / 2048 / 8192 slots a CTA, 64 experts, in us: 1024 slots
  // 5.4 / 4.5 / 4.6 / 4.6, 4096 5.5 / 5.6 / 6.7 / 7.4, 16384 5.7 / 5.7 / 6.8 / 12.7.
  int ctas = 1;
  while (ctas < most && (int64_t)ctas * kPlanThreads < a.n) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, moe_plan_kernel<BITS>, a);
}

// A ballot a bit of the experts' numbers: the fewest bits against 11, 131072 slots: 64 experts
// 13.3 / 14.7 us, 200 14.8 / 15.6; 8192 slots, 8 experts 5.9 / 6.9.
cudaError_t launch_moe_plan(const PlanArgs& a, cudaStream_t st) {
  if (a.E < 1 << 5) return run_plan<5>(a, st);
  if (a.E < 1 << 7) return run_plan<7>(a, st);
  if (a.E < 1 << 9) return run_plan<9>(a, st);
  return run_plan<11>(a, st);
}

// Columns an access takes: 8, 4, 2 or 1, the most that the width, the rows'
// strides and their bases allow (one access then stays within a row, aligned).
// 8192 tokens, eight rows each: 90 us at 4000 columns (8), 98 at 4004 (4), 114
// at 4002 (2), 272 at 4001 (1).
struct RowAlign {
  int64_t bits;
  explicit RowAlign(int64_t N) : bits(N) {}
  RowAlign& row(const void* p, int64_t ld) {
    bits |= (int64_t)(reinterpret_cast<uintptr_t>(p) / 2) | ld;
    return *this;
  }
  template <typename F>
  cudaError_t go(F&& f) const {
    if (bits % 8 == 0) return f(std::integral_constant<int, 8>{});
    if (bits % 4 == 0) return f(std::integral_constant<int, 4>{});
    if (bits % 2 == 0) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
  }
};

// f with combine_batch(k) as a compile-time number.
template <typename F>
static cudaError_t by_batch(int k, F&& f) {
  switch (combine_batch(k)) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    default: return f(std::integral_constant<int, kCombineBatch>{});
  }
}

cudaError_t launch_moe_combine(const CombineArgs& args, cudaStream_t st) {
  return RowAlign(args.N).row(args.ye, args.ldye).row(args.y, args.ldy).go([&](auto vec) {
    return by_batch(args.k, [&](auto batch) {
      constexpr int kVec = decltype(vec)::value, kBatch = decltype(batch)::value;
      CombineArgs a = args;
      a.geom = combine_geom(a.N, kVec);
      return launch_pdl(moe_combine_kernel<kVec, kBatch>, (unsigned)combine_ctas(a.T, a.geom, kBatch),
                        (unsigned)combine_threads(a.geom), 0, st, a);
    });
  });
}

cudaError_t launch_moe_combine_bwd(const CombineBwdArgs& args, int num_sms, cudaStream_t st) {
  const RowAlign rows = RowAlign(args.N).row(args.dy, args.lddy).row(args.ye, args.ldye);
  if (!args.dye) {
    if (args.T == 0) return cudaSuccess;
    return rows.go([&](auto vec) {
      return by_batch(args.k, [&](auto batch) {
        constexpr int kVec = decltype(vec)::value, kBatch = decltype(batch)::value;
        const int64_t groups = cdiv(args.T, kCombineBatch / kBatch);
        if (args.N <= 6 * 32 * kVec)
          return launch_pdl(moe_combine_dw_kernel<kVec, kBatch, true>, (unsigned)cdiv(groups, kCombineThreads / 32),
                            kCombineThreads, 0, st, args);
        return launch_pdl(moe_combine_dw_kernel<kVec, kBatch, false>, (unsigned)groups, kCombineThreads, 0, st, args);
      });
    });
  }
  return RowAlign(rows).row(args.dye, args.lddye).go([&](auto vec) {
    constexpr int kVec = decltype(vec)::value;
    auto run = [&](auto classes) {
      constexpr int kCl = decltype(classes)::value;
      CombineBwdArgs a = args;
      a.pieces = std::max<int64_t>(cdiv(a.R, a.E * kCombinePiece * (8 / kCl)), 1);
      // and CTAs for the zeros
      const int64_t zeros =
          std::min<int64_t>(cdiv(std::max(cdiv(a.T * a.k, 32), a.R), kCombineThreads / 32), 2 * num_sms);
      const unsigned ctas = (unsigned)(a.E * a.pieces + zeros);
      return launch_pdl(moe_combine_bwd_kernel<kVec, kCl>, ctas, kCombineThreads, 0, st, a);
    };
    const int64_t classes = cdiv(args.N, 32 * kVec);
    if (classes <= 1) return run(std::integral_constant<int, 1>{});
    if (classes <= 2) return run(std::integral_constant<int, 2>{});
    if (classes <= 4) return run(std::integral_constant<int, 4>{});
    return run(std::integral_constant<int, 8>{});
  });
}

}  // namespace bfp8
