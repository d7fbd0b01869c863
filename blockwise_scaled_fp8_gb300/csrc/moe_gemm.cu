// Routed product of a mixture-of-experts layer for batches that give an
// expert few rows (decoding): row r of C is the codes of A's row src[r] / k
// (or r) against the weight of the expert whose range offs[e] .. offs[e+1]
// holds r, in the method of the 1x128 x 128x128 GEMM ("Mask a_s/b_s scale
// loads in blockwise FP8 training GEMM kernels"):
//   C[r,n] = sum over 128-wide K-blocks kb of a_s[row,kb] b_s[n/128,kb] P_kb,
// P_kb the e4m3 x e4m3 partial product, promoted per K-block into fp32.
//
// Each reached expert's weight is read once from memory, which is what bounds
// the product here.  So nothing is staged: a warp's matrix instruction takes
// 16 rows of W (its A) and 8 tokens (its B) straight from the registers that
// the loads filled.  A lane holds 16 consecutive bytes of a row per load and
// uses them as the k-slices of two instructions: the sum over k does not care
// which k a slice holds as long as both operands agree, so no byte moves
// between lanes.  The warps of a CTA split a 16-row block's K-blocks and add
// their fp32 sums in warp order through shared memory.
#include "common.cuh"
#include "kernels.h"

namespace bfp8 {

namespace {

constexpr int kRpThreads = 256;
constexpr int kRpWarps = kRpThreads / 32;
constexpr int kRpRows = 16;   // rows of W an item
constexpr int kRpUnroll = 2;  // K-blocks in flight a warp

// D (16 x 8, fp32) += A (16 x 32 e4m3, row) B (32 x 8 e4m3, column)
__device__ __forceinline__ void mma_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first n (0 .. 16) bytes of v, the others zero.
__device__ __forceinline__ uint4 first_bytes(uint4 v, int n) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = n - 4 * i;
    if (b < 4) w[i] &= b <= 0 ? 0u : (1u << (8 * b)) - 1u;
  }
  return v;
}

}  // namespace

// TN: 8-token blocks an item holds at once; an expert with more rows walks W
// again for the next 8 TN.
template <int TN>
__global__ void __launch_bounds__(kRpThreads, 2) gemm_routed_kernel(const GemmRoutedArgs a) {
  __shared__ int s_expert[kMaxGroups];
  __shared__ int s_count[kRpWarps];
  __shared__ float s_part[kRpWarps][kRpRows][8 * TN + 1];
  __shared__ int s_tok[8 * TN];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = (int)a.E;
  // the experts that hold rows, in order
  int reached = 0;
  for (int e0 = 0; e0 < E; e0 += kRpThreads) {
    const int e = e0 + tid;
    const bool on = e < E && __ldg(a.offs + e + 1) > __ldg(a.offs + e);
    const uint32_t vote = __ballot_sync(0xffffffffu, on);
    if (lane == 0) s_count[warp] = __popc(vote);
    __syncthreads();
    int at = reached;
    for (int w = 0; w < kRpWarps; ++w) {
      if (w < warp) at += s_count[w];
      reached += s_count[w];
    }
    if (on) s_expert[at + __popc(vote & ((1u << lane) - 1u))] = e;
    __syncthreads();
  }
  const int64_t Kb = cdiv(a.K, kBlock), Nb = cdiv(a.N, kBlock);
  const int blocks = (int)cdiv(a.N, kRpRows);
  const int64_t items = (int64_t)reached * blocks;
  const int g = lane >> 2, q = lane & 3;
  const bool k_tail = a.K % kBlock != 0;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int e = s_expert[item / blocks];
    const int64_t n0 = (item % blocks) * kRpRows;
    int64_t r0 = __ldg(a.offs + e), r1 = __ldg(a.offs + e + 1);
    r0 = r0 < 0 ? 0 : r0;
    r1 = r1 > a.R ? a.R : r1;
    const int64_t na = n0 + g < a.N ? n0 + g : a.N - 1, nb = n0 + g + 8 < a.N ? n0 + g + 8 : a.N - 1;
    const uint8_t* wa = a.qb + (e * a.N + na) * a.ldb + q * 16;
    const uint8_t* wb = a.qb + (e * a.N + nb) * a.ldb + q * 16;
    const float* sb = a.sb + (e * Nb + n0 / kBlock) * a.ldsb;
    for (int64_t m0 = r0; m0 < r1; m0 += 8 * TN) {
      // the A row of each of the item's tokens (-1: zeros)
      if (tid < 8 * TN) {
        int64_t tok = -1;
        if (m0 + tid < r1) {
          tok = m0 + tid;
          if (a.src) {
            const int slot = __ldg(a.src + m0 + tid);
            tok = slot >= 0 ? (int64_t)((uint32_t)slot / (uint32_t)a.k) : -1;
          }
          if (tok >= a.T) tok = -1;
        }
        s_tok[tid] = (int)tok;
      }
      __syncthreads();
      const uint8_t* xp[TN];
      int tok[TN];
      const float* sa0[TN];
      const float* sa1[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        tok[j] = s_tok[8 * j + g];
        xp[j] = a.qa + (int64_t)max(tok[j], 0) * a.lda + q * 16;
        sa0[j] = a.sa + max(s_tok[8 * j + 2 * q], 0);
        sa1[j] = a.sa + max(s_tok[8 * j + 2 * q + 1], 0);
      }
      float acc[TN][4];
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
      for (int64_t kb0 = warp; kb0 < Kb; kb0 += kRpWarps * kRpUnroll) {
        uint4 w[kRpUnroll][4], x[kRpUnroll][TN][2];
        float s0[kRpUnroll][TN], s1[kRpUnroll][TN];
#pragma unroll
        for (int u = 0; u < kRpUnroll; ++u) {
          const int64_t kb = kb0 + u * kRpWarps;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t k = kb * kBlock + h * 64;
            const bool in = k + q * 16 < a.K;
            w[u][2 * h] = in ? ld_nc_v4(wa + k) : make_uint4(0, 0, 0, 0);
            w[u][2 * h + 1] = in ? ld_nc_v4(wb + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < TN; ++j)
              x[u][j][h] = in && tok[j] >= 0 ? __ldg(reinterpret_cast<const uint4*>(xp[j] + k)) : make_uint4(0, 0, 0, 0);
          }
          const float b = kb < Kb ? __ldg(sb + kb) : 0.0f;
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            s0[u][j] = kb < Kb ? __ldg(sa0[j] + kb * a.ldsa) * b : 0.0f;
            s1[u][j] = kb < Kb ? __ldg(sa1[j] + kb * a.ldsa) * b : 0.0f;
          }
        }
#pragma unroll
        for (int u = 0; u < kRpUnroll; ++u) {
          const int64_t kb = kb0 + u * kRpWarps;
          if (k_tail && kb >= Kb - 1) {  // the bytes past K are not data
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int64_t left = a.K - (kb * kBlock + h * 64 + q * 16);
              const int n = left < 0 ? 0 : left > 16 ? 16 : (int)left;
              w[u][2 * h] = first_bytes(w[u][2 * h], n);
              w[u][2 * h + 1] = first_bytes(w[u][2 * h + 1], n);
#pragma unroll
              for (int j = 0; j < TN; ++j) x[u][j][h] = first_bytes(x[u][j][h], n);
            }
          }
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 A = w[u][2 * h], B = w[u][2 * h + 1], X = x[u][j][h];
              mma_16x8x32(d, A.x, B.x, A.y, B.y, X.x, X.y);
              mma_16x8x32(d, A.z, B.z, A.w, B.w, X.z, X.w);
            }
            acc[j][0] = fmaf(s0[u][j], d[0], acc[j][0]);
            acc[j][1] = fmaf(s1[u][j], d[1], acc[j][1]);
            acc[j][2] = fmaf(s0[u][j], d[2], acc[j][2]);
            acc[j][3] = fmaf(s1[u][j], d[3], acc[j][3]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        s_part[warp][g][8 * j + 2 * q] = acc[j][0];
        s_part[warp][g][8 * j + 2 * q + 1] = acc[j][1];
        s_part[warp][g + 8][8 * j + 2 * q] = acc[j][2];
        s_part[warp][g + 8][8 * j + 2 * q + 1] = acc[j][3];
      }
      __syncthreads();
      for (int i = tid; i < kRpRows * 8 * TN; i += kRpThreads) {
        const int nl = i % kRpRows, m = i / kRpRows;
        float sum = s_part[0][nl][m];
#pragma unroll
        for (int v = 1; v < kRpWarps; ++v) sum += s_part[v][nl][m];
        if (m0 + m < r1 && n0 + nl < a.N)
          a.c[(m0 + m) * a.ldc + n0 + nl] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
      }
      __syncthreads();  // the sums and the token list are free again
    }
  }
}

cudaError_t launch_gemm_routed(const GemmRoutedArgs& a, int num_sms, cudaStream_t st) {
  const int64_t reach = a.E < a.R ? a.E : a.R;  // experts that can hold rows
  const int64_t items = reach * cdiv(a.N, kRpRows), cap = 2 * (int64_t)num_sms;
  const unsigned grid = (unsigned)(items < cap ? items : cap);
  const int64_t rows = cdiv(a.R, a.E);  // rows an expert, spread evenly
  if (rows <= 4) return launch_pdl(gemm_routed_kernel<1>, grid, kRpThreads, 0, st, a);
  if (rows <= 12) return launch_pdl(gemm_routed_kernel<2>, grid, kRpThreads, 0, st, a);
  return launch_pdl(gemm_routed_kernel<4>, grid, kRpThreads, 0, st, a);
}

}  // namespace bfp8
