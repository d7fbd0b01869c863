/*
 * CPU check of the dispatch kernel's quantiser arithmetic (test infrastructure;
 * links the oracle's reference rounding).
 *
 * For a group with scale s the kernel keeps 1/s in two floats: yh, the
 * hardware's approximation (within one ulp), lowered by two ulps where it is
 * too large, and yl = RN(RN(1 - s*yh) * yh) >= 0, what it lacks (a negative yl
 * would lose the sign of a zero x).  For every bf16 x of the group it takes
 *   q = RN(x*yh + RN(x*yl))
 * (claimed: RNE_e4m3(q) == RNE_e4m3(clamp(RN(x/s), +-448)), the method's code,
 * sign of zero included).
 *
 * The program checks the claim for every bf16 amax (step `stride` through the
 * amax values, 1 = all of them), s = RN(max(amax, 1e-12)/448), every bf16 x
 * with |x| <= amax, both signs, and each of the four floats nearest 1/s as yh.
 * Prints "tot=<cases> bad=<mismatches>".
 *
 * usage: reciprocal_check [stride]
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

uint8_t ora_e4m3_rne(float r);
float ora_group_scale(float amax);

static float from_bits(uint32_t u) {
  float x;
  memcpy(&x, &u, 4);
  return x;
}
int main(int argc, char** argv) {
  const uint32_t stride = argc > 1 ? (uint32_t)strtoul(argv[1], NULL, 10) : 1u;
  unsigned long long tot = 0, bad = 0;
  const long n_amax = (long)((0x7F80u + stride - 1) / stride);
#pragma omp parallel for schedule(dynamic, 16) reduction(+ : tot, bad)
  for (long ia = 0; ia < n_amax; ++ia) { /* every finite non-negative bf16 */
    const uint32_t ab = (uint32_t)ia * stride;
    const float s = ora_group_scale(from_bits(ab << 16));
    const double inv = 1.0 / (double)s;
    const float yr = (float)inv;
    const float below = (double)yr > inv ? nextafterf(yr, 0.0f) : yr;
    const float above = (double)yr < inv ? nextafterf(yr, INFINITY) : yr;
    float yh[4] = {nextafterf(below, 0.0f), below, above, nextafterf(above, INFINITY)};
    float yl[4];
    for (int k = 0; k < 4; ++k) {
      if (fmaf(-s, yh[k], 1.0f) < 0.0f) { /* two ulps down (yh is a normal float) */
        uint32_t u;
        memcpy(&u, &yh[k], 4);
        yh[k] = from_bits(u - 2u);
      }
      yl[k] = fmaf(-s, yh[k], 1.0f) * yh[k];
      if (!(yl[k] >= 0.0f)) bad++;
    }
    for (uint32_t xb = 0; xb <= ab; ++xb) {
      for (int sg = 0; sg < 2; ++sg) {
        const float x = from_bits((xb << 16) | (sg ? 0x80000000u : 0u));
        const uint8_t ref = ora_e4m3_rne(x / s);
        for (int k = 0; k < 4; ++k)
          if (ora_e4m3_rne(fmaf(x, yh[k], x * yl[k])) != ref) bad++;
        tot++;
      }
    }
  }
  printf("tot=%llu bad=%llu\n", tot, bad);
  return 0;
}
