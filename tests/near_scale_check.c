/*
 * CPU check of the codes that the few-token experts layer gives its tokens
 * (test infrastructure; links the oracle's reference rounding).
 *
 * The scale is one product, s = RN(max(amax, 1e-12) * RN(1/448)), within an ulp
 * of the quantisation entries' quotient; the codes come from the quantisers'
 * one-step quotient
 *   q0 = RN(x*ny),  r = RN(s*q0 + x),  q1 = RN(r*ny + q0)   (ny near -1/s)
 * with the sign flipped.  Claimed: they are RNE_e4m3(RN(x/s)) for every bf16
 * amax, every bf16 x with |x| <= amax and every ny within an ulp of -1/s.
 * Prints "tot=<pairs> bad=<mismatches>".
 *
 * usage: near_scale_check [stride through the amax values]
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

uint8_t ora_e4m3_rne(float r);

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
  for (long ia = 0; ia < n_amax; ++ia) {
    const uint32_t ab = (uint32_t)ia * stride;
    const float s = fmaxf(from_bits(ab << 16), 1e-12f) * (1.0f / 448.0f);
    const double inv = -1.0 / (double)s;
    const float yr = (float)inv;
    const float lo = (double)yr > inv ? nextafterf(yr, -INFINITY) : yr, hi = (double)yr < inv ? nextafterf(yr, INFINITY) : yr;
    const float ny[4] = {nextafterf(lo, -INFINITY), lo, hi, nextafterf(hi, INFINITY)};
    for (uint32_t xb = 0; xb <= ab; ++xb)
      for (int sign = 0; sign < 2; ++sign, ++tot) {
        const float x = from_bits((xb << 16) | (sign ? 0x80000000u : 0u));
        const uint8_t ref = ora_e4m3_rne(x / s);
        for (int k = 0; k < 4; ++k) {
          const float q0 = x * ny[k], r = fmaf(s, q0, x), q1 = fmaf(r, ny[k], q0);
          if ((uint8_t)(ora_e4m3_rne(q1) ^ 0x80u) != ref) bad++;
        }
      }
  }
  printf("tot=%llu bad=%llu\n", tot, bad);
  return 0;
}
