/*
 * CPU check of the dispatch kernel's quotient where rows are scaled by weights
 * (test infrastructure; links the oracle's reference rounding).
 *
 * A row's values are X = RN(x w) of bf16 x and one fp32 w, its scale s =
 * RN(max(RN(amax w), 1e-12) / 448).  With 1/s = yh + yl as reciprocal_check.c
 * has it, the kernel takes q = RN(X*yh + RN(X*yl)) (claimed: RNE_e4m3(q) ==
 * RNE_e4m3(clamp(RN(X/s), +-448))).
 *
 * For `groups` pseudo-random (amax, w, yh) the program checks every bf16 x from
 * amax down to 2^-8 of it, both signs, and counts as well what one product
 * RN(X*yh) would get wrong.  Prints "tot=<cases> bad=<mismatches> one=<mismatches>".
 *
 * usage: weighted_check groups
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
static uint32_t to_bits(float x) {
  uint32_t u;
  memcpy(&u, &x, 4);
  return u;
}
static uint64_t next(uint64_t* s) { /* xorshift */
  *s ^= *s << 13;
  *s ^= *s >> 7;
  *s ^= *s << 17;
  return *s;
}

int main(int argc, char** argv) {
  const long groups = argc > 1 ? atol(argv[1]) : 1000;
  unsigned long long tot = 0, bad = 0, one = 0;
#pragma omp parallel for schedule(dynamic, 16) reduction(+ : tot, bad, one)
  for (long i = 0; i < groups; ++i) {
    uint64_t st = 0x9E3779B97F4A7C15ull * (uint64_t)(i + 1) | 1u;
    for (int k = 0; k < 8; ++k) next(&st);
    const float w = from_bits((uint32_t)(0x3C000000u + next(&st) % 0x04000000u)) * (next(&st) & 64u ? -1.0f : 1.0f);
    const uint32_t ab = 0x3000u + (uint32_t)(next(&st) % 0x1800u); /* amax 2^-31 .. 2^17 */
    const float s = ora_group_scale(from_bits(ab << 16) * fabsf(w));
    float yh = from_bits(to_bits((float)(1.0 / (double)s)) + (uint32_t)(next(&st) % 3u) - 1u);
    if (fmaf(-s, yh, 1.0f) < 0.0f) yh = from_bits(to_bits(yh) - 2u);
    const float yl = fmaf(-s, yh, 1.0f) * yh;
    for (uint32_t xb = ab - 0x400u; xb <= ab; ++xb) {
      for (int sg = 0; sg < 2; ++sg) {
        const float x = from_bits((xb << 16) | (sg ? 0x80000000u : 0u)) * w;
        const uint8_t ref = ora_e4m3_rne(x / s);
        if (ora_e4m3_rne(fmaf(x, yh, x * yl)) != ref) bad++;
        if (ora_e4m3_rne(x * yh) != ref) one++;
        tot++;
      }
    }
  }
  printf("tot=%llu bad=%llu one=%llu\n", tot, bad, one);
  return 0;
}
