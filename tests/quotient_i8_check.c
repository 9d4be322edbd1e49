/*
 * Exhaustive host check of the quotient the int8 row quantisation uses.
 *
 * With s = amax / 127 in fp32 the kernels form x / s as fma(x, hi, RN(x lo)),
 * where hi = RN(1 / s) and lo = RN(RN(1 - s hi) hi), for rows with 2^-96 <=
 * amax < 2^100, and by the IEEE division otherwise: further up lo (2^-24 of
 * 1 / s or less) becomes a subnormal number and loses its bits. The code is
 * the quotient rounded to the nearest whole number (ties to even). It has to
 * be the division's for every bf16 amax and every bf16 x with |x| <= amax.
 *
 * Checks every bf16 amax from 2^-96 to the largest finite one with every x of
 * both signs. Built with -DNO_TOP the two floats are used for all of them,
 * which must report differences (at 2^125 and above): the check can fail.
 *
 * Prints the pairs, those taken by the two floats, and the codes that differ;
 * exits 1 on a difference. Build: gcc -O2 -fopenmp -ffp-contract=off -lm
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static float bf16_value(uint32_t pattern) {
  const uint32_t w = pattern << 16;
  float f;
  memcpy(&f, &w, sizeof f);
  return f;
}

/* The kernels round by adding 1.5 * 2^23 and taking the sum's low byte. */
static int code_of(float q) {
  const float sum = q + 12582912.f;
  uint32_t w;
  memcpy(&w, &sum, sizeof w);
  return (int8_t)(w & 0xff);
}

int main(void) {
  const uint32_t first = 31u << 7, last = 0x7F7Fu;
  unsigned long long pairs = 0, two_floats = 0, differ = 0;
#pragma omp parallel for schedule(dynamic, 64) reduction(+ : pairs, two_floats, differ)
  for (uint32_t pa = first; pa <= last; ++pa) {
    const float amax = bf16_value(pa), s = amax / 127.0f;
    const float hi = 1.0f / s, lo = fmaf(-s, hi, 1.0f) * hi;
#ifdef NO_TOP
    const int fast = 1;
#else
    const int fast = amax < 0x1p100f;
#endif
    for (uint32_t px = 0; px <= pa; ++px) {
      for (int neg = 0; neg <= 1; ++neg) {
        const float x = neg ? -bf16_value(px) : bf16_value(px);
        const float q = fast ? fmaf(x, hi, x * lo) : x / s;
        const int want = (int)rintf(fminf(fmaxf(x / s, -127.f), 127.f));
        ++pairs;
        two_floats += fast;
        if (code_of(q) != want) {
          ++differ;
#pragma omp critical
          fprintf(stderr, "amax %a x %a: division %d, two floats %d\n", amax, x, want, code_of(q));
        }
      }
    }
  }
  printf("pairs %llu two_floats %llu differ %llu\n", pairs, two_floats, differ);
  return differ != 0;
}
