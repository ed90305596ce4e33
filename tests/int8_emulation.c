/* The dispatch's int8 codes, emulated operation for operation (fp32 arithmetic
 * of the CPU, fmaf): the corrected product by the reciprocal against the IEEE
 * quotient, for bf16 amax and bf16 values.
 * Sources: csrc/payload_device.cuh (int8_scale, int8_codes). */
#include <math.h>
#include <stdint.h>
#include <string.h>

static float from_bits(uint32_t b) {
  float f;
  memcpy(&f, &b, 4);
  return f;
}

static uint32_t bits(float f) {
  uint32_t b;
  memcpy(&b, &f, 4);
  return b;
}

/* Code and quotient of bf16 value bits x for amax bits m >= 0x1F80. */
static int quick_code(uint32_t x, float s, float y, float* quotient) {
  const float v = from_bits(x << 16);
  const float q0 = v * y;
  const float r = fmaf(-s, q0, v);
  const float q = fmaf(r, y, q0);
  *quotient = q;
  volatile float big = 12582912.0f;
  volatile float t = q + big;
  return (int8_t)(bits(t) & 0xffu);
}

/* For every bf16 |x| <= amax: pairs whose code differs from the rounded IEEE
 * quotient, or whose quotient differs where it is 2^-20 or more. */
int64_t int8_quick_mismatches(uint32_t m_begin, uint32_t m_end) {
  int64_t bad = 0;
  for (uint32_t m = m_begin; m < m_end; ++m) {
    const float s = from_bits(m << 16) / 127.0f;
    const float y = 1.0f / s;
    for (uint32_t x = 0; x <= m; ++x) {
      for (uint32_t sign = 0; sign <= 0x8000u; sign += 0x8000u) {
        float q;
        const int code = quick_code(x | sign, s, y, &q);
        const float ref = from_bits((x | sign) << 16) / s;
        const int want = (int)nearbyintf(ref);
        bad += code != want;
        if (fabsf(ref) >= 0x1p-20f) bad += bits(q) != bits(ref);
      }
    }
  }
  return bad;
}

/* The plain path of the amax below 2^-64, and the range of its codes: amax
 * itself gives 127. */
int64_t int8_tiny_mismatches(uint32_t m_begin, uint32_t m_end) {
  int64_t bad = 0;
  for (uint32_t m = m_begin; m < m_end; ++m) {
    const float s = from_bits(m << 16) / 127.0f;
    bad += !(s > 0.0f);
    const float q = from_bits(m << 16) / s;
    bad += (int)nearbyintf(q) != 127;
  }
  return bad;
}
