// Symmetric int8 rows: a row with largest magnitude a stands for code * s with s = a / 127 and
// code = the whole number nearest 127 v / a (ties to even), |code| <= 127.
//
// Every value quantised here is a bf16 number or the product of two, so 127 v is exact in fp32 (at
// most 8 + 8 + 7 significant bits) and the quotient is the only rounding before the code: two values
// would have to lie within 2^-24 of each other's quotient for that to move a code, and 16-bit numerators
// and denominators do not.  The codes therefore do not depend on who computes them.
#pragma once

#include "common.h"

namespace moe {

// Chunks of a row that a lane keeps, so that it is read once: 4 for rows of up to 2048 columns, 16 beyond (up to 8192).
// moe_quantize_int8 with 4 / 16, us: 32768 x 512 16 / 33, 64 x 2816 x 2048 203 / 237, 8 x 4096 x 7168 173 / 132 (1.06
// GB, 5.3 TB/s).
constexpr int kInt8Held = 16, kInt8HeldShort = 4;
constexpr int64_t kInt8Short = 8 * kInt8HeldShort * kWave;

#if defined(__HIP_DEVICE_COMPILE__)
// |v| as an integer that orders like it; infinities and NaN from kInfBits up.
constexpr uint32_t kInfBits = 0x7F800000u;
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// What the codes of a row need of its largest magnitude (as bits).
struct Int8Row {
  float a, y, up;    // a power of two away from the largest magnitude, 1 / a, and 127 times that power
  float scale;       // a / 127 of the row itself; 0 for a row of zeros, NaN for one with an infinity or a NaN
  bool none;         // its codes are 0

  __device__ __forceinline__ explicit Int8Row(uint32_t amax) {
    const float m = __uint_as_float(amax);
    none = amax == 0 || amax >= kInfBits;
    scale = amax >= kInfBits ? __uint_as_float(0x7FC00000u) : __fdiv_rn(m, 127.0f);
    // (the quotient is formed away from the ends of the range, where 127 v or 1 / a leave it)
    const float p = m > 0x1p60f ? 0x1p-80f : m < 0x1p-60f ? 0x1p80f : 1.0f;
    a = none ? 1.0f : m * p;
    y = __fdiv_rn(1.0f, a);
    up = none ? 0.0f : 127.0f * p;
  }
  // The code of v in the low byte of the result.  q = fl32(127 v / a) by one correction step (Markstein);
  // adding 1.5 * 2^23 rounds it to a whole number, ties to even, whose two's complement ends the bits.
  __device__ __forceinline__ uint32_t code(float v) const {
    const float n = v * up, q0 = n * y;
    const float q = fmaf(fmaf(-q0, a, n), y, q0);
    return none ? 0u : __float_as_uint(q + 12582912.0f);
  }
  __device__ __forceinline__ uint32_t codes4(float v0, float v1, float v2, float v3) const {
    const uint32_t lo = __builtin_amdgcn_perm(code(v1), code(v0), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(code(v3), code(v2), 0x04000C0Cu);
    return lo | hi;
  }
};

// 8 bf16 values of a 16-byte chunk.
__device__ __forceinline__ void chunk_values(uint4 raw, float (&v)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t chunk_amax(uint4 raw) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
  return m;
}
__device__ __forceinline__ uint2 chunk_codes(const Int8Row& r, uint4 raw) {
  float v[8];
  chunk_values(raw, v);
  return make_uint2(r.codes4(v[0], v[1], v[2], v[3]), r.codes4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  return m;
}
// A row of n chunks by one wavefront: chunk q is src[at(q)], its codes go to dst[at(q)].  The chunks are read once and
// kept where they fit HELD a lane, else read again.
template <int HELD, class At>
__device__ __forceinline__ void int8_row(const uint4* __restrict__ src, int64_t n, At at, uint2* __restrict__ dst,
                                         float* __restrict__ scale) {
  const int lane = threadIdx.x & 63;
  uint4 v[HELD];
  auto load = [&](int64_t q0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int64_t q = q0 + i * kWave + lane;
      if (q0 + i * kWave < n) v[i] = src[at(q < n ? q : n - 1)];
      else v[i] = make_uint4(0, 0, 0, 0);
    }
  };
  uint32_t m = 0;
  for (int64_t q0 = 0; q0 < n; q0 += HELD * kWave) {
    load(q0);
#pragma unroll
    for (int i = 0; i < HELD; ++i) m = max(m, chunk_amax(v[i]));
  }
  const Int8Row c(wave_max(m));
  for (int64_t q0 = 0; q0 < n; q0 += HELD * kWave) {
    if (n > HELD * kWave) load(q0);
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int64_t q = q0 + i * kWave + lane;
      if (q < n) dst[at(q)] = chunk_codes(c, v[i]);
    }
  }
  if (lane == 0) *scale = c.scale;
}
#endif

}  // namespace moe
