// MXFP4: 32 neighbouring elements of a row share a power of two X = 2^(e - 127)
// held as one byte e (E8M0; 255 is NaN), and an element is a 4-bit E2M1 code
// (sign, 2 exponent bits with bias 1, 1 mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6)
// standing for its value times X (OCP Microscaling Formats specification).
//
// X is 2^(E - 2), E the exponent of the block's largest magnitude rounded to one
// mantissa bit: a largest magnitude of at least 1.75 * 2^n counts as 2^(n+1), so
// |v / X| < 7 for every element and the rounding to the nearest code (ties to
// the even one) is off by at most half a step everywhere; with the plain floor
// of the exponent, magnitudes between 7 X and 8 X would be cut to 6 X.  X is at
// least 2^-126 (an fp32 normal; an all-zero block has e = 1).  A block that
// holds an infinity or a NaN gets e = 255 and codes 0: it reads back as NaN.
//
// Storage: two codes a byte, the even element in the low half; scale bytes in
// planes of 128 columns: byte b of word (c, row) belongs to the columns
// [128 c + 32 b, + 32) of that row, words of a plane in row order.  The GEMMs
// load the words of a tile's rows for one 128-wide K step, which are then
// neighbours in memory, and each lane of a 16x16x128 MFMA takes one byte.
#pragma once

#include "common.h"

namespace moe {

// A quantising (or reading) workgroup of 256 lanes takes kFp4Rows rows of kFp4Cols
// columns of a matrix, each wavefront 4 of the rows, 1 KB of bf16 at a time;
// workgroups of one matrix: row blocks, and in each its column blocks.
constexpr int kFp4Rows = 16, kFp4Cols = 512;
__host__ __device__ inline int64_t quantize_fp4_blocks(int64_t rows, int64_t cols) {
  return (rows + kFp4Rows - 1) / kFp4Rows * ((cols + kFp4Cols - 1) / kFp4Cols);
}

#if defined(__HIP_DEVICE_COMPILE__)
// Scale byte of a block whose largest magnitude has the fp32 bits `top` (sign cleared).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const int e = (int)((top + 0x200000u) >> 23) - 2;
  return (uint32_t)(e < 1 ? 1 : e);
}

// 8 values as E2M1 codes of scale byte e (1..254, or 255: codes 0), element i in
// bits 4i..4i+3, by the hardware conversion (nearest, ties to the even code).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], uint32_t e) {
  const float x = __uint_as_float(e << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], x, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], x, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], x, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], x, 3);
  return e == 255u ? 0u : w;
}

// Largest magnitude (fp32 bits) of 8 packed bf16 values; a NaN ranks above infinity.
__device__ __forceinline__ uint32_t abs_top_bf16x8(uint4 r) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = max(m, (w[i] << 16) & 0x7FFF0000u);
    m = max(m, w[i] & 0x7FFF0000u);
  }
  return m;
}

// A lane's chunk of 8 bf16 values, 4 consecutive lanes (4-aligned) holding one
// 32-element block: its 8 codes, and the block's scale byte in *e.  Every lane
// of the 4 must be active.
__device__ __forceinline__ uint32_t mx_quant_chunk(uint4 raw, uint32_t* e) {
  uint32_t m = abs_top_bf16x8(raw);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  *e = mx_scale_byte(m);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return e2m1x8(v, *e);
}

// The scale word of 128 columns from the scale bytes e that 16 consecutive
// lanes (16-aligned) hold, 4 lanes a block: valid in the first of the 16.
__device__ __forceinline__ uint32_t mx_scale_word(uint32_t e) {
  uint32_t w = e | ((uint32_t)__shfl_down((int)e, 4) << 8);    // lanes 0..3: blocks 0, 1; lanes 8..11: blocks 2, 3
  return w | ((uint32_t)__shfl_down((int)w, 8) << 16);
}

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// Workgroup b of matrix mat [rows, cols] (lane tid of 256): its codes and scale
// words.  ONCE: non-temporal loads and stores, for matrices that are read once and
// whose codes are not read soon.
template <bool ONCE>
__device__ __forceinline__ void quantize_fp4_block(const uint4* __restrict__ src, int rows, int cols, int64_t b,
                                                   int64_t mat, int tid, uint32_t* __restrict__ dst,
                                                   uint32_t* __restrict__ scales) {
  const int nblk = (cols + kFp4Cols - 1) / kFp4Cols, ncol = cols / 128, lane = tid & 63;
  const int64_t nchunk = cols / 8;                      // 16-byte chunks of a row; also its code words
  const int64_t c = b % nblk * (kFp4Cols / 8) + lane;   // (16 lanes a 128-column group: whole or past the row)
  const int r0 = (int)(b / nblk) * kFp4Rows + (tid >> 6) * 4;
  uint4 raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r0 + i < rows && c < nchunk) {
      const u32x4_t* q = reinterpret_cast<const u32x4_t*>(src + (mat * rows + r0 + i) * nchunk + c);
      const u32x4_t v = ONCE ? __builtin_nontemporal_load(q) : *q;
      raw[i] = make_uint4(v.x, v.y, v.z, v.w);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t e;
    const uint32_t w = mx_quant_chunk(raw[i], &e);
    const uint32_t sw = mx_scale_word(e);
    if (r0 + i < rows && c < nchunk) {
      uint32_t* q = dst + (mat * rows + r0 + i) * nchunk + c;
      if (ONCE) __builtin_nontemporal_store(w, q);
      else *q = w;
      if ((lane & 15) == 0) scales[(mat * ncol + c / 16) * rows + r0 + i] = sw;
    }
  }
}
#endif

}  // namespace moe
