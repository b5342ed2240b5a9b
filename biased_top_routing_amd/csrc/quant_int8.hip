// Quantisation of bf16 rows to int8 codes with one scale a row (int8.h): the weight preparation of the
// int8 experts, their activations, and the SwiGLU intermediates between their two GEMMs.
#include "common.h"
#include "int8.h"
#include "kernels.h"

namespace moe {
namespace {

// One wavefront a row: the row's chunks of 16 bytes are read once and kept where they fit kHeld a lane (8192
// columns), else read again.  A row may consist of `group` pieces of nchunk chunks, `stride` chunks apart (the
// same row of `group` matrices).  limit (nullable): rows from *limit on are left alone.
constexpr int kHeld = 16;

__global__ __launch_bounds__(256) void quantize_int8_kernel(const uint4* __restrict__ src, int64_t rows,
                                                            int rows_mat, int group, int64_t nchunk,
                                                            const int32_t* __restrict__ limit,
                                                            uint2* __restrict__ dst, float* __restrict__ scales) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows || (limit && row >= *limit)) return;
  const int64_t mat = row / rows_mat, r = row % rows_mat;
  const int64_t first = (mat * group * rows_mat + r) * nchunk, stride = rows_mat * nchunk;
  const int64_t n = group * nchunk;
  auto at = [&](int64_t q) { return group == 1 ? first + q : first + q / nchunk * stride + q % nchunk; };
  uint4 v[kHeld];
  auto load = [&](int64_t q0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t q = q0 + i * kWave + lane;
      if (q0 + i * kWave < n) v[i] = src[at(q < n ? q : n - 1)];
      else v[i] = make_uint4(0, 0, 0, 0);
    }
  };
  uint32_t m = 0;
  for (int64_t q0 = 0; q0 < n; q0 += kHeld * kWave) {
    load(q0);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) m = max(m, chunk_amax(v[i]));
  }
  const Int8Row c(wave_max(m));
  for (int64_t q0 = 0; q0 < n; q0 += kHeld * kWave) {
    if (n > kHeld * kWave) load(q0);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t q = q0 + i * kWave + lane;
      if (q < n) dst[at(q)] = chunk_codes(c, v[i]);
    }
  }
  if (lane == 0) scales[row] = c.scale;
#endif
}

}  // namespace

moe_status launch_quantize_rows_int8(const bf16_t* src, int64_t rows, int cols, const int32_t* limit, uint8_t* dst,
                                     float* scales, hipStream_t st) {
  if (rows == 0) return MOE_OK;
  hipLaunchKernelGGL(quantize_int8_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, (const uint4*)src, rows,
                     (int)(rows < INT32_MAX ? rows : INT32_MAX), 1, (int64_t)cols / 8, limit, (uint2*)dst, scales);
  return launch_status();
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_int8(const void* src_bf16, int32_t n_mat, int32_t rows, int32_t cols, int32_t group,
                                        int8_t* dst, float* scales, void* stream) {
  if (n_mat < 0 || rows < 0 || cols <= 0 || cols % 8 || group < 1 || n_mat % group) return MOE_ERR_SHAPE;
  const int64_t n = (int64_t)(n_mat / group) * rows;
  if (n >= (int64_t)1 << 26) return MOE_ERR_SHAPE;   // (a wavefront a row, in a grid of fewer than 2^32 lanes)
  if (n == 0) return MOE_OK;
  if (!src_bf16 || !dst || !scales) return MOE_ERR_NULL;
  if (misaligned(src_bf16, 16) || misaligned(dst, 8) || misaligned(scales, 4)) return MOE_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(quantize_int8_kernel, dim3((unsigned)((n + 3) / 4)), dim3(256), 0, as_stream(stream),
                     (const uint4*)src_bf16, n, rows, group, (int64_t)cols / 8, (const int32_t*)nullptr, (uint2*)dst,
                     scales);
  return launch_status();
}
