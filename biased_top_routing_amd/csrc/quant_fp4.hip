// moe_quantize_fp4 / moe_dequantize_fp4: MXFP4 codes and scale bytes of bf16
// matrices (format: fp4.h), and back.  Used offline for the expert weights, and
// inside moe_expert_ffn for the rows of x.
//
// Both directions only move bytes: 2 in and 17/32 out an element, or the reverse
// (32 matrices of 4096 x 7168, both ways: 771 us, 5.5 TB/s; with 64 rows of one
// 128-column group a workgroup 999 us, 925 us with non-temporal accesses).
#include "common.h"
#include "fp4.h"
#include "kernels.h"

namespace moe {

namespace {

__global__ __launch_bounds__(256) void quantize_fp4_kernel(const uint4* __restrict__ src, int rows, int cols,
                                                           uint32_t* __restrict__ dst,
                                                           uint32_t* __restrict__ scales) {
#if defined(__HIP_DEVICE_COMPILE__)
  quantize_fp4_block<true>(src, rows, cols, blockIdx.x, blockIdx.y, threadIdx.x, dst, scales);
#endif
}

__global__ __launch_bounds__(256) void dequantize_fp4_kernel(const uint32_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int rows, int cols,
                                                             uint4* __restrict__ dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nblk = (cols + kFp4Cols - 1) / kFp4Cols, ncol = cols / 128;
  const int64_t mat = blockIdx.y, nchunk = cols / 8;
  const int64_t c = blockIdx.x % nblk * (kFp4Cols / 8) + lane;
  const int r0 = blockIdx.x / nblk * kFp4Rows + wave * 4;
  if (c >= nchunk) return;
  uint32_t w[4], e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = min(r0 + i, rows - 1);
    w[i] = codes[(mat * rows + r) * nchunk + c];
    e[i] = scales[((mat * ncol + c / 16) * rows + r) * 4 + (c % 16) / 4];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // X as fp32: e = 0 is the subnormal 2^-127, e = 255 a NaN
    const float x = __uint_as_float(e[i] == 0u ? 0x00400000u : e[i] == 255u ? 0x7FC00000u : e[i] << 23);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t code = w[i] >> (8 * j + 4 * b);
        const uint32_t ex = (code >> 1) & 3u, m = code & 1u;
        // E2M1 magnitude: m / 2 for exponent 0, else (1 + m / 2) 2^(ex - 1)
        const float mag = ex == 0u ? 0.5f * (float)m : __uint_as_float(((ex + 126u) << 23) | (m << 22));
        // (a two-bit significand times a power of two: exact in bf16)
        h[b] = __float_as_uint((code & 8u ? -mag : mag) * x) >> 16;
      }
      o[j] = h[0] | (h[1] << 16);
    }
    if (r0 + i < rows)
      __builtin_nontemporal_store(u32x4_t{o[0], o[1], o[2], o[3]},
                                  reinterpret_cast<u32x4_t*>(dst + (mat * rows + r0 + i) * nchunk + c));
  }
#endif
}

moe_status check_fp4(const void* bf16, const uint8_t* codes, const uint8_t* scales, int32_t n_mat, int32_t rows,
                     int32_t cols) {
  if (!bf16 || !codes || !scales) return MOE_ERR_NULL;
  if (n_mat < 0 || n_mat > 65535 || rows < 0 || cols <= 0 || cols % 128) return MOE_ERR_SHAPE;
  if (quantize_fp4_blocks(rows, cols) >= ((int64_t)1 << 24)) return MOE_ERR_SHAPE;   // x 256 lanes: a grid's 32 bits
  if (misaligned(bf16, 16) || misaligned(codes, 4) || misaligned(scales, 4)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_fp4(const void* src_bf16, int32_t n_mat, int32_t rows, int32_t cols, uint8_t* dst,
                                       uint8_t* scales, void* stream) {
  const moe_status st = check_fp4(src_bf16, dst, scales, n_mat, rows, cols);
  if (st != MOE_OK) return st;
  if (n_mat == 0 || rows == 0) return MOE_OK;
  hipLaunchKernelGGL(quantize_fp4_kernel, dim3((unsigned)quantize_fp4_blocks(rows, cols), (unsigned)n_mat), dim3(256),
                     0, as_stream(stream), (const uint4*)src_bf16, rows, cols, (uint32_t*)dst, (uint32_t*)scales);
  return launch_status();
}

extern "C" moe_status moe_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int32_t n_mat, int32_t rows,
                                         int32_t cols, void* dst_bf16, void* stream) {
  const moe_status st = check_fp4(dst_bf16, codes, scales, n_mat, rows, cols);
  if (st != MOE_OK) return st;
  if (n_mat == 0 || rows == 0) return MOE_OK;
  const dim3 grid((unsigned)quantize_fp4_blocks(rows, cols), (unsigned)n_mat);
  hipLaunchKernelGGL(dequantize_fp4_kernel, grid, dim3(256), 0, as_stream(stream), (const uint32_t*)codes, scales, rows,
                     cols, (uint4*)dst_bf16);
  return launch_status();
}
