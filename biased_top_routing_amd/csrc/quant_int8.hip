// Quantisation of bf16 rows to int8 codes with one scale a row (int8.h): the weight preparation of the
// int8 experts, their activations, and the SwiGLU intermediates between their two GEMMs.
#include <algorithm>

#include "common.h"
#include "int8.h"
#include "kernels.h"

namespace moe {
namespace {

// One wavefront a row.  A row may consist of `group` pieces of nchunk chunks, `stride` chunks apart (the same row of
// `group` matrices).
template <int HELD>
__global__ __launch_bounds__(256) void quantize_int8_kernel(const uint4* __restrict__ src, int64_t rows, int rows_mat,
                                                            int group, int64_t nchunk, uint2* __restrict__ dst,
                                                            float* __restrict__ scales) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int64_t first = (row / rows_mat * group * rows_mat + row % rows_mat) * nchunk, stride = rows_mat * nchunk;
  int8_row<HELD>(src, group * nchunk,
                 [&](int64_t q) { return group == 1 ? first + q : first + q / nchunk * stride + q % nchunk; }, dst,
                 scales + row);
#endif
}

// Two sets of rows, the first one's up to *limit (h of the routed rows, of which a share has fewer than there is room
// for, and of the shared experts: one launch of 4.4 us saved a call).
template <int HELD>
__global__ __launch_bounds__(256) void quantize_int8_pair_kernel(Int8Rows a, Int8Rows b, int64_t a_blocks,
                                                                 const int32_t* __restrict__ limit) {
#if defined(__HIP_DEVICE_COMPILE__)
  const bool second = blockIdx.x >= a_blocks;
  const Int8Rows& s = second ? b : a;
  const int64_t row = ((int64_t)blockIdx.x - (second ? a_blocks : 0)) * 4 + (threadIdx.x >> 6);
  if (row >= (second ? s.rows : (int64_t)*limit)) return;
  const int64_t n = s.cols / 8;
  int8_row<HELD>((const uint4*)s.src + row * n, n, [](int64_t q) { return q; }, (uint2*)s.dst + row * n, s.scales + row);
#endif
}

}  // namespace

moe_status launch_quantize_int8_pair(const Int8Rows& a, const Int8Rows& b, const int32_t* limit, hipStream_t st) {
  const int64_t na = (a.rows + 3) / 4, nb = (b.rows + 3) / 4;
  if (na + nb == 0) return MOE_OK;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(na + nb)), dim3(256), 0, st, a, b, na, limit);
  };
  // by the routed rows, of which there are more (24576 of 1408 columns and 4096 of 2816: 31.6 us, 16 held 42.8)
  if (a.cols <= kInt8Short) go(quantize_int8_pair_kernel<kInt8HeldShort>);
  else go(quantize_int8_pair_kernel<kInt8Held>);
  return launch_status();
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_int8(const void* src_bf16, int32_t n_mat, int32_t rows, int32_t cols, int32_t group,
                                        int8_t* dst, float* scales, void* stream) {
  if (n_mat < 0 || rows < 0 || cols <= 0 || cols % 8 || group < 1 || n_mat % group) return MOE_ERR_SHAPE;
  const int64_t n = (int64_t)(n_mat / group) * rows;
  if ((n + 3) / 4 >= (int64_t)1 << 24) return MOE_ERR_SHAPE;   // (four rows a workgroup of 256, fewer than 2^32 lanes)
  if (n == 0) return MOE_OK;
  if (!src_bf16 || !dst || !scales) return MOE_ERR_NULL;
  if (misaligned(src_bf16, 16) || misaligned(dst, 8) || misaligned(scales, 4)) return MOE_ERR_UNSUPPORTED;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((n + 3) / 4)), dim3(256), 0, as_stream(stream), (const uint4*)src_bf16, n,
                       rows, group, (int64_t)cols / 8, (uint2*)dst, scales);
  };
  if ((int64_t)group * cols <= kInt8Short) go(quantize_int8_kernel<kInt8HeldShort>);
  else go(quantize_int8_kernel<kInt8Held>);
  return launch_status();
}
