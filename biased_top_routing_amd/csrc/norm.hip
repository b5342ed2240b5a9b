// Root-mean-square norm with the residual's addition and 8-bit output, and its gradients.
//
//   h = x + residual (rounded to the activation type, as it is stored), y = h w r, r = (mean(h^2) + eps)^-1/2
//   int8: code = round(127 h w / max|h w|), scale = r max|h w| / 127  (a row's factor r cancels in the code)
//   E4M3: per 1 x 128 tile, scale = r max|h w| / 448
//   backward, u = h r, g = dy w:  dx = r (g - u mean(g u)) + dh,  dw = sum_t dy u
// Both read and write each element once: they are bound by memory.  A row's chunks of 16 bytes stay in
// registers between its sums and its outputs.  H = 7168, bf16: 32011 rows with residual, E4M3 codes and the normed rows
// 364 us, 5.7 TB/s read and written (a large copy: 4.8); gradients of 16384 rows with dh 180 us, 5.3 TB/s; one row with
// int8 codes 3.7 us in its kernel.
#include <algorithm>

#include "common.h"
#include "int8.h"
#include "kernels.h"
#include "norm_layout.h"

namespace moe {
namespace {

enum { kNoCodes = 0, kCodesInt8 = 1, kCodesFp8 = 2 };

#if defined(__HIP_DEVICE_COMPILE__)
// A 16-byte chunk of a row: 8 bf16 or 4 fp32 values.
template <bool F32>
struct Chunk {
  static constexpr int N = F32 ? 4 : 8;
  static __device__ __forceinline__ void get(uint4 raw, float (&v)[N]) {
    if constexpr (F32) {
      v[0] = __uint_as_float(raw.x); v[1] = __uint_as_float(raw.y);
      v[2] = __uint_as_float(raw.z); v[3] = __uint_as_float(raw.w);
    } else {
      chunk_values(raw, v);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[N]) {
    if constexpr (F32)
      return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
      return make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
  }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ float inv_rms(float sum, int H, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, (float)H) + eps));
}

__device__ __forceinline__ int live_rows(const int32_t* n_tokens, int T) {
  return n_tokens ? min(max(*n_tokens, 0), T) : T;
}
#endif

// NW wavefronts a row (NW == 1: four rows a workgroup), CPL chunks a lane held; rows of more chunks are read
// again for their outputs (from h where it is stored: it may lie over residual or x).
template <bool F32, int CODES, int NW, int CPL>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void norm_kernel(
    const int32_t* __restrict__ n_tokens, const uint4* x, const uint4* residual, const uint4* __restrict__ weight,
    float eps, int T, int H, uint4* h_out, uint4* __restrict__ y, uint2* __restrict__ codes, float* __restrict__ scale) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Chunk<F32>;
  constexpr int N = C::N, TH = 64 * NW;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = NW == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  const int tid = NW == 1 ? lane : threadIdx.x;
  if (t >= live_rows(n_tokens, T)) return;              // (the whole row's wavefronts)
  const int nchunk = H / N;
  const int64_t at = t * nchunk;
  const bool held = nchunk <= CPL * TH;
  uint4 hv[CPL];
  // the row's h of chunks c0 + i * TH + tid: formed (and stored), or read back
  auto load_h = [&](int c0, bool first) {
    uint4 rv[CPL];
    const uint4* src = !first && h_out ? h_out : x;
    const bool add = residual && !(!first && h_out);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * TH + tid;
      hv[i] = c < nchunk ? src[at + c] : make_uint4(0, 0, 0, 0);
      if (add) rv[i] = c < nchunk ? residual[at + c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * TH + tid;
      if (add) {
        float a[N], b[N];
        C::get(hv[i], a);
        C::get(rv[i], b);
#pragma unroll
        for (int j = 0; j < N; ++j) a[j] += b[j];
        hv[i] = C::put(a);
      }
      if (first && h_out && c < nchunk) h_out[at + c] = hv[i];
    }
  };
  // ---- the row's sums
  float sum = 0.f;
  uint32_t amax = 0;
  for (int c0 = 0; c0 < nchunk; c0 += CPL * TH) {
    load_h(c0, true);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * TH + tid;
      float a[N];
      C::get(hv[i], a);
#pragma unroll
      for (int j = 0; j < N; ++j) sum = fmaf(a[j], a[j], sum);
      if constexpr (CODES == kCodesInt8) {
        if (c < nchunk) {
          float w[N];
          C::get(weight[c], w);
#pragma unroll
          for (int j = 0; j < N; ++j) amax = max(amax, abs_bits(a[j] * w[j]));
        }
      }
    }
  }
  sum = wave_sum(sum);
  if constexpr (CODES == kCodesInt8) amax = wave_max(amax);
  if constexpr (NW > 1) {
    __shared__ float sum_s[NW];
    __shared__ uint32_t amax_s[NW];
    if (lane == 0) sum_s[wave] = sum, amax_s[wave] = amax;
    __syncthreads();
    sum = 0.f;
    amax = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += sum_s[w], amax = max(amax, amax_s[w]);
  }
  const float r = inv_rms(sum, H, eps);
  const Int8Row row(amax);
  if (CODES == kCodesInt8 && tid == 0) scale[t] = row.scale * r;
  // ---- its outputs
  for (int c0 = 0; c0 < nchunk; c0 += CPL * TH) {
    if (!held) load_h(c0, false);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * TH + tid;
      float p[N], w[N];
      C::get(hv[i], p);
      C::get(c < nchunk ? weight[c] : make_uint4(0, 0, 0, 0), w);
#pragma unroll
      for (int j = 0; j < N; ++j) p[j] *= w[j];
      if constexpr (CODES == kCodesFp8) {               // (16 lanes hold a tile: wholly inside or outside the row)
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(p[j]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
        // (a tile below the smallest bf16 number counts as zeros: its scale has too few bits, or none, to divide by)
        const float sc = m < 0x1p-133f ? 1.0f : __fdiv_rn(m, 448.0f), inv = __fdiv_rn(1.0f, sc);
        float q[N];
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = div_by_scale(p[j], sc, inv);
        if (c < nchunk) {
          codes[at + c] = make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
          if ((tid & 15) == 0) scale[t * (H / 128) + c / 16] = sc * r;
        }
      }
      if (c >= nchunk) continue;
      if constexpr (CODES == kCodesInt8)
        codes[at + c] = make_uint2(row.codes4(p[0], p[1], p[2], p[3]), row.codes4(p[4], p[5], p[6], p[7]));
      if (y) {
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] *= r;
        y[at + c] = C::put(p);
      }
    }
  }
#endif
}

// ------------------------------------------------------------------ gradients
// r and m = mean(g u) of every live row (rows too long for the registers of one workgroup).
constexpr int kNormRowsThreads = 512;   // (2^23 rows make a grid of fewer than 2^32 lanes)
template <bool F32>
__global__ __launch_bounds__(kNormRowsThreads) void norm_bwd_rows_kernel(const int32_t* __restrict__ n_tokens,
                                                             const uint4* __restrict__ h,
                                                             const uint4* __restrict__ weight, float eps,
                                                             const uint4* __restrict__ dy, int T, int H,
                                                             float2* __restrict__ rm) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Chunk<F32>;
  constexpr int N = C::N;
  const int64_t t = blockIdx.x;
  if (t >= live_rows(n_tokens, T)) return;
  const int nchunk = H / N, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float hh = 0.f, gh = 0.f;
  for (int c = threadIdx.x; c < nchunk; c += kNormRowsThreads) {
    float a[N], d[N], w[N];
    C::get(h[t * nchunk + c], a);
    C::get(dy[t * nchunk + c], d);
    C::get(weight[c], w);
#pragma unroll
    for (int j = 0; j < N; ++j) hh = fmaf(a[j], a[j], hh), gh = fmaf(d[j] * w[j], a[j], gh);
  }
  hh = wave_sum(hh);
  gh = wave_sum(gh);
  constexpr int NW = kNormRowsThreads / 64;
  __shared__ float hh_s[NW], gh_s[NW];
  if (lane == 0) hh_s[wave] = hh, gh_s[wave] = gh;
  __syncthreads();
  if (threadIdx.x == 0) {
    hh = gh = 0.f;
    for (int i = 0; i < NW; ++i) hh += hh_s[i], gh += gh_s[i];
    const float r = inv_rms(hh, H, eps);
    rm[t] = make_float2(r, __fdiv_rn(gh * r, (float)H));
  }
#endif
}

// Workgroup (b, panel) takes the rows b, b + gridDim.x, ...: dx of the panel's columns, and its sum of dy u over
// those rows in part[b].  FUSED: one panel holds the row, and the workgroup forms r and m itself.  NW wavefronts a row;
// NW == 1: every wavefront takes rows of its own, and their sums are added in order at the end.
template <bool F32, bool FUSED, int NW>
__global__ __launch_bounds__(kNormBwdThreads) void norm_bwd_kernel(
    const int32_t* __restrict__ n_tokens, const uint4* __restrict__ h, const uint4* __restrict__ weight, float eps,
    const uint4* dy, const uint4* dh, const float2* __restrict__ rm, int T, int H, uint4* dx, float* __restrict__ part) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Chunk<F32>;
  constexpr int N = C::N, TH = 64 * NW, CPL = kNormBwdChunks, ROWS = kNormBwdThreads / TH;
  static_assert(NW == 1 || ROWS == 1, "the wavefronts of a row meet at the workgroup's barrier");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nchunk = H / N, c0 = blockIdx.y * TH * CPL + threadIdx.x % TH;
  const int live = live_rows(n_tokens, T);
  float dw[CPL][N];
  uint4 wv[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    wv[i] = c0 + i * TH < nchunk ? weight[c0 + i * TH] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = 0.f;
  }
  __shared__ float hh_s[2][NW], gh_s[2][NW];
  int turn = 0;                                         // (two sets: a row's sums are read while the next are written)
  for (int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / TH; t < T; t += (int64_t)gridDim.x * ROWS) {
    const int64_t at = t * nchunk;
    if (t >= live) {
#pragma unroll
      for (int i = 0; i < CPL; ++i)
        if (c0 + i * TH < nchunk) dx[at + c0 + i * TH] = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 hv[CPL], dv[CPL], ev[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const bool in = c0 + i * TH < nchunk;
      hv[i] = in ? h[at + c0 + i * TH] : make_uint4(0, 0, 0, 0);
      dv[i] = in ? dy[at + c0 + i * TH] : make_uint4(0, 0, 0, 0);
      ev[i] = in && dh ? dh[at + c0 + i * TH] : make_uint4(0, 0, 0, 0);
    }
    float r, m;
    if constexpr (FUSED) {
      float hh = 0.f, gh = 0.f;
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        float a[N], d[N], w[N];
        C::get(hv[i], a);
        C::get(dv[i], d);
        C::get(wv[i], w);
#pragma unroll
        for (int j = 0; j < N; ++j) hh = fmaf(a[j], a[j], hh), gh = fmaf(d[j] * w[j], a[j], gh);
      }
      hh = wave_sum(hh);
      gh = wave_sum(gh);
      if constexpr (NW > 1) {
        if (lane == 0) hh_s[turn][wave] = hh, gh_s[turn][wave] = gh;
        __syncthreads();
        hh = gh = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) hh += hh_s[turn][i], gh += gh_s[turn][i];
        turn ^= 1;
      }
      r = inv_rms(hh, H, eps);
      m = __fdiv_rn(gh * r, (float)H);
    } else {
      r = rm[t].x;
      m = rm[t].y;
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      if (c0 + i * TH >= nchunk) continue;
      float a[N], d[N], w[N], e[N];
      C::get(hv[i], a);
      C::get(dv[i], d);
      C::get(wv[i], w);
      C::get(ev[i], e);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float u = a[j] * r;
        dw[i][j] = fmaf(d[j], u, dw[i][j]);
        e[j] = fmaf(r, d[j] * w[j] - u * m, e[j]);
      }
      dx[at + c0 + i * TH] = C::put(e);
    }
  }
  if constexpr (ROWS > 1) {                             // the first wavefront adds the others' sums to its own
    __shared__ float dw_s[ROWS - 1][CPL][N][64];
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) dw_s[wave - 1][i][j][lane] = dw[i][j];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j)
        for (int w = 0; w < ROWS - 1; ++w) dw[i][j] += dw_s[w][i][j][lane];
  }
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    if (c0 + i * TH >= nchunk) continue;
    float4* out = reinterpret_cast<float4*>(part + (int64_t)blockIdx.x * H + (int64_t)(c0 + i * TH) * N);
#pragma unroll
    for (int j = 0; j < N; j += 4) out[j / 4] = make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
  }
#endif
}

// dweight[j] = sum over the nb partials, in a fixed order: 16 strided sums, then those in order.
__global__ __launch_bounds__(1024) void norm_bwd_sum_kernel(const float* __restrict__ part, int nb, int H,
                                                            float* __restrict__ dweight) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int j = blockIdx.x * 64 + lane;
  float v = 0.f;
  if (j < H)
#pragma unroll 8
    for (int b = q; b < nb; b += 16) v += part[(int64_t)b * H + j];
  s[q][lane] = v;
  __syncthreads();
  if (q == 0 && j < H) {
    v = 0.f;
    for (int i = 0; i < 16; ++i) v += s[i][lane];
    dweight[j] = v;
  }
}

moe_status norm_check(const moe_cfg* cfg, const int32_t* n_tokens, float eps) {
  const moe_status st = validate_share(cfg);
  if (st != MOE_OK) return st;
  if (!(eps > 0.0f) || !(eps <= 3.402823466e38f)) return MOE_ERR_SHAPE;
  return misaligned(n_tokens, 4) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_norm(const moe_cfg* cfg, const int32_t* n_tokens, const void* x, const void* residual,
                               const void* weight, float eps, void* h, void* y, void* codes, float* code_scale,
                               void* stream) {
  const moe_status st = norm_check(cfg, n_tokens, eps);
  if (st != MOE_OK) return st;
  const bool i8 = cfg->wgt == MOE_INT8, f8 = cfg->wgt == MOE_FP8_E4M3, f32 = cfg->act == MOE_F32;
  if (codes && !i8 && !f8) return MOE_ERR_UNSUPPORTED;
  if (cfg->T == 0) return MOE_OK;
  if (!x || !weight || (!y && !codes) || (codes && !code_scale)) return MOE_ERR_NULL;
  for (const void* q : {x, residual, weight, (const void*)h, (const void*)y, (const void*)codes})
    if (misaligned(q, 16)) return MOE_ERR_UNSUPPORTED;
  if (misaligned(code_scale, 4)) return MOE_ERR_UNSUPPORTED;
  // Just enough lanes for a row, so that what is in flight on a CU is many rows' loads: the lane's chunks and the
  // wavefronts of a row by its length alone.  With residual, int8 codes and normed rows, us, wavefronts x chunks a lane:
  //              1 x 4   1 x 16   2 x 4   4 x 4   8 x 2   8 x 4
  //   4096 x 1024  8.7     16.2     9.9    12.3    14.9    19.1
  //   4096 x 2048 14.2     23.4    14.9    16.9    17.9    20.6
  //   4096 x 4096 29.5     36.7    23.8    25.3    26.0    27.4   (1 x 4 reads h again)
  //    512 x 7168 17.0     17.8    11.0     8.2     7.4     8.0
  //  16384 x 7168  245      239     218     189     184     184
  const int64_t nchunk = (int64_t)cfg->H * act_bytes(cfg) / 16;
  auto go = [&](auto kernel, int rows, int threads) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((cfg->T + rows - 1) / rows)), dim3(threads), 0, as_stream(stream), n_tokens,
                       (const uint4*)x, (const uint4*)residual, (const uint4*)weight, eps, cfg->T, cfg->H, (uint4*)h,
                       (uint4*)y, (uint2*)codes, code_scale);
  };
  auto shape = [&](auto f, auto c) {
    constexpr bool F = decltype(f)::value;
    constexpr int C = decltype(c)::value;
    if (nchunk <= 256) go(norm_kernel<F, C, 1, 4>, 4, 256);
    else if (nchunk <= 512) go(norm_kernel<F, C, 2, 4>, 1, 128);
    else if (nchunk <= 1024) go(norm_kernel<F, C, 8, 2>, 1, 512);
    else go(norm_kernel<F, C, 8, 4>, 1, 512);
  };
  using std::integral_constant;
  if (f32) shape(integral_constant<bool, true>{}, integral_constant<int, kNoCodes>{});
  else if (codes && i8) shape(integral_constant<bool, false>{}, integral_constant<int, kCodesInt8>{});
  else if (codes) shape(integral_constant<bool, false>{}, integral_constant<int, kCodesFp8>{});
  else shape(integral_constant<bool, false>{}, integral_constant<int, kNoCodes>{});
  return launch_status();
}

extern "C" moe_status moe_norm_backward(const moe_cfg* cfg, const int32_t* n_tokens, const void* h, const void* weight,
                                        float eps, const void* dy, const void* dh, void* dx, float* dweight, void* ws,
                                        size_t ws_bytes, void* stream) {
  const moe_status st = norm_check(cfg, n_tokens, eps);
  if (st != MOE_OK) return st;
  if (!weight || !dweight || !ws || (cfg->T > 0 && (!h || !dy || !dx))) return MOE_ERR_NULL;
  for (const void* q : {h, weight, dy, dh, (const void*)dx, (const void*)ws})
    if (misaligned(q, 16)) return MOE_ERR_UNSUPPORTED;
  if (misaligned(dweight, 4)) return MOE_ERR_UNSUPPORTED;
  const NormBwdLayout L(cfg);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  hipStream_t s = as_stream(stream);
  char* base = static_cast<char*>(ws);
  float2* rm = reinterpret_cast<float2*>(base + L.off_rm);
  float* part = reinterpret_cast<float*>(base + L.off_part);
  auto go = [&](auto f) {
    constexpr bool F = decltype(f)::value;
    const dim3 grid((unsigned)L.blocks, (unsigned)L.panels);
    auto panel = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(kNormBwdThreads), 0, s, n_tokens, (const uint4*)h, (const uint4*)weight, eps,
                         (const uint4*)dy, (const uint4*)dh, rm, cfg->T, cfg->H, (uint4*)dx, part);
    };
    if (L.panels > 1) {
      hipLaunchKernelGGL(norm_bwd_rows_kernel<F>, dim3((unsigned)cfg->T), dim3(kNormRowsThreads), 0, s, n_tokens,
                         (const uint4*)h, (const uint4*)weight, eps, (const uint4*)dy, cfg->T, cfg->H, rm);
      panel(norm_bwd_kernel<F, false, 4>);
    } else if (L.rows > 1) {
      panel(norm_bwd_kernel<F, true, 1>);
    } else {
      panel(norm_bwd_kernel<F, true, 4>);
    }
  };
  if (cfg->T > 0) {
    if (cfg->act == MOE_F32) go(std::integral_constant<bool, true>{});
    else go(std::integral_constant<bool, false>{});
    const moe_status e = launch_status();
    if (e != MOE_OK) return e;
  }
  hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3((unsigned)((cfg->H + 63) / 64)), dim3(1024), 0, s, part,
                     cfg->T > 0 ? L.blocks : 0, cfg->H, dweight);
  return launch_status();
}
