// Backward of the layer: the bandwidth-bound steps (combine, slot sum), the
// gate and balance-loss gradient of the router, and the four C entry points.
// The expert and router GEMMs are in gemm_bwd.hip.
//
// With the expert choice fixed, y_t = y_shared_t + sum_j w_tj y_perm[inv_tj] and
// w_tj = scale * s_{t,e_tj} / sum_j' s_{t,e_tj'} (DeepSeek-V3 Technical
// Report：中英对照解读, §2 and §3; the bias only ranks experts: reading notes,
// Method §1).  The sequence-wise balance loss follows the reading stated in
// moe.h (the pages keep such a loss with a very small weight but print no
// formula).  Every reduction below runs in a fixed order, so repeated calls
// give identical bits.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "bwd_layout.h"
#include "common.h"
#include "ffn_layout.h"
#include "kernels.h"
#include "route_topk.h"

namespace moe {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

constexpr int kMaxTopK = 32;   // validate_cfg bounds k

// One workgroup per token, one lane per 16-byte chunk of the row (up to 1024
// lanes): for each slot j, d_topk_w[t,j] = <dy_t, y_perm[inv_tj]> (fp32,
// per-wave shuffle sums, then the waves in order) and dy_perm[inv_tj] =
// topk_w[t,j] * dy_t.
constexpr int kMaxWaves = 16;
__global__ __launch_bounds__(1024) void combine_bwd_kernel(const uint4* __restrict__ dy,
                                                          const uint4* __restrict__ y_perm,
                                                          const int32_t* __restrict__ inv,
                                                          const float* __restrict__ topk_w, int k,
                                                          int64_t nchunk, uint4* __restrict__ dy_perm,
                                                          float* __restrict__ d_w) {
  __shared__ float red[kMaxWaves][kMaxTopK];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j = 0; j < k; ++j) {
    const int64_t p = inv[t * k + j];
    const float wj = topk_w[t * k + j];
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < nchunk; c += blockDim.x) {
      float d[8], y[8], o[8];
      bf16x8_to_f32(dy[t * nchunk + c], d);
      bf16x8_to_f32(y_perm[p * nchunk + c], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s = fmaf(d[i], y[i], s);
        o[i] = wj * d[i];
      }
      dy_perm[p * nchunk + c] = f32_to_bf16x8(o);
    }
    s = wave_sum(s);
    if (lane == 0) red[wave][j] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < k) {
    const int j = threadIdx.x, nw = (int)(blockDim.x / kWave);
    float v = red[0][j];
    for (int w = 1; w < nw; ++w) v += red[w][j];
    d_w[t * k + j] = v;
  }
}

// dx_t = sum_j dx_perm[inv_tj] + dx_shared_t + dx_router_t (fp32, in that order), bf16 out;
// one lane per 16-byte chunk of the row.
__global__ __launch_bounds__(1024) void dispatch_bwd_kernel(const uint4* __restrict__ dx_perm,
                                                           const uint4* __restrict__ dx_shared,
                                                           const float4* __restrict__ dx_router,
                                                           const int32_t* __restrict__ inv, int k,
                                                           int64_t nchunk, uint4* __restrict__ dx) {
  const int64_t t = blockIdx.x;
  for (int64_t c = threadIdx.x; c < nchunk; c += blockDim.x) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[8];
    for (int j = 0; j < k; ++j) {
      bf16x8_to_f32(dx_perm[(int64_t)inv[t * k + j] * nchunk + c], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
    if (dx_shared) {
      bf16x8_to_f32(dx_shared[t * nchunk + c], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
    if (dx_router) {
      const float4 a = dx_router[(t * nchunk + c) * 2], b = dx_router[(t * nchunk + c) * 2 + 1];
      acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
      acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
    }
    dx[t * nchunk + c] = f32_to_bf16x8(acc);
  }
}

// ---- the same two steps over a share of the batch: absent slots have inv = -1

#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ uint4 cvt_bf16x8(const float* f) {
  return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
}
#endif

// As in the share's combine: a token costs the rows it has, up to 512 lanes a
// token with 2 chunks each in flight; every wavefront finds the present slots for
// itself (lane j holds slot j, k <= 32).  The gate gradient of a slot is summed by
// wavefront, then over the wavefronts in order.  Every row is read and written
// once: non-temporal (T = 16384, H = 7168, an eighth of the experts: both kernels
// together 279 us, 5.6 TB/s, against 300 us with plain loads and stores; whole
// batches of T = 8192 650 against 695 us).
constexpr int kLocalLanes = 512, kLocalU = 2;
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ float4 ld_once(const float4* p) {
  const uint4 v = ld_once(reinterpret_cast<const uint4*>(p));
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void st_once(uint4* p, uint4 v) {
  __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_t*>(p));
}
__global__ __launch_bounds__(kLocalLanes) void combine_local_bwd_kernel(const uint4* __restrict__ dy,
                                                                       const uint4* __restrict__ y_perm,
                                                                       const int32_t* __restrict__ inv,
                                                                       const float* __restrict__ topk_w, int k,
                                                                       int64_t nchunk, uint4* __restrict__ dy_perm,
                                                                       float* __restrict__ d_w) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int U = kLocalU;
  __shared__ float red[kLocalLanes / kWave][kMaxTopK];
  const int64_t t = blockIdx.x;
  const int TH = blockDim.x, j = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t p = j < k ? inv[t * k + j] : -1;
  const float w = p >= 0 ? topk_w[t * k + j] : 0.f;
  const uint64_t here = __ballot(p >= 0);
  if (!here) {                                          // (the whole workgroup)
    if ((int)threadIdx.x < k) d_w[t * k + threadIdx.x] = 0.f;
    return;
  }
  const int64_t base = wave * kWave;                    // first chunk of this wavefront
  uint4 dv[U];                                          // dy of the first U chunks, kept over the slots
#pragma unroll
  for (int u = 0; u < U; ++u) dv[u] = ld_once(&dy[t * nchunk + min(base + u * TH + j, nchunk - 1)]);
  for (uint64_t left = here; left; left &= left - 1) {
    const int s = __builtin_ctzll(left);
    const int64_t row = __builtin_amdgcn_readlane(p, s);
    const float g = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), s));
    float sum = 0.f;
    for (int64_t c0 = base; c0 < nchunk; c0 += U * TH) {
      uint4 r[U], e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = min(c0 + u * TH + j, nchunk - 1);
        r[u] = ld_once(&y_perm[row * nchunk + c]);
        e[u] = c0 == base ? dv[u] : dy[t * nchunk + c];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c0 + u * TH + j >= nchunk) continue;
        float d[8], y[8], o[8];
        bf16x8_to_f32(e[u], d);
        bf16x8_to_f32(r[u], y);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          sum = fmaf(d[q], y[q], sum);
          o[q] = g * d[q];
        }
        st_once(&dy_perm[row * nchunk + c0 + u * TH + j], cvt_bf16x8(o));
      }
    }
    sum = wave_sum(sum);
    if (j == 0) red[wave][s] = sum;
  }
  __syncthreads();
  if ((int)threadIdx.x < k) {                           // (the first wavefront: lane j has slot j)
    float v = 0.f;
    if (p >= 0) {
      v = red[0][j];
      for (int i = 1; i * kWave < TH; ++i) v += red[i][j];
    }
    d_w[t * k + j] = v;
  }
#endif
}

__global__ __launch_bounds__(kLocalLanes) void dispatch_local_bwd_kernel(const uint4* __restrict__ dx_perm,
                                                                        const uint4* __restrict__ dx_shared,
                                                                        const float4* __restrict__ dx_router,
                                                                        const int32_t* __restrict__ inv, int k,
                                                                        int64_t nchunk, uint4* __restrict__ dx) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int U = kLocalU;
  const int64_t t = blockIdx.x;
  const int TH = blockDim.x, j = threadIdx.x & 63;
  const int32_t p = j < k ? inv[t * k + j] : -1;
  const uint64_t here = __ballot(p >= 0);
  for (int64_t c0 = threadIdx.x & ~63; c0 < nchunk; c0 += U * TH) {   // (whole wavefronts)
    float acc[U][8];
    uint4 r[U];
    int64_t c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      c[u] = min(c0 + u * TH + j, nchunk - 1);          // past the end: the last chunk again, not stored
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[u][q] = 0.f;
    }
    auto add = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        bf16x8_to_f32(r[u], v);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[u][q] += v[q];
      }
    };
    float4 ra[U], rb[U];
    if (dx_router) {                                    // (requested first, added last)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ra[u] = ld_once(&dx_router[(t * nchunk + c[u]) * 2]);
        rb[u] = ld_once(&dx_router[(t * nchunk + c[u]) * 2 + 1]);
      }
    }
    for (uint64_t left = here; left; left &= left - 1) {
      const int64_t row = __builtin_amdgcn_readlane(p, __builtin_ctzll(left));
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = ld_once(&dx_perm[row * nchunk + c[u]]);
      add();
    }
    if (dx_shared) {
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = ld_once(&dx_shared[t * nchunk + c[u]]);
      add();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float* a = acc[u];
      if (dx_router) {
        a[0] += ra[u].x; a[1] += ra[u].y; a[2] += ra[u].z; a[3] += ra[u].w;
        a[4] += rb[u].x; a[5] += rb[u].y; a[6] += rb[u].z; a[7] += rb[u].w;
      }
      if (c0 + u * TH + j < nchunk) st_once(&dx[t * nchunk + c[u]], cvt_bf16x8(a));
    }
  }
#endif
}

// up to kLocalLanes lanes a token, whole wavefronts
dim3 local_block(int64_t nchunk) {
  return dim3((unsigned)std::min<int64_t>(align_up((size_t)nchunk, kWave), kLocalLanes));
}

constexpr int kMaxEPL = 8;   // experts per lane: E <= 512

// f(EPL) with the experts a lane that E needs, rounded up to a power of two
template <typename F>
void by_epl(int E, F f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, kMaxEPL>{});
}

// Statistics of one chunk of kSeqChunk tokens of one sequence: per expert, how
// often it was selected and the sum of its normalised affinity s_te / sum_e' s_te'
// (of a token whose affinities are all 0: nothing).
// Each wave takes every fourth token, the rows of TU of them loaded at once; the waves' sums are added in order.
// EPL: experts a lane, E <= 64 * EPL.
template <int EPL>
__global__ __launch_bounds__(256) void seq_stats_kernel(const float* __restrict__ s, const int32_t* __restrict__ idx,
                                                        int T, int E, int k, int L, int nchunk,
                                                        int32_t* __restrict__ cnt, float* __restrict__ psum) {
  __shared__ int32_t c_lds[512];
  __shared__ float p_lds[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b = blockIdx.x / nchunk, ch = blockIdx.x % nchunk;
  const int t0 = b * L + ch * kSeqChunk, t1 = min(b * L + L, t0 + kSeqChunk);
  for (int e = threadIdx.x; e < E; e += blockDim.x) c_lds[e] = 0;
  __syncthreads();
  constexpr int TU = EPL >= 8 ? 4 : EPL >= 4 ? 8 : 16;
  float acc[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
  for (int tb = t0 + wave; tb < t1; tb += 4 * TU) {
    float v[TU][EPL];
    int sel[TU];
#pragma unroll
    for (int u = 0; u < TU; ++u) {
      const int t = tb + 4 * u;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        v[u][i] = t < t1 && e < E ? s[(int64_t)t * E + e] : 0.f;
      }
      sel[u] = t < t1 && lane < k ? idx[(int64_t)t * k + lane] : -1;
    }
#pragma unroll
    for (int u = 0; u < TU; ++u) {
      if (tb + 4 * u >= t1) break;
      float rs = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) rs += v[u][i];
      rs = wave_sum(rs);
#pragma unroll
      for (int i = 0; i < EPL; ++i) acc[i] += rs == 0.f ? 0.f : v[u][i] / rs;
      if ((unsigned)sel[u] < (unsigned)E) atomicAdd(&c_lds[sel[u]], 1);       // integer counts: order-free
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e < E) p_lds[wave][e] = acc[i];
  }
  __syncthreads();
  const int64_t out = (int64_t)blockIdx.x * E;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    cnt[out + e] = c_lds[e];
    psum[out + e] = ((p_lds[0][e] + p_lds[1][e]) + p_lds[2][e]) + p_lds[3][e];
  }
}

// Per (sequence, expert): f = E / (k L) * count, P = psum / L; the coefficient
// alpha / nseq * f / L of d L_bal / d s' and the loss alpha / nseq * sum f P.
// One workgroup; every thread sums its (b, e) pairs in a fixed order, then a
// fixed tree over the threads.
__global__ __launch_bounds__(256) void seq_coef_kernel(const int32_t* __restrict__ cnt, const float* __restrict__ psum,
                                                       int E, int k, int L, int nseq, int nchunk, float alpha,
                                                       float* __restrict__ coef, float* __restrict__ loss) {
  __shared__ float red[256];
  float mine = 0.f;
  for (int q = threadIdx.x; q < nseq * E; q += blockDim.x) {
    const int b = q / E, e = q % E;
    int c = 0;
    float ps = 0.f;
    for (int ch = 0; ch < nchunk; ++ch) {
      c += cnt[((int64_t)b * nchunk + ch) * E + e];
      ps += psum[((int64_t)b * nchunk + ch) * E + e];
    }
    const float f = (float)E / ((float)k * (float)L) * (float)c;
    coef[q] = alpha / (float)nseq * f / (float)L;
    mine += f * (ps / (float)L);
  }
  red[threadIdx.x] = mine;
  __syncthreads();
  for (int w = 128; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) *loss = nseq > 0 ? alpha / (float)nseq * red[0] : 0.0f;
}

// One wavefront per token: ds_e from the gates (selected experts) and from the
// balance loss (every expert, through s' = s / sum s), dlogit = ds s (1 - s),
// stored bf16 for the router GEMMs.
__global__ __launch_bounds__(256) void route_grad_kernel(const float* __restrict__ s, const int32_t* __restrict__ idx,
                                                         const float* __restrict__ d_w, const float* __restrict__ coef,
                                                         int T, int E, int k, int L, float scale,
                                                         bf16_t* __restrict__ dlogit) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int b = t / L;
  float v[kMaxEPL], ds[kMaxEPL], rs = 0.f, gs = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxEPL; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? s[(int64_t)t * E + e] : 0.f;
    ds[i] = coef && e < E ? coef[(int64_t)b * E + e] : 0.f;   // d L_bal / d s'_te
    rs += v[i];
  }
  rs = wave_sum(rs);
  // (ds grows as the sums shrink: where one leaves the range, the affinities are taken 2^80 times as large and ds by as much
  // smaller; what is a number without it keeps its bits)
  const float up_r = rs < 0x1p-60f ? 0x1p80f : 1.0f;
  rs *= up_r;
#pragma unroll
  for (int i = 0; i < kMaxEPL; ++i) gs += ds[i] * (v[i] * up_r);
  gs = wave_sum(gs);
#pragma unroll
  for (int i = 0; i < kMaxEPL; ++i) ds[i] = rs == 0.f ? 0.f : ds[i] / rs - gs / (rs * rs);
  // gates over the selected experts (an id outside [0, E) is none)
  int sel = lane < k ? idx[(int64_t)t * k + lane] : -1;
  if ((unsigned)sel >= (unsigned)E) sel = -1;
  const float ss = sel >= 0 ? s[(int64_t)t * E + sel] : 0.f;
  const float dwj = sel >= 0 ? d_w[(int64_t)t * k + lane] : 0.f;
  float S = wave_sum(ss);
  const float up = S == 0.f ? up_r : S < 0x1p-60f ? 0x1p80f : 1.0f, to_up = up_r / up;
  S *= up;
  const float B1 = wave_sum(dwj * (ss * up));
#pragma unroll
  for (int i = 0; i < kMaxEPL; ++i) ds[i] *= to_up;
  const float dsel = S == 0.f ? 0.f : scale / S * (dwj - B1 / S);   // (no affinity at all: no gradient)
  for (int j = 0; j < k; ++j) {
    const int ej = __shfl(sel, j);
    const float dj = __shfl(dsel, j);
#pragma unroll
    for (int i = 0; i < kMaxEPL; ++i)
      if (ej == lane + 64 * i) ds[i] += dj;
  }
#pragma unroll
  for (int i = 0; i < kMaxEPL; ++i) {
    const int e = lane + 64 * i;
    if (e < E) dlogit[(int64_t)t * E + e] = f32_to_bf16(ds[i] * (v[i] * up) * (1.0f - v[i]));
  }
}

#if defined(__HIP_DEVICE_COMPILE__)
// The sum over a wavefront, by DPP and four scalar reads (six shuffles go through LDS).
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f32<kDppXor1>(v);
  v += dpp_f32<kDppXor2>(v);
  v += dpp_f32<kDppHalfMirror>(v);
  v += dpp_f32<kDppMirror>(v);
  auto at = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
  return (at(0) + at(16)) + (at(32) + at(48));
}
#endif

// loss = scale * the sum of n partial losses, in a fixed order; a null loss is not written.
struct SeqLoss {
  const float* part;
  int n;
  float scale;
  float* loss;
};
// Up to this many are added by one of the wavefronts of the next kernel (a launch saved: T = 4096, E = 64, H = 2048
// 35.3 -> 33.5 us), more by a workgroup (a wavefront would take a wait for memory for every 64 of them).
constexpr int kLossInline = 1024;

// ... with the flags of moe_route: ds_e of the gates (MOE_GATES_RAW: scale * dw, not through their sum) and of the
// balance loss, through the softmax (dlogit_e = s_e (ds_e - sum s ds)) or the sigmoid.  The products d_e = s_e ds_e are
// formed, of the affinities' shares s / sum s: ds itself has no bound where the sum is small.  dlogit is stored as the sum of
// two bf16 numbers, the nearest and what it leaves (17 bits and more: the products of the router's gradients then stay
// within 2^-17 of fp32 ones), in rows of 2 * Ep, zero behind E.
template <bool SOFTMAX, int EPL>
__global__ __launch_bounds__(256) void route_grad_flags_kernel(const float* __restrict__ s,
                                                               const int32_t* __restrict__ idx,
                                                               const float* __restrict__ d_w,
                                                               const float* __restrict__ coef, int T, int E, int Ep,
                                                               int k, int L, float scale, bool raw,
                                                               bf16_t* __restrict__ dlogit, SeqLoss seq) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  if (t == 0 && seq.loss) {
    float v = 0.f;
    for (int i = lane; i < seq.n; i += 64) v += seq.part[i];
    v = row_sum(v);
    if (lane == 0) *seq.loss = seq.n > 0 ? seq.scale * v : 0.f;
  }
  const int b = t / L;
  float v[EPL], d[EPL], rs = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? s[(int64_t)t * E + e] : 0.f;
    d[i] = coef && e < E ? coef[(int64_t)b * E + e] : 0.f;   // d L_bal / d s'_te
    rs += v[i];
  }
  if (coef) {
    float n[EPL], mean = 0.f;
    rs = row_sum(rs);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      n[i] = rs != 0.f ? v[i] / rs : 0.f;                     // (all affinities 0: none of the gradient either)
      mean = fmaf(n[i], d[i], mean);
    }
    mean = row_sum(mean);
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = n[i] * (d[i] - mean);
  }
  // gates over the selected experts (an id outside [0, E) is none)
  int sel = lane < k ? idx[(int64_t)t * k + lane] : -1;
  if ((unsigned)sel >= (unsigned)E) sel = -1;
  const float ss = sel >= 0 ? s[(int64_t)t * E + sel] : 0.f;
  const float dwj = sel >= 0 ? d_w[(int64_t)t * k + lane] : 0.f;
  const float S = row_sum(ss);
  const float share = raw ? ss : S != 0.f ? ss / S : 0.f;
  const float B = raw ? 0.f : row_sum(dwj * share);
  const float dsel = scale * share * (dwj - B);
  for (int j = 0; j < k; ++j) {
    const int ej = __builtin_amdgcn_readlane(sel, j);
    const float dj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(dsel), j));
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (ej == lane + 64 * i) d[i] += dj;
  }
  float sum = 0.f;
  if constexpr (SOFTMAX) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += d[i];
    sum = row_sum(sum);
  }
  bf16_t* out = dlogit + (int64_t)t * 2 * Ep;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e >= Ep) continue;
    const float dl = e < E ? SOFTMAX ? d[i] - v[i] * sum : d[i] * (1.0f - v[i]) : 0.f;
    const bf16_t hi = f32_to_bf16(dl);
    out[e] = hi;
    out[Ep + e] = f32_to_bf16(dl - bf16_to_f32(hi));
  }
#endif
}

// seq_coef_kernel spread over the chip: workgroup (b, 64 experts from e0), each of its wavefronts a quarter of the
// sequence's chunks, and the partial loss of the 64 in part_loss (T = 16384, E = 256, 4 sequences: 71 us by one
// workgroup).
__global__ __launch_bounds__(256) void seq_coef_part_kernel(const int32_t* __restrict__ cnt,
                                                            const float* __restrict__ psum, int E, int k, int L,
                                                            int nseq, int nchunk, float alpha, float* __restrict__ coef,
                                                            float* __restrict__ part_loss) {
  const int ne = (E + 63) / 64, b = blockIdx.x / ne, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x % ne * 64 + lane;
  __shared__ int c_s[4][64];
  __shared__ float p_s[4][64];
  int c = 0;
  float ps = 0.f;
  if (e < E)
#pragma unroll 8
    for (int ch = wave; ch < nchunk; ch += 4) {
      c += cnt[((int64_t)b * nchunk + ch) * E + e];
      ps += psum[((int64_t)b * nchunk + ch) * E + e];
    }
  c_s[wave][lane] = c;
  p_s[wave][lane] = ps;
  __syncthreads();
  if (wave > 0) return;
  c = c_s[0][lane] + c_s[1][lane] + c_s[2][lane] + c_s[3][lane];
  ps = p_s[0][lane] + p_s[1][lane] + p_s[2][lane] + p_s[3][lane];
  const float f = (float)E / ((float)k * (float)L) * (float)c;
  if (e < E) coef[(int64_t)b * E + e] = alpha / (float)nseq * f / (float)L;
  const float sum = wave_sum(e < E ? f * (ps / (float)L) : 0.f);
  if (lane == 0) part_loss[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void seq_loss_kernel(SeqLoss seq) {
  __shared__ float s[16];
  float v = 0.f;
  for (int i = threadIdx.x; i < seq.n; i += 1024) v += seq.part[i];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.f;
    for (int i = 0; i < 16; ++i) v += s[i];
    *seq.loss = seq.scale * v;
  }
}

// Weight gradients of a batch without tokens.
__global__ __launch_bounds__(256) void zero_kernel(float* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.f;
}

moe_status launch_zero(float* p, int64_t n, hipStream_t st) {
  hipLaunchKernelGGL(zero_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 2048)), dim3(256), 0, st, p, n);
  return launch_status();
}

bool bwd_dtypes_ok(const moe_cfg* c) { return c->act == MOE_BF16 && c->wgt == MOE_BF16; }

// one lane per 16-byte chunk of a row, whole wavefronts, at most 1024 lanes
dim3 row_block(int64_t nchunk) {
  return dim3((unsigned)std::min<int64_t>(align_up((size_t)nchunk, kWave), kMaxWaves * kWave));
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_combine_backward(const moe_cfg* cfg, const void* dy, const void* y_perm,
                                           const int32_t* inv, const float* topk_w, void* dy_perm,
                                           float* d_topk_w, void* stream) {
  moe_status st = validate_cfg(cfg);
  if (st != MOE_OK) return st;
  if (!bwd_dtypes_ok(cfg)) return MOE_ERR_UNSUPPORTED;
  if (!dy || !y_perm || !inv || !topk_w || !dy_perm || !d_topk_w) return MOE_ERR_NULL;
  if (cfg->T == 0) return MOE_OK;
  const int64_t nchunk = (int64_t)cfg->H * 2 / 16;
  hipLaunchKernelGGL(combine_bwd_kernel, dim3((unsigned)cfg->T), row_block(nchunk), 0, as_stream(stream), (const uint4*)dy,
                     (const uint4*)y_perm, inv, topk_w, cfg->k, nchunk, (uint4*)dy_perm, d_topk_w);
  return launch_status();
}

extern "C" moe_status moe_combine_local_backward(const moe_cfg* cfg, const void* dy, const void* y_perm,
                                                 const int32_t* inv, const float* topk_w, void* dy_perm,
                                                 float* d_topk_w, void* stream) {
  moe_status st = validate_share(cfg);
  if (st != MOE_OK) return st;
  if (!bwd_dtypes_ok(cfg)) return MOE_ERR_UNSUPPORTED;
  if (cfg->T == 0) return MOE_OK;
  if (!dy || !y_perm || !inv || !topk_w || !dy_perm || !d_topk_w) return MOE_ERR_NULL;
  if (misaligned(dy, 16) || misaligned(y_perm, 16) || misaligned(dy_perm, 16) || misaligned(inv, 4) ||
      misaligned(topk_w, 4) || misaligned(d_topk_w, 4))
    return MOE_ERR_UNSUPPORTED;
  const int64_t nchunk = (int64_t)cfg->H * 2 / 16;
  hipLaunchKernelGGL(combine_local_bwd_kernel, dim3((unsigned)cfg->T), local_block(nchunk), 0, as_stream(stream),
                     (const uint4*)dy, (const uint4*)y_perm, inv, topk_w, cfg->k, nchunk, (uint4*)dy_perm, d_topk_w);
  return launch_status();
}

namespace {

// Both expert backward entry points; saved == nullptr: recompute g, u.
moe_status expert_ffn_backward(const moe_cfg* cfg, const void* x_perm, const void* x, const int32_t* offsets,
                               const moe_expert_weights* w, const moe_ffn_saved* saved, const void* dy_perm,
                               const void* dy, void* dx_perm, void* dx_shared, const moe_expert_grads* grads,
                               void* ws, size_t ws_bytes, void* stream) {
  moe_status st = validate_cfg(cfg);
  if (st != MOE_OK) return st;
  if (!bwd_dtypes_ok(cfg)) return MOE_ERR_UNSUPPORTED;
  if (!x_perm || !x || !offsets || !w || !dy_perm || !dy || !dx_perm || !grads || !ws) return MOE_ERR_NULL;
  if (!w->w_gate_up || !w->w_down || !grads->w_gate_up || !grads->w_down) return MOE_ERR_NULL;
  if (cfg->S > 0 && (!w->ws_gate_up || !w->ws_down || !dx_shared || !grads->ws_gate_up || !grads->ws_down))
    return MOE_ERR_NULL;
  const int64_t widest = std::max<int64_t>(cfg->H, 2LL * std::max(cfg->S, 1) * cfg->I);
  if ((int64_t)cfg->T * widest * 2 > INT32_MAX || 2LL * cfg->S * cfg->I * cfg->H * 2 > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (saved && (!saved->g || !saved->u || (cfg->S > 0 && (!saved->gs || !saved->us)))) return MOE_ERR_NULL;
  if (ws_bytes < FfnBwdLayout(cfg).total) return MOE_ERR_WORKSPACE;
  if (cfg->T == 0) {
    const int64_t down = (int64_t)cfg->H * cfg->I;         // (gate and up together: twice as many)
    const hipStream_t s = as_stream(stream);
    if ((st = launch_zero(grads->w_gate_up, 2 * cfg->E * down, s)) != MOE_OK) return st;
    if ((st = launch_zero(grads->w_down, cfg->E * down, s)) != MOE_OK || cfg->S == 0) return st;
    if ((st = launch_zero(grads->ws_gate_up, 2 * cfg->S * down, s)) != MOE_OK) return st;
    return launch_zero(grads->ws_down, cfg->S * down, s);
  }
  return launch_ffn_bwd_bf16(cfg, (const bf16_t*)x_perm, (const bf16_t*)x, offsets, w, saved,
                             (const bf16_t*)dy_perm, (const bf16_t*)dy, (bf16_t*)dx_perm, (bf16_t*)dx_shared, grads,
                             ws, as_stream(stream));
}

}  // namespace

extern "C" moe_status moe_expert_ffn_backward(const moe_cfg* cfg, const void* x_perm, const void* x,
                                              const int32_t* offsets, const moe_expert_weights* w,
                                              const void* dy_perm, const void* dy, void* dx_perm, void* dx_shared,
                                              const moe_expert_grads* grads, void* ws, size_t ws_bytes,
                                              void* stream) {
  return expert_ffn_backward(cfg, x_perm, x, offsets, w, nullptr, dy_perm, dy, dx_perm, dx_shared, grads, ws,
                             ws_bytes, stream);
}

extern "C" moe_status moe_expert_ffn_backward_saved(const moe_cfg* cfg, const void* x_perm, const void* x,
                                                    const int32_t* offsets, const moe_expert_weights* w,
                                                    const moe_ffn_saved* saved, const void* dy_perm, const void* dy,
                                                    void* dx_perm, void* dx_shared, const moe_expert_grads* grads,
                                                    void* ws, size_t ws_bytes, void* stream) {
  if (!saved) return MOE_ERR_NULL;
  return expert_ffn_backward(cfg, x_perm, x, offsets, w, saved, dy_perm, dy, dx_perm, dx_shared, grads, ws,
                             ws_bytes, stream);
}

namespace {

// Both entry points; with_flags: the call that takes moe_route's flags.
moe_status route_backward(const moe_cfg* cfg, bool with_flags, uint32_t flags, const void* x, const void* w_router,
                          const float* scores, const int32_t* topk_idx, const float* d_topk_w, float alpha,
                          int32_t seq_len, float* dx_router, float* dw_router, float* loss, void* ws, size_t ws_bytes,
                          void* stream) {
  moe_status st = validate_cfg(cfg);
  if (st != MOE_OK) return st;
  if (!bwd_dtypes_ok(cfg)) return MOE_ERR_UNSUPPORTED;
  if (with_flags) {
    if (!flags || (flags & ~(MOE_SOFTMAX | MOE_GATES_RAW))) return MOE_ERR_UNSUPPORTED;
    if (misaligned(x, 16) || misaligned(w_router, 16) || misaligned(ws, 16) || misaligned(scores, 4) ||
        misaligned(topk_idx, 4) || misaligned(d_topk_w, 4) || misaligned(dx_router, 4) || misaligned(dw_router, 16) ||
        misaligned(loss, 4))
      return MOE_ERR_UNSUPPORTED;
  }
  if (!x || !w_router || !scores || !topk_idx || !d_topk_w || !dw_router || !loss || !ws) return MOE_ERR_NULL;
  if (!(alpha >= 0.0f) || !isfinite(alpha)) return MOE_ERR_SHAPE;
  if (seq_len < 0 || (seq_len > 0 && cfg->T % seq_len != 0)) return MOE_ERR_SHAPE;
  const RouteBwdLayout L(cfg, seq_len, with_flags ? 2 : 1);
  if (with_flags && (cfg->T >= 1 << 23 || (int64_t)L.nseq * ((cfg->E + 63) / 64) >= 1 << 24)) return MOE_ERR_SHAPE;
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  hipStream_t s = as_stream(stream);
  char* base = static_cast<char*>(ws);
  int32_t* cnt = reinterpret_cast<int32_t*>(base + L.off_cnt);
  float* psum = reinterpret_cast<float*>(base + L.off_psum);
  float* coef = reinterpret_cast<float*>(base + L.off_coef);
  bf16_t* dlogit = reinterpret_cast<bf16_t*>(base + L.off_dlogit);
  float* part = reinterpret_cast<float*>(base + L.off_part);
  if (cfg->T == 0) {
    hipLaunchKernelGGL(seq_coef_kernel, dim3(1), dim3(256), 0, s, cnt, psum, cfg->E, cfg->k, 1, 0, 0, 0.0f, coef,
                       loss);
    if ((st = launch_status()) != MOE_OK) return st;
    return launch_zero(dw_router, (int64_t)cfg->E * cfg->H, s);
  }
  const bool bal = alpha > 0.0f;
  if (bal) {
    by_epl(cfg->E, [&](auto epl) {
      hipLaunchKernelGGL((seq_stats_kernel<decltype(epl)::value>), dim3((unsigned)(L.nseq * L.nchunk)), dim3(256), 0, s,
                         scores, topk_idx, cfg->T, cfg->E, cfg->k, L.seq_len, L.nchunk, cnt, psum);
    });
    if ((st = launch_status()) != MOE_OK) return st;
  }
  SeqLoss seq{reinterpret_cast<float*>(base + L.off_loss), bal ? L.nseq * ((cfg->E + 63) / 64) : 0, alpha / (float)L.nseq,
              loss};
  if (with_flags) {
    if (bal)
      hipLaunchKernelGGL(seq_coef_part_kernel, dim3((unsigned)seq.n), dim3(256), 0, s, cnt, psum, cfg->E, cfg->k,
                         L.seq_len, L.nseq, L.nchunk, alpha, coef, (float*)(base + L.off_loss));
    if (seq.n > kLossInline) {
      hipLaunchKernelGGL(seq_loss_kernel, dim3(1), dim3(1024), 0, s, seq);
      seq.loss = nullptr;
    }
  } else {
    hipLaunchKernelGGL(seq_coef_kernel, dim3(1), dim3(256), 0, s, cnt, psum, cfg->E, cfg->k, L.seq_len,
                       bal ? L.nseq : 0, L.nchunk, alpha, coef, loss);
  }
  if ((st = launch_status()) != MOE_OK) return st;
  const dim3 tokens((unsigned)((cfg->T + 3) / 4));
  if (!with_flags) {
    hipLaunchKernelGGL(route_grad_kernel, tokens, dim3(256), 0, s, scores, topk_idx, d_topk_w, bal ? coef : nullptr,
                       cfg->T, cfg->E, cfg->k, L.seq_len, cfg->route_scale, dlogit);
    if ((st = launch_status()) != MOE_OK) return st;
    return launch_router_bwd_gemms(cfg, (const bf16_t*)x, (const bf16_t*)w_router, dlogit, part, L.nsplit, dw_router,
                                   dx_router, s);
  }
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, tokens, dim3(256), 0, s, scores, topk_idx, d_topk_w, bal ? coef : nullptr, cfg->T, cfg->E,
                       L.Ep, cfg->k, L.seq_len, cfg->route_scale, (flags & MOE_GATES_RAW) != 0, dlogit, seq);
  };
  by_epl(cfg->E, [&](auto epl) {
    if (flags & MOE_SOFTMAX) launch(route_grad_flags_kernel<true, decltype(epl)::value>);
    else launch(route_grad_flags_kernel<false, decltype(epl)::value>);
  });
  if ((st = launch_status()) != MOE_OK) return st;
  return launch_router_bwd_gemms2(cfg, L, (const bf16_t*)x, (const bf16_t*)w_router, dlogit, part, dw_router, dx_router, s);
}

}  // namespace

extern "C" moe_status moe_route_backward(const moe_cfg* cfg, const void* x, const void* w_router,
                                         const float* scores, const int32_t* topk_idx, const float* d_topk_w,
                                         float alpha, int32_t seq_len, float* dx_router, float* dw_router,
                                         float* loss, void* ws, size_t ws_bytes, void* stream) {
  return route_backward(cfg, false, 0, x, w_router, scores, topk_idx, d_topk_w, alpha, seq_len, dx_router, dw_router, loss,
                        ws, ws_bytes, stream);
}

extern "C" moe_status moe_route_backward_flags(const moe_cfg* cfg, uint32_t flags, const void* x, const void* w_router,
                                               const float* scores, const int32_t* topk_idx, const float* d_topk_w,
                                               float alpha, int32_t seq_len, float* dx_router, float* dw_router,
                                               float* loss, void* ws, size_t ws_bytes, void* stream) {
  return route_backward(cfg, true, flags, x, w_router, scores, topk_idx, d_topk_w, alpha, seq_len, dx_router, dw_router,
                        loss, ws, ws_bytes, stream);
}

extern "C" moe_status moe_dispatch_backward(const moe_cfg* cfg, const void* dx_perm, const void* dx_shared,
                                            const float* dx_router, const int32_t* inv, void* dx, void* stream) {
  moe_status st = validate_cfg(cfg);
  if (st != MOE_OK) return st;
  if (!bwd_dtypes_ok(cfg)) return MOE_ERR_UNSUPPORTED;
  if (!dx_perm || !inv || !dx || (cfg->S > 0 && !dx_shared)) return MOE_ERR_NULL;
  if (cfg->T == 0) return MOE_OK;
  const int64_t nchunk = (int64_t)cfg->H * 2 / 16;
  hipLaunchKernelGGL(dispatch_bwd_kernel, dim3((unsigned)cfg->T), row_block(nchunk), 0, as_stream(stream),
                     (const uint4*)dx_perm, cfg->S > 0 ? (const uint4*)dx_shared : nullptr,
                     (const float4*)dx_router, inv, cfg->k, nchunk, (uint4*)dx);
  return launch_status();
}

extern "C" moe_status moe_dispatch_local_backward(const moe_cfg* cfg, const void* dx_perm, const void* dx_shared,
                                                  const float* dx_router, const int32_t* inv, void* dx,
                                                  void* stream) {
  moe_status st = validate_share(cfg);
  if (st != MOE_OK) return st;
  if (!bwd_dtypes_ok(cfg)) return MOE_ERR_UNSUPPORTED;
  if (cfg->T == 0) return MOE_OK;
  if (!dx_perm || !inv || !dx || (cfg->S > 0 && !dx_shared)) return MOE_ERR_NULL;
  if (misaligned(dx_perm, 16) || (cfg->S > 0 && misaligned(dx_shared, 16)) || misaligned(dx_router, 16) ||
      misaligned(dx, 16) || misaligned(inv, 4))
    return MOE_ERR_UNSUPPORTED;
  const int64_t nchunk = (int64_t)cfg->H * 2 / 16;
  hipLaunchKernelGGL(dispatch_local_bwd_kernel, dim3((unsigned)cfg->T), local_block(nchunk), 0, as_stream(stream),
                     (const uint4*)dx_perm, cfg->S > 0 ? (const uint4*)dx_shared : nullptr,
                     (const float4*)dx_router, inv, cfg->k, nchunk, (uint4*)dx);
  return launch_status();
}
