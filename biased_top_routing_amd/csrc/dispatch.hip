// moe_dispatch: per-expert load count, expert-sorted stable permutation of the
// (token, slot) pairs, and the permuted activation rows.
//
// Tokens are dispatched to the experts they selected and combined back later
// (DeepSeek-V3 Technical Report：中英对照解读, §2.2); each expert's load is
// counted over the whole batch (qwbw.cn essay on the DeepSeek-V3 report,
// load-balancing section).  On one GPU dispatch is a permutation.
//
// Design: no atomics.  Flat pair ids f = t*k + j are cut into segments of
// kSegPairs, one wavefront each.  Inside a wavefront the lanes holding the same
// expert find each other with ballots over the bits of the expert id, so each
// pair learns how many earlier pairs of its segment share its expert, and one
// leader lane per expert updates the segment's LDS counter.  A column scan over
// segments turns the per-segment counts into stable destinations.
#include <mutex>

#include "common.h"
#include "ffn_layout.h"
#include "fp4.h"
#include "kernels.h"

namespace moe {

__device__ __forceinline__ uint64_t lanes_below() {
  const int lane = threadIdx.x & (kWave - 1);
  return lane == 0 ? 0ull : (~0ull >> (64 - lane));
}

// Lanes of this wavefront whose (valid) expert id equals mine.
__device__ __forceinline__ uint64_t same_expert_lanes(int e, bool valid, int nbits) {
  uint64_t m = __ballot(valid);
  for (int b = 0; b < nbits; ++b) {
    const bool bit = (e >> b) & 1;
    const uint64_t on = __ballot(valid && bit);
    m &= bit ? on : ~on;
  }
  return m;
}

// The expert ids of segment `seg` held by this lane (pair lo + 64 it + lane),
// all loaded before any is used; -1 past the last pair.
__device__ __forceinline__ void load_segment(const int32_t* __restrict__ idx, int64_t seg, int64_t N,
                                             int (&ev)[kSegPairs / kWave]) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t lo = seg * kSegPairs;
#pragma unroll
  for (int it = 0; it < kSegPairs / kWave; ++it) {
    const int64_t f = lo + it * kWave + lane;
    ev[it] = f < N ? idx[f] : -1;
  }
}

__global__ __launch_bounds__(256) void count_kernel(const int32_t* __restrict__ idx, int64_t N,
                                                    int E, int nbits, int64_t nseg,
                                                    int32_t* __restrict__ segcounts) {
  extern __shared__ int32_t cnt_all[];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int32_t* cnt = cnt_all + wave * E;
  const int64_t seg = (int64_t)blockIdx.x * 4 + wave;
  for (int e = lane; e < E; e += kWave) cnt[e] = 0;
  __syncthreads();
  int ev[kSegPairs / kWave];
  load_segment(idx, seg, N, ev);
#pragma unroll
  for (int it = 0; it < kSegPairs / kWave; ++it) {
    const bool valid = (unsigned)ev[it] < (unsigned)E;   // (an id outside [0, E) is not counted)
    const int e = valid ? ev[it] : 0;
    const uint64_t m = same_expert_lanes(e, valid, nbits);
    if (valid && (m & lanes_below()) == 0) cnt[e] += __popcll(m);
  }
  __syncthreads();
  if (seg < nseg)
    for (int e = lane; e < E; e += kWave) segcounts[seg * E + e] = cnt[e];
}

// Column scan over segments: segcounts[s][e] becomes the number of pairs of
// expert e in segments before s; counts[e] the total; offsets the exclusive
// prefix of counts over experts.
__global__ __launch_bounds__(1024) void scan_kernel(int32_t* __restrict__ segcounts, int64_t nseg,
                                                    int E, int Ep2, int32_t* __restrict__ counts,
                                                    int32_t* __restrict__ offsets) {
  extern __shared__ int32_t sm[];
  const int P = 1024 / Ep2;                 // parts per expert column
  int32_t* part_sum = sm;                   // [P][Ep2]
  int32_t* tot = sm + P * Ep2;              // [Ep2]
  const int tid = threadIdx.x;
  const int e = tid % Ep2, part = tid / Ep2;
  const int64_t chunk = (nseg + P - 1) / P;
  const int64_t s0 = part * chunk;
  const int64_t s1 = s0 + chunk < nseg ? s0 + chunk : nseg;
  // (the column is walked in batches of kScanBatch segments whose loads are all
  // issued before any is added)
  constexpr int kScanBatch = 16;
  int32_t acc = 0;
  if (e < E)
    for (int64_t b = s0; b < s1; b += kScanBatch) {
      int32_t c[kScanBatch];
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) c[i] = b + i < s1 ? segcounts[(b + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) acc += c[i];
    }
  part_sum[part * Ep2 + e] = acc;
  __syncthreads();
  int32_t run = 0;
  for (int p = 0; p < part; ++p) run += part_sum[p * Ep2 + e];
  if (e < E)
    for (int64_t b = s0; b < s1; b += kScanBatch) {
      int32_t c[kScanBatch];
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) c[i] = b + i < s1 ? segcounts[(b + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i)
        if (b + i < s1) {
          segcounts[(b + i) * E + e] = run;
          run += c[i];
        }
    }
  if (part == 0) {
    int32_t total = 0;
    for (int p = 0; p < P; ++p) total += part_sum[p * Ep2 + e];
    tot[e] = e < E ? total : 0;
    if (e < E) counts[e] = total;
  }
  __syncthreads();
  for (int d = 1; d < Ep2; d <<= 1) {     // inclusive scan of tot over experts
    int32_t v = 0;
    if (part == 0 && e >= d) v = tot[e - d];
    __syncthreads();
    if (part == 0) tot[e] += v;
    __syncthreads();
  }
  if (part == 0 && e < E) offsets[e + 1] = tot[e];
  if (tid == 0) offsets[0] = 0;
}

__global__ __launch_bounds__(256) void rank_kernel(const int32_t* __restrict__ idx, int64_t N, int E,
                                                   int nbits, int64_t nseg,
                                                   const int32_t* __restrict__ segprefix,
                                                   const int32_t* __restrict__ offsets,
                                                   int32_t* __restrict__ perm,
                                                   int32_t* __restrict__ inv) {
  extern __shared__ int32_t cnt_all[];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int32_t* cnt = cnt_all + wave * E;
  const int64_t seg = (int64_t)blockIdx.x * 4 + wave;
  if (seg < nseg)
    for (int e = lane; e < E; e += kWave) cnt[e] = offsets[e] + segprefix[seg * E + e];
  __syncthreads();
  const int64_t lo = seg * kSegPairs;
  int ev[kSegPairs / kWave];
  load_segment(idx, seg, N, ev);
#pragma unroll
  for (int it = 0; it < kSegPairs / kWave; ++it) {
    const int64_t f = lo + it * kWave + lane;
    const bool valid = (unsigned)ev[it] < (unsigned)E;   // (an id outside [0, E) is not counted)
    const int e = valid ? ev[it] : 0;
    const uint64_t m = same_expert_lanes(e, valid, nbits);
    const int32_t base = valid ? cnt[e] : 0;
    const int32_t pos = base + __popcll(m & lanes_below());
    if (valid && (m & lanes_below()) == 0) cnt[e] = base + __popcll(m);
    if (valid) {
      perm[pos] = (int32_t)f;
      inv[f] = pos;
    }
  }
}

// ---- the same over a share: some pairs are absent
// Present are the pairs of the first *n_tokens tokens (nullptr: all T) whose
// expert id less `first` lies in [0, E).
struct Window {
  const int32_t* n_tokens;
  int first, T, k;
};

// Pairs [0, limit) belong to live tokens.
__device__ __forceinline__ int64_t live_pairs(const Window& w, int64_t N) {
  return w.n_tokens ? (int64_t)min(max(*w.n_tokens, 0), w.T) * w.k : N;
}

// One workgroup per segment, a quarter of its pairs per wavefront (a wavefront
// alone walks its 16 rounds of ballots one after the other: at 131072 pairs the
// whole dispatch takes 18 us longer with one).
constexpr int kQuarter = kSegPairs / 4;

// The share's experts of this lane's pairs (lo + 64 it + lane), -1 for absent ones;
// every id is asked for before the live count is looked at.
__device__ __forceinline__ void load_quarter(const int32_t* __restrict__ idx, int64_t lo, int64_t N, const Window& w,
                                             int E, int (&ev)[kQuarter / kWave]) {
  const int lane = threadIdx.x & (kWave - 1);
  uint32_t id[kQuarter / kWave];
#pragma unroll
  for (int it = 0; it < kQuarter / kWave; ++it) {
    const int64_t f = lo + it * kWave + lane;
    id[it] = f < N ? (uint32_t)idx[f] : ~0u;
  }
  const int64_t limit = live_pairs(w, N);
#pragma unroll
  for (int it = 0; it < kQuarter / kWave; ++it) {
    const uint32_t e = id[it] - (uint32_t)w.first;
    ev[it] = lo + it * kWave + lane < limit && e < (uint32_t)E ? (int)e : -1;
  }
}

// Counts the wavefront's pairs by expert in cnt (zeroed), and gives each present
// one the number of earlier ones of its expert.
__device__ __forceinline__ void count_quarter(const int (&ev)[kQuarter / kWave], int nbits, int32_t* cnt,
                                              int (&before)[kQuarter / kWave]) {
#pragma unroll
  for (int it = 0; it < kQuarter / kWave; ++it) {
    const bool here = ev[it] >= 0;
    const int e = here ? ev[it] : 0;
    const uint64_t m = same_expert_lanes(e, here, nbits);
    const int32_t base = here ? cnt[e] : 0;
    before[it] = base + __popcll(m & lanes_below());
    if (here && (m & lanes_below()) == 0) cnt[e] = base + __popcll(m);
  }
}

__global__ __launch_bounds__(256) void count_local_kernel(const int32_t* __restrict__ idx, int64_t N, int E, int nbits,
                                                          Window win, int32_t* __restrict__ segcounts) {
  extern __shared__ int32_t cnt_all[];                  // [4][E]
  const int wave = threadIdx.x >> 6;
  const int64_t seg = blockIdx.x;
  for (int e = threadIdx.x; e < 4 * E; e += 256) cnt_all[e] = 0;
  int ev[kQuarter / kWave], before[kQuarter / kWave];
  load_quarter(idx, seg * kSegPairs + wave * kQuarter, N, win, E, ev);
  __syncthreads();
  count_quarter(ev, nbits, cnt_all + wave * E, before);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256)
    segcounts[seg * E + e] = cnt_all[e] + cnt_all[E + e] + cnt_all[2 * E + e] + cnt_all[3 * E + e];
}

// SUM: segcounts are the segments' counts as they were taken, and every workgroup
// adds up what it needs of them (at most kSumCounts, E <= 256) instead of waiting for
// scan_kernel; workgroup 0 writes counts and offsets (bf16 rows, the whole dispatch
// with scan_kernel and without: T = 16384, k = 8, H = 7168, 32 of 256 experts held 83.2
// and 79.0 us; H = 1024, all 256 held, 32768 counts 72.5 and 70.4; T = 4096, k = 6, H =
// 2048, 8 of 64 held 17.4 and 14.3).
constexpr int kSumCounts = 32768;

template <bool SUM>
__global__ __launch_bounds__(256) void rank_local_kernel(const int32_t* __restrict__ idx, int64_t N, int E, int nbits,
                                                         Window win, const int32_t* __restrict__ segcounts, int nseg,
                                                         int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
  extern __shared__ int32_t cnt_all[];                  // [4][E] counts, then [4][E] first rows
  __shared__ int32_t all_s[256], earlier_s[256], wave_s[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t seg = blockIdx.x, lo = seg * kSegPairs + wave * kQuarter;
  for (int e = threadIdx.x; e < 4 * E; e += 256) cnt_all[e] = 0;
  int ev[kQuarter / kWave], before[kQuarter / kWave];
  load_quarter(idx, lo, N, win, E, ev);
  if constexpr (SUM) {                                  // a power of two of threads an expert
    const int e = threadIdx.x & ((1 << nbits) - 1), part = threadIdx.x >> nbits, parts = 256 >> nbits;
    int32_t all = 0, earlier = 0;
    if (e < E) {
#pragma unroll 8
      for (int b = part; b < nseg; b += parts) {
        const int32_t c = segcounts[b * E + e];
        all += c;
        earlier += b < seg ? c : 0;
      }
    }
    all_s[threadIdx.x] = all;
    earlier_s[threadIdx.x] = earlier;
  }
  __syncthreads();
  count_quarter(ev, nbits, cnt_all + wave * E, before);
  if constexpr (SUM) {
    const int e = threadIdx.x, step = 1 << nbits;
    int32_t all = 0, earlier = 0;
    if (e < E)
      for (int i = e; i < 256; i += step) all += all_s[i], earlier += earlier_s[i];
    int32_t upto = all;                                 // inclusive scan over the experts
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 63) wave_s[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; ++w) upto += wave_s[w];
    if (seg == 0) {
      if (e < E) counts[e] = all, offsets[e + 1] = upto;
      if (e == 0) offsets[0] = 0;
    }
    earlier_s[e] = upto - all + earlier;                // (all entries have been read: the barrier above)
  }
  __syncthreads();
  int32_t* first = cnt_all + 4 * E;
  for (int e = threadIdx.x; e < E; e += 256) {
    int32_t at = SUM ? earlier_s[e] : offsets[e] + segcounts[seg * E + e];
    for (int w = 0; w < 4; ++w) {
      first[w * E + e] = at;
      at += cnt_all[w * E + e];
    }
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kQuarter / kWave; ++it) {
    const int64_t f = lo + it * kWave + lane;
    if (f >= N) continue;
    int32_t pos = -1;
    if (ev[it] >= 0) {
      pos = first[wave * E + ev[it]] + before[it];
      perm[pos] = (int32_t)f;
    }
    inv[f] = pos;
  }
}

// One wavefront per token: load the token's row once, store it to each of its
// k destination rows.  16-byte chunks; CPL chunks per lane per pass.  Plain
// stores: with x read from HBM (the Infinity Cache flushed before the launch)
// non-temporal ones were 11% slower, and a training step, which reads the
// permuted rows back, ran at the same speed with either.  LOCAL (here and in the
// quantising copies below): absent pairs (inv = -1) are skipped, and a token
// without any present one is not read.
#ifndef MOE_PERMUTE_NT
#define MOE_PERMUTE_NT 0
#endif
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void st_stream(uint4* p, uint4 v) {
#if MOE_PERMUTE_NT
  __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_t*>(p));
#else
  *p = v;
#endif
}
template <int CPL, bool LOCAL>
__global__ __launch_bounds__(256) void permute_rows_kernel(const uint4* __restrict__ src,
                                                           const int32_t* __restrict__ inv, int T,
                                                           int k, int64_t nchunk,
                                                           uint4* __restrict__ dst) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int32_t myp = lane < k ? inv[t * k + lane] : LOCAL ? -1 : 0;
  if (LOCAL && !__any(myp >= 0)) return;
  for (int64_t c0 = 0; c0 < nchunk; c0 += (int64_t)CPL * kWave) {
    uint4 v[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int64_t c = c0 + i * kWave + lane;
      v[i] = src[t * nchunk + (c < nchunk ? c : nchunk - 1)];   // tail lanes reload the last chunk
    }
    for (int j = 0; j < k; ++j) {
      const int64_t p = __shfl(myp, j);
      if (LOCAL && p < 0) continue;
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const int64_t c = c0 + i * kWave + lane;
        if (c >= nchunk) continue;
        // (a share's rows: non-temporal, T = 16384, H = 7168, an eighth of the experts
        // 92 -> 83 us the whole dispatch, every expert of T = 8192 230 -> 201 us, both with
        // x partly in the memory-side cache; not measured with x cold, as the plain stores above)
        if constexpr (LOCAL)
          __builtin_nontemporal_store(u32x4_t{v[i].x, v[i].y, v[i].z, v[i].w},
                                      reinterpret_cast<u32x4_t*>(&dst[p * nchunk + c]));
        else
          st_stream(&dst[p * nchunk + c], v[i]);
      }
    }
  }
}

// 1 x 128 E4M3 quantisation of a chunk of 8 bf16 values held by this lane;
// 16 consecutive lanes hold one tile.  Returns the 8 codes packed and the
// tile's scale (sc = amax / 448, or 1 for an all-zero tile).
__device__ __forceinline__ uint2 quant_chunk_1x128(uint4 raw, float* sc_out) {
  float v[8];
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32((bf16_t)(w[i] & 0xFFFF));
    v[2 * i + 1] = bf16_to_f32((bf16_t)(w[i] >> 16));
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off));
  const float sc = amax == 0.f ? 1.0f : __fdiv_rn(amax, 448.0f);
  const float y = __fdiv_rn(1.0f, sc);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = div_by_scale(v[i], sc, y);   // fl32(v / sc)
  *sc_out = sc;
  return make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
}

// fp8 dispatch: quantise the token's bf16 row per 1x128 tile once, then store
// the codes and scales to each of its k destination rows.
template <int CPL, bool LOCAL>
__global__ __launch_bounds__(256) void permute_rows_fp8_kernel(const uint4* __restrict__ src,
                                                               const int32_t* __restrict__ inv,
                                                               int T, int k, int H,
                                                               uint2* __restrict__ dst,
                                                               float* __restrict__ dst_scale) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;      // whole wavefront exits together
  const int64_t nchunk = H / 8, ntile = H / 128;
  const int32_t myp = lane < k ? inv[t * k + lane] : LOCAL ? -1 : 0;
  if (LOCAL && !__any(myp >= 0)) return;
  for (int64_t c0 = 0; c0 < nchunk; c0 += (int64_t)CPL * kWave) {
    uint2 q[CPL];
    float sc[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int64_t c = c0 + i * kWave + lane;
      // a 16-lane tile group is wholly inside or outside the row (H % 128 == 0)
      const uint4 raw = c < nchunk ? src[t * nchunk + c] : make_uint4(0, 0, 0, 0);
      q[i] = quant_chunk_1x128(raw, &sc[i]);
    }
    for (int j = 0; j < k; ++j) {
      const int64_t p = __shfl(myp, j);
      if (LOCAL && p < 0) continue;
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const int64_t c = c0 + i * kWave + lane;
        if (c < nchunk) {
          dst[p * nchunk + c] = q[i];
          if ((lane & 15) == 0) dst_scale[p * ntile + c / 16] = sc[i];
        }
      }
    }
  }
}

// MXFP4 dispatch (format: fp4.h): quantise the token's bf16 row once, then store
// the codes and the scale words of its 128-column groups to each of its k
// destination rows (a row's scale words lie ntile planes of T*k words apart).
template <int CPL, bool LOCAL>
__global__ __launch_bounds__(256) void permute_rows_fp4_kernel(const uint4* __restrict__ src,
                                                               const int32_t* __restrict__ inv,
                                                               int T, int k, int H,
                                                               uint32_t* __restrict__ dst,
                                                               uint32_t* __restrict__ dst_scale) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;      // whole wavefront exits together
  const int64_t nchunk = H / 8, P = (int64_t)T * k;
  const int32_t myp = lane < k ? inv[t * k + lane] : LOCAL ? -1 : 0;
  if (LOCAL && !__any(myp >= 0)) return;
  for (int64_t c0 = 0; c0 < nchunk; c0 += (int64_t)CPL * kWave) {
    uint32_t q[CPL], sw[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int64_t c = c0 + i * kWave + lane;
      // a 16-lane group of 128 columns is wholly inside or outside the row (H % 128 == 0)
      const uint4 raw = c < nchunk ? src[t * nchunk + c] : make_uint4(0, 0, 0, 0);
      uint32_t e;
      q[i] = mx_quant_chunk(raw, &e);
      sw[i] = mx_scale_word(e);
    }
    for (int j = 0; j < k; ++j) {
      const int64_t p = __shfl(myp, j);
      if (LOCAL && p < 0) continue;
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const int64_t c = c0 + i * kWave + lane;
        if (c < nchunk) {
          dst[p * nchunk + c] = q[i];
          if ((lane & 15) == 0) dst_scale[c / 16 * P + p] = sw[i];
        }
      }
    }
  }
#endif
}

// Row quantisation without permutation (shared-expert input, tests).
__global__ __launch_bounds__(256) void quantize_rows_kernel(const uint4* __restrict__ src,
                                                            int64_t rows, int cols,
                                                            uint2* __restrict__ dst,
                                                            float* __restrict__ dst_scale) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= rows) return;
  const int64_t nchunk = cols / 8, ntile = cols / 128;
  for (int64_t c0 = 0; c0 < nchunk; c0 += kWave) {
    const int64_t c = c0 + lane;
    float sc;
    const uint4 raw = c < nchunk ? src[r * nchunk + c] : make_uint4(0, 0, 0, 0);
    const uint2 q = quant_chunk_1x128(raw, &sc);
    if (c < nchunk) {
      dst[r * nchunk + c] = q;
      if ((lane & 15) == 0) dst_scale[r * ntile + c / 16] = sc;
    }
  }
}

moe_status launch_quantize_rows(const bf16_t* src, int64_t rows, int cols, fp8_t* dst, float* scales,
                                hipStream_t st) {
  if (rows == 0) return MOE_OK;
  hipLaunchKernelGGL(quantize_rows_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st,
                     (const uint4*)src, rows, cols, (uint2*)dst, scales);
  return launch_status();
}

// 128 x 128 weight blocks: one workgroup per block.
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const bf16_t* __restrict__ src,
                                                              int rows, int cols,
                                                              uint8_t* __restrict__ dst,
                                                              float* __restrict__ scales) {
  __shared__ float red[4];
  const int nbc = cols / 128, nbr = rows / 128;
  const int64_t blk = blockIdx.x;
  const int64_t mat = blk / ((int64_t)nbr * nbc);
  const int br = (int)((blk / nbc) % nbr), bc = (int)(blk % nbc);
  const bf16_t* s = src + mat * (int64_t)rows * cols;
  uint8_t* d = dst + mat * (int64_t)rows * cols;
  float v[64];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = threadIdx.x + 256 * i;          // 2048 chunks of 8 values
    const int r = q >> 4, cc = q & 15;
    const uint4 raw = *reinterpret_cast<const uint4*>(s + (int64_t)(br * 128 + r) * cols + bc * 128 + cc * 8);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v[8 * i + 2 * h] = bf16_to_f32((bf16_t)(w[h] & 0xFFFF));
      v[8 * i + 2 * h + 1] = bf16_to_f32((bf16_t)(w[h] >> 16));
    }
#pragma unroll
    for (int h = 0; h < 8; ++h) amax = fmaxf(amax, fabsf(v[8 * i + h]));
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float sc = amax == 0.f ? 1.0f : __fdiv_rn(amax, 448.0f);
  const float y = __fdiv_rn(1.0f, sc);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = threadIdx.x + 256 * i;
    const int r = q >> 4, cc = q & 15;
    float t[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) t[h] = div_by_scale(v[8 * i + h], sc, y);   // fl32(v / sc)
    *reinterpret_cast<uint2*>(d + (int64_t)(br * 128 + r) * cols + bc * 128 + cc * 8) =
        make_uint2(e4m3x4(t[0], t[1], t[2], t[3]), e4m3x4(t[4], t[5], t[6], t[7]));
  }
  if (threadIdx.x == 0) scales[(mat * nbr + br) * nbc + bc] = sc;
}

// ---- a small share in one launch
// Row formats of the copy.
enum { kRowsCopy = 0, kRowsFp8 = 1, kRowsFp4 = 2, kRowsNone = 3 };

// Workgroup t < T does token t, workgroup T the counts.  A pair's row is the
// number of pairs that come before it, ordered by (expert, pair id): with the
// key expert * N + f of every pair, absent ones last, the keys below its own.
// Every workgroup holds all N <= kSmallPairs keys in its registers, kSmallPer a
// lane, and counts by ballot: k * kSmallPer compares a wavefront (8 slots: 128).
// That repeats the counting T times, and saves the two launches that compute it once.
// Measured, one launch against three (bf16, every expert held): T = 128, k = 8, H =
// 7168: 8.7 and 15.8 us; at 4096 pairs, T = 512, k = 8, H = 7168: 17.9 and 21.8 us (an
// eighth of the experts held: 10.0 and 13.3), T = 4096, k = 1, H = 1024: 13.8 and 13.7
// us.  More pairs would need more than 16 keys a lane.
constexpr int kSmallThreads = 256, kSmallPer = 16, kSmallPairs = kSmallThreads * kSmallPer;

template <int ROWS>
__global__ __launch_bounds__(kSmallThreads) void dispatch_small_kernel(
    const int32_t* __restrict__ idx, const uint4* __restrict__ x, int N, int E, int64_t nchunk, Window win,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ perm, int32_t* __restrict__ inv,
    void* __restrict__ x_perm, void* __restrict__ x_scale) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int k = win.k, limit = (int)live_pairs(win, N);
  const uint32_t absent = (uint32_t)E * (uint32_t)N;   // E <= 512, N <= 4096: below 2^31
  auto key = [&](int f) {
    const uint32_t e = f < limit ? (uint32_t)idx[f] - (uint32_t)win.first : ~0u;
    return e < (uint32_t)E ? e * (uint32_t)N + (uint32_t)f : absent;
  };
  if ((int)blockIdx.x == win.T) {                       // counts and offsets
    __shared__ int32_t cnt[512];
    for (int e = tid; e < 512; e += kSmallThreads) cnt[e] = 0;
    __syncthreads();
    for (int f = tid; f < N; f += kSmallThreads) {
      const uint32_t q = key(f);
      if (q < absent) atomicAdd(&cnt[q / (uint32_t)N], 1);   // (integer counts: the order does not matter)
    }
    __syncthreads();
    const int c0 = cnt[tid], c1 = cnt[tid + 256];
    for (int d = 1; d < 512; d <<= 1) {                 // inclusive scan, two entries a thread
      const int v0 = tid >= d ? cnt[tid - d] : 0, v1 = tid + 256 >= d ? cnt[tid + 256 - d] : 0;
      __syncthreads();
      cnt[tid] += v0;
      cnt[tid + 256] += v1;
      __syncthreads();
    }
    if (tid == 0) offsets[0] = 0;
    if (tid < E) counts[tid] = c0, offsets[tid + 1] = cnt[tid];
    if (tid + 256 < E) counts[tid + 256] = c1, offsets[tid + 257] = cnt[tid + 256];
    return;
  }
  const int64_t t = blockIdx.x;
  __shared__ int32_t below[4][32];
  __shared__ int32_t dest[32];
  // the row's first chunks are on their way while the pairs are counted
  constexpr int U = 4;
  const uint4* row = x + t * nchunk;
  uint4 v[U];
  auto load = [&](int64_t c0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * kSmallThreads + tid;
      v[u] = c < nchunk ? row[c] : make_uint4(0, 0, 0, 0);
    }
  };
  uint32_t q[kSmallPer];
#pragma unroll
  for (int i = 0; i < kSmallPer; ++i) {
    const int f = tid + i * kSmallThreads;
    q[i] = f < N ? key(f) : absent;
  }
  const uint32_t own = lane < k ? key((int)t * k + lane) : absent;   // the token's pairs, one a lane
  if constexpr (ROWS != kRowsNone) {
    if ((int)t * k < limit) load(0);
  }
  for (int j = 0; j < k; ++j) {
    const uint32_t mine = (uint32_t)__builtin_amdgcn_readlane((int)own, j);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSmallPer; ++i) n += __popcll(__ballot(q[i] < mine));
    if (lane == 0) below[wave][j] = mine < absent ? n : -1;
  }
  __syncthreads();
  if (tid < k) {
    const int f = (int)t * k + tid;
    int32_t p = -1;
    if (below[0][tid] >= 0) {
      p = below[0][tid] + below[1][tid] + below[2][tid] + below[3][tid];
      perm[p] = f;
    }
    inv[f] = p;
    dest[tid] = p;
  }
  if constexpr (ROWS == kRowsNone) return;
  __syncthreads();
  bool any = false;
  for (int j = 0; j < k; ++j) any |= dest[j] >= 0;
  if (!any) return;
  for (int64_t c0 = 0; c0 < nchunk; c0 += U * kSmallThreads) {
    if (c0 > 0) load(c0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * kSmallThreads + tid;
      // (quantised rows: a 16-lane group of 128 columns is wholly inside or outside the row)
      uint2 w8;
      float sc;
      uint32_t w4, sw;
      if constexpr (ROWS == kRowsFp8) w8 = quant_chunk_1x128(v[u], &sc);
      if constexpr (ROWS == kRowsFp4) {
        uint32_t e;
        w4 = mx_quant_chunk(v[u], &e);
        sw = mx_scale_word(e);
      }
      if (c >= nchunk) continue;
      for (int j = 0; j < k; ++j) {
        const int64_t p = dest[j];
        if (p < 0) continue;
        if constexpr (ROWS == kRowsCopy) static_cast<uint4*>(x_perm)[p * nchunk + c] = v[u];
        if constexpr (ROWS == kRowsFp8) {
          static_cast<uint2*>(x_perm)[p * nchunk + c] = w8;
          if ((lane & 15) == 0) static_cast<float*>(x_scale)[p * (nchunk / 16) + c / 16] = sc;
        }
        if constexpr (ROWS == kRowsFp4) {
          static_cast<uint32_t*>(x_perm)[p * nchunk + c] = w4;
          if ((lane & 15) == 0) static_cast<uint32_t*>(x_scale)[c / 16 * N + p] = sw;
        }
      }
    }
  }
#endif
}

static moe_status dispatch_small(const moe_cfg* cfg, const Window& win, const int32_t* topk_idx, const void* x,
                                 int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* x_perm,
                                 float* x_perm_scale, hipStream_t s) {
  const int64_t nchunk = (int64_t)cfg->H * act_bytes(cfg) / 16;
  const int N = (int)pairs(cfg);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)cfg->T + 1), dim3(kSmallThreads), 0, s, topk_idx, (const uint4*)x, N,
                       cfg->E, nchunk, win, counts, offsets, perm, inv, x_perm, (void*)x_perm_scale);
  };
  if (!x_perm) go(dispatch_small_kernel<kRowsNone>);
  else if (cfg->wgt == MOE_MXFP4) go(dispatch_small_kernel<kRowsFp4>);
  else if (cfg->wgt == MOE_FP8_E4M3) go(dispatch_small_kernel<kRowsFp8>);
  else go(dispatch_small_kernel<kRowsCopy>);
  return launch_status();
}

// The kernels of moe_dispatch, with the per-segment counts in `segc`
// (dispatch_segments(cfg) * E int32, no contents required).  Arguments checked.
template <bool LOCAL>
static moe_status dispatch_launch(const moe_cfg* cfg, const Window& win, const int32_t* topk_idx, const void* x,
                                  int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* x_perm,
                                  float* x_perm_scale, int32_t* segc, hipStream_t s) {
  moe_status st;
  const bool fp8 = cfg->wgt == MOE_FP8_E4M3, fp4 = cfg->wgt == MOE_MXFP4;
  const int64_t N = pairs(cfg);
  const int64_t nseg = dispatch_segments(cfg);
  const int E = cfg->E;
  int nbits = 0;
  while ((1 << nbits) < E) ++nbits;
  int Ep2 = 1;
  while (Ep2 < E) Ep2 <<= 1;
  auto permute = [&]() -> moe_status {
    if (!x_perm) return MOE_OK;
    const unsigned tblocks = (unsigned)((cfg->T + 3) / 4);
    if (fp4) {
      hipLaunchKernelGGL((permute_rows_fp4_kernel<8, LOCAL>), dim3(tblocks), dim3(256), 0, s, (const uint4*)x, inv,
                         cfg->T, cfg->k, cfg->H, (uint32_t*)x_perm, (uint32_t*)x_perm_scale);
    } else if (fp8) {
      hipLaunchKernelGGL((permute_rows_fp8_kernel<8, LOCAL>), dim3(tblocks), dim3(256), 0, s, (const uint4*)x, inv,
                         cfg->T, cfg->k, cfg->H, (uint2*)x_perm, x_perm_scale);
    } else {
      const int64_t nchunk = (int64_t)cfg->H * act_bytes(cfg) / 16;
      hipLaunchKernelGGL((permute_rows_kernel<16, LOCAL>), dim3(tblocks), dim3(256), 0, s, (const uint4*)x, inv,
                         cfg->T, cfg->k, nchunk, (uint4*)x_perm);
    }
    return launch_status();
  };
  const unsigned blocks = (unsigned)((nseg + 3) / 4);
  if (nseg > 0) {
    if constexpr (LOCAL)
      hipLaunchKernelGGL(count_local_kernel, dim3((unsigned)nseg), dim3(256), 4 * E * sizeof(int32_t), s, topk_idx, N,
                         E, nbits, win, segc);
    else
      hipLaunchKernelGGL(count_kernel, dim3(blocks), dim3(256), 4 * E * sizeof(int32_t), s, topk_idx, N,
                         E, nbits, nseg, segc);
    if ((st = launch_status()) != MOE_OK) return st;
  }
  if (LOCAL && nseg > 0 && E <= 256 && nseg * E <= kSumCounts) {
    hipLaunchKernelGGL(rank_local_kernel<true>, dim3((unsigned)nseg), dim3(256), 8 * E * sizeof(int32_t), s, topk_idx,
                       N, E, nbits, win, segc, (int)nseg, counts, offsets, perm, inv);
    if ((st = launch_status()) != MOE_OK) return st;
    return permute();
  }
  const int P = 1024 / Ep2;
  hipLaunchKernelGGL(scan_kernel, dim3(1), dim3(1024), (size_t)(P + 1) * Ep2 * sizeof(int32_t), s, segc,
                     nseg, E, Ep2, counts, offsets);
  if ((st = launch_status()) != MOE_OK) return st;
  if (nseg == 0) return MOE_OK;
  if constexpr (LOCAL)
    hipLaunchKernelGGL(rank_local_kernel<false>, dim3((unsigned)nseg), dim3(256), 8 * E * sizeof(int32_t), s, topk_idx,
                       N, E, nbits, win, segc, (int)nseg, counts, offsets, perm, inv);
  else
    hipLaunchKernelGGL(rank_kernel, dim3(blocks), dim3(256), 4 * E * sizeof(int32_t), s, topk_idx, N, E,
                       nbits, nseg, segc, offsets, perm, inv);
  if ((st = launch_status()) != MOE_OK) return st;
  return permute();
}

static moe_status dispatch_check(const moe_cfg* cfg, const int32_t* topk_idx, const void* x, int32_t* counts,
                                 int32_t* offsets, int32_t* perm, int32_t* inv, void* x_perm, float* x_perm_scale) {
  moe_status st = validate_cfg(cfg);
  if (st != MOE_OK) return st;
  const bool fp4 = cfg->wgt == MOE_MXFP4, scaled = fp4 || cfg->wgt == MOE_FP8_E4M3;
  // x_perm == nullptr: indices only (the expert FFN gathers the rows itself)
  if (!topk_idx || !counts || !offsets || !perm || !inv) return MOE_ERR_NULL;
  if (x_perm && (!x || (scaled && !x_perm_scale))) return MOE_ERR_NULL;
  if (fp4 && x_perm && (misaligned(x, 16) || misaligned(x_perm, 16) || misaligned(x_perm_scale, 4)))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_dispatch(const moe_cfg* cfg, const int32_t* topk_idx, const void* x,
                                   int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv,
                                   void* x_perm, float* x_perm_scale, void* ws, size_t ws_bytes,
                                   void* stream) {
  moe_status st = dispatch_check(cfg, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale);
  if (st != MOE_OK) return st;
  if (!ws) return MOE_ERR_NULL;
  if (ws_bytes < dispatch_ws_bytes(cfg)) return MOE_ERR_WORKSPACE;
  return dispatch_launch<false>(cfg, Window{}, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale,
                                static_cast<int32_t*>(ws), as_stream(stream));
}

extern "C" moe_status moe_dispatch_local(const moe_cfg* cfg, int32_t first_expert, const int32_t* n_tokens,
                                         const int32_t* topk_idx, const void* x, int32_t* counts, int32_t* offsets,
                                         int32_t* perm, int32_t* inv, void* x_perm, float* x_perm_scale, void* ws,
                                         size_t ws_bytes, void* stream) {
  moe_status st = validate_share(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T > 0) {   // (an empty batch's tensors may have no address)
    st = dispatch_check(cfg, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale);
    if (st != MOE_OK) return st;
  } else if (!counts || !offsets) {
    return MOE_ERR_NULL;
  }
  // (the kernels take the unsigned difference id - first_expert: with the share below 2^31 no negative id wraps into it)
  if (first_expert < 0 || (int64_t)first_expert + cfg->E > (int64_t)1 << 31) return MOE_ERR_SHAPE;
  if (!ws) return MOE_ERR_NULL;
  if (ws_bytes < dispatch_ws_bytes(cfg)) return MOE_ERR_WORKSPACE;
  for (const void* q : {(const void*)n_tokens, (const void*)topk_idx, (const void*)counts, (const void*)offsets,
                        (const void*)perm, (const void*)inv, (const void*)x_perm_scale, (const void*)ws})
    if (misaligned(q, 4)) return MOE_ERR_UNSUPPORTED;
  if (x_perm && (misaligned(x, 16) || misaligned(x_perm, 16))) return MOE_ERR_UNSUPPORTED;
  const Window win{n_tokens, first_expert, cfg->T, cfg->k};
  if (pairs(cfg) <= kSmallPairs)
    return dispatch_small(cfg, win, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale, as_stream(stream));
  return dispatch_launch<true>(cfg, win, topk_idx, x, counts, offsets, perm,
                               inv, x_perm, x_perm_scale, static_cast<int32_t*>(ws), as_stream(stream));
}

// ------------------------------------------------ dispatch without a workspace
// The per-segment counts live in a fixed array of device memory that belongs
// to the library (one copy per GPU, held until the process ends).  Host code
// never passes the array's name to a kernel: on the host it only stands for
// the symbol; the array's device address on each GPU comes from
// hipGetSymbolAddress, taken once per device with that device current.
namespace moe {
namespace {
__device__ __align__(256) int32_t scratch[kDispatchScratchBytes / sizeof(int32_t)];

constexpr int kMaxDevices = 64;
std::mutex scratch_mu;
int32_t* scratch_ptr[kMaxDevices];   // device address of `scratch` per device, once known

moe_status scratch_on_current_device(int32_t** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_LAUNCH;
  std::lock_guard<std::mutex> lock(scratch_mu);
  if (!scratch_ptr[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return MOE_ERR_LAUNCH;
    scratch_ptr[dev] = static_cast<int32_t*>(p);
  }
  *out = scratch_ptr[dev];
  return MOE_OK;
}
}  // namespace
}  // namespace moe

extern "C" moe_status moe_dispatch_noalloc(const moe_cfg* cfg, const int32_t* topk_idx, const void* x,
                                           int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv,
                                           void* x_perm, float* x_perm_scale, void* stream) {
  moe_status st = dispatch_check(cfg, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale);
  if (st != MOE_OK) return st;
  if ((size_t)dispatch_segments(cfg) * cfg->E * sizeof(int32_t) > kDispatchScratchBytes) return MOE_ERR_SCRATCH;
  int32_t* segc = nullptr;
  if ((st = scratch_on_current_device(&segc)) != MOE_OK) return st;
  return dispatch_launch<false>(cfg, Window{}, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale, segc,
                                as_stream(stream));
}

extern "C" moe_status moe_quantize_fp8(const void* src_bf16, int32_t n_mat, int32_t rows, int32_t cols,
                                       int32_t block_rows, uint8_t* dst, float* scales, void* stream) {
  if (!src_bf16 || !dst || !scales) return MOE_ERR_NULL;
  if (n_mat < 0 || rows < 0 || cols <= 0 || cols % 128) return MOE_ERR_SHAPE;
  if (block_rows != 1 && block_rows != 128) return MOE_ERR_UNSUPPORTED;
  if (rows % block_rows) return MOE_ERR_SHAPE;
  if (n_mat == 0 || rows == 0) return MOE_OK;
  hipStream_t s = as_stream(stream);
  if (block_rows == 1)
    return launch_quantize_rows((const bf16_t*)src_bf16, (int64_t)n_mat * rows, cols, dst, scales, s);
  const int64_t nblk = (int64_t)n_mat * (rows / 128) * (cols / 128);
  if (nblk >= ((int64_t)1 << 31)) return MOE_ERR_SHAPE;
  hipLaunchKernelGGL(quantize_blocks_kernel, dim3((unsigned)nblk), dim3(256), 0, s, (const bf16_t*)src_bf16,
                     rows, cols, dst, scales);
  return launch_status();
}
