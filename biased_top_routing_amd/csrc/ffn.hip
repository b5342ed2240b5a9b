// moe_expert_ffn: the routed experts on their segments of the permuted rows and
// the shared experts on every token, each a SwiGLU FFN
// (DeepSeek-V3 Technical Report：中英对照解读, §2 Architecture: shared experts
// every token passes through plus routed experts picked by top-k).
//
// This file holds the entry point, the device-side tile-table builder of the
// grouped GEMMs, and the fp32 expert kernels of the small fp32 configuration.
#include <algorithm>

#include "common.h"
#include "ffn_layout.h"
#include "fp4.h"
#include "kernels.h"

namespace moe {

// ------------------------------------------------------------ tile tables
// Segments 0..E-1 are the routed experts (rows offsets[e]..offsets[e+1] of the
// permuted rows); segment E is the shared experts over all T tokens.  Each
// segment contributes ceil(rows / bm) row tiles times its column tiles, with
// the row height bm of the GEMM the table is for.
// Inside a segment the row tiles are cut into groups of kGroupRowTiles; a
// group's tiles are listed column-tile-major.  Tiles that run at the same time
// on one XCD (consecutive entries, or runs of them: grouped_tile_at) then cover
// a few row tiles times a few column tiles, so both their activation rows and
// their weight rows are shared in that XCD's L2, also for segments far larger
// than the number of tiles in flight.  Every workgroup computes the prefix sums over segments in LDS
// (at most 513 segments) and writes its own share of the entries.
struct TileTables {
  int E, S, T, bm1, bm1_alt, bm2, bm2_alt, nt1, nt1s, nt2;
  TileDesc *t1, *t2;     // t2 == nullptr: the first table only
  int32_t* hdr;
  bool fp4_choose;       // MXFP4: bm1 and bm2 are the lowest of the heights, the rows that are there decide
};

// Block b of nb blocks of 1024 threads.
__device__ void build_tiles_block(const int32_t* __restrict__ offsets, const TileTables& p, int b, int nb) {
  __shared__ int32_t pre1[1024], pre2[1024], mt1_s[1024], mt2_s[1024], row0_s[1024], rows_s[1024], hb1_s[1024],
      hb2_s[1024];
  __shared__ int32_t wave1[16], wave2[16];
  const int E = p.E, nt1 = p.nt1, nt1s = p.nt1s, nt2 = p.nt2;
  TileDesc *t1 = p.t1, *t2 = p.t2;
  int32_t* hdr = p.hdr;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nseg = E + (p.S > 0 ? 1 : 0);
  int bm1 = p.bm1, bm2 = p.bm2;
  int rows = p.T, row0 = 0;
  if (tid < E) {
    row0 = offsets[tid];
    rows = offsets[tid + 1] - row0;
  }
  if (p.fp4_choose) {                                   // the tiles of the routed segments at each height
    __shared__ int32_t tiles_s[3][16];
    int n[3] = {0, 0, 0};
    if (tid < E) {
      n[0] = (rows + kFp4LowBM - 1) / kFp4LowBM;
      n[1] = (rows + kFp4BM - 1) / kFp4BM;
      n[2] = (rows + kFp4HighBM - 1) / kFp4HighBM;
    }
#pragma unroll
    for (int h = 0; h < 3; ++h) {
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) n[h] += __shfl_xor(n[h], d);
      if (lane == 0) tiles_s[h][wave] = n[h];
    }
    __syncthreads();
    int sum[3] = {0, 0, 0};
#pragma unroll
    for (int h = 0; h < 3; ++h)
#pragma unroll
      for (int w = 0; w < 16; ++w) sum[h] += tiles_s[h][w];
    bm1 = bm2 = fp4_tile_rows(sum[0], sum[1], sum[2]);
  }
  int c1 = 0, c2 = 0;
  if (tid < nseg) {
    const int mt1 = (rows + bm1 - 1) / bm1, mt2 = (rows + bm2 - 1) / bm2;
    // as many tiles of bm1_alt rows cover the segment: use that height
    hb1_s[tid] = p.bm1_alt > 0 && (int64_t)mt1 * p.bm1_alt >= rows ? p.bm1_alt : bm1;
    hb2_s[tid] = p.bm2_alt > 0 && (int64_t)mt2 * p.bm2_alt >= rows ? p.bm2_alt : bm2;
    c1 = mt1 * (tid < E ? nt1 : nt1s);
    c2 = mt2 * nt2;
    mt1_s[tid] = mt1;
    mt2_s[tid] = mt2;
    row0_s[tid] = row0;
    rows_s[tid] = rows;
  }
  // exclusive prefixes over the segments: within each wavefront, then over the wavefronts
  int v1 = c1, v2 = c2;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u1 = __shfl_up(v1, d), u2 = __shfl_up(v2, d);
    if (lane >= d) v1 += u1, v2 += u2;
  }
  if (lane == 63) wave1[wave] = v1, wave2[wave] = v2;
  __syncthreads();
  int total1 = 0, total2 = 0, base1 = 0, base2 = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    if (w == wave) base1 = total1, base2 = total2;
    total1 += wave1[w];
    total2 += wave2[w];
  }
  pre1[tid] = base1 + v1 - c1;
  pre2[tid] = base2 + v2 - c2;
  __syncthreads();
  if (tid == 0 && b == 0) {
    hdr[0] = total1;
    hdr[1] = t2 ? total2 : 0;
    if (p.fp4_choose) hdr[kFp4TileRows] = bm1;
    // tiles of the routed segments (they come first; the shared ones follow)
    hdr[4] = p.S > 0 ? pre1[E] : total1;
    hdr[5] = t2 ? (p.S > 0 ? pre2[E] : total2) : 0;
  }
  for (int pass = 0; pass < (t2 ? 2 : 1); ++pass) {   // t2 == nullptr: the first table only
    const int* pre = pass == 0 ? pre1 : pre2;
    const int total = pass == 0 ? total1 : total2;
    TileDesc* out = pass == 0 ? t1 : t2;
    for (int L = b * 1024 + tid; L < total; L += nb * 1024) {
      int lo = 0, hi = nseg;           // last g with pre[g] <= L and a non-empty segment
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= L) lo = mid;
        else hi = mid;
      }
      int g = lo;
      // skip empty segments that share the same prefix value
      while (g + 1 < nseg && pre[g + 1] <= L) ++g;
      const int local = L - pre[g];
      const int mt = pass == 0 ? mt1_s[g] : mt2_s[g];
      const int bm = pass == 0 ? hb1_s[g] : hb2_s[g];
      const int ncol = (pass == 0 ? (g < E ? nt1 : nt1s) : nt2);
      const int q = local / (kGroupRowTiles * ncol);             // row-tile group (all earlier ones full)
      const int idx = local - q * kGroupRowTiles * ncol;
      const int gs = min(kGroupRowTiles, mt - q * kGroupRowTiles);
      const int nt = idx / gs, rt = q * kGroupRowTiles + idx % gs;
      TileDesc d;
      d.seg = g;
      d.row0 = row0_s[g] + rt * bm;
      d.rows = min(bm, rows_s[g] - rt * bm);
      d.nt = nt;
      out[L] = d;
    }
  }
}

__global__ __launch_bounds__(1024) void build_tiles_kernel(const int32_t* __restrict__ offsets, TileTables p) {
  build_tiles_block(offsets, p, blockIdx.x, gridDim.x);
}

// The tables of an MXFP4 call and x in MXFP4 (fp4.h) in one launch: blocks [0, nb)
// build, the others quantise, 4 groups of 256 lanes each.  (Two launches of a few
// microseconds each stood before the GEMMs: T = 1, H = 7168, 8 experts and a shared
// one 59.0 -> 56.5 us the whole call.)
__global__ __launch_bounds__(1024) void build_tiles_quantize_fp4_kernel(const int32_t* __restrict__ offsets,
                                                                       TileTables p, int nb,
                                                                       const uint4* __restrict__ x, int rows,
                                                                       int cols, int64_t blocks,
                                                                       uint32_t* __restrict__ dst,
                                                                       uint32_t* __restrict__ scales) {
#if defined(__HIP_DEVICE_COMPILE__)
  if ((int)blockIdx.x < nb) {
    build_tiles_block(offsets, p, blockIdx.x, nb);
    return;
  }
  const int64_t b = ((int64_t)blockIdx.x - nb) * 4 + (threadIdx.x >> 8);
  if (b < blocks) quantize_fp4_block<false>(x, rows, cols, b, 0, threadIdx.x & 255, dst, scales);
#endif
}

// Blocks that fill the larger of two tables of at most max1 and max2 entries.
static unsigned table_blocks(int64_t max1, int64_t max2) {
  return (unsigned)std::min<int64_t>(std::max<int64_t>((std::max(max1, max2) + 1023) / 1024, 1), 64);
}

moe_status launch_build_tile_tables(const moe_cfg* c, const int32_t* offsets, int bm1, int bm1_alt, int nt1,
                                    int nt1s, TileDesc* t1, int64_t max1, int bm2, int bm2_alt, int nt2, TileDesc* t2,
                                    int64_t max2, int32_t* hdr, hipStream_t st) {
  const TileTables p{c->E, c->S, c->T, bm1, bm1_alt, bm2, bm2_alt, nt1, nt1s, nt2, t1, t2, hdr, false};
  hipLaunchKernelGGL(build_tiles_kernel, dim3(table_blocks(max1, max2)), dim3(1024), 0, st, offsets, p);
  return launch_status();
}

static TileTables ffn_tables(const moe_cfg* c, const FfnLayout& L, char* base) {
  return TileTables{c->E, c->S, c->T, L.bm1, L.bm1_alt, L.bm2, L.bm2_alt, (int)L.nt1, (int)L.nt1s, (int)L.nt2,
                    reinterpret_cast<TileDesc*>(base + L.off_t1), reinterpret_cast<TileDesc*>(base + L.off_t2),
                    reinterpret_cast<int32_t*>(base + L.off_hdr), c->wgt == MOE_MXFP4 && L.bm1 != kFp4RowsBM};
}

moe_status launch_build_tiles(const moe_cfg* c, const int32_t* offsets, void* ws, hipStream_t st) {
  const FfnLayout L(c);
  hipLaunchKernelGGL(build_tiles_kernel, dim3(table_blocks(L.max1, L.max2)), dim3(1024), 0, st, offsets,
                     ffn_tables(c, L, static_cast<char*>(ws)));
  return launch_status();
}

moe_status launch_build_tiles_quantize_fp4(const moe_cfg* c, const int32_t* offsets, const bf16_t* x, void* ws,
                                           hipStream_t st) {
  const FfnLayout L(c);
  char* base = static_cast<char*>(ws);
  const unsigned nb = table_blocks(L.max1, L.max2);
  const int64_t blocks = quantize_fp4_blocks(c->T, c->H);
  hipLaunchKernelGGL(build_tiles_quantize_fp4_kernel, dim3(nb + (unsigned)((blocks + 3) / 4)), dim3(1024), 0, st,
                     offsets, ffn_tables(c, L, base), (int)nb, (const uint4*)x, c->T, c->H, blocks,
                     (uint32_t*)(base + L.off_xq), (uint32_t*)(base + L.off_xqs));
  return launch_status();
}

// ------------------------------------------------------------ fp32 experts
__device__ __forceinline__ int expert_of_row(const int32_t* offsets, int E, int64_t row) {
  int lo = 0, hi = E;                  // last e with offsets[e] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= row) lo = mid;
    else hi = mid;
  }
  while (lo + 1 < E && offsets[lo + 1] <= row) ++lo;
  return lo;
}

// h[row, c] = silu(<a_row, Wg_c>) * <a_row, Wu_c>; one thread per (row, c).
// offsets == nullptr: shared experts (h width S*I, column c -> expert c / I).
// rowmap != nullptr: operand row `row` is row rowmap[row] / k of a (the
// expert-sorted order gathered from x).
__global__ __launch_bounds__(256) void gateup_f32_kernel(const float* __restrict__ a, int64_t nrows,
                                                         const int32_t* __restrict__ rowmap, int k,
                                                         const int32_t* __restrict__ offsets, int E,
                                                         const float* __restrict__ W, int H, int I,
                                                         int hw, float* __restrict__ h) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= nrows * hw) return;
  const int64_t row = id / hw;
  if (offsets && row >= offsets[E]) return;   // behind the last present pair of a share
  const int c = (int)(id % hw);
  const int ex = offsets ? expert_of_row(offsets, E, row) : c / I;
  const int cc = c % I;
  const float* wg = W + ((int64_t)ex * 2 * I + cc) * H;
  const float* wu = wg + (int64_t)I * H;
  const int64_t arow = rowmap ? (int64_t)(rowmap[row] / k) : row;
  const float4* ar = reinterpret_cast<const float4*>(a + arow * H);
  float g = 0.f, u = 0.f;
  for (int i = 0; i < H / 4; ++i) {
    const float4 x = ar[i];
    const float4 p = reinterpret_cast<const float4*>(wg)[i];
    const float4 q = reinterpret_cast<const float4*>(wu)[i];
    g = fmaf(x.x, p.x, g); g = fmaf(x.y, p.y, g); g = fmaf(x.z, p.z, g); g = fmaf(x.w, p.w, g);
    u = fmaf(x.x, q.x, u); u = fmaf(x.y, q.y, u); u = fmaf(x.z, q.z, u); u = fmaf(x.w, q.w, u);
  }
  h[row * hw + c] = g / (1.0f + expf(-g)) * u;
}

// y[row, n] = sum_k h[row, k] * W_d[k / I][n][k % I]; one thread per (row, n).
__global__ __launch_bounds__(256) void down_f32_kernel(const float* __restrict__ h, int64_t nrows,
                                                       const int32_t* __restrict__ offsets, int E,
                                                       const float* __restrict__ W, int H, int I,
                                                       int kw, float* __restrict__ y) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= nrows * H) return;
  const int64_t row = id / H;
  if (offsets && row >= offsets[E]) return;   // behind the last present pair of a share
  const int n = (int)(id % H);
  const float* Wb = offsets ? W + (int64_t)expert_of_row(offsets, E, row) * H * I : W;
  const float* hr = h + row * kw;
  float acc = 0.f;
  for (int k0 = 0; k0 < kw; k0 += I) {
    const float4* wr = reinterpret_cast<const float4*>(Wb + (int64_t)(k0 / I) * H * I + (int64_t)n * I);
    const float4* hq = reinterpret_cast<const float4*>(hr + k0);
    for (int i = 0; i < I / 4; ++i) {
      const float4 x = hq[i], w = wr[i];
      acc = fmaf(x.x, w.x, acc); acc = fmaf(x.y, w.y, acc);
      acc = fmaf(x.z, w.z, acc); acc = fmaf(x.w, w.w, acc);
    }
  }
  y[row * H + n] = acc;
}

moe_status launch_ffn_f32(const moe_cfg* c, const float* x_perm, const int32_t* perm,
                          const int32_t* offsets, const moe_expert_weights* w, const float* x,
                          float* y_perm, float* y_shared, void* ws, int phase, hipStream_t st) {
  const FfnLayout L(c);
  char* base = static_cast<char*>(ws);
  float* hp = reinterpret_cast<float*>(base + L.off_hp);
  float* hs = reinterpret_cast<float*>(base + L.off_hs);
  const int64_t P = pairs(c);
  auto blocks = [](int64_t n) { return dim3((unsigned)((n + 255) / 256)); };
  if (phase == MOE_FFN_ALL || phase == MOE_FFN_GATE_UP) {
    hipLaunchKernelGGL(gateup_f32_kernel, blocks(P * c->I), dim3(256), 0, st, perm ? x : x_perm, P, perm,
                       c->k, offsets, c->E, (const float*)w->w_gate_up, c->H, c->I, c->I, hp);
    if (c->S > 0)
      hipLaunchKernelGGL(gateup_f32_kernel, blocks((int64_t)c->T * c->S * c->I), dim3(256), 0, st, x,
                         (int64_t)c->T, (const int32_t*)nullptr, 1, (const int32_t*)nullptr, c->E,
                         (const float*)w->ws_gate_up, c->H, c->I, c->S * c->I, hs);
  }
  if (phase == MOE_FFN_ALL || phase == MOE_FFN_DOWN) {
    hipLaunchKernelGGL(down_f32_kernel, blocks(P * c->H), dim3(256), 0, st, hp, P, offsets, c->E,
                       (const float*)w->w_down, c->H, c->I, c->I, y_perm);
    if (c->S > 0)
      hipLaunchKernelGGL(down_f32_kernel, blocks((int64_t)c->T * c->H), dim3(256), 0, st, hs, (int64_t)c->T,
                         (const int32_t*)nullptr, c->E, (const float*)w->ws_down, c->H, c->I,
                         c->S * c->I, y_shared);
  }
  return launch_status();
}

}  // namespace moe

using namespace moe;

namespace {

// The MXFP4 kernels load 16-byte chunks of rows and codes and 4-byte scale words.
bool fp4_misaligned(const moe_cfg* c, const void* x_perm, const void* x_perm_scale, const moe_expert_weights* w,
                    const void* x, const void* y_perm, const void* y_shared, const void* ws) {
  const void* chunks[] = {x_perm, w->w_gate_up, w->w_down, c->S > 0 ? w->ws_gate_up : nullptr,
                          c->S > 0 ? w->ws_down : nullptr, x, y_perm, c->S > 0 ? y_shared : nullptr, ws};
  for (const void* q : chunks)
    if (misaligned(q, 16)) return true;
  const void* words[] = {x_perm_scale, w->w_gate_up_scale, w->w_down_scale,
                         c->S > 0 ? w->ws_gate_up_scale : nullptr, c->S > 0 ? w->ws_down_scale : nullptr};
  for (const void* q : words)
    if (misaligned(q, 4)) return true;
  return false;
}

// Both FFN entry points: routed gate/up rows from x_perm (perm == nullptr) or
// gathered from x through perm.
moe_status expert_ffn(const moe_cfg* cfg, const void* x_perm, const float* x_perm_scale,
                      const int32_t* perm, const int32_t* offsets, const moe_expert_weights* w,
                      const void* x, void* y_perm, void* y_shared, const moe_ffn_saved* saved, void* ws,
                      size_t ws_bytes, int phase, void* stream) {
  moe_status st = validate_cfg(cfg);
  if (st != MOE_OK) return st;
  if (phase != MOE_FFN_ALL && phase != MOE_FFN_GATE_UP && phase != MOE_FFN_DOWN)
    return MOE_ERR_UNSUPPORTED;
  const bool gate_up = phase != MOE_FFN_DOWN;
  if (!w || !offsets || !y_perm || !ws || !w->w_gate_up || !w->w_down) return MOE_ERR_NULL;
  if (!perm && !x_perm) return MOE_ERR_NULL;
  if (perm && gate_up && !x) return MOE_ERR_NULL;
  if (cfg->S > 0 && (!x || !y_shared || !w->ws_gate_up || !w->ws_down)) return MOE_ERR_NULL;
  const bool fp8 = cfg->wgt == MOE_FP8_E4M3, fp4 = cfg->wgt == MOE_MXFP4, scaled = fp8 || fp4;
  if (scaled && ((!perm && !x_perm_scale) || !w->w_gate_up_scale || !w->w_down_scale)) return MOE_ERR_NULL;
  if (scaled && cfg->S > 0 && (!w->ws_gate_up_scale || !w->ws_down_scale)) return MOE_ERR_NULL;
  if (saved) {
    if (cfg->act != MOE_BF16 || cfg->wgt != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (!saved->g || !saved->u || (cfg->S > 0 && (!saved->gs || !saved->us))) return MOE_ERR_NULL;
  }
  // gathered rows are addressed by 32-bit byte offsets into x (one row past
  // the end marks a dropped row)
  if (perm && cfg->act != MOE_F32 &&
      ((int64_t)cfg->T + 1) * cfg->H * (fp4 ? 1 : fp8 ? 2 : 2 * (int64_t)act_bytes(cfg)) / 2 > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (fp4 && fp4_misaligned(cfg, x_perm, x_perm_scale, w, x, y_perm, y_shared, ws)) return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < FfnLayout(cfg).total) return MOE_ERR_WORKSPACE;
  if (cfg->T == 0) return MOE_OK;
  hipStream_t s = as_stream(stream);
  if (cfg->act == MOE_F32)
    return launch_ffn_f32(cfg, (const float*)x_perm, perm, offsets, w, (const float*)x, (float*)y_perm,
                          (float*)y_shared, ws, phase, s);
  if (fp4)
    return launch_ffn_fp4(cfg, (const uint8_t*)x_perm, (const uint8_t*)x_perm_scale, perm, offsets, w, (const bf16_t*)x,
                          (bf16_t*)y_perm, (bf16_t*)y_shared, ws, phase, s);
  if (!fp8)
    return launch_ffn_bf16(cfg, (const bf16_t*)x_perm, perm, offsets, w, (const bf16_t*)x,
                           (bf16_t*)y_perm, (bf16_t*)y_shared, phase == MOE_FFN_DOWN ? nullptr : saved, ws,
                           phase, s);
  return launch_ffn_fp8(cfg, (const fp8_t*)x_perm, x_perm_scale, perm, offsets, w, (const bf16_t*)x,
                        (bf16_t*)y_perm, (bf16_t*)y_shared, ws, phase, s);
}

}  // namespace

extern "C" moe_status moe_expert_ffn(const moe_cfg* cfg, const void* x_perm, const float* x_perm_scale,
                                     const int32_t* offsets, const moe_expert_weights* w, const void* x,
                                     void* y_perm, void* y_shared, void* ws, size_t ws_bytes, int phase,
                                     void* stream) {
  if (!x_perm) return MOE_ERR_NULL;
  return expert_ffn(cfg, x_perm, x_perm_scale, nullptr, offsets, w, x, y_perm, y_shared, nullptr, ws, ws_bytes,
                    phase, stream);
}

extern "C" moe_status moe_expert_ffn_gather(const moe_cfg* cfg, const void* x, const int32_t* perm,
                                            const int32_t* offsets, const moe_expert_weights* w,
                                            void* y_perm, void* y_shared, void* ws, size_t ws_bytes,
                                            int phase, void* stream) {
  if (!perm) return MOE_ERR_NULL;
  return expert_ffn(cfg, nullptr, nullptr, perm, offsets, w, x, y_perm, y_shared, nullptr, ws, ws_bytes, phase,
                    stream);
}

extern "C" moe_status moe_expert_ffn_save(const moe_cfg* cfg, const void* x_perm, const int32_t* perm,
                                          const int32_t* offsets, const moe_expert_weights* w, const void* x,
                                          void* y_perm, void* y_shared, const moe_ffn_saved* saved, void* ws,
                                          size_t ws_bytes, int phase, void* stream) {
  if (!saved || (!x_perm && !perm)) return MOE_ERR_NULL;
  return expert_ffn(cfg, x_perm, nullptr, x_perm ? nullptr : perm, offsets, w, x, y_perm, y_shared, saved, ws,
                    ws_bytes, phase, stream);
}
