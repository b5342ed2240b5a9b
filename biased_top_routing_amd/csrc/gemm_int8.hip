// int8 expert GEMMs of the layer on gfx950 (rows: int8.h): activations with one scale a token, weights with one
// a row (an output channel).
//
// C[i][j] = sum_k a[i][k] w[j][k] over whole numbers, exactly, in the 32-bit accumulators of
// v_mfma_i32_16x16x64_i8 (K < 2^17, so that 128 * 128 * K stays below 2^31); the two scales multiply it once, in
// the epilogue.
//   gate/up  h = silu(g) u with g, u = C sa sw, rounded to bf16 (the layer's activation type; a row's int8 scale
//            needs all of its columns, which several workgroups compute: the rows are quantised between the GEMMs)
//   down     y = C sh sw, stored as bf16.  The shared experts are one FFN of S I columns: their K ranges follow
//            each other in one accumulator, so W_d has one scale a channel for all of them.
#include <algorithm>

#include "common.h"
#include "ffn_layout.h"
#include "gemm_common.h"
#include "int8.h"
#include "kernels.h"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

namespace {

enum { kGateUpI8 = 1, kDownI8 = 2 };

struct Int8Params {
  const uint8_t* a_routed;    // gate/up: x_perm codes [P, H]; down: h codes [P, I]
  const float* sa_routed;     // their scales [P]
  const uint8_t* a_shared;    // gate/up: x codes [T, H]; down: h_shared codes [T, S*I]
  const float* sa_shared;     // [T]
  const uint8_t* w_routed;    // gate/up: w_gate_up; down: w_down (codes)
  const float* sw_routed;     // [E, 2I]; [E, H]
  const uint8_t* w_shared;
  const float* sw_shared;     // [S, 2I]; [H]
  bf16_t* out_routed;         // gate/up: h [P, I]; down: y_perm
  bf16_t* out_shared;
  const TileDesc* tiles;
  const int32_t* ntiles;
  const int32_t* perm;        // gate/up: non-null -> routed rows gathered from a_shared / sa_shared
  int T, H, E, S, I, k;
};

#if defined(__HIP_DEVICE_COMPILE__)
constexpr int NI8 = 4;          // MFMA column blocks of a wavefront
typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ i32x4_t mfma_i8(i32x4_t w, i32x4_t a, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, c, 0, 0, 0);
}

// Entry L of the tile table, read through the scalar cache.
__device__ __forceinline__ TileDesc tile_at(const Int8Params& p, int L) {
  typedef const __attribute__((address_space(4))) int32_t* cptr;
  const cptr t = (cptr)(uintptr_t)(p.tiles + L);
  return TileDesc{t[0], t[1], t[2], t[3]};
}

// One tile's operands (all wavefront-uniform).
template <int MODE>
struct OperandsI8 {
  const uint8_t *A, *W;
  const float *SA, *SW;         // scales of row 0 of the tile (gathered: of token 0), of the tile's expert
  int lda, ldw;                 // bytes between rows
  int a_rows;                   // rows the A descriptor covers
  int a_bytes, w_bytes;
  int w_one;                    // one expert's weights, bytes
  int nk1, nexp;                // 128-wide K slices of one expert; experts whose K ranges follow each other
  int ncols;                    // output columns of the segment
  int ex, c0;                   // the tile's expert among the shared ones, and its first weight row there
  bool shared, gather;

  __device__ __forceinline__ OperandsI8(const Int8Params& p, const TileDesc& d) {
    shared = d.seg == p.E;
    // routed gate/up rows gathered from the quantised x: row row0 + r of the expert-sorted order is token
    // perm[row0 + r] / k
    gather = MODE == kGateUpI8 && !shared && p.perm != nullptr;
    const int K1 = MODE == kDownI8 ? p.I : p.H;
    nk1 = K1 / 128;
    nexp = MODE == kDownI8 && shared ? p.S : 1;
    lda = nexp * K1;
    ldw = K1;
    const int a_base = gather ? 0 : d.row0;
    a_rows = gather ? p.T : d.rows;
    A = (shared || gather ? p.a_shared : p.a_routed) + (int64_t)a_base * lda;
    SA = (shared || gather ? p.sa_shared : p.sa_routed) + a_base;
    const int nrow_w = MODE == kGateUpI8 ? 2 * p.I : p.H;      // weight rows of one expert
    w_one = nrow_w * ldw;
    ncols = MODE == kGateUpI8 ? (shared ? p.S * p.I : p.I) : p.H;
    // (a gate/up tile's 128 columns lie in one expert: I is a multiple of 128)
    ex = MODE == kGateUpI8 && shared ? d.nt * 128 / p.I : 0;
    c0 = MODE == kGateUpI8 ? d.nt * 128 - ex * p.I : d.nt * 256;
    W = shared ? p.w_shared : p.w_routed + d.seg * (int64_t)w_one;
    SW = (shared ? p.sw_shared : p.sw_routed + d.seg * (int64_t)nrow_w) + ex * nrow_w;
    a_bytes = a_rows * lda;
    w_bytes = (shared ? p.S : 1) * w_one;
  }

  // weight row (in its expert) of row r of part `part` of the tile's columns (BN weight rows a part), the
  // last one for rows past the columns
  template <int BN>
  __device__ __forceinline__ int wrow(const Int8Params& p, int part, int r) const {
    if constexpr (MODE == kGateUpI8) return c0 + part * (BN / 2) + (r < BN / 2 ? r : r - BN / 2 + p.I);
    else return min(c0 + part * BN + r, ncols - 1);
  }
};

// The order of a wavefront's columns: block ni, MFMA row 4 g + r is column 8 g + 4 (ni mod 2) + r of its 32 gate
// columns (ni < 2) or of the up columns BN / 2 further on, or of its first or second 32 output columns, so that a
// lane holds 8 neighbouring columns of a row in two blocks: 16 bytes of bf16.  The tile column whose LDS row lane
// l16 reads is col_lane + col_off.
__device__ __forceinline__ int col_lane(int l16) { return 8 * (l16 >> 2) + (l16 & 3); }
template <int MODE, int BN>
__device__ __forceinline__ constexpr int col_off(int ni) {
  return (ni / 2) * (MODE == kGateUpI8 ? BN / 2 : 32) + (ni % 2) * 4;
}
// Physical 16-byte chunk of logical chunk c of 8 in LDS row r of the weights: 8 lanes' rows (4, and 4 that lie 8
// further on) meet no bank twice.
__device__ __forceinline__ int swz_w(int r, int c) { return c ^ ((r & 3) | (((r >> 3) & 1) << 2)); }

// Workgroup barrier for LDS: this wavefront's LDS operations are done; loads and stores in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(kLgkmWaitZero);
  asm volatile("s_barrier" ::: "memory");
}
#endif

// One workgroup of WM x WN wavefronts a tile (PARTS > 1: a part of one) of WM * MI * 16 token rows x WN * 64
// weight rows.  K advances 128 bytes a slice through a ring of STAGES LDS stages filled by direct-to-LDS loads
// (16-byte chunks, XOR swizzle per row), one barrier a slice.
template <int MODE, int WM, int WN, int MI, int STAGES, int PARTS>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_int8_kernel(Int8Params p) {
  constexpr int NT = 64 * WM * WN, BM = WM * MI * 16, BN = WN * 64, BK = 128, CPR = BK / 16;
  static_assert(PARTS * BN == kInt8BN2 && BN / 2 * PARTS == kInt8BNH, "the tiles of the table, in parts");
  constexpr int A_CH = BM * CPR / NT, B_CH = BN * CPR / NT, PER = A_CH + B_CH;   // loads per thread per slice
  static_assert(BM * CPR % NT == 0 && BN * CPR % NT == 0 && PER * (STAGES - 2) < 64, "whole loads per thread");
  constexpr int STAGE = (BM + BN) * BK;
  static_assert(STAGES * STAGE <= 163840, "LDS of a CU");
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(16))) uint8_t lds[STAGES * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN, l16 = lane & 15, g = lane >> 4;
  // (the parts of a tile go to one XCD)
  const int part = (blockIdx.x >> 3) % PARTS, b = (blockIdx.x >> 3) / PARTS * 8 + (blockIdx.x & 7);
  const int L = grouped_tile_at(b, __builtin_amdgcn_readfirstlane(p.ntiles[0]),
                                __builtin_amdgcn_readfirstlane(p.ntiles[4]), kStripeInt8);
  if (L < 0) return;
  const TileDesc d = tile_at(p, L);
  const OperandsI8<MODE> o(p, d);
  // (rows past the tile's lie past the descriptor: the range check drops their loads)
  int a_off[A_CH], b_off[B_CH];
#pragma unroll
  for (int i = 0; i < A_CH; ++i) {
    const int c = i * NT + tid, r = c / CPR;
    a_off[i] = (r >= d.rows ? o.a_rows + 1 : o.gather ? p.perm[d.row0 + r] / p.k : r) * o.lda + swz<CPR>(r, c % CPR) * 16;
  }
#pragma unroll
  for (int i = 0; i < B_CH; ++i) {
    const int c = i * NT + tid, r = c / CPR;
    b_off[i] = o.ex * o.w_one + o.template wrow<BN>(p, part, r) * o.ldw + swz_w(r, c % CPR) * 16;
  }
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(o.A, o.a_bytes), rw = make_rsrc(o.W, o.w_bytes);
  const int ns = o.nexp * o.nk1;
  auto issue = [&](int stage, int kt) {
    const int ex = MODE == kDownI8 ? kt / o.nk1 : 0, ak = kt * BK, wk = ex * o.w_one + (kt - ex * o.nk1) * BK;
    uint8_t* sb = lds + stage * STAGE + wave * 1024;
#pragma unroll
    for (int i = 0; i < A_CH; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(sb + i * NT * 16), 16, a_off[i], ak, 0, 0);
#pragma unroll
    for (int i = 0; i < B_CH; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(sb + BM * BK + i * NT * 16), 16, b_off[i], wk, 0, 0);
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < ns) issue(s, s);
  i32x4_t acc[MI][NI8];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI8; ++ni) acc[mi][ni] = i32x4_t{0, 0, 0, 0};
  const int arow0 = wm * MI * 16 + l16, brow = wn * (MODE == kGateUpI8 ? 32 : 64) + col_lane(l16);
  const bool has_rows = wm * MI * 16 < d.rows;
  int cur = 0;
  for (int kt = 0; kt < ns; ++kt) {
    // the loads of slice kt have landed once only the later slices' remain
    const int later = min(ns - 1, kt + STAGES - 2) - kt;
    if (STAGES > 3 && later >= 2) wait_vm<PER * (STAGES > 3 ? 2 : 0)>();
    else if (STAGES > 2 && later >= 1) wait_vm<PER * (STAGES > 2 ? 1 : 0)>();
    else wait_vm<0>();
    lds_barrier();
    if (kt + STAGES - 1 < ns) issue(cur == 0 ? STAGES - 1 : cur - 1, kt + STAGES - 1);
    const uint8_t* base = lds + cur * STAGE;
    if (has_rows) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        i32x4_t fb[NI8];
#pragma unroll
        for (int ni = 0; ni < NI8; ++ni)
          fb[ni] = *reinterpret_cast<const i32x4_t*>(base + (BM + brow + col_off<MODE, BN>(ni)) * BK +
                                                     swz_w(col_lane(l16), kk * 4 + g) * 16);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          const i32x4_t fa = *reinterpret_cast<const i32x4_t*>(base + (arow0 + mi * 16) * BK +
                                                              swz<CPR>(arow0, kk * 4 + g) * 16);
#pragma unroll
          for (int ni = 0; ni < NI8; ++ni) acc[mi][ni] = mfma_i8(fb[ni], fa, acc[mi][ni]);
        }
      }
    }
    cur = cur == STAGES - 1 ? 0 : cur + 1;
  }
  // acc[mi][ni][r] holds C[i][j] with i = arow0 + 16 mi (token row), j in the order of col_off
  bf16_t* out = o.shared ? p.out_shared : p.out_routed;
  float sw[NI8][4];
#pragma unroll
  for (int ni = 0; ni < NI8; ++ni)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      sw[ni][r] = o.SW[o.template wrow<BN>(p, part, wn * (MODE == kGateUpI8 ? 32 : 64) + 8 * g + col_off<MODE, BN>(ni) + r)];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const int i = arow0 + mi * 16;
    if (i >= d.rows) continue;
    const float sa = o.SA[o.gather ? p.perm[d.row0 + i] / p.k : i];
    bf16_t* row = out + (d.row0 + i) * (int64_t)o.ncols;
    if constexpr (MODE == kGateUpI8) {
      float h[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float gv = (float)acc[mi][q / 4][q % 4] * (sa * sw[q / 4][q % 4]);
        const float uv = (float)acc[mi][q / 4 + 2][q % 4] * (sa * sw[q / 4 + 2][q % 4]);
        h[q] = gv * gate_sigmoid(gv) * uv;
      }
      *reinterpret_cast<uint4*>(row + d.nt * 128 + part * (BN / 2) + wn * 32 + 8 * g) =
          make_uint4(cvt_bf16x2(h[0], h[1]), cvt_bf16x2(h[2], h[3]), cvt_bf16x2(h[4], h[5]), cvt_bf16x2(h[6], h[7]));
    } else {
#pragma unroll
      for (int b2 = 0; b2 < 2; ++b2) {
        float y[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          y[q] = (float)acc[mi][2 * b2 + q / 4][q % 4] * (sa * sw[2 * b2 + q / 4][q % 4]);
        const int col = d.nt * 256 + part * BN + wn * 64 + b2 * 32 + 8 * g;
        if (col < o.ncols)
          *reinterpret_cast<uint4*>(row + col) =
              make_uint4(cvt_bf16x2(y[0], y[1]), cvt_bf16x2(y[2], y[3]), cvt_bf16x2(y[4], y[5]), cvt_bf16x2(y[6], y[7]));
      }
    }
  }
#endif
}

template <int MODE>
moe_status launch_gemm_int8(const FfnLayout& L, int64_t max_tiles, const Int8Params& p, hipStream_t st) {
  const unsigned grid = (unsigned)grouped_grid(max_tiles, kStripeInt8);
  if (grid == 0) return MOE_OK;
  if (L.bm1 == kInt8RowsBM) hipLaunchKernelGGL((gemm_int8_kernel<MODE, 1, 1, 2, 4, 4>), dim3(4 * grid), dim3(64), 0, st, p);
  else hipLaunchKernelGGL((gemm_int8_kernel<MODE, 2, 4, 8, 2, 1>), dim3(grid), dim3(512), 0, st, p);
  return launch_status();
}

}  // namespace

moe_status launch_ffn_int8(const moe_cfg* c, const uint8_t* x_perm, const float* x_perm_scale, const int32_t* perm,
                           const int32_t* offsets, const moe_expert_weights* w, const bf16_t* x, const uint8_t* x_codes,
                           const float* x_scale, bf16_t* y_perm, bf16_t* y_shared, void* ws, int phase,
                           hipStream_t st) {
  const FfnLayout L(c);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const int32_t* hdr = reinterpret_cast<const int32_t*>(base + L.off_hdr);
  auto bytes = [](const void* q) { return static_cast<const uint8_t*>(q); };
  auto floats = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  bf16_t* hb = reinterpret_cast<bf16_t*>(base + L.off_hb);
  bf16_t* hbs = reinterpret_cast<bf16_t*>(base + L.off_hbs);
  moe_status s;
  Int8Params p{};
  p.T = c->T; p.H = c->H; p.E = c->E; p.S = c->S; p.I = c->I; p.k = c->k;
  if (phase == MOE_FFN_ALL || phase == MOE_FFN_GATE_UP) {
    if ((s = launch_build_tiles(c, offsets, ws, st)) != MOE_OK) return s;
    // x once in int8: the shared experts' operand, and the routed one when its rows are gathered
    if (!x_codes && (c->S > 0 || perm)) {
      s = launch_quantize_rows_int8(x, c->T, c->H, nullptr, base + L.off_xq, floats(L.off_xqs), st);
      if (s != MOE_OK) return s;
      x_codes = base + L.off_xq;
      x_scale = floats(L.off_xqs);
    }
    p.perm = perm;
    p.a_routed = x_perm; p.sa_routed = x_perm_scale;
    p.a_shared = x_codes; p.sa_shared = x_scale;
    p.w_routed = bytes(w->w_gate_up); p.sw_routed = w->w_gate_up_scale;
    p.w_shared = bytes(w->ws_gate_up); p.sw_shared = w->ws_gate_up_scale;
    p.out_routed = hb; p.out_shared = hbs;
    p.tiles = reinterpret_cast<const TileDesc*>(base + L.off_t1);
    p.ntiles = hdr;
    if ((s = launch_gemm_int8<kGateUpI8>(L, L.max1, p, st)) != MOE_OK) return s;
    // (rows behind the last present pair of a share hold nothing)
    s = launch_quantize_rows_int8(hb, pairs(c), c->I, offsets + c->E, base + L.off_hp, floats(L.off_hps), st);
    if (s != MOE_OK) return s;
    if (c->S > 0 && (s = launch_quantize_rows_int8(hbs, c->T, c->S * c->I, nullptr, base + L.off_hs, floats(L.off_hss),
                                                   st)) != MOE_OK)
      return s;
  }
  if (phase == MOE_FFN_ALL || phase == MOE_FFN_DOWN) {
    p.perm = nullptr;
    p.a_routed = base + L.off_hp; p.sa_routed = floats(L.off_hps);
    p.a_shared = base + L.off_hs; p.sa_shared = floats(L.off_hss);
    p.w_routed = bytes(w->w_down); p.sw_routed = w->w_down_scale;
    p.w_shared = bytes(w->ws_down); p.sw_shared = w->ws_down_scale;
    p.out_routed = y_perm; p.out_shared = y_shared;
    p.tiles = reinterpret_cast<const TileDesc*>(base + L.off_t2);
    p.ntiles = hdr + 1;
    if ((s = launch_gemm_int8<kDownI8>(L, L.max2, p, st)) != MOE_OK) return s;
  }
  return MOE_OK;
}

}  // namespace moe
