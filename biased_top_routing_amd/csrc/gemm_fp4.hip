// MXFP4 expert GEMMs of the layer on gfx950 (format: fp4.h): activations and
// weights are E2M1 codes with one power-of-two scale per 32 elements of K.
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 takes a 128-wide K step of both
// operands with their scale bytes and accumulates in fp32: lane l holds the 32
// elements [32 (l / 16), + 32) of row l % 16, one scale block, so each lane
// brings its operand's 16 code bytes and one scale byte, and no scaling is left
// to the vector ALU.  The MFMA takes the weight fragment as its first operand,
// so a lane's four results are four adjacent weight columns of one token row.
//   gate/up  h = silu(X W_g^T) * (X W_u^T), quantised per 32 columns of h in
//            the epilogue from the fp32 accumulators (one rounding, to E2M1)
//   down     Y = h W_d^T, stored as bf16
//
// Tiling: a workgroup of WM x WN wavefronts computes a (WM*MI*16) x (WN*64)
// tile; each wavefront owns MI x 4 MFMA blocks.  K advances 256 elements (128
// bytes of codes) per slice through a ring of LDS stages filled by direct-to-LDS
// buffer loads (16-byte chunks, XOR swizzle per row), the rows' scale words of
// the slice's two 128-wide steps beside them.  K is a multiple of 128: the last
// slice of an odd number of steps runs its first step only (its second half
// holds bytes of the next row or nothing, and is not read).  The shared experts'
// down GEMM walks the experts one after the other, each with its own slices.
// The gate/up tile's 256 weight rows are the 128 gate rows and the 128 up rows
// of 128 h columns; a wavefront holds gate and up of 32 of them, one scale block.
// All LDS is one array: with several LDS objects the compiler makes every LDS
// read wait for the direct-to-LDS loads in flight.
#include "common.h"
#include "ffn_layout.h"
#include "fp4.h"
#include "gemm_common.h"
#include "kernels.h"

namespace moe {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4v_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

namespace {

enum { kGateUp4 = 1, kDown4 = 2 };

struct Fp4Params {
  const uint8_t* a_routed;    // gate/up: x_perm codes [P, H/2]; down: h codes [P, I/2]
  const uint8_t* sa_routed;   // their scale words [K/128][P]
  const uint8_t* a_shared;    // gate/up: x codes [T, H/2]; down: h_shared codes [T, S*I/2]
  const uint8_t* sa_shared;
  const uint8_t* w_routed;    // gate/up: w_gate_up; down: w_down (codes)
  const uint8_t* sw_routed;   // their scale words [K/128][rows] per expert
  const uint8_t* w_shared;
  const uint8_t* sw_shared;
  uint8_t* out_routed;        // gate/up: h codes; down: y_perm (bf16)
  uint8_t* out_routed_scale;  // gate/up: h scale words
  uint8_t* out_shared;
  uint8_t* out_shared_scale;
  const TileDesc* tiles;
  const int32_t* ntiles;
  const int32_t* perm;        // gate/up: non-null -> routed rows gathered from a_shared / sa_shared
  int T, H, E, S, I, k;
};

#if defined(__HIP_DEVICE_COMPILE__)
// 16 code bytes (32 elements of K) of an LDS row; a 4-bit operand fills the first half of the MFMA's registers.
__device__ __forceinline__ i32x8_t frag4(const uint8_t* p) {
  const i32x4v_t a = *reinterpret_cast<const i32x4v_t*>(p);
  return i32x8_t{a.x, a.y, a.z, a.w, 0, 0, 0, 0};
}

__device__ __forceinline__ f32x4_t mfma_fp4(i32x8_t w, i32x8_t a, f32x4_t c, int sw, int sa) {
  constexpr int kE2M1 = 4;   // operand format selector
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, kE2M1, kE2M1, 0, sw, 0, sa);
}
#endif

template <int MODE, int WM, int WN, int MI, int STAGES>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_fp4_kernel(Fp4Params p) {
  constexpr int NI = 4;
  constexpr int NW = WM * WN, NT = 64 * NW;
  constexpr int BM = WM * MI * 16, BN = WN * NI * 16;
  constexpr int BK = 128, CPR = BK / 16;               // bytes and 16-byte chunks of a row per slice
  constexpr int A_CH = BM * CPR / NT, B_CH = BN * CPR / NT;
  static_assert(BM * CPR % NT == 0 && BN * CPR % NT == 0, "whole loads per thread");
  constexpr int SC_W = 2 * (BM + BN);                  // scale words of a slice: A steps 0, 1, then B steps 0, 1
  static_assert(2 * BM % 64 == 0 && 2 * BN % 64 == 0, "a wavefront's scale load is all A or all B");
  constexpr int SC_CH = (SC_W + NT - 1) / NT;
  constexpr int PER = A_CH + B_CH + SC_CH;             // loads per thread per slice
  static_assert(MODE != kGateUp4 || BN == 256, "a gate/up tile is 128 columns of h");
  constexpr int SC_OFF = (BM + BN) * BK;
  constexpr int STAGE = SC_OFF + SC_CH * NT * 4;
  // epilogue staging over the finished ring: down, (MI*16) x 64 bf16 per wavefront; gate/up, 64 code bytes
  // and 4 scale bytes per tile row
  constexpr int STG_PITCH = NI * 16 * 2 + 16;
  constexpr int H_PITCH = 64 + 16;
  constexpr int STG_BYTES = MODE == kDown4 ? NW * MI * 16 * STG_PITCH : BM * (H_PITCH + 4);
  constexpr int LDS_BYTES = STAGES * STAGE > STG_BYTES ? STAGES * STAGE : STG_BYTES;
  static_assert(LDS_BYTES <= 163840, "LDS of a CU");
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS_BYTES];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, g = lane >> 4;

  // ------------------------------------------------------------ which tile
  const int L = grouped_tile<kStripeFp4>(p.ntiles);
  if (L < 0) return;
  const TileDesc d = p.tiles[L];
  const int seg = __builtin_amdgcn_readfirstlane(d.seg);
  const int row0 = __builtin_amdgcn_readfirstlane(d.row0);
  const int rows = __builtin_amdgcn_readfirstlane(d.rows);
  const int nt = __builtin_amdgcn_readfirstlane(d.nt);
  const bool shared = seg == p.E;
  // Routed gate/up rows gathered from the quantised x: row row0 + r of the
  // expert-sorted order is token perm[row0 + r] / k (codes and scales).
  const bool gather = MODE == kGateUp4 && !shared && p.perm != nullptr;

  // ------------------------------------------------------------ operands
  const int K1 = MODE == kDown4 ? p.I : p.H;            // K of one expert
  const int nexp = MODE == kDown4 && shared ? p.S : 1;  // experts whose K ranges follow each other
  const int lda = nexp * K1 / 2, ldw = K1 / 2;          // bytes
  const int a_total = shared || gather ? p.T : p.T * p.k;   // rows of the A tensor (scale plane length)
  const int a_base = gather ? 0 : row0;
  const int a_rows = gather ? p.T : rows;               // rows the A descriptor covers
  const uint8_t* A = (shared || gather ? p.a_shared : p.a_routed) + (int64_t)a_base * lda;
  const uint8_t* SA = (shared || gather ? p.sa_shared : p.sa_routed) + (int64_t)a_base * 4;
  const int nrow_w = MODE == kGateUp4 ? 2 * p.I : p.H;  // weight rows of one expert
  const int64_t w_one = (int64_t)nrow_w * ldw, sw_one = (int64_t)nrow_w * (K1 / 32);
  const uint8_t* W = shared ? p.w_shared : p.w_routed + seg * w_one;
  const uint8_t* SW = shared ? p.sw_shared : p.sw_routed + seg * sw_one;
  const int w_bytes = (int)((shared ? p.S : 1) * w_one), sw_bytes = (int)((shared ? p.S : 1) * sw_one);
  const int ncols = MODE == kGateUp4 ? (shared ? p.S * p.I : p.I) : p.H;
  const int sa_stride = a_total * 4, sw_stride = nrow_w * 4;   // bytes between the scale planes of K steps
  const int sa_bytes = (nexp * K1 / 128) * sa_stride - a_base * 4;

  // weight row (within the descriptor: all shared experts together) of tile column row r
  auto weight_row = [&](int r) {
    if constexpr (MODE == kGateUp4) {
      const bool up = r >= BN / 2;
      const int c = min(nt * (BN / 2) + (up ? r - BN / 2 : r), ncols - 1);
      return (c / p.I) * 2 * p.I + (up ? p.I : 0) + c % p.I;
    } else {
      return min(nt * BN + r, ncols - 1);
    }
  };
  // row of A for tile row r, or one past the descriptor (the range check drops the load)
  auto a_row = [&](int r) {
    int src = r < rows ? r : a_rows + 1;
    if (MODE == kGateUp4 && gather && r < rows) src = p.perm[row0 + r] / p.k;
    return src;
  };

  // ------------------------------------------------------------ load offsets
  int a_off[A_CH], b_off[B_CH], s_off[SC_CH];
#pragma unroll
  for (int i = 0; i < A_CH; ++i) {
    const int q = (i * NW + wave) * 64 + lane, r = q / CPR, pc = q % CPR;
    a_off[i] = a_row(r) * lda + swz<CPR>(r, pc) * 16;
  }
#pragma unroll
  for (int i = 0; i < B_CH; ++i) {
    const int q = (i * NW + wave) * 64 + lane, r = q / CPR, pc = q % CPR;
    b_off[i] = weight_row(r) * ldw + swz<CPR>(r, pc) * 16;
  }
  constexpr int kDrop = 0x7FFFFFFF;                     // past every descriptor
#pragma unroll
  for (int i = 0; i < SC_CH; ++i) {
    const int q = (i * NW + wave) * 64 + lane;
    if (q < 2 * BM) {
      const int r = q % BM;
      s_off[i] = r < rows ? (q / BM) * sa_stride + a_row(r) * 4 : kDrop;
    } else if (q < SC_W) {
      const int r = (q - 2 * BM) % BN;
      int wr = weight_row(r);
      int eoff = 0;
      if constexpr (MODE == kGateUp4) {                 // scale words are kept per expert
        eoff = (wr / nrow_w) * (int)sw_one;
        wr %= nrow_w;
      }
      s_off[i] = eoff + (q - 2 * BM) / BN * sw_stride + wr * 4;
    } else {
      s_off[i] = kDrop;
    }
  }
  const __amdgpu_buffer_rsrc_t rsrc_a = make_rsrc(A, a_rows * lda);
  const __amdgpu_buffer_rsrc_t rsrc_w = make_rsrc(W, w_bytes);
  const __amdgpu_buffer_rsrc_t rsrc_sa = make_rsrc(SA, sa_bytes);
  const __amdgpu_buffer_rsrc_t rsrc_sw = make_rsrc(SW, sw_bytes);
  typedef __attribute__((address_space(3))) void lds_void_t;
  const int nk1 = (K1 + 255) / 256, nk = nexp * nk1;    // slices of one expert, of all
  auto issue = [&](int stage, int kt) {
    const int ex = MODE == kDown4 ? kt / nk1 : 0, j = MODE == kDown4 ? kt - ex * nk1 : kt;
    const int ak = ex * ldw + j * BK, wk = ex * (int)w_one + j * BK;
    const int as = (ex * (K1 / 128) + 2 * j) * sa_stride, ws = ex * (int)sw_one + 2 * j * sw_stride;
    uint8_t* sb = lds + stage * STAGE;
#pragma unroll
    for (int i = 0; i < A_CH; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_a, (lds_void_t*)(sb + (i * NW + wave) * 1024), 16, a_off[i], ak, 0,
                                               0);
#pragma unroll
    for (int i = 0; i < B_CH; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_w, (lds_void_t*)(sb + BM * BK + (i * NW + wave) * 1024), 16,
                                               b_off[i], wk, 0, 0);
#pragma unroll
    for (int i = 0; i < SC_CH; ++i) {
      lds_void_t* dst = (lds_void_t*)(sb + SC_OFF + (i * NW + wave) * 256);
      if ((i * NW + wave) * 64 < 2 * BM)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_sa, dst, 4, s_off[i], as, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_sw, dst, 4, s_off[i], ws, 0, 0);
    }
  };

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < nk) issue(s, s);

  f32x4_t acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // LDS rows of this lane's operands; lane group g supplies the elements [32g, 32g + 32) of a step
  const int arow0 = wm * MI * 16 + l16;
  int b_rd[NI];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    int brow;
    if constexpr (MODE == kGateUp4)   // blocks 0, 1: gate rows of h columns wn*32 + ...; 2, 3: the matching up rows
      brow = (ni < 2 ? 0 : BN / 2) + wn * 32 + (ni % 2) * 16;
    else
      brow = wn * NI * 16 + ni * 16;
    b_rd[ni] = brow + l16;
  }
  const bool has_rows = wm * MI * 16 < rows;

  int cur = 0, left = K1 / 128;                         // K steps left of the current expert
  for (int kt = 0; kt < nk; ++kt) {
    wait_slices<PER>(min(nk - 1, kt + STAGES - 2) - kt);
    __builtin_amdgcn_s_waitcnt(kLgkmWaitZero);          // this wavefront's reads of the stage issued into next
    asm volatile("s_barrier" ::: "memory");
    if (kt + STAGES - 1 < nk) issue(cur == 0 ? STAGES - 1 : cur - 1, kt + STAGES - 1);
    if (has_rows) {
      const uint8_t* base = lds + cur * STAGE;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        if (kk == 1 && left < 2) break;
        const int ch = swz<CPR>(l16, kk * 4 + g) * 16;
        const uint8_t* sca = base + SC_OFF + kk * BM * 4 + g;
        const uint8_t* scb = base + SC_OFF + (2 * BM + kk * BN) * 4 + g;
        i32x8_t fb[NI];
        int sb[NI];
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          fb[ni] = frag4(base + BM * BK + b_rd[ni] * BK + ch);
          sb[ni] = scb[b_rd[ni] * 4];
        }
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          const i32x8_t fa = frag4(base + (arow0 + mi * 16) * BK + ch);
          const int sa = sca[(arow0 + mi * 16) * 4];
#pragma unroll
          for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = mfma_fp4(fb[ni], fa, acc[mi][ni], sb[ni], sa);
        }
      }
    }
    left -= 2;
    if (left <= 0) left = K1 / 128;
    cur = cur == STAGES - 1 ? 0 : cur + 1;
  }

  // ------------------------------------------------------------ epilogue
  // acc[mi][ni][r] holds C[i][j] with i = arow0 + 16 mi (token row), j = 16 ni + 4 (lane / 16) + r
  __syncthreads();   // every wavefront is done with the ring
  if constexpr (MODE == kGateUp4) {
    uint8_t* hc = lds;                                  // [BM][H_PITCH] codes
    uint8_t* hsc = lds + BM * H_PITCH;                  // [BM][4] scale bytes
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      float v[8];
      uint32_t m = 0;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float gv = acc[mi][b][r], uv = acc[mi][b + 2][r];
          const float h = gv * gate_sigmoid(gv) * uv;
          v[b * 4 + r] = h;
          m = max(m, __float_as_uint(h) & 0x7FFFFFFFu);
        }
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      const uint32_t e = mx_scale_byte(m);
      const uint32_t w = e2m1x8(v, e);                  // block 0's four codes, then block 1's
      const int i = arow0 + mi * 16;
      uint8_t* dst = hc + i * H_PITCH + wn * 16 + g * 2;
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w;
      *reinterpret_cast<uint16_t*>(dst + 8) = (uint16_t)(w >> 16);
      if (g == 0) hsc[i * 4 + wn] = (uint8_t)e;
    }
    __syncthreads();
    uint8_t* out = shared ? p.out_shared : p.out_routed;
    uint32_t* out_s = reinterpret_cast<uint32_t*>(shared ? p.out_shared_scale : p.out_routed_scale);
    const int64_t plane = shared ? p.T : (int64_t)p.T * p.k;
    for (int q = tid; q < BM * 4; q += NT) {            // 4 lanes a row, 16 bytes each
      const int i = q >> 2, c = q & 3;
      if (i < rows)
        *reinterpret_cast<uint4*>(out + (row0 + i) * (int64_t)(ncols / 2) + nt * 64 + c * 16) =
            *reinterpret_cast<const uint4*>(hc + i * H_PITCH + c * 16);
    }
    for (int i = tid; i < rows; i += NT)
      out_s[nt * plane + row0 + i] = *reinterpret_cast<const uint32_t*>(hsc + i * 4);
  } else {
    // a lane holds 4 adjacent columns of a row; through LDS the wavefront stores
    // whole 128-byte row segments, 16 bytes a lane
    uint8_t* stg = lds + wave * (MI * 16 * STG_PITCH);
    bf16_t* out = reinterpret_cast<bf16_t*>(shared ? p.out_shared : p.out_routed);
    const int col = nt * BN + wn * 64 + (lane & 7) * 8;   // ncols is a multiple of 128: the segment is whole or absent
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        *reinterpret_cast<uint2*>(stg + (mi * 16 + l16) * STG_PITCH + (ni * 16 + 4 * g) * 2) =
            uint2{cvt_bf16x2(acc[mi][ni][0], acc[mi][ni][1]), cvt_bf16x2(acc[mi][ni][2], acc[mi][ni][3])};
    // (the wavefront reads back only what it wrote; its LDS operations complete in order)
    __builtin_amdgcn_s_waitcnt(kLgkmWaitZero);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int it = 0; it < MI * 2; ++it) {
      const int lr = it * 8 + (lane >> 3);
      const int i = wm * MI * 16 + lr;
      const uint4 v = *reinterpret_cast<const uint4*>(stg + lr * STG_PITCH + (lane & 7) * 16);
      if (i < rows && col < ncols) *reinterpret_cast<uint4*>(out + (row0 + i) * (int64_t)ncols + col) = v;
    }
  }
#endif
}

// Tile shapes <WM, WN, MI, STAGES>: large batches, and few rows per expert.
#define MOE_FP4_TILE 2, 4, 8, 2
#define MOE_FP4_DEC_TILE 1, 4, 2, 4

template <int MODE>
moe_status launch_gemm_fp4(const FfnLayout& L, int64_t max_tiles, const Fp4Params& p, hipStream_t st) {
  const int64_t grid = grouped_grid(max_tiles, kStripeFp4);
  if (grid == 0) return MOE_OK;
  if (L.bm1 == kFp4DecBM)
    hipLaunchKernelGGL((gemm_fp4_kernel<MODE, MOE_FP4_DEC_TILE>), dim3((unsigned)grid), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((gemm_fp4_kernel<MODE, MOE_FP4_TILE>), dim3((unsigned)grid), dim3(512), 0, st, p);
  return launch_status();
}

}  // namespace

moe_status launch_ffn_fp4(const moe_cfg* c, const uint8_t* x_perm, const uint8_t* x_perm_scale, const int32_t* perm,
                          const int32_t* offsets, const moe_expert_weights* w, const bf16_t* x, bf16_t* y_perm,
                          bf16_t* y_shared, void* ws, int phase, hipStream_t st) {
  const FfnLayout L(c);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const int32_t* hdr = reinterpret_cast<const int32_t*>(base + L.off_hdr);
  auto bytes = [](const void* q) { return static_cast<const uint8_t*>(q); };
  moe_status s;
  Fp4Params p{};
  p.T = c->T; p.H = c->H; p.E = c->E; p.S = c->S; p.I = c->I; p.k = c->k;
  if (phase == MOE_FFN_ALL || phase == MOE_FFN_GATE_UP) {
    if ((s = launch_build_tiles(c, offsets, ws, st)) != MOE_OK) return s;
    // x once in MXFP4: the shared experts' operand, and the routed one when its rows are gathered
    if ((c->S > 0 || perm) &&
        (s = launch_quantize_fp4(x, 1, c->T, c->H, base + L.off_xq, base + L.off_xqs, st)) != MOE_OK)
      return s;
    p.perm = perm;
    p.a_routed = x_perm; p.sa_routed = x_perm_scale;
    p.a_shared = base + L.off_xq; p.sa_shared = base + L.off_xqs;
    p.w_routed = bytes(w->w_gate_up); p.sw_routed = bytes(w->w_gate_up_scale);
    p.w_shared = bytes(w->ws_gate_up); p.sw_shared = bytes(w->ws_gate_up_scale);
    p.out_routed = base + L.off_hp; p.out_routed_scale = base + L.off_hps;
    p.out_shared = base + L.off_hs; p.out_shared_scale = base + L.off_hss;
    p.tiles = reinterpret_cast<const TileDesc*>(base + L.off_t1);
    p.ntiles = hdr;
    if ((s = launch_gemm_fp4<kGateUp4>(L, L.max1, p, st)) != MOE_OK) return s;
  }
  if (phase == MOE_FFN_ALL || phase == MOE_FFN_DOWN) {
    p.perm = nullptr;
    p.a_routed = base + L.off_hp; p.sa_routed = base + L.off_hps;
    p.a_shared = base + L.off_hs; p.sa_shared = base + L.off_hss;
    p.w_routed = bytes(w->w_down); p.sw_routed = bytes(w->w_down_scale);
    p.w_shared = bytes(w->ws_down); p.sw_shared = bytes(w->ws_down_scale);
    p.out_routed = reinterpret_cast<uint8_t*>(y_perm); p.out_routed_scale = nullptr;
    p.out_shared = reinterpret_cast<uint8_t*>(y_shared); p.out_shared_scale = nullptr;
    p.tiles = reinterpret_cast<const TileDesc*>(base + L.off_t2);
    p.ntiles = hdr + 1;
    if ((s = launch_gemm_fp4<kDown4>(L, L.max2, p, st)) != MOE_OK) return s;
  }
  return MOE_OK;
}

}  // namespace moe
