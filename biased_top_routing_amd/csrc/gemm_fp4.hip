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
// Large batches: tiles of 128, 256 or 288 token rows x 256 weight rows, one workgroup
// of 2 x 4 wavefronts a CU, each wavefront 4 x 4 to 9 x 4 MFMA blocks, and the
// workgroups stay: each takes a 32nd of its XCD's contiguous share of the table (one
// expert's tiles run on one XCD at the same time and meet in its L2), and the loads
// run through the tiles without a break.  K advances two 128-wide steps (128 bytes of
// codes a row: whole cache lines; by single steps, in half lines, gate/up takes 7%
// and down 8% longer) per slice through two LDS stages filled by direct-to-LDS buffer
// loads (16-byte chunks, XOR swizzle per row), the rows' scale words of both steps
// beside them.  There is one barrier a slice, before the MFMAs of its last row block:
// the next slice has landed by then, this one's last fragments have been read, and
// the loads of the slice after next go out into its stage, one after each row block's
// MFMAs.  A 4-bit MFMA takes half the time of an 8-bit one on the same operand bytes,
// so the fragment reads are kept ahead of it: the token rows' 2 blocks, the weights' a
// K step.  When a tile's last slice is multiplied the next tile's first one is on its
// way, and its epilogue runs over it.
//   T = 16384, H = 7168, I = 2048, 256 experts, 8 + 1 a token: gate/up 2.51 ms (3.45
// PFLOP/s), down 1.42 ms (3.05 PFLOP/s, 2.1 GB of y among it).  The MFMAs alone, from
// registers, reach 7.0 PFLOP/s on such operands (the chip's power limit; 9.8 on
// zeros).  Of gate/up's time they are 1.2 ms; the LDS reads, the barriers and the
// epilogue add 0.2 ms each, and the rest is operand loads that do not hide: with
// 256-row tiles the kernel takes 1.8 ms without them and 2.2 ms without the MFMAs.
// Measured without gain: 3 or 4 stages of single steps (deeper, but half lines), runs
// of tiles dealt to the XCDs instead of shares, a K walk that starts elsewhere in
// each tile, cache hints on the weights (slower), wave priorities, waits that leave
// the stores out, row blocks skipped where a tile is short (branches between the
// MFMAs: 2% to 10% slower, with MFMA work saved).
//
// 128-row tiles leave room for 3 stages: two slices are on their way, and a slice takes
// 1.3 us where the others take 2 whatever rows they hold (64 rows an expert on that
// layer: the whole call 1.21 ms against 1.44 with 256-row tiles).
//
// Few rows per expert: the GEMMs stream the weights.  Tiles of 32 rows in 4 parts of 64
// weight rows, a workgroup of one wavefront each, 3 stages of two K steps, 4 of them a
// CU, which nothing but their own loads holds up (layer above, the whole call in us
// with 4 wavefronts a workgroup and 4 stages / 2 and 3 / 1 and 3: T = 1 53.4 / 52.7 /
// 50.2, 16 419 / 406 / 406, 128 996 / 983 / 983, 512 1066 / 1056 / 1064; H = 2048, I =
// 1408, T = 2, 6 + 2 a token 29.7 / 25.5 / 25.4).  T = 128 reads its 5.9 GB at 6.0 TB/s.
//
// The shared experts' down GEMM walks the experts one after the other.  The
// gate/up tile's 256 weight rows are the 128 gate rows and the 128 up rows of 128
// h columns; a wavefront holds gate and up of 32 of them, one scale block.
// All LDS is one array: with several LDS objects the compiler makes every LDS
// read wait for the direct-to-LDS loads in flight.
#include <algorithm>
#include <type_traits>

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
  const int32_t* tile_rows;   // rows per tile
  const int32_t* perm;        // gate/up: non-null -> routed rows gathered from a_shared / sa_shared
  int T, H, E, S, I, k;
};

constexpr int kHPitch = 64 + 16;         // a tile row's 64 bytes of h codes in LDS
constexpr int align64(int n) { return (n + 63) / 64 * 64; }

#if defined(__HIP_DEVICE_COMPILE__)
constexpr int NI4 = 4;          // MFMA column blocks of a wavefront
constexpr int kDrop = 0x7FFFFFFF;   // a byte offset past every descriptor: the range check drops the load
typedef __attribute__((address_space(3))) void lds_void_t;

// 16 code bytes (32 elements of K) of an LDS row; a 4-bit operand fills the first half of the MFMA's registers.
__device__ __forceinline__ i32x8_t frag4(const uint8_t* p) {
  const i32x4v_t a = *reinterpret_cast<const i32x4v_t*>(p);
  return i32x8_t{a.x, a.y, a.z, a.w, 0, 0, 0, 0};
}

__device__ __forceinline__ f32x4_t mfma_fp4(i32x8_t w, i32x8_t a, f32x4_t c, int sw, int sa) {
  constexpr int kE2M1 = 4;   // operand format selector
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, kE2M1, kE2M1, 0, sw, 0, sa);
}

// Waits until at most min(n, MAX) slices' loads (PER instructions each) of this wavefront are outstanding.
template <int PER, int MAX>
__device__ __forceinline__ void wait_loads(int n) {
  static_assert(PER * MAX < 64, "vmcnt range");
  if constexpr (MAX == 0) wait_vm<0>();
  else if (n >= MAX) wait_vm<PER * MAX>();
  else wait_loads<PER, MAX - 1>(n);
}

// v as a value that the compiler cannot compute ahead of this point (what a tile's
// begin and epilogue derive from the lane would otherwise be computed before the
// loops and held, or spilled, through them).
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Entry L of the tile table, read through the scalar cache.
__device__ __forceinline__ TileDesc tile_at(const Fp4Params& p, int L) {
  typedef const __attribute__((address_space(4))) int32_t* cptr;
  const cptr t = (cptr)(uintptr_t)(p.tiles + L);
  return TileDesc{t[0], t[1], t[2], t[3]};
}

// One tile's operands (all wavefront-uniform).
template <int MODE>
struct Operands4 {
  const uint8_t *A, *SA, *W, *SW;
  int lda, ldw;                 // bytes between rows
  int a_rows;                   // rows the A descriptor covers
  int a_bytes, w_bytes, sa_bytes, sw_bytes;
  int sa_stride, sw_stride;     // bytes between the scale planes of K steps
  int64_t w_one;                // one expert's weights and scale words, bytes
  int sw_one;
  int nk1, nexp;                // 128-wide K steps of one expert; experts whose K ranges follow each other
  int ncols;                    // output columns of the segment
  int ex, c0;                   // the tile's expert among the shared ones, and its first weight row there
  bool shared, gather;

  __device__ __forceinline__ Operands4(const Fp4Params& p, const TileDesc& d) {
    shared = d.seg == p.E;
    // routed gate/up rows gathered from the quantised x: row row0 + r of the
    // expert-sorted order is token perm[row0 + r] / k (codes and scales)
    gather = MODE == kGateUp4 && !shared && p.perm != nullptr;
    const int K1 = MODE == kDown4 ? p.I : p.H;
    nk1 = K1 / 128;
    nexp = MODE == kDown4 && shared ? p.S : 1;
    lda = nexp * K1 / 2;
    ldw = K1 / 2;
    const int a_total = shared || gather ? p.T : p.T * p.k;   // rows of the A tensor (scale plane length)
    const int a_base = gather ? 0 : d.row0;
    a_rows = gather ? p.T : d.rows;
    A = (shared || gather ? p.a_shared : p.a_routed) + (int64_t)a_base * lda;
    SA = (shared || gather ? p.sa_shared : p.sa_routed) + (int64_t)a_base * 4;
    const int nrow_w = MODE == kGateUp4 ? 2 * p.I : p.H;      // weight rows of one expert
    w_one = (int64_t)nrow_w * ldw;
    sw_one = nrow_w * (K1 / 32);
    W = shared ? p.w_shared : p.w_routed + d.seg * w_one;
    SW = shared ? p.sw_shared : p.sw_routed + d.seg * (int64_t)sw_one;
    a_bytes = a_rows * lda;
    w_bytes = (int)((shared ? p.S : 1) * w_one);
    sw_bytes = (shared ? p.S : 1) * sw_one;
    sa_stride = a_total * 4;
    sw_stride = nrow_w * 4;
    sa_bytes = nexp * nk1 * sa_stride - a_base * 4;
    ncols = MODE == kGateUp4 ? (shared ? p.S * p.I : p.I) : p.H;
    // (a gate/up tile's 128 columns lie in one expert: I is a multiple of 128)
    ex = MODE == kGateUp4 && shared ? d.nt * 128 / p.I : 0;
    c0 = MODE == kGateUp4 ? d.nt * 128 - ex * p.I : d.nt * 256;
  }

  // weight row (in its expert) of row r of part `part` of the tile's columns (BN weight rows a part), the
  // last one for rows past the columns
  template <int BN>
  __device__ __forceinline__ int wrow(const Fp4Params& p, int part, int r) const {
    if constexpr (MODE == kGateUp4) return c0 + part * (BN / 2) + (r < BN / 2 ? r : r - BN / 2 + p.I);
    else return min(c0 + part * BN + r, ncols - 1);
  }
};

// The order of a wavefront's columns: block ni, MFMA row 4 g + r is column
// 8 g + 4 (ni mod 2) + r of its 32 gate columns (ni < 2) or of the up columns BN / 2
// further on, or of its first or second 32 output columns, so that a lane holds 8
// neighbouring columns of a row in two blocks: 4 bytes of codes, 16 of bf16.  The
// tile column whose LDS row lane l16 reads is col_lane + col_off.
__device__ __forceinline__ int col_lane(int l16) { return 8 * (l16 >> 2) + (l16 & 3); }
template <int MODE, int BN>
__device__ __forceinline__ constexpr int col_off(int ni) {
  return (ni / 2) * (MODE == kGateUp4 ? BN / 2 : 32) + (ni % 2) * 4;
}
// Physical 16-byte chunk of logical chunk c of 8 in LDS row r of the weights: 8
// lanes' rows (4, and 4 that lie 8 further on) meet no bank twice.
__device__ __forceinline__ int swz_w(int r, int c) { return c ^ ((r & 3) | (((r >> 3) & 1) << 2)); }

// SwiGLU of one row block: acc[b] gate, acc[b + 2] up; the codes of this lane's 8 h
// values (neighbouring columns), and the scale byte of the row's 32 columns, which
// the 4 lanes l16, + 16, + 32, + 48 hold together.
__device__ __forceinline__ uint32_t swiglu_codes(const f32x4_t (&acc)[NI4], uint32_t* e) {
  float v[8];
  uint32_t m = 0;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float gv = acc[b][r], uv = acc[b + 2][r];
      const float h = gv * gate_sigmoid(gv) * uv;
      v[b * 4 + r] = h;
      m = max(m, __float_as_uint(h) & 0x7FFFFFFFu);
    }
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  *e = mx_scale_byte(m);
  return e2m1x8(v, *e);
}

// Workgroup barrier for LDS: this wavefront's LDS operations are done; loads and
// stores in flight stay in flight (__syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(kLgkmWaitZero);
  asm volatile("s_barrier" ::: "memory");
}

// A wavefront's gate/up row block in LDS: codes [row][kHPitch] and scale bytes [row][4].
__device__ __forceinline__ void stage_h(uint8_t* hc, uint8_t* hsc, int row, int wn, int g, uint32_t w, uint32_t e) {
  *reinterpret_cast<uint32_t*>(hc + row * kHPitch + wn * 16 + g * 4) = w;
  if (g == 0) hsc[row * 4 + wn] = (uint8_t)e;
}

// The staged gate/up tile, or its quarter `part` (WN = 1), to memory: 16 bytes a lane,
// WN lanes a row, and the rows' scale words, or bytes of them.
template <int NT, int WN>
__device__ __forceinline__ void store_h(const Fp4Params& p, const TileDesc& d, int part, bool shared, const uint8_t* hc,
                                        const uint8_t* hsc, int tid) {
  const int hw = shared ? p.S * p.I / 2 : p.I / 2;      // bytes of an h row
  uint8_t* out = shared ? p.out_shared : p.out_routed;
  uint8_t* out_s = shared ? p.out_shared_scale : p.out_routed_scale;
  const int64_t plane = shared ? p.T : (int64_t)p.T * p.k;
  for (int q = tid; q < d.rows * WN; q += NT) {
    const int i = q / WN, c = q % WN;
    *reinterpret_cast<uint4*>(out + (d.row0 + i) * (int64_t)hw + d.nt * 64 + (part * WN + c) * 16) =
        *reinterpret_cast<const uint4*>(hc + i * kHPitch + c * 16);
  }
  using scales_t = std::conditional_t<WN == 4, uint32_t, uint8_t>;
  for (int i = tid; i < d.rows; i += NT)
    *reinterpret_cast<scales_t*>(out_s + (d.nt * plane + d.row0 + i) * 4 + part * WN) =
        *reinterpret_cast<const scales_t*>(hsc + i * 4);
}

// 16 rows x 64 columns of a wavefront's down tile as bf16, through its own two 1 KB
// pieces of LDS (8 rows each, `dist` bytes apart, 16-byte chunks XOR swizzled), so
// that whole 128-byte row segments are stored, 16 bytes a lane.  (A wavefront reads
// back only what it wrote; its LDS operations complete in order.)
__device__ __forceinline__ void store_y(uint8_t* stg, int dist, const f32x4_t (&acc)[NI4], bf16_t* out, int64_t row0,
                                        int i0, int rows, int col0, int ncols, int lane) {
  const int l16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int b = 0; b < NI4; b += 2)
    *reinterpret_cast<uint4*>(stg + (l16 >> 3) * dist + (l16 & 7) * 128 + ((2 * b + g) ^ (l16 & 7)) * 16) =
        make_uint4(cvt_bf16x2(acc[b][0], acc[b][1]), cvt_bf16x2(acc[b][2], acc[b][3]),
                   cvt_bf16x2(acc[b + 1][0], acc[b + 1][1]), cvt_bf16x2(acc[b + 1][2], acc[b + 1][3]));
  __builtin_amdgcn_s_waitcnt(kLgkmWaitZero);
  __builtin_amdgcn_wave_barrier();
  const int col = col0 + (lane & 7) * 8;   // (ncols is a multiple of 128: the segment is whole or absent)
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int lr = it * 8 + (lane >> 3), i = i0 + lr;
    const uint4 v =
        *reinterpret_cast<const uint4*>(stg + it * dist + (lane >> 3) * 128 + ((lane & 7) ^ (lane >> 3)) * 16);
    if (i < rows && col < ncols) *reinterpret_cast<uint4*>(out + (row0 + i) * ncols + col) = v;
  }
  __builtin_amdgcn_s_waitcnt(kLgkmWaitZero);
  __builtin_amdgcn_wave_barrier();
}
#endif

// ------------------------------------------------------------------ large batches
constexpr int kFp4Threads = 512;
constexpr int kFp4Lds = 160256;

#if defined(__HIP_DEVICE_COMPILE__)
// The GEMM over tiles of BM rows, in kFp4Lds bytes of LDS.
template <int MODE, int BM, int STAGES>
__device__ __forceinline__ void gemm_fp4_tiles(const Fp4Params& p, uint8_t* lds) {
  constexpr int WM = 2, WN = 4, MI = BM / (WM * 16);
  constexpr int NT = kFp4Threads, NW = NT / 64, BN = 256;
  static_assert(WM * WN == NW && WM * MI * 16 == BM && BN == kFp4BN2, "tile shape");
  constexpr int BK = 128, CPR = BK / 16;               // bytes (two K steps) and 16-byte chunks of a row per slice
  constexpr int RPL = NT / CPR;                        // rows a load of all threads covers
  constexpr int A_CH = (BM + RPL - 1) / RPL, B_CH = BN / RPL;   // loads per thread; A's last one covers AX rows
  // of a step's scale words wavefronts 0-3 load A's first 256, wavefronts 4-7 B's; past 256 rows (32 of
  // them) A's last load is wavefronts 0-3's alone
  constexpr int ASC = BM > 256 ? BM : 256, AX = ASC - 256;
  static_assert(BN == 256 && NT == 512 && (AX == 0 || (AX == RPL / 2 && STAGES == 2)), "the loads of a slice");
  constexpr int PER = A_CH + B_CH + 2;                 // loads per thread per slice (every wavefront's, unless AX)
  constexpr int SCP = (ASC + BN) * 4;                  // a step's scale words: A's, B's
  constexpr int B_OFF = BM * BK, SC_OFF = B_OFF + BN * BK, STAGE = SC_OFF + 2 * SCP;
  constexpr int PERM_OFF = STAGES * STAGE;                  // the next tile's perm entries (gathered rows)
  constexpr int LDS_BYTES = PERM_OFF + align64(BM) * 4;
  static_assert(LDS_BYTES <= kFp4Lds, "LDS");
  // the epilogue's staging: the weights' part of the stage that is filled next
  static_assert(BM * (kHPitch + 4) <= BN * BK && B_CH >= 2, "the epilogue's staging");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, g = lane >> 4;

  // ------------------------------------------------------------ this workgroup's tiles
  // XCD x = b mod 8 takes an equal contiguous share of the shared tiles and then
  // one of the routed tiles; its workgroups take them in turn.
  const int n_real = __builtin_amdgcn_readfirstlane(p.ntiles[0]), n_rt = __builtin_amdgcn_readfirstlane(p.ntiles[4]);
  const int xcd = blockIdx.x & 7, per_s = (n_real - n_rt + 7) >> 3, per_r = (n_rt + 7) >> 3;
  const int s_cnt = min(max(n_real - n_rt - xcd * per_s, 0), per_s);
  const int r_cnt = min(max(n_rt - xcd * per_r, 0), per_r);
  const int step = gridDim.x >> 3;
  // the n-th of this workgroup: round n takes the next `step` positions of the share, turned by 5 n
  // (an expert's row tiles of one column follow each other, the last one shorter: without the turn
  // a workgroup might get only long ones; 32 + 5 shares no divisor with their number, at most 8)
  auto place = [&](int n) { return n * step + ((int)(blockIdx.x >> 3) + 5 * n) % step; };
  auto entry = [&](int q) { return q < s_cnt ? n_rt + xcd * per_s + q : xcd * per_r + q - s_cnt; };
  int nq = 0, q = place(0);                            // position in the XCD's share
  const int q_end = s_cnt + r_cnt;
  if (q >= q_end) return;

  // ------------------------------------------------------------ the loads
  // The stream of slices runs a slice ahead of the products, through the tiles.
  TileDesc ld = tile_at(p, entry(q)), nd = ld;         // the tile being loaded, the one after it
  bool more = false;                                   // nd is one
  int left_l = 0, in_l = 0;                            // experts of ld to load yet, K steps of the current one
  int ls = 0;                                          // stage the next slice goes to
  int ak = 0, wk = 0, sk = 0;                          // scalar offsets of the next slice: A, W, scale words
  // A: an offset a load where rows are gathered, else one and the rows' distance; W: one,
  // the rows' distance, and what lies between gate and up rows
  constexpr int A_OFF = MODE == kGateUp4 ? A_CH : 1;
  int a_off[A_OFF], b_off = 0, s_off = 0, a_dist = 0, w_dist = 0, w_gap = 0;
  int s_step = 0, a_skip = 0, w_skip = 0, s_skip = 0, nk1 = 1;   // scale plane distance; extra steps to the next expert
  // the scale words of A's last AX rows: wavefront 4 loads those of a slice's first step, 5 the second's,
  // 64 rows each (the rows before them twice)
  int sx_off = 0, sa_step = 0;
  int s_first = 0;                                     // down: first byte of this wavefront's scale words
  const uint8_t *baseA = nullptr, *baseW = nullptr, *baseS = nullptr, *baseSA = nullptr;
  int bytesA = 0, bytesW = 0, bytesS = 0, bytesSA = 0;   // 0 when the stream has ended: its loads are dropped
  // the perm entries of a gathered tile's rows into LDS
  auto load_perm = [&](const TileDesc& d) {
    if (MODE == kGateUp4 && p.perm != nullptr && d.seg != p.E && wave < align64(BM) / 64)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(p.perm + d.row0, d.rows * 4),
                                               (lds_void_t*)(lds + PERM_OFF + wave * 256), 4, tid * 4, 0, 0, 0);
  };
  // start loading ld: its perm entries, if any, are in LDS
  auto begin = [&]() {
    const Operands4<MODE> o(p, ld);
    const int32_t* rows = reinterpret_cast<const int32_t*>(lds + PERM_OFF);
    const int tid = opaque(threadIdx.x), lr = tid / CPR;
    const int ca = swz<CPR>(lr, tid % CPR) * 16, cw = swz_w(lr, tid % CPR) * 16;
    static_assert(RPL % 16 == 0, "a thread's rows have one swizzle");
    // (rows past the tile's lie past the descriptor: the range check drops their loads)
    if constexpr (MODE == kGateUp4) {
#pragma unroll
      for (int i = 0; i < A_CH; ++i) {
        const int r = lr + i * RPL;
        a_off[i] = (r >= ld.rows ? o.a_rows + 1 : o.gather ? rows[r] / p.k : r) * o.lda + ca;
      }
    } else {
      a_off[0] = lr * o.lda + ca;
      a_dist = RPL * o.lda;
    }
    b_off = (int)(o.ex * o.w_one) + (o.c0 + lr) * o.ldw + cw;
    w_dist = RPL * o.ldw;
    w_gap = MODE == kGateUp4 ? (p.I - 128) * o.ldw : 0;
    const bool sa = wave < NW / 2;                     // this wavefront loads A's scale words, else B's
    if constexpr (MODE == kGateUp4) {
      const int xr = BM - 64 + (tid & 63);
      if (sa) s_off = tid < ld.rows ? (o.gather ? rows[tid] / p.k : tid) * 4 : kDrop;
      else s_off = o.ex * o.sw_one + (o.c0 + tid - BN + (tid - BN >= 128 ? p.I - 128 : 0)) * 4;
      sx_off = xr < ld.rows ? (o.gather ? rows[xr] / p.k : xr) * 4 + (wave == NW / 2 + 1 ? o.sa_stride : 0) : kDrop;
    } else {                                           // (what lies past the tile is read where it is there, not used)
      s_first = sa ? wave * 256 : o.c0 * 4 + (wave - NW / 2) * 256;
    }
    sa_step = o.sa_stride;
    baseSA = o.SA; bytesSA = o.sa_bytes;
    baseA = o.A; bytesA = o.a_bytes;
    baseW = o.W; bytesW = o.w_bytes;
    baseS = sa ? o.SA : o.SW;
    bytesS = sa ? o.sa_bytes : o.sw_bytes;
    s_step = sa ? o.sa_stride : o.sw_stride;
    // from the slice after an expert's last one (which may hold one step only) to the next expert's first
    const int over = (o.nk1 + 1) / 2 * 2 - o.nk1;
    a_skip = -over * 64;
    w_skip = (int)o.w_one - o.nk1 * 64 - over * 64;
    s_skip = sa ? -over * s_step : o.sw_one - (o.nk1 + over) * s_step;
    ak = wk = sk = 0;
    in_l = nk1 = o.nk1;
    left_l = o.nexp;
    q = place(++nq);
    more = q < q_end;
    if (more) nd = tile_at(p, entry(q));
  };
  // Load i of PER of the stream's next slice.  (Only offsets that lie inside the
  // descriptor whatever the lane go through the scalar offset: the range check
  // compares the lane's offset with what the scalar one leaves of it.)
  auto issue_part = [&](int i) {
    uint8_t* sb = lds + ls * STAGE + wave * 1024;
    // (the down kernel has no registers to keep what the lane and scalars give at once)
    const unsigned lane4 = (opaque(threadIdx.x) & 63) * 4;
    const unsigned s_lane = MODE == kGateUp4 ? (unsigned)s_off : lane4 + (unsigned)s_first;
    const unsigned sx_lane =
        MODE == kGateUp4 ? (unsigned)sx_off : lane4 + (unsigned)((BM - 64) * 4 + (wave == NW / 2 + 1 ? sa_step : 0));
    if (AX > 0 && i == A_CH - 1 && wave >= NW / 2) {   // (rows past the tile: the scale words of the last ones instead)
      if (wave < NW / 2 + 2)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            make_rsrc(baseSA, bytesSA),
            (lds_void_t*)(lds + ls * STAGE + SC_OFF + (wave - NW / 2) * SCP + (BM - 64) * 4), 4, (int)sx_lane,
            ak / 64 * sa_step, 0, 0);
    } else if (i < A_CH)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(baseA, bytesA), (lds_void_t*)(sb + i * NW * 1024), 16,
                                               MODE == kGateUp4 ? a_off[i % A_OFF] : a_off[0] + i * a_dist, ak, 0, 0);
    else if (i < A_CH + B_CH)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          make_rsrc(baseW, bytesW), (lds_void_t*)(sb + B_OFF + (i - A_CH) * NW * 1024), 16,
          b_off + (i - A_CH) * w_dist + ((i - A_CH) * RPL >= 128 ? w_gap : 0), wk, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          make_rsrc(baseS, bytesS),
          (lds_void_t*)(lds + ls * STAGE + SC_OFF + (i - A_CH - B_CH) * SCP + wave * 256 +
                        (wave < NW / 2 ? 0 : AX * 4)),
          4, (int)(s_lane + (unsigned)((i - A_CH - B_CH) * s_step)), sk, 0, 0);
  };
  // After a slice's loads.
  auto advance = [&]() {
    ak += BK;
    wk += BK;
    sk += 2 * s_step;
    in_l -= 2;
    if (in_l <= 0) {
      --left_l;
      in_l = nk1;
      if (MODE == kDown4) {                            // the next shared expert's K range
        ak += a_skip;
        wk += w_skip;
        sk += s_skip;
      }
    }
    ls = ls == STAGES - 1 ? 0 : ls + 1;
  };
  // Before a slice's loads: the next tile is begun where the last one has ended.
  auto prepare = [&]() {
    if (left_l > 0) return;
    if (!more) {
      bytesA = bytesW = bytesS = bytesSA = 0;
      ak = wk = sk = 0;
      return;
    }
    ld = nd;
    begin();
    if (MODE == kGateUp4 && p.perm != nullptr) {
      lds_barrier();                                   // all have read this tile's entries: on to the next one's
      if (more) load_perm(nd);
    }
  };

  // ------------------------------------------------------------ the products
  // this lane's fragments in a stage: tile rows arow0 + 16 mi and brow + col_off(ni);
  // lane group g supplies the elements [32g, 32g + 32) of a step (the swizzles are the
  // same for every block, and a row's second step is 64 bytes away by exclusive or)
  const int arow0 = wm * MI * 16 + l16;
  const int brow = wn * (MODE == kGateUp4 ? 32 : 64) + col_lane(l16);
  const int a_lane = arow0 * BK + swz<CPR>(l16, g) * 16;
  const int b_lane = B_OFF + brow * BK + swz_w(col_lane(l16), g) * 16;
  const int sa_lane = SC_OFF + arow0 * 4 + g, sb_lane = SC_OFF + (ASC + brow) * 4 + g;
  constexpr int NB = MI % 3 == 0 ? 3 : 4, D = 2;       // A fragments held, and read ahead
  static_assert(MI % NB == 0 && D < NB && MI >= NI4, "the buffers rotate within a step; B's next step is read in one");
  f32x4_t acc[MI][NI4];
  i32x8_t fa[NB], fb[NI4], fbn[NI4];
  int ra[NB], rb[NI4], rbn[NI4];
  auto clear = [&]() {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI4; ++ni) acc[mi][ni] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };
  auto read_a = [&](const uint8_t* stage, int kk, int mi) {
    fa[mi % NB] = frag4(stage + (a_lane ^ (kk * 64)) + mi * 16 * BK);
    ra[mi % NB] = stage[sa_lane + kk * SCP + mi * 64];
  };
  auto read_b = [&](const uint8_t* stage, int kk, int ni) {
    fbn[ni] = frag4(stage + (b_lane ^ (kk * 64)) + col_off<MODE, BN>(ni) * BK);
    rbn[ni] = stage[sb_lane + kk * SCP + col_off<MODE, BN>(ni) * 4];
  };
  auto next_b = [&]() {
#pragma unroll
    for (int ni = 0; ni < NI4; ++ni) {
      fb[ni] = fbn[ni];
      rb[ni] = rbn[ni];
    }
  };
  auto read_first = [&](const uint8_t* stage) {        // a slice's first fragments
#pragma unroll
    for (int ni = 0; ni < NI4; ++ni) read_b(stage, 0, ni);
#pragma unroll
    for (int i = 0; i < D; ++i) read_a(stage, 0, i);
  };
  auto multiply = [&](int mi) {
#pragma unroll
    for (int ni = 0; ni < NI4; ++ni)
      acc[mi][ni] = mfma_fp4(fb[ni], fa[mi % NB], acc[mi][ni], rb[ni], ra[mi % NB]);
  };
  // K step KK of the slice in stage `here`; of the second one all but the last row
  // block, which is multiplied over the barrier.  The loads of the slice to come go
  // out one after each row block of the first step.
  auto products = [&](auto kkc, const uint8_t* here) {
    constexpr int KK = decltype(kkc)::value;
#pragma unroll
    for (int mi = 0; mi < MI - KK; ++mi) {
      if (mi + D < MI) read_a(here, KK, mi + D);
      else if (KK == 0) read_a(here, 1, mi + D - MI);
      if (KK == 0 && mi < NI4) read_b(here, 1, mi);
      __builtin_amdgcn_sched_barrier(0);
      multiply(mi);
      if (KK == 0) {
#pragma unroll
        for (int i = 2 + (PER - 2) * mi / MI; i < 2 + (PER - 2) * (mi + 1) / MI; ++i) issue_part(i);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (KK == 0) {
      next_b();
      advance();
    }
  };
  load_perm(ld);
  wait_vm<0>();
  lds_barrier();
  begin();
  lds_barrier();
  if (more) load_perm(nd);
#pragma unroll
  for (int i = 0; i < PER; ++i) issue_part(i);
  advance();
#pragma unroll
  for (int s = 2; s < STAGES; ++s) {
    if (left_l <= 0) {                                 // (the next tile's perm entries)
      wait_vm<0>();
      lds_barrier();
    }
    prepare();
#pragma unroll
    for (int i = 0; i < PER; ++i) issue_part(i);
    advance();
  }
  clear();

  int nc = 0, qc = place(1);                           // the tile after the one being computed
  TileDesc cd = tile_at(p, entry(place(0))), after = cd;
  if (qc < q_end) after = tile_at(p, entry(qc));
  const int steps1 = (MODE == kDown4 ? p.I : p.H) / 128;   // K steps of an expert
  auto experts = [&]() { return MODE == kDown4 && cd.seg == p.E ? p.S : 1; };
  int cs = 0, left = steps1, exps = experts();         // stage of the next slice; K steps left of the expert, experts
  bool half = false;                                   // a slice's last row block is to be multiplied
  bool done = false;                                   // ... and it is the tile's last slice
  while (true) {
    // The slice's one barrier: the next slice has landed, everywhere (it was asked for a
    // slice ago), and this one's stage is free; loading into it begins.
    wait_vm<PER * (STAGES - 2)>();
    lds_barrier();
    prepare();
    const uint8_t* here = lds + cs * STAGE;
    cs = cs == STAGES - 1 ? 0 : cs + 1;
    read_first(here);                                  // (not into the buffer in use; after the last slice unused)
    __builtin_amdgcn_sched_barrier(0);
    if (half) multiply(MI - 1);
    issue_part(0);
    issue_part(1);
    next_b();
    if (done) {
      // acc[mi][ni][r] holds C[i][j] with i = arow0 + 16 mi (token row), j in the order of col_off
      const bool shared = cd.seg == p.E;
      const int tid = opaque(threadIdx.x), lane = tid & 63, l16 = lane & 15, g = lane >> 4;
      if constexpr (MODE == kGateUp4) {
        uint8_t* hc = lds + ls * STAGE + B_OFF;
        uint8_t* hsc = hc + BM * kHPitch;
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          uint32_t e;
          const uint32_t w = swiglu_codes(acc[mi], &e);
          stage_h(hc, hsc, wm * MI * 16 + l16 + mi * 16, wn, g, w, e);
        }
        lds_barrier();
        store_h<NT, WN>(p, cd, 0, shared, hc, hsc, tid);
        lds_barrier();                                 // the staging is read: its loads may go out
      } else {
        bf16_t* out = reinterpret_cast<bf16_t*>(shared ? p.out_shared : p.out_routed);
        // (stored straight from the registers, in halves or by exchange in whole row
        // segments, the stores come in one burst in front of the next loads: 3% slower)
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
          store_y(lds + ls * STAGE + B_OFF + wave * 1024, NW * 1024, acc[mi], out, cd.row0, (wm * MI + mi) * 16,
                  cd.rows, cd.nt * BN + wn * 64, p.H, lane);
      }
      if (qc >= q_end) break;
      cd = after;
      qc = place(++nc + 1);
      if (qc < q_end) after = tile_at(p, entry(qc));
      exps = experts();
      clear();
    }
    half = wm * MI * 16 < cd.rows;
    if (!half) {                                       // no rows here, perhaps some in the next tile
#pragma unroll
      for (int i = 2; i < PER; ++i) issue_part(i);
      advance();
    } else {
      products(std::integral_constant<int, 0>{}, here);
      if (left >= 2) products(std::integral_constant<int, 1>{}, here);
      else half = false;                               // a slice of one step: what was read ahead is not used
    }
    left -= 2;
    done = false;
    if (left <= 0) {
      left = steps1;
      done = --exps == 0;
    }
  }
}
#endif

// The table's builder chose the tiles' height from the rows that are there.
template <int MODE>
__global__ __launch_bounds__(kFp4Threads, 1) void gemm_fp4_kernel(Fp4Params p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(16))) uint8_t lds[kFp4Lds];
  const int bm = __builtin_amdgcn_readfirstlane(*p.tile_rows);
  if (bm == kFp4LowBM) gemm_fp4_tiles<MODE, kFp4LowBM, 3>(p, lds);
  else if (bm == kFp4BM) gemm_fp4_tiles<MODE, kFp4BM, 2>(p, lds);
  else gemm_fp4_tiles<MODE, kFp4HighBM, 2>(p, lds);
#endif
}

// ------------------------------------------------------------------ few rows per expert
template <int MODE>
__global__ __launch_bounds__(64, 1) void gemm_fp4_rows_kernel(Fp4Params p) {
  constexpr int BM = kFp4RowsBM, STAGES = 3, PARTS = 4;
  constexpr int MI = BM / 16, NT = 64, BN = 64;
  static_assert(PARTS * BN == kFp4BN2, "the tiles of the table, in quarters");
  constexpr int BK = 128, CPR = BK / 16;               // bytes (two K steps) and 16-byte chunks of a row per slice
  constexpr int A_CH = BM * CPR / NT, B_CH = BN * CPR / NT;
  static_assert(BM * CPR % NT == 0 && BN * CPR % NT == 0, "whole loads per thread");
  // scale words of a slice: A's of step 0, of step 1, then B's likewise
  constexpr int SC_CH = (2 * (BM + BN) + NT - 1) / NT;
  static_assert(2 * BM % 64 == 0, "a scale load is all A or all B");
  constexpr int PER = A_CH + B_CH + SC_CH;             // loads per thread per slice
  constexpr int SC_OFF = (BM + BN) * BK, STAGE = SC_OFF + SC_CH * NT * 4;
  constexpr int LDS_BYTES = STAGES * STAGE;
  static_assert(LDS_BYTES <= 163840, "LDS of a CU");
  static_assert(BM * (kHPitch + 4) <= LDS_BYTES && 2048 <= LDS_BYTES, "the epilogue's staging");
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS_BYTES];
  const int lane = threadIdx.x, l16 = lane & 15, g = lane >> 4;
  // (the parts of a tile go to one XCD)
  const int part = (blockIdx.x >> 3) % PARTS, b = (blockIdx.x >> 3) / PARTS * 8 + (blockIdx.x & 7);
  const int L = grouped_tile_at(b, __builtin_amdgcn_readfirstlane(p.ntiles[0]),
                                __builtin_amdgcn_readfirstlane(p.ntiles[4]), kStripeFp4);
  if (L < 0) return;
  const TileDesc d = tile_at(p, L);
  const Operands4<MODE> o(p, d);
  auto a_row = [&](int r) { return r >= d.rows ? o.a_rows + 1 : o.gather ? p.perm[d.row0 + r] / p.k : r; };
  int a_off[A_CH], b_off[B_CH], s_off[SC_CH];
#pragma unroll
  for (int i = 0; i < A_CH; ++i) {
    const int c = i * NT + lane, r = c / CPR;
    a_off[i] = a_row(r) * o.lda + swz<CPR>(r, c % CPR) * 16;
  }
#pragma unroll
  for (int i = 0; i < B_CH; ++i) {
    const int c = i * NT + lane, r = c / CPR;
    b_off[i] = (int)(o.ex * o.w_one) + o.template wrow<BN>(p, part, r) * o.ldw + swz_w(r, c % CPR) * 16;
  }
#pragma unroll
  for (int i = 0; i < SC_CH; ++i) {
    const int c = i * NT + lane, cb = c - 2 * BM;
    if (c < 2 * BM) s_off[i] = c % BM < d.rows ? c / BM * o.sa_stride + a_row(c % BM) * 4 : kDrop;
    else if (cb < 2 * BN)
      s_off[i] = o.ex * o.sw_one + cb / BN * o.sw_stride + o.template wrow<BN>(p, part, cb % BN) * 4;
    else s_off[i] = kDrop;
  }
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(o.A, o.a_bytes), rw = make_rsrc(o.W, o.w_bytes),
                               rsa = make_rsrc(o.SA, o.sa_bytes), rsw = make_rsrc(o.SW, o.sw_bytes);
  // slices of one expert (the last one of an odd number of steps holds one step: its
  // second half is bytes of the next row or nothing, and is not read), of all
  const int ns1 = (o.nk1 + 1) / 2, ns = o.nexp * ns1;
  auto issue = [&](int stage, int kt) {
    const int ex = MODE == kDown4 ? kt / ns1 : 0, j = MODE == kDown4 ? kt - ex * ns1 : kt;
    const int ak = ex * o.ldw + j * BK, wk = ex * (int)o.w_one + j * BK;
    const int as = (ex * o.nk1 + 2 * j) * o.sa_stride, ws = ex * o.sw_one + 2 * j * o.sw_stride;
    uint8_t* sb = lds + stage * STAGE;
#pragma unroll
    for (int i = 0; i < A_CH; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(sb + i * 1024), 16, a_off[i], ak, 0, 0);
#pragma unroll
    for (int i = 0; i < B_CH; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(sb + BM * BK + i * 1024), 16, b_off[i], wk, 0, 0);
#pragma unroll
    for (int i = 0; i < SC_CH; ++i) {
      lds_void_t* dst = (lds_void_t*)(sb + SC_OFF + i * 256);
      if (i * 64 < 2 * BM) __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, dst, 4, s_off[i], as, 0, 0);
      else __builtin_amdgcn_raw_ptr_buffer_load_lds(rsw, dst, 4, s_off[i], ws, 0, 0);
    }
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < ns) issue(s, s);
  f32x4_t acc[MI][NI4];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI4; ++ni) acc[mi][ni] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int cur = 0, left = o.nk1;                           // K steps left of the current expert
  for (int kt = 0; kt < ns; ++kt) {
    wait_loads<PER, STAGES - 2>(min(ns - 1, kt + STAGES - 2) - kt);
    lds_barrier();
    if (kt + STAGES - 1 < ns) issue(cur == 0 ? STAGES - 1 : cur - 1, kt + STAGES - 1);
    const uint8_t* base = lds + cur * STAGE;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      if (kk == 1 && left < 2) break;
      const int ch = swz<CPR>(l16, kk * 4 + g) * 16, chw = swz_w(col_lane(l16), kk * 4 + g) * 16;
      const uint8_t* sca = base + SC_OFF + kk * BM * 4 + g;
      const uint8_t* scb = base + SC_OFF + (2 * BM + kk * BN) * 4 + g;
      i32x8_t fb[NI4];
      int sb[NI4];
#pragma unroll
      for (int ni = 0; ni < NI4; ++ni) {
        const int r = col_lane(l16) + col_off<MODE, BN>(ni);
        fb[ni] = frag4(base + BM * BK + r * BK + chw);
        sb[ni] = scb[r * 4];
      }
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        const i32x8_t fa = frag4(base + (l16 + mi * 16) * BK + ch);
        const int sa = sca[(l16 + mi * 16) * 4];
#pragma unroll
        for (int ni = 0; ni < NI4; ++ni) acc[mi][ni] = mfma_fp4(fb[ni], fa, acc[mi][ni], sb[ni], sa);
      }
    }
    left -= 2;
    if (left <= 0) left = o.nk1;
    cur = cur == STAGES - 1 ? 0 : cur + 1;
  }
  lds_barrier();                                       // the ring has been read
  if constexpr (MODE == kGateUp4) {
    uint8_t* hsc = lds + BM * kHPitch;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      uint32_t e;
      const uint32_t w = swiglu_codes(acc[mi], &e);
      stage_h(lds, hsc, l16 + mi * 16, 0, g, w, e);
    }
    lds_barrier();
    store_h<NT, 1>(p, d, part, o.shared, lds, hsc, lane);
  } else {
    bf16_t* out = reinterpret_cast<bf16_t*>(o.shared ? p.out_shared : p.out_routed);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
      store_y(lds, 1024, acc[mi], out, d.row0, mi * 16, d.rows, d.nt * kFp4BN2 + part * BN, p.H, lane);
  }
#endif
}

template <int MODE>
moe_status launch_gemm_fp4(const FfnLayout& L, int64_t max_tiles, const Fp4Params& p, hipStream_t st) {
  if (max_tiles == 0) return MOE_OK;
  if (L.bm1 == kFp4RowsBM) {
    const unsigned parts = 4 * (unsigned)grouped_grid(max_tiles, kStripeFp4);
    hipLaunchKernelGGL(gemm_fp4_rows_kernel<MODE>, dim3(parts), dim3(64), 0, st, p);
    return launch_status();
  }
  // one workgroup a CU (its LDS leaves no room for two), whole rounds of the 8 XCDs
  const int64_t grid = std::min<int64_t>(std::max(cu_count() / 8 * 8, 8), (int64_t)align_up((size_t)max_tiles, 8));
  hipLaunchKernelGGL(gemm_fp4_kernel<MODE>, dim3((unsigned)grid), dim3(kFp4Threads), 0, st, p);
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
  p.tile_rows = hdr + kFp4TileRows;
  p.T = c->T; p.H = c->H; p.E = c->E; p.S = c->S; p.I = c->I; p.k = c->k;
  if (phase == MOE_FFN_ALL || phase == MOE_FFN_GATE_UP) {
    // the tile tables, and x once in MXFP4: the shared experts' operand, and the routed one when its rows are gathered
    if (c->S > 0 || perm) s = launch_build_tiles_quantize_fp4(c, offsets, x, ws, st);
    else s = launch_build_tiles(c, offsets, ws, st);
    if (s != MOE_OK) return s;
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
