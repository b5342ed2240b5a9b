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
//
// Large batches: resident workgroups of 8 wavefronts, one a CU, each 144 or 64 rows x 64 columns of a tile of 288 or
// 128 x 256, whose direct-to-LDS loads run ahead through the tiles.  288 rows (2 stages of 128 columns, all that LDS
// holds) load the fewest bytes an operation; 128 rows (3 stages) waste fewer of short segments: the table's builder
// counts both and chooses (int8_tile_rows, ffn_layout.h).  T = 16384, H = 7168, 256 experts, 8 + 1 a token, I = 2048:
// gate/up 3.9 ms, down 2.15 ms, 2.1 POP/s over the whole call, at 1.8 GHz with the MFMAs busy 64% and 56% (a product of
// two large square matrices by the library reaches 2.3).  16 x 16 x 64 blocks: from registers alone they reach 4.2 to
// 4.3 POP/s on such operands, 32 x 32 x 32 ones 3.6 (4.9 either on zeros: the clock follows the power).
// Few rows an expert (the rule beside kInt8RowsAvg): 32-row tiles, bound by reading the weights once, 6.9 TB/s.
// 4 wavefronts of 128 x 128 7.0 ms a call against 6.2, loads staged through registers 6.8, weights touched ahead in
// the L2 7.3 to 8.5, loads issued before the stores 6.6; another K order a tile and another XCD run, none.
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
  const int32_t* tile_rows;   // rows per tile, and whether weights are read once (header entries kTileRows, kTileOnce)
  const int32_t* perm;        // gate/up: non-null -> routed rows gathered from a_shared / sa_shared
  int T, H, E, S, I, k;
};

#if defined(__HIP_DEVICE_COMPILE__)
constexpr int NI8 = 4;          // MFMA column blocks of a wavefront (few rows)
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

// The order of a wavefront's columns: blocks ni and ni + 1 (ni even) share 32 neighbouring columns, MFMA row 4 g + r
// of block ni being column 8 g + 4 (ni mod 2) + r of them, so that a lane holds 8 neighbouring columns of a row in two
// blocks: 16 bytes of bf16.  The first half of a gate/up wavefront's blocks are gate columns, the other half the up
// columns BN / 2 further on.  The tile column whose LDS row lane l16 reads is col_lane + col_off.
__device__ __forceinline__ int col_lane(int l16) { return 8 * (l16 >> 2) + (l16 & 3); }
template <int MODE, int NI, int BN>
__device__ __forceinline__ constexpr int col_off(int ni) {
  if (MODE == kGateUpI8) return (ni / (NI / 2)) * (BN / 2) + (ni % (NI / 2)) / 2 * 32 + (ni % 2) * 4;
  return (ni / 2) * 32 + (ni % 2) * 4;
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

// ------------------------------------------------------------------ large batches
constexpr int kInt8Threads = 512;
constexpr int kInt8Lds = 147456;

#if defined(__HIP_DEVICE_COMPILE__)
// v as a value that the compiler cannot compute ahead of this point (what a tile's begin and epilogue derive from the
// lane would otherwise be computed before the loops and held, or spilled, through them).
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The GEMM over tiles of BM rows; ONCE: weights past the caches.
template <int MODE, int BM, int STAGES, bool ONCE>
__device__ __forceinline__ void gemm_int8_tiles(const Int8Params& p, uint8_t* lds) {
  constexpr int WM = 2, WN = 4, NT = kInt8Threads, NW = NT / 64, BN = 256;
  constexpr int MI = BM / (WM * 16), NI = BN / (WN * 16), HALF = NI / 2;
  static_assert(WM * WN == NW && WM * MI * 16 == BM && BN == kInt8BN2, "tile shape");
  constexpr int BK = 128, CPR = BK / 16;               // bytes (two K steps) and 16-byte chunks of a row per slice
  constexpr int RPL = NT / CPR;                        // rows a load of all threads covers
  // loads per thread per slice; an odd number of 32 rows: A's last load is the first half of the wavefronts' alone
  constexpr int A_CH = (BM + RPL - 1) / RPL, B_CH = BN / RPL, PER = A_CH + B_CH;
  constexpr bool A_HALF = BM % RPL != 0;
  static_assert(RPL % 16 == 0 && BN % RPL == 0 && BM % (RPL / 2) == 0 && (!A_HALF || STAGES == 2), "the loads of a slice");
  constexpr int B_OFF = BM * BK, STAGE = B_OFF + BN * BK;
  static_assert(STAGES * STAGE <= kInt8Lds && B_CH >= 2, "LDS; the pieces that the down GEMM's outputs pass through");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, g = lane >> 4;

  // ------------------------------------------------------------ this workgroup's tiles
  // XCD x = b mod 8 takes an equal contiguous share of the shared tiles and then one of the routed tiles; its
  // workgroups take them in turn.
  const int n_real = __builtin_amdgcn_readfirstlane(p.ntiles[0]), n_rt = __builtin_amdgcn_readfirstlane(p.ntiles[4]);
  const int xcd = blockIdx.x & 7, per_s = (n_real - n_rt + 7) >> 3, per_r = (n_rt + 7) >> 3;
  const int s_cnt = min(max(n_real - n_rt - xcd * per_s, 0), per_s);
  const int r_cnt = min(max(n_rt - xcd * per_r, 0), per_r);
  const int step = gridDim.x >> 3;
  // the n-th of this workgroup: round n takes the next `step` positions of the share, turned by 5 n (an expert's row
  // tiles of one column follow each other, the last one shorter: without the turn a workgroup might get only long
  // ones)
  auto place = [&](int n) { return n * step + ((int)(blockIdx.x >> 3) + 5 * n) % step; };
  auto entry = [&](int q) { return q < s_cnt ? n_rt + xcd * per_s + q : xcd * per_r + q - s_cnt; };
  const int q_end = s_cnt + r_cnt;
  int nq = 0;                                          // the tile being loaded
  if (place(0) >= q_end) return;

  // ------------------------------------------------------------ the loads
  // The stream of slices runs STAGES - 1 slices ahead of the products, through the tiles.
  int ls = 0;                                          // stage the next slice goes to
  int left = 0;                                        // slices of the tile to load yet
  int in_l = 0, nk1 = 1;                               // slices of its current expert to load yet, of each
  int ak = 0, wk = 0, w_skip = 0;                      // scalar offsets of the next slice; to the next expert's first
  // A: an offset a load where rows are gathered, else one and the rows' distance; W: one, the rows' distance, and
  // what lies between gate and up rows
  constexpr int A_OFF = MODE == kGateUpI8 ? A_CH : 1;
  int a_off[A_OFF], b_off = 0, a_dist = 0, w_dist = 0, w_gap = 0;
  int pn[A_OFF];                                       // perm entries of this lane's rows in the tile after it
  const uint8_t *baseA = nullptr, *baseW = nullptr;
  int bytesA = 0, bytesW = 0;                          // 0 when the stream has ended: its loads are dropped
  const int lr = tid / CPR;
  auto load_perm = [&](int q) {
    if (MODE != kGateUpI8 || p.perm == nullptr || q >= q_end) return;
    const TileDesc d = tile_at(p, entry(q));
    if (d.seg == p.E) return;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(p.perm + d.row0, d.rows * 4);
#pragma unroll
    for (int i = 0; i < A_OFF; ++i) pn[i] = __builtin_amdgcn_raw_buffer_load_b32(r, (lr + i * RPL) * 4, 0, 0);
  };
  // the next tile's loads begin, if there is one
  auto next_tile = [&]() {
    const int q = place(nq);
    left = 0x7FFFFFFF;
    ak = wk = 0;
    bytesA = bytesW = 0;
    if (q >= q_end) return;
    const TileDesc d = tile_at(p, entry(q));
    const OperandsI8<MODE> o(p, d);
    const int ca = swz<CPR>(lr, tid % CPR) * 16, cw = swz_w(lr, tid % CPR) * 16;
    // (rows past the tile's lie past the descriptor: the range check drops their loads)
    if constexpr (MODE == kGateUpI8) {
#pragma unroll
      for (int i = 0; i < A_CH; ++i) {
        const int r = lr + i * RPL;
        a_off[i] = (r >= d.rows ? o.a_rows + 1 : o.gather ? pn[i] / p.k : r) * o.lda + ca;
      }
    } else {
      a_off[0] = lr * o.lda + ca;
      a_dist = RPL * o.lda;
    }
    b_off = o.ex * o.w_one + (o.c0 + lr) * o.ldw + cw;
    w_dist = RPL * o.ldw;
    w_gap = MODE == kGateUpI8 ? (p.I - 128) * o.ldw : 0;
    baseA = o.A; bytesA = o.a_bytes;
    baseW = o.W; bytesW = o.w_bytes;
    w_skip = o.w_one - o.nk1 * BK;
    in_l = nk1 = o.nk1;
    left = o.nk1 * o.nexp;
    load_perm(place(++nq));
  };
  // Load i of PER of the stream's next slice.  (Down: rows past the columns' end lie past the descriptor with the last
  // expert's scalar offset, and inside it, in the next expert's rows, with the others': read, but never stored.)
  struct Stream {                                      // (in scalar registers)
    __amdgpu_buffer_rsrc_t a, w;
    int ak, wk;
  };
  auto stream = [&]() {
    return Stream{make_rsrc(baseA, bytesA), make_rsrc(baseW, bytesW), __builtin_amdgcn_readfirstlane(ak),
                  __builtin_amdgcn_readfirstlane(wk)};
  };
  auto load_part = [&](const Stream& s, int i) {
    lds_void_t* dst =
        (lds_void_t*)(lds + ls * STAGE + wave * 1024 + (i < A_CH ? i * NT * 16 : B_OFF + (i - A_CH) * NT * 16));
    if (A_HALF && i == A_CH - 1 && wave >= NW / 2) return;
    if (i < A_CH)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s.a, dst, 16, MODE == kGateUpI8 ? a_off[i % A_OFF] : a_off[0] + i * a_dist,
                                               s.ak, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          s.w, dst, 16, b_off + (i - A_CH) * w_dist + ((i - A_CH) * RPL >= 128 ? w_gap : 0), s.wk, 0,
          ONCE ? kNonTemporal : 0);
  };
  // After a slice's loads.
  auto advance = [&]() {
    ak += BK;
    wk += BK;
    --left;
    ls = ls == STAGES - 1 ? 0 : ls + 1;
    if (MODE == kDownI8 && --in_l == 0) {              // the next shared expert's K range
      in_l = nk1;
      wk += w_skip;
    }
  };

  // ------------------------------------------------------------ the products
  // this lane's fragments in a stage: tile rows arow0 + 16 mi and brow + col_off(ni); lane group g supplies the
  // elements [16g, 16g + 16) of a step (the swizzles are the same for every block, and a row's second step is 64 bytes
  // away by exclusive or)
  const int arow0 = wm * MI * 16 + l16;
  const int brow = wn * (MODE == kGateUpI8 ? BN / WN / 2 : BN / WN) + col_lane(l16);
  const int a_lane = arow0 * BK + swz<CPR>(l16, g) * 16;
  const int b_lane = B_OFF + brow * BK + swz_w(col_lane(l16), g) * 16;
  constexpr int NB = MI % 3 == 0 ? 3 : 4, D = 2, R = NB - D;   // A fragments held, read ahead, multiplied over the barrier
  static_assert(MI % NB == 0 && MI >= NI, "the buffers rotate within a step; B's next step is read in one");
  i32x4_t fa[NB], fb[2][NI];                           // fragments of token rows; of the weights, in either K step
  auto read_a = [&](const uint8_t* stage, int kk, int mi) {
    fa[mi % NB] = *reinterpret_cast<const i32x4_t*>(stage + (a_lane ^ (kk * 64)) + mi * 16 * BK);
  };
  auto read_b = [&](const uint8_t* stage, int kk, int ni) {
    fb[kk][ni] = *reinterpret_cast<const i32x4_t*>(stage + (b_lane ^ (kk * 64)) + col_off<MODE, NI, BN>(ni) * BK);
  };
  int cs = 0;                                          // stage of the current slice
  auto read_first = [&]() {                            // a slice's first fragments
    const uint8_t* here = lds + cs * STAGE;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) read_b(here, 0, ni);
#pragma unroll
    for (int i = 0; i < D; ++i) read_a(here, 0, i);
  };
  auto load_slice = [&]() {
    if (left == 0) next_tile();
    const Stream s = stream();
#pragma unroll
    for (int i = 0; i < PER; ++i) load_part(s, i);
    advance();
  };
  // What follows a slice's reads: the next slice has landed, everywhere, and this one's stage is free.
  auto turn = [&]() {
    wait_vm<PER * (STAGES - 2)>();
    lds_barrier();
    cs = cs == STAGES - 1 ? 0 : cs + 1;
  };
  load_perm(place(0));
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) load_slice();
  wait_vm<PER * (STAGES - 2)>();
  lds_barrier();

  const int steps1 = (MODE == kDownI8 ? p.I : p.H) / BK;   // slices of an expert
  for (int nc = 0, qc = place(0); qc < q_end; qc = place(++nc)) {
    const TileDesc cd = tile_at(p, entry(qc));
    const int slices = MODE == kDownI8 && cd.seg == p.E ? p.S * steps1 : steps1;
    if (wm * MI * 16 >= cd.rows) {                     // no rows for this wavefront: it only loads
      for (int kt = 0; kt < slices; ++kt) {
        load_slice();
        turn();
      }
      continue;
    }
    const OperandsI8<MODE> o(p, cd);
    const int cl = wn * (MODE == kGateUpI8 ? BN / WN / 2 : BN / WN) + 8 * g;
    // the scales of this lane's columns and rows
    float sw[NI][4], sa[MI];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const int c = cl + col_off<MODE, NI, BN>(ni);    // (4 columns: all there, or none)
      const float* q = o.SW + (MODE == kGateUpI8 ? o.template wrow<BN>(p, 0, c) : min(o.c0 + c, o.ncols - 4));
#pragma unroll
      for (int r = 0; r < 4; ++r) sw[ni][r] = q[r];
    }
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      const int i = min(arow0 + mi * 16, cd.rows - 1);
      sa[mi] = o.SA[o.gather ? p.perm[cd.row0 + i] / p.k : i];
    }
    i32x4_t acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = i32x4_t{0, 0, 0, 0};
    // row block mi of a K step, what else is to be issued between the products
    auto multiply = [&](int mi, const i32x4_t (&b)[NI], auto also) {
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        acc[mi][ni] = mfma_i8(b[ni], fa[mi % NB], acc[mi][ni]);
        also(ni);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    read_first();
    for (int kt = 0; kt < slices; ++kt) {
      if (left == 0) next_tile();
      const uint8_t* here = lds + cs * STAGE;
      const Stream s = stream();
      // the slice's first K step, the loads of the slice to come between its products
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
        multiply(mi, fb[0], [&](int ni) {
          if (ni == 0) read_a(here, mi + D < MI ? 0 : 1, (mi + D) % MI);
          if (ni == 1 && mi < NI) read_b(here, 1, mi);
          const int i = PER * mi / MI + ni - 2;
          if (ni >= 2 && i < PER * (mi + 1) / MI) load_part(s, i);
        });
      advance();
      // the second, its last R row blocks over the barrier and the next slice's first reads
#pragma unroll
      for (int mi = 0; mi < MI - R; ++mi)
        multiply(mi, fb[1], [&](int ni) {
          if (ni == 0 && mi + D < MI) read_a(here, 1, mi + D);
        });
      turn();
      read_first();                                    // (not into the buffers in use; after a tile's last slice unused)
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < R; ++i) multiply(MI - R + i, fb[1], [](int) {});
    }
    static_assert(PER <= 2 * MI && NI == 4, "the loads fit between the products");
    // acc[mi][ni][r] holds C[i][j] with i = arow0 + 16 mi (token row), j in the order of col_off
    bf16_t* out = (o.shared ? p.out_shared : p.out_routed) + cd.row0 * (int64_t)o.ncols;
    const int lane = opaque(threadIdx.x) & 63, l16 = lane & 15, g = lane >> 4;
    auto packed = [](const float (&v)[8]) {
      return make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
    };
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      float v[8];
      if constexpr (MODE == kGateUpI8) {
        const int i = wm * MI * 16 + l16 + mi * 16;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gv = (float)acc[mi][e / 4][e % 4] * (sa[mi] * sw[e / 4][e % 4]);
          const float uv = (float)acc[mi][e / 4 + HALF][e % 4] * (sa[mi] * sw[e / 4 + HALF][e % 4]);
          v[e] = gv * gate_sigmoid(gv) * uv;
        }
        if (i < cd.rows) *reinterpret_cast<uint4*>(out + i * (int64_t)o.ncols + cd.nt * 128 + cl) = packed(v);
      } else {
        // 16 rows x 64 columns through two 1 KB pieces of the stage that is filled next, which only this wavefront's
        // own loads fill (8 rows each, 16-byte chunks XOR swizzled), so that whole 128-byte row segments are stored
        // (1.5% faster than halves of them).  (It reads back only what it wrote; its LDS operations complete in order.)
        uint8_t* stg = lds + ls * STAGE + B_OFF + wave * 1024;
#pragma unroll
        for (int b = 0; b < NI; b += 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = (float)acc[mi][b + e / 4][e % 4] * (sa[mi] * sw[b + e / 4][e % 4]);
          *reinterpret_cast<uint4*>(stg + (l16 >> 3) * NW * 1024 + (l16 & 7) * 128 + ((2 * b + g) ^ (l16 & 7)) * 16) =
              packed(v);
        }
        __builtin_amdgcn_s_waitcnt(kLgkmWaitZero);
        __builtin_amdgcn_wave_barrier();
        const int col = cd.nt * 256 + wn * 64 + (lane & 7) * 8;   // (ncols is a multiple of 128: whole segments)
#pragma unroll
        for (int it = 0; it < 2; ++it) {
          const int i = wm * MI * 16 + mi * 16 + it * 8 + (lane >> 3);
          const uint4 y = *reinterpret_cast<const uint4*>(stg + it * NW * 1024 + (lane >> 3) * 128 +
                                                         ((lane & 7) ^ (lane >> 3)) * 16);
          typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
          if (i < cd.rows && col < o.ncols)            // (non-temporal: 1% faster)
            __builtin_nontemporal_store(u32x4_t{y.x, y.y, y.z, y.w},
                                        reinterpret_cast<u32x4_t*>(out + i * (int64_t)o.ncols + col));
        }
        __builtin_amdgcn_s_waitcnt(kLgkmWaitZero);
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
}
#endif

// The table's builder chose the tiles' height from the rows that are there.
template <int MODE>
__global__ __launch_bounds__(kInt8Threads, 1) void gemm_int8_kernel(Int8Params p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(16))) uint8_t lds[kInt8Lds];
  const int bm = __builtin_amdgcn_readfirstlane(*p.tile_rows);
  const int once = __builtin_amdgcn_readfirstlane(p.tile_rows[kTileOnce - kTileRows]);
  if (bm != kTileLowBM) gemm_int8_tiles<MODE, kTileHighBM, 2, false>(p, lds);
  else if (once) gemm_int8_tiles<MODE, kTileLowBM, 3, true>(p, lds);
  else gemm_int8_tiles<MODE, kTileLowBM, 3, false>(p, lds);
#endif
}

// ------------------------------------------------------------------ few rows per expert
// The weights are read once, and past the caches (non-temporal loads: T = 128, H = 7168, 256 experts the whole call 1831
// -> 1650 us, 6.9 TB/s; T = 1 97 -> 87; 4 / 3 stages a workgroup 87 / 81).
// One workgroup of WM x WN wavefronts a tile (PARTS > 1: a part of one) of WM * MI * 16 token rows x WN * 64
// weight rows.  K advances 128 bytes a slice through a ring of STAGES LDS stages filled by direct-to-LDS loads
// (16-byte chunks, XOR swizzle per row), one barrier a slice.
template <int MODE, int WM, int WN, int MI, int STAGES, int PARTS>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_int8_rows_kernel(Int8Params p) {
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
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(sb + BM * BK + i * NT * 16), 16, b_off[i], wk, 0,
                                               kNonTemporal);
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
          fb[ni] = *reinterpret_cast<const i32x4_t*>(base + (BM + brow + col_off<MODE, NI8, BN>(ni)) * BK +
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
      sw[ni][r] = o.SW[o.template wrow<BN>(
          p, part, wn * (MODE == kGateUpI8 ? 32 : 64) + 8 * g + col_off<MODE, NI8, BN>(ni) + r)];
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
  if (max_tiles == 0) return MOE_OK;
  if (L.bm1 == kInt8RowsBM) {
    const unsigned parts = 4 * (unsigned)grouped_grid(max_tiles, kStripeInt8);
    hipLaunchKernelGGL((gemm_int8_rows_kernel<MODE, 1, 1, 2, 3, 4>), dim3(parts), dim3(64), 0, st, p);
    return launch_status();
  }
  // one workgroup a CU (its LDS leaves no room for two), whole rounds of the 8 XCDs
  const int64_t grid = std::min<int64_t>(std::max(cu_count() / 8 * 8, 8), (int64_t)align_up((size_t)max_tiles, 8));
  hipLaunchKernelGGL(gemm_int8_kernel<MODE>, dim3((unsigned)grid), dim3(kInt8Threads), 0, st, p);
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
  p.tile_rows = hdr + kTileRows;
  p.T = c->T; p.H = c->H; p.E = c->E; p.S = c->S; p.I = c->I; p.k = c->k;
  if (phase == MOE_FFN_ALL || phase == MOE_FFN_GATE_UP) {
    // the tile tables, and x once in int8, unless the caller has it: the shared experts' operand, and the routed one
    // when its rows are gathered
    const bool quantise = !x_codes && (c->S > 0 || perm);
    s = quantise ? launch_build_tiles_quantize_int8(c, offsets, x, ws, st) : launch_build_tiles(c, offsets, ws, st);
    if (s != MOE_OK) return s;
    if (quantise) {
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
    s = launch_quantize_int8_pair(
        Int8Rows{hb, pairs(c), c->I, base + L.off_hp, floats(L.off_hps)},
        Int8Rows{hbs, c->S > 0 ? c->T : 0, c->S * c->I, base + L.off_hs, floats(L.off_hss)}, offsets + c->E, st);
    if (s != MOE_OK) return s;
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
