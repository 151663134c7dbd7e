// mx_linear.hip -- the linear on microscaled (MX) codes, gfx950 matrix cores.
//
//   y[m][n] = bf16( sum_b 2^(sa_mb + sw_nb - 254) sum_{k in block b} a_mk w_nk )
//
// The scaled matrix instructions multiply elements of either type and apply
// the two blocks' powers of two themselves, so codes and scale bytes go from
// memory to the matrix cores as they are: no decoding, no separate scaling.
//
// Operand layout of v_mfma_scale_f32_32x32x64_f8f6f4: lane (r = lane % 32,
// g = lane / 32) supplies row r.  4-bit elements: 16 bytes, block g of the
// two.  8-bit elements: bytes 16 g .. 16 g + 15 of block 0, then of block 1.
// Either way the lane's scale byte is that of block g.  Any assignment of
// the row's blocks to (instruction, g) will do that both operands share.
// (16x16x128: r = lane % 16, four groups g; 4-bit block g; 8-bit bytes 16 g of
// each 64-element half; scale of block g.)  The 32 x 32 form does the same
// work with half of the operand reads: 8.1 against 6.5 PFLOP/s for 4-bit
// elements, registers only.
//
// Two kernels.  Many rows: 64, 128 or 256 square tiles.  Codes go from memory
// straight to LDS, in stages of 128 bytes of a row (whole lines of the L2),
// several stages in a ring; the waves read fragments one step ahead of the
// products.  Few rows: no tile has enough of them to share, the weights are
// streamed once, K split over the waves of a workgroup.
//
// Measured (one MI355X): 32760 x 15360 x 5120, e2m1 both: 1.22-1.29 ms, 4.0-4.2
// PFLOP/s; e2m1 x e4m3: 1.87-1.91 ms, 2.7 PFLOP/s; e4m3 both: 2.03-2.18 ms, 2.4-2.5
// PFLOP/s; 32760 x 5120 x 13824, e4m3 x e2m1: 1.68 ms, 2.76 PFLOP/s.  The matrix instructions alone, on random registers,
// keep 6.6, 4.3 and 3.9 PFLOP/s on this card: power, not issue, is what bounds
// them (about 1.8 GHz under this load; the matrix cores are busy 57% of the
// time), and the requests for the next stage, drained at each barrier, take
// most of the rest (without them 1.04 ms); a quarter of them are for scales.  At the first of those sizes four
// waves of 128 x 128 took 1.26 ms, stages of 128 elements (64-byte pieces) with
// four of them in LDS 1.38, 256 x 128 tiles with three stages 1.51, 128 tiles
// 1.63.  2 x 30720 x 5120: 16.5 us, 5.1 TB/s of weights, the rate of a large
// copy.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "mx_codec.h"
#include "mx_stage.h"
#include "oq_internal.h"

namespace oq {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
// output pieces at any row length and address of y: the memory takes them at
// two-byte alignment
typedef uint32_t u32x4_y __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_y __attribute__((ext_vector_type(2), aligned(2)));

// Tile rows per group of the tile order: an XCD's resident tiles share 4 row
// blocks and 8 column blocks, and the 4 row blocks stay in its L2 while the
// columns pass (8 rows: 2% slower; 16: 7% to 17%).
constexpr int kGroupM = 4;

// A workgroup of 2 x WN waves computes a (64 IB) x (32 WN JB) tile; each wave
// a (32 IB) x (32 JB) block of it.
template <int FA, int FW, int WN_, int IB_, int JB_, int WGS_, int KS_, int NST_>
struct MxTile {
  static constexpr int WN = WN_, IB = IB_, JB = JB_, WGS = WGS_, NST = NST_;
  static constexpr int THREADS = 128 * WN;
  static constexpr int TM = 64 * IB, TN = 32 * WN * JB;
  static constexpr int KS = KS_;                                        // elements of K a stage
  static constexpr int STEPS = KS / 64;                                 // products in depth
  static constexpr int RA = KS / (FA ? 1 : 2), RW = KS / (FW ? 1 : 2);  // row bytes a stage
  static constexpr int AB = TM * RA, STAGE = AB + TN * RW;
  static constexpr int SROWS = TM + TN;
  static constexpr int SBUF = 4 * SROWS * 4;     // scales of 16 blocks: 4 planes of one word a row
  static constexpr int SPG = 512 / KS;           // stages that one such group lasts
  static constexpr int EPI = 32 * 64 * JB;       // a wave's 32 output rows on their way out
  static constexpr int SC0 = NST * STAGE, LDS = SC0 + 2 * SBUF;
  static_assert(2 * WN * EPI <= SC0, "the output goes through the stages' LDS");
  static_assert(LDS * WGS <= 160 * 1024, "LDS of one CU");
};

typedef __attribute__((address_space(3))) void lds_void;

// 64 lanes x 16 bytes from memory straight to LDS, lane after lane from `dst`
// (uniform); lanes outside the buffer write zeros.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rs, uint8_t *dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)dst, 16, off, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_and_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Group-major tile order: index g -> tile (tm, tn), kGroupM tile rows per
// group, column-major inside a group.
__device__ __forceinline__ void tile_of(int g, int nbm, int nbn, int &tm, int &tn) {
  const int gsz = kGroupM * nbn, grp = g / gsz, first = grp * kGroupM;
  const int gm = (nbm - first) < kGroupM ? (nbm - first) : kGroupM;
  tm = first + (g % gsz) % gm;
  tn = (g % gsz) / gm;
}

template <int FMT>
struct Frag {
  u32x4 v[FMT ? 2 : 1];
  __device__ __forceinline__ i32x8 op() const {
    const u32x4 h = v[FMT ? 1 : 0];
    return i32x8{(int)v[0][0], (int)v[0][1], (int)v[0][2], (int)v[0][3],
                 (int)h[0],    (int)h[1],    (int)h[2],    (int)h[3]};
  }
};

template <int FA, int FW, class TL>
__global__ __launch_bounds__(TL::THREADS, TL::WGS *TL::THREADS / 256) void mx_tile_kernel(
    const uint8_t *__restrict__ A, const uint8_t *__restrict__ As, const uint8_t *__restrict__ W,
    const uint8_t *__restrict__ Ws, int M, int N, int K, uint16_t *__restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int IB = TL::IB, JB = TL::JB, RA = TL::RA, RW = TL::RW;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int TH = TL::THREADS;
  const int wm = wave / TL::WN, wn = wave % TL::WN, r = lane & 31, g = lane >> 5;
  const int rowA = K / (FA ? 1 : 2), rowW = K / (FW ? 1 : 2), nb = K / 32;
  const int T = (K + TL::KS - 1) / TL::KS;
  const int nbm = (M + TL::TM - 1) / TL::TM, nbn = (N + TL::TN - 1) / TL::TN;
  const int count = nbm * nbn;

  // Loads of a stage: piece idx = tid + TH k of an operand
  using PieceA = MxPieces<RA, TH>;
  using PieceW = MxPieces<RW, TH>;
  constexpr int PA = TL::TM * PieceA::C, PW = TL::TN * PieceW::C;  // pieces
  constexpr int LA = PA / TH, LW = PW / TH, NL = LA + LW;
  // pieces requested in the last step of a stage, the others in the first of the
  // next (all of them in one burst: 3% slower)
  constexpr int LL = TL::STEPS == 4 ? NL / 2 : NL;
  constexpr int NST = TL::NST;
  static_assert(PA % TH == 0 && PW % TH == 0, "whole rounds of requests");
  const int ba0 = PieceA::byte(tid), bw0 = PieceW::byte(tid);
  const int uw = __builtin_amdgcn_readfirstlane(wave);
  const int la0 = uw * 1024, lw0 = TL::AB + uw * 1024;
  // Fragments.  Of a stage's 2 STEPS blocks, step j multiplies blocks j and
  // STEPS + j; lane (r, g) takes 4-bit block STEPS g + j, piece STEPS g + j
  // of the row, or of 8-bit blocks j (h = 0) and STEPS + j (h = 1) piece
  // 2 j + 4 h + g.  Pieces differ in the bits of j and h alone, which the
  // swizzle leaves exclusive-or apart.
  const int arow = wm * 32 * IB + r, wrow = wn * 32 * JB + r;
  const int fa0 = arow * RA + (((FA ? g : TL::STEPS * g) ^ mx_swizzle<RA>(r)) << 4);
  const int fw0 = TL::AB + wrow * RW + (((FW ? g : TL::STEPS * g) ^ mx_swizzle<RW>(r)) << 4);
  // the lane's scale bytes of a stage: blocks STEPS g .. STEPS g + STEPS - 1
  const int sp = TL::STEPS == 4 ? g * TL::SROWS * 4 : 2 * g;
  const int sa0 = TL::SC0 + 4 * arow + sp, sw0 = TL::SC0 + 4 * (TL::TM + wrow) + sp;

  struct Tile {
    int m0, n0, mr, nr;  // origin, rows and columns inside the matrix
    __amdgpu_buffer_rsrc_t a[LA], w[LW];  // of each round of requests
  };
  // each XCD takes a contiguous run of the tile order; rows past the last lie
  // outside the buffers
  auto tile_at = [&](int v) {
    const int xcd = v & 7, per = count >> 3, rem = count & 7;
    int tm, tn;
    tile_of(xcd * per + (xcd < rem ? xcd : rem) + (v >> 3), nbm, nbn, tm, tn);
    Tile x;
    x.m0 = tm * TL::TM, x.n0 = tn * TL::TN;
    x.mr = M - x.m0 < TL::TM ? M - x.m0 : TL::TM, x.nr = N - x.n0 < TL::TN ? N - x.n0 : TL::TN;
#pragma unroll
    for (int k = 0; k < LA; k++)
      x.a[k] = __builtin_amdgcn_make_buffer_rsrc(
          (void *)(A + (int64_t)x.m0 * rowA + PieceA::base(rowA, k)), 0, PieceA::size(x.mr, rowA, k), 0x00027000);
#pragma unroll
    for (int k = 0; k < LW; k++)
      x.w[k] = __builtin_amdgcn_make_buffer_rsrc(
          (void *)(W + (int64_t)x.n0 * rowW + PieceW::base(rowW, k)), 0, PieceW::size(x.nr, rowW, k), 0x00027000);
    return x;
  };
  // piece k of stage t of a tile into LDS stage `buf`: activations first.
  // Rows past the last, pieces past K and stages past the last lie outside the
  // buffers.
  const uint32_t offA = PieceA::row(tid) * rowA + ba0, offW = PieceW::row(tid) * rowW + bw0;
  auto load_piece = [&](const Tile &x, int t, int buf, int k) {
    uint8_t *b = lds + buf * TL::STAGE;
    if (k < LA)
      load_to_lds(x.a[k], b + la0 + k * (16 * TH), PieceA::offset(offA, ba0, rowA, t));
    else
      load_to_lds(x.w[k - LA], b + lw0 + (k - LA) * (16 * TH), PieceW::offset(offW, bw0, rowW, t));
  };

  for (int v = blockIdx.x; v < count; v += gridDim.x) {
    const Tile x = tile_at(v);
    const int m0 = x.m0, n0 = x.n0;

    // Scales: 32 blocks of a row are loaded at once (one request to the L2 for
    // most; their address has no alignment), 16 a time go to LDS.  A last,
    // partial group of 16 goes byte by byte, zero past K.
    constexpr int LS = (TL::SROWS + TH - 1) / TH;
    u32x4 sts[LS][2];
    auto group_rows = [&](const Tile &x, auto f) {
#pragma unroll
      for (int i = 0; i < LS; i++) {
        const int row = tid + TH * i;
        if (LS * TH == TL::SROWS || row < TL::SROWS) {
          const bool isw = row >= TL::TM;
          const int lr = isw ? row - TL::TM : row, n = (isw ? x.nr : x.mr) - 1;
          f(i, row, (isw ? Ws : As) + (int64_t)((isw ? x.n0 : x.m0) + (lr < n ? lr : n)) * nb);
        }
      }
    };
    auto load_groups = [&](const Tile &x, int grp) {  // grp even
      group_rows(x, [&](int i, int, const uint8_t *p) {
#pragma unroll
        for (int h = 0; h < 2; h++)
          if (16 * (grp + h) + 16 <= nb) {
            u32x4 s;
            __builtin_memcpy(&s, p + 16 * (grp + h), 16);
            sts[i][h] = s;
          }
      });
    };
    auto store_group = [&](const Tile &x, int grp) {
      uint8_t *b = lds + TL::SC0 + (grp & 1) * TL::SBUF;
      if (16 * grp + 16 <= nb) {
        auto put = [&](int h) {
          group_rows(x, [&](int i, int row, const uint8_t *) {
#pragma unroll
            for (int p = 0; p < 4; p++) *(uint32_t *)(b + (p * TL::SROWS + row) * 4) = sts[i][h][p];
          });
        };
        if (grp & 1) put(1);  // a constant index in each case: registers
        else put(0);
      } else {
        group_rows(x, [&](int, int row, const uint8_t *p) {
#pragma unroll 1
          for (int k = 0; k < 16; k++)
            b[((k >> 2) * TL::SROWS + row) * 4 + (k & 3)] = 16 * grp + k < nb ? p[16 * grp + k] : 0;
        });
      }
    };

    f32x16 acc[JB][IB];
#pragma unroll
    for (int j = 0; j < JB; j++)
#pragma unroll
      for (int i = 0; i < IB; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[j][i][e] = 0.f;

    Frag<FA> a[2][IB];
    Frag<FW> w[2][JB];
    int sa[IB], sw[JB], sa1[IB], sw1[JB];
    // LDS read k of a step's fragments, in the order its products need them
    constexpr int NRA = FA ? 2 : 1, NRW = FW ? 2 : 1, NR = JB * NRW + IB * NRA;
    auto read_frag = [&](int buf, int step, int k) {
      const uint8_t *b = lds + buf * TL::STAGE;
      const bool isa = k >= NRW && k < NRW + IB * NRA;  // w[0], every a, the other w
      if (isa) {
        const int i = (k - NRW) / NRA, h = (k - NRW) % NRA;
        a[step & 1][i].v[h] =
            *(const u32x4 *)(b + (fa0 ^ (FA ? step << 5 | h << 6 : step << 4)) + i * 32 * RA);
      } else {
        const int q = k < NRW ? k : k - IB * NRA, j = q / NRW, h = q % NRW;
        w[step & 1][j].v[h] =
            *(const u32x4 *)(b + (fw0 ^ (FW ? step << 5 | h << 6 : step << 4)) + j * 32 * RW);
      }
    };
    // scale bytes of stage t, read k: block STEPS g + j of it in byte j
    auto read_scale = [&](int t, int k) {
      const int blk = t * (TL::KS / 32);
      const uint8_t *b = lds + ((blk >> 4) & 1) * TL::SBUF + ((blk >> 2) & 3) * (TL::SROWS * 4);
      const bool isa = k >= 1 && k < 1 + IB;
      const int x = isa ? k - 1 : k < 1 ? 0 : k - IB;
      const uint8_t *p = b + (isa ? sa0 : sw0) + 128 * x;
      (isa ? sa1 : sw1)[x] = TL::STEPS == 4 ? *(const int *)p : *(const uint16_t *)p;
    };
    auto take_scales = [&] {
#pragma unroll
      for (int i = 0; i < IB; i++) sa[i] = sa1[i];
#pragma unroll
      for (int j = 0; j < JB; j++) sw[j] = sw1[j];
    };
    // product k of step S, column blocks first
    auto multiply = [&](auto step, int k) {
      constexpr int S = decltype(step)::value;
      const int j = k / IB, i = k % IB;
      acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          w[S & 1][j].op(), a[S & 1][i].op(), acc[j][i], FW ? 0 : 4, FA ? 0 : 4, S, sw[j], S, sa[i]);
    };

    wait_and_sync<63>();  // the previous tile's output has left LDS
    load_groups(x, 0);
#pragma unroll
    for (int t = 0; t < NST; t++)
#pragma unroll
      for (int k = 0; k < (t == NST - 1 ? LL : NL); k++) load_piece(x, t, t, k);
    store_group(x, 0);
    wait_and_sync<(NST - 2) * NL + LL>();
#pragma unroll
    for (int k = 0; k < NR; k++) read_frag(0, 0, k);
#pragma unroll
    for (int k = 0; k < IB + JB; k++) read_scale(0, k);
    take_scales();

    // One stage t: in each step but the last the next step's fragments are
    // read.  Before the last step a barrier sees stage t + 1 arrived and this
    // stage's LDS buffer read for the last time; in the last step the first
    // fragments and the scales of stage t + 1 are read, and from there to the
    // end of its first step stage t + NST is requested into this stage's buffer.
    // Each memory operation is pinned behind a product, evenly, so that the
    // matrix cores always have the next one.
    constexpr int NM = IB * JB;
    int cur = 0;
    auto step = [&](int t, int nxt, int prv, auto c) {
      constexpr int S = decltype(c)::value;
      constexpr bool LAST = S == TL::STEPS - 1;
      constexpr int R = LAST ? NR + IB + JB : NR;
      constexpr int L0 = LAST ? 0 : LL, L1 = LAST ? LL : S == 0 ? NL : LL;
#pragma unroll
      for (int k = 0; k < NM; k++) {
        multiply(c, k);
#pragma unroll
        for (int o = k * R / NM; o < (k + 1) * R / NM; o++) {
          if (!LAST) read_frag(cur, S + 1, o);
          else if (o < NR) read_frag(nxt, 0, o);
          else read_scale(t + 1, o - NR);
        }
        // pieces 0 .. LL of stage t + NST, or LL .. NL of the stage before it
#pragma unroll
        for (int o = L0 + k * (L1 - L0) / NM; o < L0 + (k + 1) * (L1 - L0) / NM; o++)
          load_piece(x, LAST ? t + NST : t + NST - 1, LAST ? cur : prv, o);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int t = 0; t < T; t++) {
      const int ph = t & (TL::SPG - 1), grp = t / TL::SPG;
      const bool more = (grp + 1) * 16 < nb;
      // (branches only here: the products below stay one block, in order)
      if (more && ph == 0 && (grp & 1)) load_groups(x, grp + 1);
      if (more && ph == TL::SPG / 2) store_group(x, grp + 1);
      const int nxt = cur + 1 == NST ? 0 : cur + 1, prv = cur == 0 ? NST - 1 : cur - 1;
      step(t, nxt, prv, std::integral_constant<int, 0>{});
      if constexpr (TL::STEPS == 4) {
        step(t, nxt, prv, std::integral_constant<int, 1>{});
        step(t, nxt, prv, std::integral_constant<int, 2>{});
      }
      wait_and_sync<(NST - 2) * NL>();
      step(t, nxt, prv, std::integral_constant<int, TL::STEPS - 1>{});
      take_scales();
      cur = nxt;
    }
    wait_and_sync<0>();  // the requests past the last stage are done, every buffer is free

    // Epilogue: 32 output rows of the wave's block at a time through the
    // wave's own LDS region (16-byte pieces XOR-swizzled by the row), out as
    // whole rows in 16-byte pieces.  Lane (r, g) holds row r, columns
    // 32 j + 8 q + 4 g + (0..3).
    uint8_t *reg = lds + wave * TL::EPI;
    constexpr int PPR = 4 * JB;  // pieces per row
    int lane_ = lane;  // opaque: keeps the addresses below out of the K loop's registers
    asm volatile("" : "+v"(lane_));
    const int er = lane_ & 31, eg = lane_ >> 5, c = lane_ % PPR;
    const int mw = m0 + wm * 32 * IB, n = n0 + wn * 32 * JB + 8 * c;
#pragma unroll
    for (int i = 0; i < IB; i++) {
#pragma unroll
      for (int j = 0; j < JB; j++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const bf16x2 p0 = {(__bf16)acc[j][i][4 * q], (__bf16)acc[j][i][4 * q + 1]};
          const bf16x2 p1 = {(__bf16)acc[j][i][4 * q + 2], (__bf16)acc[j][i][4 * q + 3]};
          *(u32x2 *)(reg + er * (64 * JB) + (((4 * j + q) ^ (er & (PPR - 1))) << 4) + 8 * eg) =
              u32x2{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1)};
        }
      __builtin_amdgcn_wave_barrier();  // LDS works in order within a wave
      const int m1 = mw + 32 * i;
#pragma unroll
      for (int k = 0; k < (32 * PPR + 63) / 64; k++) {
        const int rr = lane_ / PPR + k * (64 / PPR);
        const u32x4 o = *(const u32x4 *)(reg + rr * (64 * JB) + ((c ^ (rr & (PPR - 1))) << 4));
        uint16_t *yp = Y + (int64_t)(m1 + rr) * N + n;
        if (m1 + rr >= M || n >= N) continue;
        if (n + 8 <= N) {
          __builtin_nontemporal_store(o, (u32x4_y *)yp);
        } else {
#pragma unroll 1
          for (int e = 0; e < 8; e++) {
            const uint32_t d = e & 4 ? (e & 2 ? o[3] : o[2]) : e & 2 ? o[1] : o[0];
            if (n + e < N) yp[e] = (uint16_t)(d >> (16 * (e & 1)));
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Few rows: a workgroup of 8 waves computes 16 NB columns for 16 MB rows, the
// waves taking every eighth 256-element chunk of K, straight from memory to
// registers: the weights are read once and nothing is shared but the
// activations, which the caches hold.  The waves' sums meet in LDS, in wave
// order.
template <int FA, int FW, int MB, int NB>
__global__ __launch_bounds__(512) void mx_rows_kernel(
    const uint8_t *__restrict__ A, const uint8_t *__restrict__ As, const uint8_t *__restrict__ W,
    const uint8_t *__restrict__ Ws, int M, int N, int K, uint16_t *__restrict__ Y) {
  constexpr int WAVES = 8;
  __shared__ f32x4 part[WAVES][MB * NB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * NB), m0 = blockIdx.y * (16 * MB);
  const int rowA = K / (FA ? 1 : 2), rowW = K / (FW ? 1 : 2), nb = K / 32, C = (K + 255) / 256;
  const int mr = M - m0 < 16 * MB ? M - m0 : 16 * MB, nr = N - n0 < 16 * NB ? N - n0 : 16 * NB;
  // rows past the last and pieces past K lie outside the buffers: zeros
  const __amdgpu_buffer_rsrc_t ba = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(A + (int64_t)m0 * rowA), 0, mr * rowA, 0x00027000);
  const __amdgpu_buffer_rsrc_t bw = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(W + (int64_t)n0 * rowW), 0, nr * rowW, 0x00027000);

  // a row's operand of step 0 or 1 of a chunk
  auto load = [&](auto fmt, __amdgpu_buffer_rsrc_t b, int row, int rowb, int step) {
    constexpr int F = decltype(fmt)::value;
    Frag<F> f;
    const int at = step * (F ? 128 : 64) + 16 * g, off = row * rowb + at;
#pragma unroll
    for (int h = 0; h < (F ? 2 : 1); h++)
      f.v[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             b, at + 64 * h < rowb ? off + 64 * h : 0x7ffffff0, 0, 0));
    return f;
  };
  // the row's 8 scale bytes of a chunk, zero past K; the lane's are bytes g and 4 + g
  auto scales = [&](const uint8_t *p, int row, int last, int c) {
    p += (int64_t)(row < last ? row : last) * nb + 8 * c;
    u32x2 s = {0, 0};
    if (8 * c + 8 <= nb) {
      __builtin_memcpy(&s, p, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (8 * c + i < nb) s[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
    return s;
  };

  f32x4 acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; j++)
#pragma unroll
    for (int i = 0; i < MB; i++) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint8_t *as = As + (int64_t)m0 * nb, *ws = Ws + (int64_t)n0 * nb;
  for (int c = wave; c < C; c += WAVES) {
    Frag<FW> w[NB][2];
    Frag<FA> a[MB][2];
    u32x2 sw[NB], sa[MB];
#pragma unroll
    for (int j = 0; j < NB; j++) {
#pragma unroll
      for (int h = 0; h < 2; h++)
        w[j][h] = load(std::integral_constant<int, FW>{}, bw, 16 * j + r, rowW, 2 * c + h);
      sw[j] = scales(ws, 16 * j + r, nr - 1, c);
    }
#pragma unroll
    for (int i = 0; i < MB; i++) {
#pragma unroll
      for (int h = 0; h < 2; h++)
        a[i][h] = load(std::integral_constant<int, FA>{}, ba, 16 * i + r, rowA, 2 * c + h);
      sa[i] = scales(as, 16 * i + r, mr - 1, c);
    }
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int j = 0; j < NB; j++)
#pragma unroll
        for (int i = 0; i < MB; i++)
          acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              w[j][h].op(), a[i][h].op(), acc[j][i], FW ? 0 : 4, FA ? 0 : 4, 0,
              (int)(sw[j][h] >> (8 * g)), 0, (int)(sa[i][h] >> (8 * g)));
  }
#pragma unroll
  for (int j = 0; j < NB; j++)
#pragma unroll
    for (int i = 0; i < MB; i++) part[wave][j * MB + i][lane] = acc[j][i];
  __syncthreads();
#pragma unroll
  for (int b0 = 0; b0 < NB * MB; b0 += WAVES) {
    const int blk = b0 + wave;
    if (blk >= NB * MB) break;
    f32x4 y = part[0][blk][lane];
#pragma unroll
    for (int v = 1; v < WAVES; v++) y += part[v][blk][lane];
    const int m = m0 + 16 * (blk % MB) + r, n = n0 + 16 * (blk / MB) + 4 * g;  // four columns of a row
    if (m >= M) continue;
    uint16_t *yp = Y + (int64_t)m * N + n;
    if (n + 4 <= N) {
      const bf16x2 p0 = {(__bf16)y[0], (__bf16)y[1]}, p1 = {(__bf16)y[2], (__bf16)y[3]};
      *(u32x2_y *)yp = u32x2{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1)};
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (n + e < N) yp[e] = __builtin_bit_cast(uint16_t, (__bf16)y[e]);
    }
  }
}

template <int FA, int FW, int MB, int NB>
hipError_t launch_rows(const MxLinearArgs &a) {
  const int64_t gx = (a.N + 16 * NB - 1) / (16 * NB), gy = (a.M + 16 * MB - 1) / (16 * MB);
  if (gx > (1 << 22) || gy > 65535) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx_rows_kernel<FA, FW, MB, NB>), dim3((unsigned)gx, (unsigned)gy), dim3(512), 0,
                     a.stream, a.a_codes, a.a_scales, a.w_codes, a.w_scales, (int)a.M, (int)a.N,
                     a.K, a.y);
  return hipGetLastError();
}

template <int FA, int FW, class TL>
hipError_t launch_tiles(const MxLinearArgs &a, int cus) {
  static std::atomic<uint64_t> lds_set{0};  // per instantiation and device
  hipError_t e = ensure_lds_limit((const void *)mx_tile_kernel<FA, FW, TL>, TL::LDS, lds_set);
  if (e != hipSuccess) return e;
  const int64_t tiles = ((a.M + TL::TM - 1) / TL::TM) * ((a.N + TL::TN - 1) / TL::TN);
  if (tiles > INT32_MAX / 2) return hipErrorInvalidValue;
  const int64_t slots = (int64_t)cus * TL::WGS;
  hipLaunchKernelGGL((mx_tile_kernel<FA, FW, TL>), dim3((unsigned)(tiles < slots ? tiles : slots)),
                     dim3(TL::THREADS), TL::LDS, a.stream, a.a_codes, a.a_scales, a.w_codes, a.w_scales,
                     (int)a.M, (int)a.N, a.K, a.y);
  return hipGetLastError();
}

// Which kernel, by the number of 64 x 64, 128 x 128 tiles that the output has
// (us at K = 5120, e2m1 on both sides):
//   rows, up to 32 rows, or so few 64 tiles that they leave half of the CUs
//     without one (64 x 5120: 10.9 against 16.6); 32 columns a workgroup where
//     that still gives a workgroup to half of the CUs, else 16 (1 x 5120: 6.0
//     against 6.8; 64 x 1024 at K = 16384: 34 against 28.7)
//   64 tiles as long as all of them are resident, two a CU with three stages
//     each (128 x 5120: 13.1, 128 tiles 16.9; 256 x 13824, three a CU: 38, 30)
//   128 tiles, two a CU, or 256 tiles, one a CU: whichever needs less time for
//     its rounds over the CUs, a round of 128 tiles taken as 0.6 of one of 256
//     tiles (measured 0.54 at K = 512, 0.64 at K = 5120).  128 tiles: 509 x
//     13824: 26, 256 tiles 34; 6000 x 6000 at K = 3200, 5 against 3 rounds:
//     118, 125.  256 tiles: 2048 x 5120: 36, 128 tiles 44; 32768 x 4096 at K =
//     2048: 155, 187
template <int FA, int FW>
hipError_t launch_pair(const MxLinearArgs &a, int cus) {
  // a stage: 128 bytes of a row (64 of 4-bit weights against 8-bit
  // activations), so that a row's request is a whole line of the L2, and the
  // same matrix-core time either way (8-bit elements run at half rate);
  // 64-byte pieces in a deeper ring: 1.38 against 1.24 ms at 32760 x 15360 x 5120
  constexpr int KS = FA || FW ? 128 : 256;
  auto tiles = [&](int64_t t) { return ((a.M + t - 1) / t) * ((a.N + t - 1) / t); };
  const int64_t small = tiles(64);
  if ((a.M <= 32 && a.N <= 1 << 26) || 2 * small <= cus) {
    const bool wide = 2 * ((a.M + 63) / 64) * ((a.N + 31) / 32) > cus;
    if (a.M <= 16) return wide ? launch_rows<FA, FW, 1, 2>(a) : launch_rows<FA, FW, 1, 1>(a);
    if (a.M <= 32) return wide ? launch_rows<FA, FW, 2, 2>(a) : launch_rows<FA, FW, 2, 1>(a);
    return wide ? launch_rows<FA, FW, 4, 2>(a) : launch_rows<FA, FW, 4, 1>(a);
  }
  if (small <= 2 * cus) return launch_tiles<FA, FW, MxTile<FA, FW, 2, 1, 1, 2, KS, 3>>(a, cus);
  auto rounds = [](int64_t t, int64_t slots) { return (t + slots - 1) / slots; };
  if (3 * rounds(tiles(128), 2 * cus) <= 5 * rounds(tiles(256), cus))
    return launch_tiles<FA, FW, MxTile<FA, FW, 2, 2, 2, 2, KS, 2>>(a, cus);
  // three stages where they fit: 1.68 against 1.70 ms at 32760 x 5120 x 13824
  constexpr int NST = (FA || FW) && !(FA && FW) ? 3 : 2;
  return launch_tiles<FA, FW, MxTile<FA, FW, 4, 4, 2, 1, KS, NST>>(a, cus);
}

}  // namespace

hipError_t launch_mx_linear(const MxLinearArgs &a) {
  // CUs of the current device, asked once a device
  static std::atomic<int> known[64];
  int cus = 0, dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return hipErrorInvalidDevice;
  const bool slot = dev >= 0 && dev < 64;
  if (slot) cus = known[dev].load(std::memory_order_relaxed);
  if (cus <= 0) {
    const hipError_t e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    if (slot) known[dev].store(cus, std::memory_order_relaxed);
  }
  if (a.a_format == 0) return a.w_format == 0 ? launch_pair<0, 0>(a, cus) : launch_pair<0, 1>(a, cus);
  return a.w_format == 0 ? launch_pair<1, 0>(a, cus) : launch_pair<1, 1>(a, cus);
}

}  // namespace oq
