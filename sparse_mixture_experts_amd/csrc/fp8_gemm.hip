// fp8_gemm.hip -- products of e4m3 codes with one fp32 scale per 128
// reduction elements (activations: per row; weights: per 128 x 128 block),
// grouped by expert:
//   y[p][n] = sum_b sa[b][r] sw[e][n / 128][b] sum_{k in block b} a[r][k] w[e][n][k],
// r = row_map[p] (or p), e the expert whose range of rows holds p.
//
// The sum over one block is one v_mfma_f32_16x16x128_f8f6f4 or four
// v_mfma_f32_16x16x32_f16 (fp8_common.h), started from zero, whose four
// results per lane one fma each brings to the running fp32 sum with the
// block's scale: 16 vector cycles beside 32 or 64 matrix cycles.  Operand a
// holds 16 weight rows n and operand b 16 token rows, so a lane's results are
// 4 consecutive outputs of one token and its scale is one value.  Lane group
// g = lane / 16 holds bytes 16 g .. +15 and 64 + 16 g .. +15 of the 128 (of
// both operands).
//
// Four kernels, by rows per expert: the decode kernel (16 rows a tile), the
// tile kernel (32, 48 or 64), and for the 8-bit instruction the wide and the
// huge one (128 and 256); a fifth holds the tile and the wide one, for experts
// of unequal numbers of rows.  Where an expert has few rows the weights' bytes
// are the bound, so they are loaded as they lie in memory, whole 128-byte
// rows, several blocks ahead of their use, and turned into the operand's
// layout through LDS.  (Loaded in the operand's layout directly, neighbouring
// lanes are in different rows and every load met 64 cache lines: about 28 ns
// of a CU's address path each, which bounded all four kernels.)
#include <algorithm>
#include <climits>

#include "fp8_common.h"
#include "launch.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kNW = kThreads / kWave;
constexpr int kNT = 4;                    // 16-row weight tiles per wave of the tile kernel
constexpr int kBN = kNW * kNT * 16;       // weight rows per workgroup (256)
constexpr int kPieces = kFp8Block / 16;   // 16-byte pieces per row and block (8)
constexpr int kWideRows = 128;            // rows of the wide tile
constexpr int kWideFrom = 96;             // rows of an expert from which the mixed kernel takes them
constexpr int kBigTile = 1 << 30;         // my_work: a wide tile among small ones

__device__ __forceinline__ uint4 keep(const uint4 &v, bool ok) {
  return make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
}

// 16 bytes per lane from memory to consecutive places of LDS (1 KB a wave).
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;
__device__ __forceinline__ void to_lds(const uint8_t *src, uint8_t *dst) {
  __builtin_amdgcn_global_load_lds((global_void *)src, (lds_void *)dst, 16, 0, 0);
}
// Rows of 128 codes in LDS: piece c (16 bytes) of row m lies at place
// c ^ (m % 8), which puts the pieces that 8 lanes read together, one of 8
// rows each, on different banks.  Byte offset of piece c of row m:
__device__ __forceinline__ uint32_t piece_at(int m, int c) { return uint32_t(m * kFp8Block + ((c ^ (m & 7)) * 16)); }
// A wave's 1 KB covers 8 rows; the piece that lane l brings for its place.
__device__ __forceinline__ int piece_of_lane(int l) { return (l % kPieces) ^ (l / kPieces); }

// Two weight tiles hold 32 rows in turn by fours: row r of tile nt is row
// 8 (r / 4) + 4 (nt % 2) + r % 4 of the pair's, so that a lane's results of
// the two are 8 neighbouring outputs: 16 bytes of 16-bit ones, 64 a row and
// store, where single tiles wrote 8 and 32 (8192 x 5632 x 2048: 125 us, 115
// with pairs).  pair_key: the exchange of a row's pieces in LDS that keeps
// reads in this order on different banks.
__device__ __forceinline__ int pair_row(int nt, int r) { return nt / 2 * 32 + 8 * (r / 4) + 4 * (nt % 2) + r % 4; }
__device__ __forceinline__ int pair_key(int m) { return (m & 3) | ((m >> 3) & 1) << 2; }

// One 16 x 128 tile of weight codes on its way from memory to the operand
// layout.  Loaded as it lies in memory (8 lanes to the 128 bytes of a row, so
// that an instruction meets 8 cache lines; in the operand's own layout
// neighbouring lanes are in different rows, and each load met 64), it is
// turned around through a piece of LDS that only this wave uses.
constexpr int kTileBytes = 16 * kFp8Block;
template <bool PAIR>
__device__ __forceinline__ uint32_t weight_at(int m, int c) {
  return PAIR ? uint32_t(m * kFp8Block + (c ^ pair_key(m)) * 16) : piece_at(m, c);
}
struct WeightTile {
  uint4 v[2];
  // base: the tile's first row; k0: the block's first code.  Past the end of
  // the reduction the codes are zero (a stray one may be a NaN).
  __device__ __forceinline__ void load(const uint8_t *base, int K, int k0) {
    const int lane = lane_id(), k = min(k0 + lane % kPieces * 16, K - 16);
    const uint32_t o = uint32_t(lane / kPieces) * uint32_t(K) + uint32_t(k);
    v[0] = *reinterpret_cast<const uint4 *>(base + o);
    v[1] = *reinterpret_cast<const uint4 *>(base + 8 * int64_t(K) + o);
  }
  // PAIR: for reads in the order of pair_row
  template <bool PAIR = false>
  __device__ __forceinline__ void put(uint8_t *lds, int K, int k0) const {
    const int lane = lane_id(), m = lane / kPieces, c = lane % kPieces;
    const bool ok = k0 + c * 16 < K;
    *reinterpret_cast<uint4 *>(lds + weight_at<PAIR>(m, c)) = keep(v[0], ok);
    *reinterpret_cast<uint4 *>(lds + weight_at<PAIR>(m + 8, c)) = keep(v[1], ok);
  }
};
// Tile nt of those that follow one another in `lds`.
template <bool PAIR = false>
__device__ __forceinline__ i32x8 tile_operand(const uint8_t *lds, int nt) {
  const int lr = lane_id() & 15, lg = lane_id() >> 4, m = PAIR ? pair_row(nt, lr) : nt * 16 + lr;
  return join8(*reinterpret_cast<const uint4 *>(lds + weight_at<PAIR>(m, lg)),
               *reinterpret_cast<const uint4 *>(lds + weight_at<PAIR>(m, lg + 4)));
}

// What a projection writes: the product, or the gated unit of two of them
// (as e4m3 codes per 128 columns from the tile kernel, as fp32 rows from the
// decode kernel).
constexpr int kPlain = 0, kGated = 1;

struct Fp8Args {
  const void *a;             // codes [a_rows][K]
  const float *as;           // [blocks][a_rows]
  int64_t a_rows;
  const int32_t *row_map;    // null: row p is p
  int rows, N, K;            // output rows, output columns, reduction
  int T, n_routed;           // layer: rows past n_routed are shared experts' (token (p - n_routed) % T)
  const uint8_t *w0, *w1;    // [E][N][K]; gated: gate (or [gate | up]) and up
  const float *s0, *s1;      // [E][ceil(N/128)][ceil(K/128)]
  int fused;                 // gated: w0 holds [gate | up]
  int round, geglu;          // gated: per-op rounding mode, tanh-GELU gate
  int E;
  const int32_t *expert_off; // null: one expert has all rows
  const PlanItem *tiles;     // layer: the work plan (expert_off unused)
  const int32_t *counters;
  void *out;                 // plain: [rows][N] out_dtype; gated: h (codes or fp32) [rows][N]
  int out_dtype;
  float *hs;                 // gated tile kernel: h scales [ceil(N/128)][rows]
};

// Tiles of bm rows that n rows (any count of an int) take.
__device__ __forceinline__ int tiles_in(int n, int bm) { return int((unsigned(n) + unsigned(bm) - 1) / unsigned(bm)); }

// This workgroup's row tile and column block (false: none is left).  Each
// XCD takes one contiguous range of the work, ordered in groups of 8 column
// blocks with the tiles of an expert together, so that what neighbours share
// (a tile's rows, an expert's weights) is read into one L2.
//
// Without a plan the tiles are found here, by every wave: the experts' rows
// in tiles of bm are counted 64 at a time, one prefix sum gives the number of
// tiles, and the lane whose range holds this one's number looks it up.
// Ranges are read as if clamped to [0, rows].
//
// `wide`: experts with at least that many rows are in tiles of kWideRows
// (their rows come with kBigTile), which all go before the others' tiles: a
// long workgroup that starts last would be waited for.
template <bool MIXED = false>
__device__ __forceinline__ bool my_work(const Fp8Args &a, int bm, int nbx, PlanItem &t, int &bx, int wide = 0) {
  int lin = int(blockIdx.x);
  const int lane = lane_id();
  int n_tiles, incl = 0, n = 0, e0 = 0, e1 = 0;
  bool big = false;  // MIXED: this workgroup's tile is a wide one
  auto range = [&](int e, int &lo, int &hi) {
    lo = min(max(a.expert_off[e], 0), a.rows);
    hi = min(max(a.expert_off[e + 1], lo), a.rows);
  };
  if (a.tiles) {
    n_tiles = a.counters[1];
  } else if (a.expert_off) {
    const int per = (a.E + kWave - 1) / kWave;
    e0 = lane * per, e1 = min(e0 + per, a.E);
    int nw = 0;
    for (int e = e0; e < e1; ++e) {
      int lo, hi;
      range(e, lo, hi);
      if (MIXED && hi - lo >= wide) nw += tiles_in(hi - lo, kWideRows);
      else n += tiles_in(hi - lo, bm);
    }
    if constexpr (MIXED) {
      const int inclw = wave_incl_scan(nw), first = read_lane_i(inclw, kWave - 1) * nbx;
      big = lin < first;
      if (!big) lin -= first;
      incl = wave_incl_scan(big ? nw : n);
      n = big ? nw : n;
    } else {
      incl = wave_incl_scan(n);
    }
    n_tiles = read_lane_i(incl, kWave - 1);
  } else {
    n_tiles = tiles_in(a.rows, bm);
  }
  const int work = n_tiles * nbx;  // the grid has at least as many workgroups
  if (lin >= work) return false;
  int tile;
  item_tile_block(xcd_contiguous(lin, work), n_tiles, nbx, min(nbx, kColGroup), tile, bx);
  if (a.tiles) {
    t = a.tiles[tile];
  } else if (a.expert_off) {
    const int m = big ? kWideRows : bm;
    int at = incl - n, fe = 0, frow = 0, frows = 0;
    if (tile >= at && tile < incl) {
      for (int e = e0; e < e1; ++e) {
        int lo, hi;
        range(e, lo, hi);
        const int k = MIXED && (hi - lo >= wide) != big ? 0 : tiles_in(hi - lo, m);
        if (tile < at + k) {
          fe = e;
          frow = lo + (tile - at) * m;
          frows = min(m, hi - frow);
          break;
        }
        at += k;
      }
    }
    const int src = __builtin_ctzll(__ballot(incl > tile));
    t.expert = read_lane_i(fe, src);
    t.row0 = read_lane_i(frow, src);
    t.rows = read_lane_i(frows, src);
  } else {
    t.expert = 0;
    t.row0 = tile * bm;
    t.rows = min(bm, a.rows - t.row0);
  }
  t.expert = __builtin_amdgcn_readfirstlane(t.expert);
  t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  if (MIXED && big) t.rows |= kBigTile;
  return true;
}

// Source row of output row p, or -1 when the map points outside.
__device__ __forceinline__ int source_row(const Fp8Args &a, int p) {
  int r = p;
  if (a.T && p >= a.n_routed) r = (p - a.n_routed) % a.T;
  else if (a.row_map) r = a.row_map[p];
  return unsigned(r) < unsigned(a.a_rows) ? r : -1;
}

// Four consecutive outputs of one row.
__device__ __forceinline__ void store4(const Fp8Args &a, int64_t at, const fp8_acc &v) {
  if (a.out_dtype == MOE_DT_F32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = a.out_dtype == MOE_DT_F16 ? f32_to_f16_bits(v[i]) : f32_to_bf16_bits(v[i]);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
        make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
}

// Eight consecutive outputs of one row, 16 bits each.
__device__ __forceinline__ void store8(const Fp8Args &a, int64_t at, const fp8_acc &u, const fp8_acc &v) {
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = a.out_dtype == MOE_DT_F16 ? f32_to_f16_bits(u[i]) : f32_to_bf16_bits(u[i]);
    h[4 + i] = a.out_dtype == MOE_DT_F16 ? f32_to_f16_bits(v[i]) : f32_to_bf16_bits(v[i]);
  }
  *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at) =
      make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

// The tile of 16 RB token rows (32, 48 or 64) by 256 weight rows.  Weights
// and rows are requested two blocks ahead of their use, into two sets of
// registers: with one block in flight a workgroup waited out a memory round
// trip per block.  EXACT: see Fp8Operand.  Bound by the weights' bytes: gate
// and up of 512 experts of 2048 x 512 at 40 rows each (1.07 GB) take 238 us
// with the exact sums, 4.5 TB/s, and down (0.54 GB and 168 MB of results)
// 151 us, 4.7 TB/s, where a large copy reaches 5.1.
template <int RB, bool EXACT>
struct TileLds {
  static constexpr int BM = RB == 2 ? 32 : 64;  // rows that are staged (zeros past the tile's)
  // rows in LDS: codes, or (EXACT) fp16, turned into it once here instead of
  // by every wave for every weight tile; 16 bytes of padding put the pieces
  // that 16 lanes read together, one of 16 rows each, on different banks
  static constexpr int XB = EXACT ? 2 : 1, ROW = kFp8Block * XB + 16;
  static constexpr int NSL = kThreads / BM;     // one scale per thread
  using Rows = uint8_t[2][BM][ROW];
  using Scales = float[2][NSL][BM];             // row scale * weight scale
  using Max = float[kNW][BM];
};
using Turn = uint8_t[kNW][kNT][kTileBytes];
template <int RB, int MODE, bool EXACT>
__device__ __forceinline__ void tile_body(const Fp8Args &a, const PlanItem &tile, int bx, typename TileLds<RB, EXACT>::Rows &sa,
                                          Turn &turn, typename TileLds<RB, EXACT>::Scales &ss,
                                          typename TileLds<RB, EXACT>::Max &rmax) {
  constexpr int BM = TileLds<RB, EXACT>::BM, XB = TileLds<RB, EXACT>::XB, NSL = TileLds<RB, EXACT>::NSL;
  constexpr bool PAIR = MODE == kPlain && !EXACT;   // (16-bit results)
  constexpr int NP = 2;                             // weight tiles that a read of the rows serves
  constexpr int PPT = BM * kPieces / kThreads;      // 16-byte pieces of the rows per thread
  constexpr int NTH = MODE == kGated ? kNT / 2 : kNT;
  constexpr int COLS = kNW * NTH * 16;              // output columns per workgroup
  // weight scale blocks that a workgroup meets: 256 rows cover two; gated:
  // one of gate rows, and two of up rows when they start inside a block
  constexpr int NS = MODE == kGated ? 3 : 2;
  static_assert(NS <= NSL && RB * 16 <= BM, "one scale per thread");
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = lane_id();
  const int lr = lane & 15, lg = lane >> 4;
  const int K = a.K, nb = (K + kFp8Block - 1) / kFp8Block;
  const int col0 = (bx * kNW + wave) * NTH * 16;    // first output column of this wave
  const int n_rows = MODE == kGated && a.fused ? 2 * a.N : a.N;  // rows of one expert's matrix
  const int nbr = (n_rows + kFp8Block - 1) / kFp8Block;

  // each weight tile's first row (clamped; what a tile past the end computes
  // is not stored) and which of the NS scales it takes
  const uint8_t *wp[kNT];
  int sidx[kNT];
  const int up0 = MODE == kGated && a.fused ? a.N : 0;
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    const bool up = MODE == kGated && nt >= NTH;
    const int col = min(col0 + (nt % NTH) * 16, a.N - 16);
    const int row = col + (up ? up0 : 0);
    wp[nt] = (up && !a.fused ? a.w1 : a.w0) + (int64_t(tile.expert) * n_rows + row) * K;
    const int blk = MODE == kGated ? (up ? 1 + row / kFp8Block - (up0 + bx * COLS) / kFp8Block : 0)
                                   : col / kFp8Block - bx * (COLS / kFp8Block);
    sidx[nt] = __builtin_amdgcn_readfirstlane(min(max(blk, 0), NS - 1));
  }
  // staging of the rows' codes: pass p of a thread -> row 32 p + tid / 8, piece tid % 8
  const int piece = tid % kPieces;
  const uint8_t *ap[PPT];
  bool aok[PPT];
#pragma unroll
  for (int p = 0; p < PPT; ++p) {
    const int m = p * (kThreads / kPieces) + tid / kPieces;
    const int r = m < tile.rows ? source_row(a, tile.row0 + m) : -1;
    aok[p] = r >= 0;
    ap[p] = static_cast<const uint8_t *>(a.a) + int64_t(max(r, 0)) * K;
  }
  // staging of the scales: thread -> scale tid / BM, row tid % BM
  const int sm = tid % BM, sn = min(tid / BM, NS - 1);
  const int srow = sm < tile.rows ? source_row(a, tile.row0 + sm) : -1;
  const float *sap = a.as + max(srow, 0), *swp;
  {
    const int blk = MODE == kGated ? (sn == 0 ? bx * COLS / kFp8Block : (up0 + bx * COLS) / kFp8Block + sn - 1)
                                   : bx * (COLS / kFp8Block) + sn;
    const float *base = MODE == kGated && sn > 0 && !a.fused ? a.s1 : a.s0;
    swp = base + (int64_t(tile.expert) * nbr + min(blk, nbr - 1)) * nb;
  }

  WeightTile wq[2][kNT];
  uint4 stg[2][PPT];
  float sga[2], sgw[2];
  // (blocks past the end repeat the last one: those loads hit the cache, and
  // keeping them keeps the waits of every step the same)
  auto load_rows = [&](int s, int r) {
    s = min(s, nb - 1);
    const int k = min(s * kFp8Block + piece * 16, K - 16);
#pragma unroll
    for (int p = 0; p < PPT; ++p) stg[r][p] = *reinterpret_cast<const uint4 *>(ap[p] + k);
    sga[r] = sap[int64_t(s) * a.a_rows];
    sgw[r] = swp[s];
  };
  auto load_weights = [&](int s, int r) {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) wq[r][nt].load(wp[nt], K, min(s, nb - 1) * kFp8Block);
  };
  auto stage = [&](int s, int r) {  // block s from registers r into buffer r
    const int k = s * kFp8Block + piece * 16;
#pragma unroll
    for (int p = 0; p < PPT; ++p) {
      const uint4 v = keep(stg[r][p], aok[p] && k < K);
      uint4 *to = reinterpret_cast<uint4 *>(&sa[r][p * (kThreads / kPieces) + tid / kPieces][piece * 16 * XB]);
      if constexpr (EXACT) to[0] = fp8_to_f16(v.x, v.y), to[1] = fp8_to_f16(v.z, v.w);
      else to[0] = v;
    }
    // (without a branch: one here lets the compiler move a step's sums past
    // it, with all its products in registers until then)
    ss[r][tid / BM][sm] = srow >= 0 ? sga[r] * sgw[r] : 0.f;
  };

  fp8_acc acc[kNT][RB];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
    for (int mt = 0; mt < RB; ++mt) acc[nt][mt] = fp8_acc{0.f, 0.f, 0.f, 0.f};

  auto step = [&](int s, auto rc) {
    constexpr int r = decltype(rc)::value;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) wq[r][nt].template put<PAIR>(turn[wave][nt], K, s * kFp8Block);
    // (the loads stay behind the last use of the registers that they fill)
    __builtin_amdgcn_sched_barrier(0);
    load_rows(s + 2, r);
    load_weights(s + 2, r);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int np = 0; np < kNT; np += NP) {
      const Fp8Operand<EXACT> w0(tile_operand<PAIR>(turn[wave][0], np)), w1(tile_operand<PAIR>(turn[wave][0], np + NP - 1));
#pragma unroll
      for (int mt = 0; mt < RB; ++mt) {
        const uint4 *row = reinterpret_cast<const uint4 *>(&sa[r][mt * 16 + lr][lg * 16 * XB]);
        const auto x = [&] {
          if constexpr (EXACT) return Fp8Operand<true>(row[0], row[1], row[8], row[9]);
          else return Fp8Operand<false>(join8(row[0], row[4]));
        }();
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          const fp8_acc d = fp8_product(q ? w1 : w0, x);
          const float sc = ss[r][sidx[np + q]][mt * 16 + lr];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[np + q][mt][i] = __builtin_fmaf(d[i], sc, acc[np + q][mt][i]);
        }
        if (EXACT && RB == 4 && mt % 2) __builtin_amdgcn_sched_barrier(0);  // (more reads ahead would not fit the registers)
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    stage(s + 1, 1 - r);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
  };
  using R0 = std::integral_constant<int, 0>;
  using R1 = std::integral_constant<int, 1>;
  load_rows(0, 0);
  load_weights(0, 0);
  load_rows(1, 1);
  load_weights(1, 1);
  stage(0, 0);
  __syncthreads();
  int st = 0;
  for (; st + 1 < nb; st += 2) {
    step(st, R0{});
    step(st + 1, R1{});
  }
  if (st < nb) step(st, R0{});

  if constexpr (MODE == kPlain) {
#pragma unroll
    for (int mt = 0; mt < RB; ++mt) {
      const int m = mt * 16 + lr;
      if (m < tile.rows) {
        // (codes of zero are not enough where a weight is a NaN)
        const bool ok = source_row(a, tile.row0 + m) >= 0;
        const fp8_acc z = {0.f, 0.f, 0.f, 0.f};
        const int64_t at = int64_t(tile.row0 + m) * a.N + col0;
        if constexpr (PAIR) {
#pragma unroll
          for (int nt = 0; nt < kNT; nt += 2)
            if (col0 + nt * 16 + 8 * lg < a.N)
              store8(a, at + nt * 16 + 8 * lg, ok ? acc[nt][mt] : z, ok ? acc[nt + 1][mt] : z);
        } else {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
            if (col0 + nt * 16 < a.N) store4(a, at + nt * 16 + 4 * lg, ok ? acc[nt][mt] : z);
        }
      }
    }
  } else {
    // h = the gated unit, its maxima over the workgroup's 128 columns, codes
    const bool ok[2] = {col0 < a.N, col0 + 16 < a.N};
#pragma unroll
    for (int mt = 0; mt < RB; ++mt) {
      float mx = 0.f;
      with_glu(a.round, a.geglu, [&](auto rt, auto gt) {
#pragma unroll
        for (int nt = 0; nt < NTH; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float h = glu_t<decltype(rt)::value, decltype(gt)::value>(acc[nt][mt][i], acc[nt + NTH][mt][i]);
            acc[nt][mt][i] = h;
            if (ok[nt]) mx = fmaxf(mx, fabsf(h));
          }
      });
      mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
      mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
      if (lg == 0) rmax[wave][mt * 16 + lr] = mx;
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < RB; ++mt) {
      const int m = mt * 16 + lr;
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < kNW; ++i) mx = fmaxf(mx, rmax[i][m]);
      const Fp8Quant q(mx);
      if (m < tile.rows) {
        const int64_t row = tile.row0 + m;
        uint8_t *h = static_cast<uint8_t *>(a.out) + row * a.N + col0 + 4 * lg;
#pragma unroll
        for (int nt = 0; nt < NTH; ++nt) {
          const fp8_acc &v = acc[nt][mt];
          if (ok[nt]) *reinterpret_cast<uint32_t *>(h + nt * 16) = fp8_pack4(q(v[0]), q(v[1]), q(v[2]), q(v[3]));
        }
        if (wave == 0 && lg == 0) a.hs[int64_t(bx) * a.rows + row] = q.scale;
      }
    }
  }
}

template <int RB, int MODE, bool EXACT>
__global__ __launch_bounds__(kThreads, 2) void fp8_tile_kernel(Fp8Args a) {
  using L = TileLds<RB, EXACT>;
  __shared__ __align__(16) typename L::Rows sa;
  __shared__ __align__(16) Turn turn;
  __shared__ typename L::Scales ss;
  __shared__ typename std::conditional<MODE == kGated, typename L::Max, float>::type rmax;
  constexpr int COLS = MODE == kGated ? kBN / 2 : kBN;
  PlanItem tile;
  int bx;
  if (my_work(a, RB * 16, (a.N + COLS - 1) / COLS, tile, bx))
    tile_body<RB, MODE, EXACT>(a, tile, bx, sa, turn, ss, reinterpret_cast<typename L::Max &>(rmax));
}

// The 128-row tile of the 8-bit instruction, for products that the matrix
// cores bound.  128 token rows by 64 weight rows per wave are 32 products of
// 32 cycles for 16 KB read from LDS and 8 KB from memory, so that with two
// waves per SIMD neither path (128 and 64 bytes a cycle) is near its limit.
// The rows go from memory to LDS without passing through registers.  4096
// rows, N = 4096, K = 2048: 50 us, 1.36 PFLOP/s (the tile kernel 66).  Neither
// memory, LDS nor the fmas alone bound it: left out one by one in timing
// copies, each changed it by a few percent.  What is left are the waits of
// two workgroups per CU at one barrier per block.
__device__ __forceinline__ void wide_body(const Fp8Args &a, const PlanItem &tile, int bx, uint8_t *sa0, uint8_t *sa1,
                                          Turn &turn, float *ssp0, float *ssp1) {
  constexpr int RB = 8, BM = RB * 16, PASS = BM * kPieces / kThreads;  // 4
  // row scale * scale of either block of 128 weight rows
  auto &ss0 = *reinterpret_cast<float (*)[2][BM]>(ssp0);
  auto &ss1 = *reinterpret_cast<float (*)[2][BM]>(ssp1);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = lane_id();
  const int lr = lane & 15, lg = lane >> 4;
  const int K = a.K, nb = (K + kFp8Block - 1) / kFp8Block;
  const int col0 = bx * kBN + wave * kNT * 16;
  const int nbr = (a.N + kFp8Block - 1) / kFp8Block;
  const uint8_t *wp[kNT];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
    wp[nt] = a.w0 + (int64_t(tile.expert) * a.N + min(col0 + nt * 16, a.N - 16)) * K;
  // pass p: row 32 p + tid / 8, the piece that belongs at place tid % 8
  const int piece = piece_of_lane(lane);
  const uint8_t *ap[PASS];
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int m = p * (kThreads / kPieces) + tid / kPieces;
    const int r = m < tile.rows ? source_row(a, tile.row0 + m) : -1;
    ap[p] = static_cast<const uint8_t *>(a.a) + int64_t(max(r, 0)) * K;
  }
  const int sm = tid % BM, sn = tid / BM;
  const int srow = sm < tile.rows ? source_row(a, tile.row0 + sm) : -1;
  const float *sap = a.as + max(srow, 0);
  const float *swp = a.s0 + (int64_t(tile.expert) * nbr + min(bx * (kBN / kFp8Block) + sn, nbr - 1)) * nb;

  WeightTile wn[kNT];  // the next block's weights
  i32x8 w[kNT];        // this one's, as operands
  float sga, sgw;
  auto load = [&](int s, uint8_t *buf) {
    s = min(s, nb - 1);
    const int k = s * kFp8Block;
    const int ka = min(k + piece * 16, K - 16);
#pragma unroll
    for (int p = 0; p < PASS; ++p)
      to_lds(ap[p] + ka, buf + (p * kNW + wave) * (kWave * 16));
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) wn[nt].load(wp[nt], K, k);
    sga = sap[int64_t(s) * a.a_rows];
    sgw = swp[s];
  };
  auto stage = [&](int s, float (&ss)[2][BM]) {  // block s: scales to LDS, weights through it
    ss[sn][sm] = srow >= 0 ? sga * sgw : 0.f;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) wn[nt].template put<true>(turn[wave][nt], K, s * kFp8Block);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) w[nt] = tile_operand<true>(turn[wave][0], nt);
  };
  fp8_acc acc[kNT][RB];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
    for (int mt = 0; mt < RB; ++mt) acc[nt][mt] = fp8_acc{0.f, 0.f, 0.f, 0.f};
  const uint32_t x0 = piece_at(lr, lg), x1 = piece_at(lr, lg + 4);
  // one block; TAIL: it reaches past the end of the reduction, where the
  // rows' codes count as zero too
  auto block = [&](int s, const uint8_t *buf, const float (&ss)[2][BM], auto tail) {
    constexpr bool TAIL = decltype(tail)::value;
    const bool ok0 = s * kFp8Block + lg * 16 < K, ok1 = s * kFp8Block + 64 + lg * 16 < K;
    auto codes = [&](const uint4 &lo, const uint4 &hi) {
      return Fp8Operand<false>(TAIL ? join8(keep(lo, ok0), keep(hi, ok1)) : join8(lo, hi));
    };
    auto rows = [&](int mt) {
      return codes(*reinterpret_cast<const uint4 *>(buf + x0 + mt * 16 * kFp8Block),
                   *reinterpret_cast<const uint4 *>(buf + x1 + mt * 16 * kFp8Block));
    };
    Fp8Operand<false> x = rows(0);
    float sc = ss[wave / 2][lr];
#pragma unroll
    for (int mt = 0; mt < RB; ++mt) {
      const Fp8Operand<false> xn = rows(mt + 1 < RB ? mt + 1 : mt);  // read while this one multiplies
      const float scn = ss[wave / 2][(mt + 1 < RB ? mt + 1 : mt) * 16 + lr];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const fp8_acc d = fp8_product(Fp8Operand<false>(w[nt]), x);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][mt][i] = __builtin_fmaf(d[i], sc, acc[nt][mt][i]);
      }
      x = xn, sc = scn;
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const int whole = K / kFp8Block;  // blocks without a tail
  load(0, sa0);
  stage(0, ss0);
  __syncthreads();
  int s = 0;
  for (; s + 1 < whole; s += 2) {
    load(s + 1, sa1);
    block(s, sa0, ss0, std::false_type{});
    stage(s + 1, ss1);
    __syncthreads();
    load(s + 2, sa0);
    block(s + 1, sa1, ss1, std::false_type{});
    stage(s + 2, ss0);
    __syncthreads();
  }
  // at most two blocks are left, the last perhaps short
  if (s < nb) {
    load(s + 1, sa1);
    block(s, sa0, ss0, std::true_type{});
    stage(s + 1, ss1);
    __syncthreads();
    if (s + 1 < nb) block(s + 1, sa1, ss1, std::true_type{});
  }
#pragma unroll
  for (int mt = 0; mt < RB; ++mt) {
    const int m = mt * 16 + lr;
    if (m < tile.rows) {
      const bool ok = source_row(a, tile.row0 + m) >= 0;
      const int64_t at = int64_t(tile.row0 + m) * a.N + 8 * lg + col0;
      const fp8_acc z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < kNT; nt += 2)
        if (col0 + nt * 16 + 8 * lg < a.N) store8(a, at + nt * 16, ok ? acc[nt][mt] : z, ok ? acc[nt + 1][mt] : z);
    }
  }
}

__global__ __launch_bounds__(kThreads, 2) void fp8_wide_kernel(Fp8Args a) {
  __shared__ __align__(16) uint8_t sa0[kWideRows * kFp8Block], sa1[kWideRows * kFp8Block];
  __shared__ __align__(16) Turn turn;
  __shared__ float ss0[kThreads], ss1[kThreads];
  PlanItem tile;
  int bx;
  if (my_work(a, kWideRows, (a.N + kBN - 1) / kBN, tile, bx)) wide_body(a, tile, bx, sa0, sa1, turn, ss0, ss1);
}

// Both in one grid, since experts' numbers of rows differ: the wide tile for
// experts with kWideFrom rows or more, the small one (the mean's size) for the
// others.  An expert with many rows in small tiles reads its weights from L2
// once per tile and pays each tile's waits.  Small tiles alone / mixed from
// 96 / 129 / 257 rows on, us: 20480 skewed rows over 512 experts of
// 1024 x 2048, about a third of them touched, 153 / 133 / 133 / 134; all
// touched 268 / 260 / 262 / 265; evenly spread 227 / 230 / 229 / 230; 4096
// rows over 128 experts of 2048 x 1024 59 / 56 / 57 / 58, over 32 experts of
// 1024 x 2048 36 / 30 / 30 / 35.
template <int RB>
__global__ __launch_bounds__(kThreads, 2) void fp8_mixed_kernel(Fp8Args a) {
  using L = TileLds<RB, false>;
  constexpr int WIDE = kWideRows * kFp8Block;
  __shared__ __align__(16) uint8_t sa0[std::max<int>(sizeof(typename L::Rows), WIDE)], sa1[WIDE];
  __shared__ __align__(16) Turn turn;
  __shared__ float ss0[2 * kThreads], ss1[kThreads];
  static_assert(sizeof(typename L::Scales) == sizeof(ss0), "the small tile's scales");
  PlanItem tile;
  int bx;
  if (!my_work<true>(a, RB * 16, (a.N + kBN - 1) / kBN, tile, bx, kWideFrom)) return;
  if (tile.rows & kBigTile) {
    tile.rows &= ~kBigTile;
    wide_body(a, tile, bx, sa0, sa1, turn, ss0, ss1);
  } else {
    tile_body<RB, kPlain, false>(a, tile, bx, reinterpret_cast<typename L::Rows &>(sa0), turn,
                                 reinterpret_cast<typename L::Scales &>(ss0),
                                 reinterpret_cast<typename L::Max &>(ss1));  // (no maxima in a plain product)
  }
}

// The 256-row tile, for large products: 8 waves of 128 token rows by 64
// weight rows, both operands from memory to LDS without passing through
// registers and read from there as they are used (24 KB for a wave's 32
// products).  One workgroup fills a CU.  8192 x 5632 x 2048: 115 us, 1.65
// PFLOP/s; the instruction alone, fed from registers with random codes,
// reaches 3.7, and a bf16 product of the library 1.2.
constexpr int kHugeRows = 256;
constexpr int kHugeThreads = 512;
__global__ __launch_bounds__(kHugeThreads, 2) void fp8_huge_kernel(Fp8Args a) {
  constexpr int RB = 8, BM = kHugeRows, PASS = BM * kPieces / kHugeThreads;  // 4
  __shared__ __align__(16) uint8_t sa0[BM * kFp8Block], sa1[BM * kFp8Block];
  __shared__ __align__(16) uint8_t sw0[kBN * kFp8Block], sw1[kBN * kFp8Block];
  __shared__ float ss0[2][BM], ss1[2][BM];  // row scale * scale of either block of 128 weight rows

  const int nbx = (a.N + kBN - 1) / kBN;
  PlanItem tile;
  int bx;
  if (!my_work(a, BM, nbx, tile, bx)) return;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave_id = __builtin_amdgcn_readfirstlane(tid / kWave), wave = wave_id % kNW;
  const int lr = lane & 15, lg = lane >> 4;
  const int K = a.K, nb = (K + kFp8Block - 1) / kFp8Block;
  const int col0 = bx * kBN + wave * kNT * 16, m0 = wave_id / kNW * RB * 16;
  const int nbr = (a.N + kFp8Block - 1) / kFp8Block;
  // pass p of either operand: row 64 p + tid / 8, the piece that belongs at place tid % 8
  const int piece = piece_of_lane(lane), piece_w = lane % kPieces ^ pair_key(tid / kPieces);
  const uint8_t *ap[PASS];
  uint32_t wo[PASS];  // rows of the tile's columns, from the first one's weights
  const uint8_t *wbase = a.w0 + (int64_t(tile.expert) * a.N + bx * kBN) * K;
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int m = p * (kHugeThreads / kPieces) + tid / kPieces;
    const int r = m < tile.rows ? source_row(a, tile.row0 + m) : -1;
    ap[p] = static_cast<const uint8_t *>(a.a) + int64_t(max(r, 0)) * K;
    wo[p] = uint32_t(min(m, a.N - 1 - bx * kBN)) * uint32_t(K);
  }
  const int sm = tid % BM, sn = tid / BM;
  const int srow = sm < tile.rows ? source_row(a, tile.row0 + sm) : -1;
  const float *sap = a.as + max(srow, 0);
  const float *swp = a.s0 + (int64_t(tile.expert) * nbr + min(bx * (kBN / kFp8Block) + sn, nbr - 1)) * nb;

  float sga, sgw;
  auto load = [&](int s, uint8_t *ba, uint8_t *bw) {
    s = min(s, nb - 1);
    const int k = min(s * kFp8Block + piece * 16, K - 16), kw = min(s * kFp8Block + piece_w * 16, K - 16);
#pragma unroll
    for (int p = 0; p < PASS; ++p) {
      const int at = (p * (kHugeThreads / kWave) + wave_id) * (kWave * 16);
      to_lds(ap[p] + k, ba + at);
      to_lds(wbase + (wo[p] + uint32_t(kw)), bw + at);
    }
    sga = sap[int64_t(s) * a.a_rows];
    sgw = swp[s];
  };
  auto stage_scale = [&](float (&ss)[2][BM]) { ss[sn][sm] = srow >= 0 ? sga * sgw : 0.f; };
  fp8_acc acc[kNT][RB];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
    for (int mt = 0; mt < RB; ++mt) acc[nt][mt] = fp8_acc{0.f, 0.f, 0.f, 0.f};
  const uint32_t r0 = piece_at(lr, lg), r1 = piece_at(lr, lg + 4);
  // one block; TAIL: it may reach past the end of the reduction, where the
  // codes count as zero in both operands (a stray one may be a NaN)
  auto block = [&](int s, const uint8_t *ba, const uint8_t *bw, const float (&ss)[2][BM], auto tail) {
    constexpr bool TAIL = decltype(tail)::value;
    const bool ok0 = s * kFp8Block + lg * 16 < K, ok1 = s * kFp8Block + 64 + lg * 16 < K;
    auto read = [&](const uint8_t *b, int row) {
      const uint4 lo = *reinterpret_cast<const uint4 *>(b + row * kFp8Block + r0);
      const uint4 hi = *reinterpret_cast<const uint4 *>(b + row * kFp8Block + r1);
      return Fp8Operand<false>(TAIL ? join8(keep(lo, ok0), keep(hi, ok1)) : join8(lo, hi));
    };
    auto read_w = [&](int nt) {
      const int m = wave * 64 + pair_row(nt, lr);
      const uint4 lo = *reinterpret_cast<const uint4 *>(bw + m * kFp8Block + (lg ^ pair_key(m)) * 16);
      const uint4 hi = *reinterpret_cast<const uint4 *>(bw + m * kFp8Block + ((lg + 4) ^ pair_key(m)) * 16);
      return Fp8Operand<false>(TAIL ? join8(keep(lo, ok0), keep(hi, ok1)) : join8(lo, hi));
    };
    const Fp8Operand<false> w[kNT] = {read_w(0), read_w(1), read_w(2), read_w(3)};
    Fp8Operand<false> x = read(ba, m0);
    float sc = ss[wave / 2][m0 + lr];
#pragma unroll
    for (int mt = 0; mt < RB; ++mt) {
      const Fp8Operand<false> xn = read(ba, m0 + min(mt + 1, RB - 1) * 16);  // read while this one multiplies
      const float scn = ss[wave / 2][m0 + min(mt + 1, RB - 1) * 16 + lr];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const fp8_acc d = fp8_product(w[nt], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][mt][i] = __builtin_fmaf(d[i], sc, acc[nt][mt][i]);
      }
      x = xn, sc = scn;
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const int whole = K / kFp8Block;  // blocks without a tail
  load(0, sa0, sw0);
  stage_scale(ss0);
  __syncthreads();
  int s = 0;
  for (; s + 1 < whole; s += 2) {
    load(s + 1, sa1, sw1);
    block(s, sa0, sw0, ss0, std::false_type{});
    stage_scale(ss1);
    __syncthreads();
    load(s + 2, sa0, sw0);
    block(s + 1, sa1, sw1, ss1, std::false_type{});
    stage_scale(ss0);
    __syncthreads();
  }
  // at most two blocks are left, the last perhaps short
  if (s < nb) {
    load(s + 1, sa1, sw1);
    block(s, sa0, sw0, ss0, std::true_type{});
    stage_scale(ss1);
    __syncthreads();
    if (s + 1 < nb) block(s + 1, sa1, sw1, ss1, std::true_type{});
  }
#pragma unroll
  for (int mt = 0; mt < RB; ++mt) {
    const int m = m0 + mt * 16 + lr;
    if (m < tile.rows) {
      const bool ok = source_row(a, tile.row0 + m) >= 0;
      const int64_t at = int64_t(tile.row0 + m) * a.N + 8 * lg + col0;
      const fp8_acc z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < kNT; nt += 2)
        if (col0 + nt * 16 + 8 * lg < a.N) store8(a, at + nt * 16, ok ? acc[nt][mt] : z, ok ? acc[nt + 1][mt] : z);
    }
  }
}

// The decode kernel: 16 token rows by WN weight tiles per wave; KW of the
// four waves split the reduction, the others take further columns.  Bound by
// the weights' bytes: 32 tokens' down (111 experts' 2048 x 768, 181 MB with
// the results) 39.6 us, 4.6 TB/s; one token's 8 experts of 1536 x 2048 (25 MB)
// 8.2 us, of which a launch and one memory round trip are about 4.  Each wave
// keeps DEPTH blocks in flight in registers (a ring in LDS filled by direct
// loads was drained by the compiler at every step, and lost).
template <int KW, int WN, int MODE>
__global__ __launch_bounds__(kThreads, 2) void fp8_decode_kernel(Fp8Args a) {
  constexpr int NTH = MODE == kGated ? WN / 2 : WN;
  constexpr int COLS = (kNW / KW) * NTH * 16;
  constexpr int DEPTH = 4;  // blocks in flight per wave
  __shared__ __align__(16) uint8_t turn[kNW][WN][kTileBytes];
  __shared__ float part[KW > 1 ? kNW : 1][KW > 1 ? WN * 4 : 1][kWave];

  const int nbx = (a.N + COLS - 1) / COLS;
  PlanItem tile;
  int bx;
  if (!my_work(a, 16, nbx, tile, bx)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int lr = lane & 15, lg = lane >> 4;
  const int kz = wave % KW;
  const int K = a.K, nb = (K + kFp8Block - 1) / kFp8Block;
  const int per = (nb + KW - 1) / KW, sbeg = min(kz * per, nb), send = min(sbeg + per, nb);
  const int col0 = (bx * (kNW / KW) + wave / KW) * NTH * 16;
  const int n_rows = MODE == kGated && a.fused ? 2 * a.N : a.N;
  const int nbr = (n_rows + kFp8Block - 1) / kFp8Block;

  const uint8_t *wp[WN];
  const float *sp[WN];  // scales of each tile's block row
#pragma unroll
  for (int nt = 0; nt < WN; ++nt) {
    const bool up = MODE == kGated && nt >= NTH;
    const int row = min(col0 + (nt % NTH) * 16, a.N - 16) + (up && a.fused ? a.N : 0);
    const bool second = up && !a.fused;
    wp[nt] = (second ? a.w1 : a.w0) + (int64_t(tile.expert) * n_rows + row) * K;
    sp[nt] = (second ? a.s1 : a.s0) + (int64_t(tile.expert) * nbr + row / kFp8Block) * nb;
  }
  const int r = lr < tile.rows ? source_row(a, tile.row0 + lr) : -1;
  const bool rok = r >= 0;
  // (rows past the tile read row 0, which the others of their kind share)
  const uint8_t *xp = static_cast<const uint8_t *>(a.a) + int64_t(max(r, 0)) * K;
  const float *sxp = a.as + max(r, 0);

  WeightTile wq[DEPTH][WN];
  uint4 xq[DEPTH][2];
  float sq[DEPTH][WN], sx[DEPTH];
  auto load = [&](int s, int d) {
    const int k0 = s * kFp8Block;
#pragma unroll
    for (int nt = 0; nt < WN; ++nt) {
      wq[d][nt].load(wp[nt], K, k0);
      sq[d][nt] = sp[nt][s];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xq[d][h] = *reinterpret_cast<const uint4 *>(xp + min(k0 + 64 * h + lg * 16, K - 16));
    sx[d] = sxp[int64_t(s) * a.a_rows];
  };
  fp8_acc acc[WN];
#pragma unroll
  for (int nt = 0; nt < WN; ++nt) acc[nt] = fp8_acc{0.f, 0.f, 0.f, 0.f};

  auto use = [&](int s, int d) {
    const int k0 = s * kFp8Block;
    const i32x8 x = join8(keep(xq[d][0], rok && k0 + lg * 16 < K), keep(xq[d][1], rok && k0 + 64 + lg * 16 < K));
    const Fp8Operand<true> xo(x);
#pragma unroll
    for (int nt = 0; nt < WN; ++nt) wq[d][nt].put(turn[wave][nt], K, k0);
    const float sxv = rok ? sx[d] : 0.f;
#pragma unroll
    for (int nt = 0; nt < WN; ++nt) {
      const fp8_acc v = fp8_product(Fp8Operand<true>(tile_operand(turn[wave][0], nt)), xo);
      const float sc = sxv * sq[d][nt];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = __builtin_fmaf(v[i], sc, acc[nt][i]);
    }
  };
  // (a wave without blocks of its own loads the last one and uses none)
  const int last = max(send - 1, sbeg < nb ? sbeg : nb - 1);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(min(sbeg + d, last), d);
  int s0 = sbeg;
  for (; s0 + DEPTH < send; s0 += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      use(s0 + d, d);
      load(min(s0 + DEPTH + d, last), d);
    }
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (s0 + d < send) use(s0 + d, d);
  if constexpr (KW > 1) {  // the parts of the reduction, added in their order
    if (kz) {
#pragma unroll
      for (int nt = 0; nt < WN; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][nt * 4 + i][lane] = acc[nt][i];
    }
    __syncthreads();
    if (kz) return;
#pragma unroll
    for (int z = 1; z < KW; ++z)
#pragma unroll
      for (int nt = 0; nt < WN; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] += part[wave + z][nt * 4 + i][lane];
  }
  if (lr >= tile.rows) return;
  const int64_t at = int64_t(tile.row0 + lr) * a.N + 4 * lg;
#pragma unroll
  for (int nt = 0; nt < NTH; ++nt) {
    const int col = col0 + nt * 16;
    if (col < a.N) {
      fp8_acc v = rok ? acc[nt] : fp8_acc{0.f, 0.f, 0.f, 0.f};
      if constexpr (MODE == kGated) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = glu(acc[nt][i], acc[nt + NTH][i], a.round, a.geglu);
      }
      store4(a, at + col, v);
    }
  }
}

// Row tiles that the experts' rows can take at most: each expert adds at most
// one partly filled tile.
int64_t most_tiles(int64_t rows, int experts, int bm) {
  return rows / bm + std::min<int64_t>(rows, experts);
}

// bm: 32, 48 or 64 rows a tile.
template <int MODE, bool EXACT>
void launch_tile(const Fp8Args &a, int bm, int64_t tiles, hipStream_t s) {
  constexpr int COLS = MODE == kGated ? kBN / 2 : kBN;
  const int64_t nbx = (a.N + COLS - 1) / COLS;
  const dim3 grid(unsigned(tiles * nbx));
  if (bm == 32) launch((fp8_tile_kernel<2, MODE, EXACT>), grid, dim3(kThreads), 0, s, a);
  else if (bm == 48) launch((fp8_tile_kernel<3, MODE, EXACT>), grid, dim3(kThreads), 0, s, a);
  else launch((fp8_tile_kernel<4, MODE, EXACT>), grid, dim3(kThreads), 0, s, a);
}
void launch_mixed(const Fp8Args &a, int bm, int64_t tiles, hipStream_t s) {
  const int64_t nbx = (a.N + kBN - 1) / kBN;
  const dim3 grid(unsigned(tiles * nbx));
  if (bm == 32) launch(fp8_mixed_kernel<2>, grid, dim3(kThreads), 0, s, a);
  else if (bm == 48) launch(fp8_mixed_kernel<3>, grid, dim3(kThreads), 0, s, a);
  else launch(fp8_mixed_kernel<4>, grid, dim3(kThreads), 0, s, a);
}
void launch_wide(const Fp8Args &a, int64_t tiles, hipStream_t s) {
  const int64_t nbx = (a.N + kBN - 1) / kBN;
  launch(fp8_wide_kernel, dim3(unsigned(tiles * nbx)), dim3(kThreads), 0, s, a);
}

void launch_huge(const Fp8Args &a, int64_t tiles, hipStream_t s) {
  const int64_t nbx = (a.N + kBN - 1) / kBN;
  launch(fp8_huge_kernel, dim3(unsigned(tiles * nbx)), dim3(kHugeThreads), 0, s, a);
}

template <int KW, int WN, int MODE>
void launch_decode_one(const Fp8Args &a, int64_t tiles, hipStream_t s) {
  constexpr int COLS = (kNW / KW) * (MODE == kGated ? WN / 2 : WN) * 16;
  const int64_t nbx = (a.N + COLS - 1) / COLS;
  launch((fp8_decode_kernel<KW, WN, MODE>), dim3(unsigned(tiles * nbx)), dim3(kThreads), 0, s, a);
}

// Waves that split the reduction of the decode kernel.
int decode_split(int K) {
  const int nb = (K + kFp8Block - 1) / kFp8Block;
  return nb >= 8 ? 4 : nb >= 4 ? 2 : 1;
}
// Output columns per workgroup of the decode kernel.
int decode_cols(int K, bool gated) { return kNW / decode_split(K) * (gated ? 1 : 2) * 16; }

template <int MODE>
void launch_decode(const Fp8Args &a, int64_t tiles, hipStream_t s) {
  const int kw = decode_split(a.K);
  if (kw == 4) launch_decode_one<4, 2, MODE>(a, tiles, s);
  else if (kw == 2) launch_decode_one<2, 2, MODE>(a, tiles, s);
  else launch_decode_one<1, 2, MODE>(a, tiles, s);
}

}  // namespace

// Rows per tile: 16 (the decode kernel), 64, or for the 8-bit instruction 128
// or 256.  Measured for K = 2048 and bf16 results, us with 16 / 64 / 128
// rows (256 where given): one matrix of N = 4096, 128 rows 10.8 / 23.6 / 33,
// 256 rows 18 / 24 / 34, 512 rows 32 / 24.5 / 35, 2048 rows 113 / 37 / 38,
// 4096 rows 211 / 66 / 51, 8192 rows - / 125 / 97 / 93; 64 matrices of
// N = 1024 with 16 rows each 25 / 26 / 35, 32 rows 38 / 27 / 36, 128 rows
// 135 / 38 / 41, 256 rows 250 / 73 / 51.  So: 16 while its workgroups fill
// the GPU at most about once over, or at most 16 rows an expert; 64 while its
// workgroups fit the GPU at once, or experts would leave a larger tile half
// empty; 256 from two of its tiles per CU on.
int fp8_tile_rows(int64_t rows, int32_t N, int32_t K, int experts, bool exact) {
  const int64_t t16 = most_tiles(rows, experts, 16), t64 = rows / 64 + experts / 2;
  const int dc = decode_cols(K, false), nbx = (N + kBN - 1) / kBN;
  if (rows <= 16LL * experts || t16 * ((N + dc - 1) / dc) <= 2560) return 16;
  if (rows <= 42LL * experts) return fp8_small_tile(rows, experts);
  if (exact || rows < 96LL * experts || t64 * nbx <= 640) return 64;
  return rows / kHugeRows * nbx >= 512 && rows >= 1024LL * experts ? 256 : 128;
}

// For experts with few rows, the smallest tile that holds the mean with room:
// rows of a tile that no token fills cost products all the same.  Gate/up and
// down of the 512-expert layer at 40 rows an expert 247 and 155 us with 64
// rows, 238 and 151 with 48, 298 and 181 with 32 (experts above the mean then
// read their weights twice).
int fp8_small_tile(int64_t rows, int experts) {
  return rows <= 26LL * experts ? 32 : rows <= 42LL * experts ? 48 : 64;
}

int64_t fp8_matmul_groups(int64_t rows, int32_t N, int32_t K, int32_t n_experts, bool offsets, bool exact) {
  const int bm = fp8_tile_rows(rows, N, K, n_experts, exact);
  const int64_t tiles = offsets ? most_tiles(rows, n_experts, bm) : (rows + bm - 1) / bm;
  const int cols = bm == 16 ? decode_cols(K, false) : kBN;
  return tiles * ((N + cols - 1) / cols);
}

static int64_t ffn_tiles(const moe_layer_desc *d, int32_t T) {
  const int bm = plan_tile_rows(d, T);
  return most_tiles(int64_t(T) * d->top_k, d->n_experts, bm) + int64_t(d->n_shared) * ((T + bm - 1) / bm);
}

int64_t fp8_ffn_groups(const moe_layer_desc *d, int32_t T) {
  const bool dec = plan_tile_rows(d, T) == 16;
  const int gc = dec ? decode_cols(d->d_model, true) : kBN / 2, dc = dec ? decode_cols(d->d_ff, false) : kBN;
  return ffn_tiles(d, T) * std::max((d->d_ff + gc - 1) / gc, (d->d_model + dc - 1) / dc);
}

void launch_fp8_matmul(int32_t rows, int32_t N, int32_t K, int32_t n_experts, int32_t a_rows, const uint8_t *a,
                       const float *a_scales, const int32_t *row_map, const int32_t *expert_off, const uint8_t *w,
                       const float *w_scales, void *y, int32_t out_dtype, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  Fp8Args g{};
  g.a = a, g.as = a_scales, g.a_rows = a_rows, g.row_map = row_map;
  g.rows = rows, g.N = N, g.K = K;
  g.w0 = w, g.s0 = w_scales;
  g.E = n_experts, g.expert_off = expert_off;
  g.out = y, g.out_dtype = out_dtype;
  const bool exact = out_dtype == MOE_DT_F32;
  const int bm = fp8_tile_rows(rows, N, K, n_experts, exact);
  const int64_t tiles = expert_off ? most_tiles(rows, n_experts, bm) : (int64_t(rows) + bm - 1) / bm;
  if (bm == 16) launch_decode<kPlain>(g, tiles, s);
  else if (exact) launch_tile<kPlain, true>(g, bm, tiles, s);
  else if (bm <= 64 && expert_off && n_experts > 1) launch_mixed(g, bm, tiles, s);
  else if (bm <= 64) launch_tile<kPlain, false>(g, bm, tiles, s);
  else if (bm == 128) launch_wide(g, tiles, s);
  else launch_huge(g, tiles, s);
}

// The codes of the decode tiles' h, behind its fp32 rows (h_bytes counts them).
static uint8_t *codes_of_h(void *h, int64_t rows, int F) { return static_cast<uint8_t *>(h) + rows * F * 4; }

// Workspace of the expert FFN: x codes and scales, h as codes and scales and
// (decode tiles) as fp32 rows.
void launch_expert_ffn_fp8(const moe_layer_desc *d, int32_t T, const void *x, const int32_t *row_map,
                           const moe_weights *w, const int32_t *counters, const PlanItem *tiles,
                           const FfnScratch &sc, float *y_sorted, void *stream, StageMarker *mk) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t max_tiles = ffn_tiles(d, T);
  const int D = d->d_model, F = d->d_ff, M = d->n_experts + d->n_shared;
  const int N = T * d->top_k, R = N + d->n_shared * T;
  const moe_proj &pg = d->gate_up_fused ? w->gate_up : w->gate;
  const int bm = plan_tile_rows(d, T);
  Fp8Args g{};
  g.row_map = row_map, g.rows = R, g.N = F, g.K = D, g.T = T, g.n_routed = N;
  g.w0 = static_cast<const uint8_t *>(pg.w), g.s0 = static_cast<const float *>(pg.scales);
  g.w1 = static_cast<const uint8_t *>(w->up.w), g.s1 = static_cast<const float *>(w->up.scales);
  g.fused = d->gate_up_fused, g.round = glu_round_mode(d), g.geglu = d->activation == MOE_ACT_GEGLU;
  g.E = M, g.tiles = tiles, g.counters = counters;
  g.a_rows = T;
  g.out = sc.h;
  Fp8Args n{};
  n.rows = R, n.N = D, n.K = F;
  n.w0 = static_cast<const uint8_t *>(w->down.w), n.s0 = static_cast<const float *>(w->down.scales);
  n.E = M, n.tiles = tiles, n.counters = counters;
  n.a = sc.h, n.a_rows = R;
  n.out = y_sorted, n.out_dtype = MOE_DT_F32;
  uint8_t *xq = static_cast<uint8_t *>(sc.x16);
  float *xs = reinterpret_cast<float *>(sc.xg);
  float *hs = reinterpret_cast<float *>(sc.hsh);
  // x is quantised once, not by every workgroup for its own rows: that saved
  // two launches on the decode tiles but repeated the work so often that it
  // lost even at one token (21.6 against 20.0 us for 128 experts of 2048 x 768,
  // top 8; 32 tokens 136 against 101 us, 256 tokens 236 against 152 us).
  launch_fp8_rows(x, d->act_dtype, T, D, xq, xs, stream);
  if (mk) mk->mark("x_fp8");
  g.a = xq, g.as = xs, g.hs = hs;
  n.as = hs;
  if (bm == 16) {  // a workgroup's 16 columns do not make a block of h: fp32 rows first
    g.out_dtype = MOE_DT_F32;
    launch_decode<kGated>(g, max_tiles, s);
    if (mk) mk->mark("gateup_fp8");
    uint8_t *hq = codes_of_h(sc.h, R, F);
    launch_fp8_rows(sc.h, MOE_DT_F32, R, F, hq, hs, stream);
    if (mk) mk->mark("h_fp8");
    n.a = hq;
    launch_decode<kPlain>(n, max_tiles, s);
    if (mk) mk->mark("down_fp8");
    return;
  }
  launch_tile<kGated, true>(g, bm, max_tiles, s);
  if (mk) mk->mark("gateup_fp8");
  launch_tile<kPlain, true>(n, bm, max_tiles, s);
  if (mk) mk->mark("down_fp8");
}

}  // namespace moe
