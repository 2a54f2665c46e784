// balance.hip -- the router's balance loss, per-expert counts, and their
// gradients (with those of the routing weights) for x, the router and its
// bias.
//
// With logits l[t][e] = x[t] . W[:, e] + bias[e], p = softmax(l), and for
// sequence b its n_b counted tokens, c_be slots at expert e and mean
// probability P_be:
//   L = 1/B' sum_b E / (k n_b) sum_e c_be P_be,   B' sequences with n_b > 0.
// Its gradient with the counts held fixed is, for a token of sequence b,
//   dl = p (g - sum_e p_e g_e),  g_e = dL E c_be / (k n_b^2 B'),
// which does not change when a constant is taken from all g_e: c_be enters as
// its difference from the mean count, an exact integer, so that nearly
// balanced experts keep the digits of their differences.  The routing
// weights' gradient adds to dl through the softmax over the selected experts
// (renormalised weights), or to g (plain ones).  Then
//   dx = dl W^T,  dW = x^T dl,  dbias = sum_t dl.
//
// The three matrix products run on the 16-bit matrix cores with fp32 sums.
// 16-bit operands enter the logits as they are.  Elsewhere fp32 values are
// cut into three bf16 pieces of 8 significant bits each (24 in all, so
// nothing is lost), fp16 values into two, and the products of pieces above
// 2^-24 of the largest are added: 3 products for bf16 layers, 5 for fp16 and
// 6 for fp32, each at 16 times the fp32 matrix rate.  dl is cut once, where
// it is made, and kept as three planes.
//
// Softmax, sums over tokens and the loss are per-wave rows and two-level sums
// in a fixed order: no floating-point atomics.
#include <algorithm>

#include "dequant_f16.h"
#include "device_common.h"
#include "launch.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;             // output rows and columns per workgroup
constexpr int kStep = 64;             // reduction elements per LDS stage
constexpr int kPieces = 3;            // bf16 pieces of an fp32 value
constexpr int kDtPieces = 3;          // operand type: three bf16 planes (beside the moe_dtype values)

// ---- the split products -----------------------------------------------------

// One operand: element (row, k) at p[row * ld + k] (KC) or p[k * ld + row].
struct Operand {
  const void *p;
  int64_t ld;
  int rows;
  int vec;  // rows start 16-byte aligned: whole pieces load as vectors
  int64_t plane = 0;  // kDtPieces: elements per plane; ld is a multiple of 8, zero past the end of a row
};
// Tokens that take part (the reduction of dW runs over tokens): null mask and
// off for all of them.
struct Tokens {
  const uint8_t *mask;
  const int32_t *off;  // [n + 1]
  int n, T;
};
__device__ __forceinline__ void token_range(const Tokens &k, int &lo, int &hi) {
  lo = 0, hi = k.T;
  if (k.off) {
    lo = min(max(k.off[0], 0), k.T);
    hi = min(max(k.off[k.n], lo), k.T);
  }
}

struct GemmArgs {
  Operand a, b;
  int K, per;          // reduction length, steps per part
  float *out;          // [parts][a.rows][b.rows]
  int64_t part;        // elements per part
  const float *bias;   // nullable, added per column
  Tokens tokens;       // MASK: reduction elements that take part
  float *bsum = nullptr;  // MASK: sum_k B(n, k), [parts][b.rows] after `bpart` elements each (null: not wanted)
  int64_t bpart = 0;
};

// Place of element (row, k) in a 64 x 64 tile of 16-bit elements in LDS.  The
// 16-byte pieces of a row are exchanged by its number so that both the reads
// (one piece each of 8 neighbouring rows) and the writes of turned-around
// elements (8 bytes each of every fourth row) meet different banks.
__device__ __forceinline__ int lds_at(int row, int k) {
  const int f = ((row >> 2) & 1) | ((((row >> 1) ^ (row >> 3)) & 1) << 1) | (((row >> 4) & 1) << 2);
  return row * kStep + (((k >> 3) ^ f) << 3) + (k & 7);
}

template <int DT>
constexpr int pieces(bool native) {
  return DT == kDtBF16 || native ? 1 : DT == kDtF16 ? 2 : kPieces;
}

// v as bf16 pieces: cut (not rounded) to 8 significant bits, the rest cut
// again; the last piece is rounded.  A value without a finite rest keeps its
// first piece alone.
template <int P>
__device__ __forceinline__ void split(float v, uint32_t (&out)[P]) {
  if constexpr (P == 1) {
    out[0] = f32_to_bf16_bits(v);
  } else {
    const uint32_t b = __float_as_uint(v);
    out[0] = b >> 16;
    float r = v - __uint_as_float(b & 0xffff0000u);
    if (!(fabsf(v) < INFINITY)) r = 0.f, out[0] = f32_to_bf16_bits(v);
    if constexpr (P == 2) {
      out[1] = f32_to_bf16_bits(r);
    } else {
      const uint32_t c = __float_as_uint(r);
      out[1] = c >> 16;
      out[2] = f32_to_bf16_bits(r - __uint_as_float(c & 0xffff0000u));
    }
  }
}

// Staging of 64 rows by 64 reduction elements of one operand.  KC: a thread
// takes 16 consecutive reduction elements of one row; else 4 x 4 elements
// (4 neighbouring rows at 4 reduction elements), turned around in registers,
// so that LDS always holds [row][k].  Loads go to clamped addresses without
// a condition and their values are touched only in store(), so that they
// stay in flight in between.  Reduction elements that do not exist (or do not
// take part) are zeroed there; rows that do not exist are not: they reach
// only results that are not stored.
// The last step of a reduction that is no multiple of 64 loads its last 64
// elements and zeroes those of the step before (`start` is where a step's
// loads begin, the same for both operands), so that a thread's offsets from
// there never change and cost no multiplication per step.
// VEC: rows are 16-byte aligned (16-bit KC and fp32: whole 16-byte pieces;
// 16-bit rows side by side: 8-byte ones).
template <int DT, bool KC, bool NATIVE, bool VEC>
struct Stage {
  static constexpr int P = pieces<DT>(NATIVE);
  static constexpr bool RAW = P == 1;  // 16-bit elements that are copied as they are
  static constexpr int W = DT == kDtF32 || !VEC ? 16 : 8;  // words: one or two elements each
  uint32_t w[W];
  uint32_t on;  // bit j: reduction element j of the four takes part
  template <bool MASK>
  __device__ __forceinline__ void load(const Operand &o, int row0, int start, int K, const Tokens &tk, int lo,
                                       int hi) {
    const int tid = threadIdx.x;
    const int64_t from = KC ? int64_t(start) : int64_t(start) * o.ld;  // uniform
    const float *pf = static_cast<const float *>(o.p) + from;
    const uint16_t *ph = static_cast<const uint16_t *>(o.p) + from;
    if constexpr (KC) {
      const int64_t row = int64_t(min(row0 + tid / 4, o.rows - 1)) * o.ld;
      const int c = tid % 4 * 16;
      if constexpr (!VEC) {
#pragma unroll
        for (int u = 0; u < 16; ++u) w[u] = word(pf, ph, row + min(c + u, K - 1 - start));
      } else {
        constexpr int C = DT == kDtF32 ? 4 : 8;  // elements of a 16-byte piece
#pragma unroll
        for (int u = 0; u < 16 / C; ++u) {
          const int64_t at = row + min(c + C * u, K - C - start);
          const uint4 q = DT == kDtF32 ? *reinterpret_cast<const uint4 *>(pf + at)
                                       : *reinterpret_cast<const uint4 *>(ph + at);
          w[4 * u] = q.x, w[4 * u + 1] = q.y, w[4 * u + 2] = q.z, w[4 * u + 3] = q.w;
        }
      }
    } else {
      const int c = tid / 16 * 4, r = row0 + tid % 16 * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = uint32_t(min(c + j, K - 1)) * uint32_t(o.ld);
        if constexpr (!VEC) {
#pragma unroll
          for (int u = 0; u < 4; ++u) w[4 * j + u] = word(pf, ph, at + uint32_t(min(r + u, o.rows - 1)));
        } else if constexpr (DT == kDtF32) {
          const uint4 q = *reinterpret_cast<const uint4 *>(pf + (at + uint32_t(min(r, o.rows - 4))));
          w[4 * j] = q.x, w[4 * j + 1] = q.y, w[4 * j + 2] = q.z, w[4 * j + 3] = q.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2 *>(ph + (at + uint32_t(min(r, o.rows - 4))));
          w[2 * j] = q.x, w[2 * j + 1] = q.y;
        }
      }
      on = 15;
      if constexpr (MASK) {
        if (tk.mask) {
          on = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) on |= uint32_t(tk.mask[start + min(c + j, K - 1)] != 0) << j;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (start + c + j < lo || start + c + j >= hi) on &= ~(1u << j);
      }
    }
  }
  static __device__ __forceinline__ uint32_t word(const float *pf, const uint16_t *ph, int64_t i) {
    if constexpr (DT == kDtF32) return __float_as_uint(pf[i]);
    else return ph[i];
  }
  // Element u of the 16: its 16 bits (16-bit types) or its value.
  __device__ __forceinline__ uint32_t half_bits(int u) const {
    if constexpr (W == 16) return w[u];
    else return u & 1 ? w[u / 2] >> 16 : w[u / 2] & 0xffffu;
  }
  __device__ __forceinline__ void cut(int u, bool ok, uint32_t (&q)[P]) const {
    if constexpr (RAW) q[0] = ok ? half_bits(u) : 0u;
    else if constexpr (DT == kDtF32) split<P>(ok ? __uint_as_float(w[u]) : 0.f, q);
    else split<P>(ok ? half_to_f32<DT>(half_bits(u)) : 0.f, q);
  }
  // into LDS; the elements k0 <= k < K of those loaded from start
  __device__ __forceinline__ void store(uint16_t (&lds)[P][kTile * kStep], int start, int k0, int K) const {
    const int tid = threadIdx.x;
    if constexpr (KC) {
      const int k = start + tid % 4 * 16;
      uint32_t o[P][8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if constexpr (RAW && W == 8) {  // K and start are multiples of 8
          const int c = k + u / 4 * 8;
          o[0][u] = c >= k0 && c < K ? w[u] : 0u;
        } else {
          const int c = k + 2 * u;
          uint32_t x[P], y[P];
          cut(2 * u, c >= k0 && c < K, x), cut(2 * u + 1, c + 1 >= k0 && c + 1 < K, y);
#pragma unroll
          for (int p = 0; p < P; ++p) o[p][u] = x[p] | (y[p] << 16);
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        uint16_t *q = lds[p];
        *reinterpret_cast<uint4 *>(q + lds_at(tid / 4, tid % 4 * 16)) =
            make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
        *reinterpret_cast<uint4 *>(q + lds_at(tid / 4, tid % 4 * 16 + 8)) =
            make_uint4(o[p][4], o[p][5], o[p][6], o[p][7]);
      }
    } else {
      const int k = start + tid / 16 * 4;
      bool ok[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) ok[j] = k + j >= k0 && k + j < K && ((on >> j) & 1u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // row i of the four
        uint32_t x[4][P];
#pragma unroll
        for (int j = 0; j < 4; ++j) cut(4 * j + i, ok[j], x[j]);
#pragma unroll
        for (int p = 0; p < P; ++p)
          *reinterpret_cast<uint2 *>(&lds[p][lds_at(tid % 16 * 4 + i, tid / 16 * 4)]) =
              make_uint2(x[0][p] | (x[1][p] << 16), x[2][p] | (x[3][p] << 16));
      }
    }
  }
};

// The same of values that lie cut into three planes already: copied as they are.
template <bool KC>
struct Stage<kDtPieces, KC, false, true> {
  static constexpr int P = kPieces;
  uint32_t w[P][8];  // (words: arrays of vectors here went to scratch memory)
  template <bool MASK>
  __device__ __forceinline__ void load(const Operand &o, int row0, int start, int K, const Tokens &, int, int) {
    const int tid = threadIdx.x;
    if constexpr (KC) {  // 16 elements of a row
      const uint16_t *base = static_cast<const uint16_t *>(o.p) + start;
      const int64_t row = int64_t(min(row0 + tid / 4, o.rows - 1)) * o.ld;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = min(tid % 4 * 16 + 8 * h, int(o.ld) - 8);
          const uint4 q = *reinterpret_cast<const uint4 *>(base + p * o.plane + (row + c));
          w[p][4 * h] = q.x, w[p][4 * h + 1] = q.y, w[p][4 * h + 2] = q.z, w[p][4 * h + 3] = q.w;
        }
    } else {  // 4 x 4 elements, two words for each reduction element
      const uint16_t *base = static_cast<const uint16_t *>(o.p) + int64_t(start) * o.ld;
      const int c = tid / 16 * 4, r = min(row0 + tid % 16 * 4, int(o.ld) - 4);
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t at = uint32_t(min(c + j, K - 1)) * uint32_t(o.ld) + uint32_t(r);
          const uint2 q = *reinterpret_cast<const uint2 *>(base + p * o.plane + at);
          w[p][2 * j] = q.x, w[p][2 * j + 1] = q.y;
        }
    }
  }
  __device__ __forceinline__ void store(uint16_t (&lds)[P][kTile * kStep], int start, int k0, int K) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if constexpr (KC) {  // (elements past K, up to a multiple of 8, are zero in memory)
        const int k = start + tid % 4 * 16;
        uint16_t *q = lds[p];
        const bool a = k >= k0 && k < K, b = k + 8 >= k0 && k + 8 < K;
        *reinterpret_cast<uint4 *>(q + lds_at(tid / 4, tid % 4 * 16)) =
            make_uint4(a ? w[p][0] : 0u, a ? w[p][1] : 0u, a ? w[p][2] : 0u, a ? w[p][3] : 0u);
        *reinterpret_cast<uint4 *>(q + lds_at(tid / 4, tid % 4 * 16 + 8)) =
            make_uint4(b ? w[p][4] : 0u, b ? w[p][5] : 0u, b ? w[p][6] : 0u, b ? w[p][7] : 0u);
      } else {
        const int k = start + tid / 16 * 4;
        uint32_t v[8];  // [reduction element][pair of rows]
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = k + j / 2 >= k0 && k + j / 2 < K ? w[p][j] : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;  // high or low halves of two words
          *reinterpret_cast<uint2 *>(&lds[p][lds_at(tid % 16 * 4 + i, tid / 16 * 4)]) =
              make_uint2(__builtin_amdgcn_perm(v[2 + (i >> 1)], v[i >> 1], sel),
                         __builtin_amdgcn_perm(v[6 + (i >> 1)], v[4 + (i >> 1)], sel));
        }
      }
    }
  }
};

// C[m][n] = sum_k A(m, k) B(n, k) over one part of the reduction, tiles of
// 64 x 64.  A wave makes 32 x 32 outputs (operand a of the matrix cores:
// columns n, so that a lane's four results are neighbours in a row of C).
// Two steps are in flight in registers while one is multiplied: a step's
// products take a fraction of a memory round trip.  NATIVE: fp16 operands
// multiplied as they are.  MASK: reduction elements outside `tokens` count as
// zeros, whatever they hold.
//
// Bound by latency more than by either rate: a step is one round through LDS
// and 8 to 48 matrix instructions a wave, with two or three workgroups per CU
// to hide it.  2048 tokens, d_model 2048, 512 experts (bf16): logits 18.3 us
// for 4.3 GFLOP and 10.5 MB read; 8192 tokens, 128 experts: dW 37 us for 12.9
// GFLOP in matrix-core products.  Tiles of 128 x 128 spilled with three
// pieces, and 4 waves per SIMD spilled too (both slower).
template <int DTA, bool KCA, int DTB, bool KCB, bool NATIVE, bool MASK, bool VECB>
__global__ __launch_bounds__(kThreads, 2) void split_gemm_kernel(GemmArgs g) {
  using SA = Stage<DTA, KCA, NATIVE, true>;
  using SB = Stage<DTB, KCB, NATIVE, VECB>;
  constexpr int PA = SA::P, PB = SB::P, S = 2;
  // Two buffers (one barrier a step, a step's elements stored while the last
  // one's are multiplied) for single pieces; with more, the second one costs
  // occupancy (8192 tokens, 128 experts, dx by this kernel: 34 us with one,
  // 39 with two).
  constexpr int BUF = PA + PB <= 2 ? 2 : 1;
  __shared__ __align__(16) uint16_t la[BUF][PA][kTile * kStep], lb[BUF][PB][kTile * kStep];
  const int lane = lane_id(), wave = threadIdx.x / kWave, lr = lane & 15, lg = lane >> 4;
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  const int wm = (wave >> 1) * 16 * S, wn = (wave & 1) * 16 * S;
  const int s0 = int(blockIdx.z) * g.per, s1 = min(s0 + g.per, (g.K + kStep - 1) / kStep);
  int lo = 0, hi = 0;
  if constexpr (MASK) token_range(g.tokens, lo, hi);
  f32x4 acc[S][S];
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // The sums of B over the reduction are its products with ones, made by the
  // waves that hold the first rows of the first row of tiles.
  const bool sums = MASK && g.bsum && m0 == 0 && wm == 0;
  f32x4 accb[S];
#pragma unroll
  for (int j = 0; j < S; ++j) accb[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);  // bf16 1.0
  SA sa[2];
  SB sb[2];
  // where step s loads from: its own elements, or the last 64 (a multiple of
  // 8 where both operands are read along the reduction)
  const int Kl = KCA && KCB ? (g.K + 7) / 8 * 8 : g.K;
  auto start_of = [&](int s) { return max(0, min(s * kStep, Kl - kStep)); };
  auto load = [&](int s, auto rc) {
    constexpr int r = decltype(rc)::value;
    sa[r].template load<MASK>(g.a, m0, start_of(s), g.K, g.tokens, lo, hi);
    sb[r].template load<MASK>(g.b, n0, start_of(s), g.K, g.tokens, lo, hi);
  };
  auto store = [&](int s, auto rc) {  // step s from its registers into its buffer
    constexpr int r = decltype(rc)::value;
    sa[r].store(la[r % BUF], start_of(s), s * kStep, g.K);
    sb[r].store(lb[r % BUF], start_of(s), s * kStep, g.K);
  };
  auto multiply = [&](auto rc) {
    constexpr int r = decltype(rc)::value % BUF;
#pragma unroll
    for (int kk = 0; kk < kStep; kk += 32) {
      uint4 fa[PA][S];
#pragma unroll
      for (int p = 0; p < PA; ++p)
#pragma unroll
        for (int i = 0; i < S; ++i)
          fa[p][i] = *reinterpret_cast<const uint4 *>(&la[r][p][lds_at(wm + i * 16 + lr, kk + lg * 8)]);
#pragma unroll
      for (int q = PB - 1; q >= 0; --q)
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const uint4 fb = *reinterpret_cast<const uint4 *>(&lb[r][q][lds_at(wn + j * 16 + lr, kk + lg * 8)]);
          if constexpr (MASK && !NATIVE) {
            if (sums)
              accb[j] = mfma_bf16(__builtin_bit_cast(bf16x8, fb), __builtin_bit_cast(bf16x8, ones), accb[j]);
          }
#pragma unroll
          for (int p = PA - 1; p >= 0; --p)
            if (p + q < kPieces)
#pragma unroll
              for (int i = 0; i < S; ++i) {
                if constexpr (NATIVE)
                  acc[i][j] = mfma_f16(__builtin_bit_cast(f16x8, fb), __builtin_bit_cast(f16x8, fa[p][i]), acc[i][j]);
                else
                  acc[i][j] =
                      mfma_bf16(__builtin_bit_cast(bf16x8, fb), __builtin_bit_cast(bf16x8, fa[p][i]), acc[i][j]);
              }
        }
    }
  };
  using R0 = std::integral_constant<int, 0>;
  using R1 = std::integral_constant<int, 1>;
  auto step = [&](int s, auto rc, auto next) {
    if constexpr (BUF == 1) {
      __syncthreads();
      store(s, rc);
      __syncthreads();
      if (s + 2 < s1) load(s + 2, rc);
      multiply(rc);
    } else {  // step s lies in its buffer
      if (s + 2 < s1) load(s + 2, rc);
      multiply(rc);
      if (s + 1 < s1) store(s + 1, next);
      __syncthreads();
    }
  };
  if (s0 < s1) {
    load(s0, R0{});
    load(min(s0 + 1, s1 - 1), R1{});
    if constexpr (BUF == 2) {
      store(s0, R0{});
      __syncthreads();
    }
    int s = s0;
    for (; s + 1 < s1; s += 2) {
      step(s, R0{}, R1{});
      step(s + 1, R1{}, R0{});
    }
    if (s < s1) step(s, R0{}, R1{});
  }
  const int N = g.b.rows;
  if (sums && lr == 0) {  // every column of the product holds the same sums
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = n0 + wn + j * 16 + 4 * lg + c;
        if (n < N) g.bsum[int64_t(blockIdx.z) * g.bpart + n] = accb[j][c];
      }
  }
  if (!g.out) return;
  float *out = g.out + int64_t(blockIdx.z) * g.part;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int m = m0 + wm + i * 16 + lr;
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int n = n0 + wn + j * 16 + 4 * lg;
      if (m >= g.a.rows || n >= N) continue;
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = acc[i][j][c] + (g.bias && n + c < N ? g.bias[n + c] : 0.f);
      float *p = out + int64_t(m) * N + n;
      if (N % 4 == 0) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n + c < N) p[c] = v[c];
      }
    }
  }
}

// dx = dl W^T for at most 64 KS experts: a workgroup keeps the pieces of its 64
// tokens' dl in registers, as operands, and runs over column tiles of W, two
// steps ahead (a reduction this short is over before a workgroup of its own
// for every 64 x 64 results has its operands).  Bound by the results: 8192
// tokens, 128 experts, d_model 2048 (67 MB) 23 us; 29 with ordinary stores,
// and 34 with a workgroup for each tile.
template <int DT, bool VECB, int KS>
__global__ __launch_bounds__(kThreads, 2) void balance_dx_kernel(GemmArgs g, int per_wg) {
  using SB = Stage<DT, true, false, VECB>;
  constexpr int PA = kPieces, PB = SB::P, S = 2;
  __shared__ __align__(16) uint16_t lb[2][PB][kTile * kStep];
  const int lane = lane_id(), wave = threadIdx.x / kWave, lr = lane & 15, lg = lane >> 4;
  const int m0 = blockIdx.y * kTile, wm = (wave >> 1) * 16 * S, wn = (wave & 1) * 16 * S;
  const int N = g.b.rows, nt0 = blockIdx.x * per_wg, nt1 = min(nt0 + per_wg, (N + kTile - 1) / kTile);
  const int Kl = (g.K + 7) / 8 * 8;
  auto start_of = [&](int s) { return max(0, min(s * kStep, Kl - kStep)); };
  uint4 fa[KS][2][PA][S];  // (elements past K meet zeros of the other operand)
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int p = 0; p < PA; ++p)
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int64_t row = min(m0 + wm + i * 16 + lr, g.a.rows - 1);
          const int k = min(start_of(s) + h * 32 + lg * 8, int(g.a.ld) - 8);
          fa[s][h][p][i] =
              *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(g.a.p) + p * g.a.plane + row * g.a.ld + k);
        }
  f32x4 acc[S][S];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  SB sb[2];
  const int total = (nt1 - nt0) * KS;  // steps: the KS of one column tile after another
  auto load = [&](int q, auto rc) {
    sb[decltype(rc)::value].template load<false>(g.b, (nt0 + q / KS) * kTile, start_of(q % KS), g.K, g.tokens, 0, 0);
  };
  auto store = [&](int q, auto rc) {
    constexpr int r = decltype(rc)::value;
    sb[r].store(lb[r], start_of(q % KS), q % KS * kStep, g.K);
  };
  auto step = [&](int q, auto rc, auto next) {
    constexpr int r = decltype(rc)::value, s = KS == 2 ? r : 0;
    if (q + 2 < total) load(q + 2, rc);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = PB - 1; b >= 0; --b)
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const uint4 fb = *reinterpret_cast<const uint4 *>(&lb[r][b][lds_at(wn + j * 16 + lr, h * 32 + lg * 8)]);
#pragma unroll
          for (int p = PA - 1; p >= 0; --p)
            if (p + b < kPieces)
#pragma unroll
              for (int i = 0; i < S; ++i)
                acc[i][j] = mfma_bf16(__builtin_bit_cast(bf16x8, fb), __builtin_bit_cast(bf16x8, fa[s][h][p][i]), acc[i][j]);
        }
    if (q + 1 < total) store(q + 1, next);
    if (s == KS - 1) {  // the column tile is complete
      const int n0 = (nt0 + q / KS) * kTile;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int m = m0 + wm + i * 16 + lr;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const int n = n0 + wn + j * 16 + 4 * lg;  // N is a multiple of 8
          if (m < g.a.rows && n < N)
            __builtin_nontemporal_store(acc[i][j], reinterpret_cast<f32x4 *>(g.out + int64_t(m) * N + n));
        }
      }
      clear();
    }
    __syncthreads();
  };
  using R0 = std::integral_constant<int, 0>;
  using R1 = std::integral_constant<int, 1>;
  clear();
  load(0, R0{});
  load(min(1, total - 1), R1{});
  store(0, R0{});
  __syncthreads();
  int q = 0;
  for (; q + 1 < total; q += 2) {
    step(q, R0{}, R1{});
    step(q + 1, R1{}, R0{});
  }
  if (q < total) step(q, R0{}, R1{});
}

// ---- rows of logits ---------------------------------------------------------

// Sequence of token t: the last b with off[b] <= t (0 without offsets), kept
// inside [0, n).
__device__ __forceinline__ int sequence_of(const Tokens &k, int t) {
  if (!k.off) return 0;
  int lo = 0, hi = k.n;  // off[lo] <= t < off[hi], for tokens inside
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (k.off[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct RowArgs {
  Tokens tokens;
  int E, K;
  int chunk;               // tokens per workgroup
  const float *parts;      // [z][T][E] partial logits, or null: `logits` holds them
  int z;
  const float *bias;       // added to the parts
  float *logits;           // [T][E]
  const int32_t *idx;      // [T][K]
  // forward: one record per (chunk of tokens, sequence), at chunk + sequence
  float *psum;             // [slots][E]
  int32_t *count;          // [slots][E]
  int32_t *ntok;           // [slots]
  int32_t *ticket;         // set to 0 for the kernel that follows
  // backward
  const int32_t *counts, *seq_tokens;  // [n][E], [n]
  const float *dloss;
  const float *dtopk;      // [T][K] or null
  int renorm;
  uint16_t *dl;            // bf16 pieces [3][T][ld], zero past E
  int ld;
};

// Waves of the row kernels, and tokens that a wave takes at a time: eight
// tokens as 8 x 1 instead of 4 x 2 took the forward rows of 2048 tokens and
// 512 experts from 11.8 to 8.9 us, the backward rows of 256 from 5.2 to 4.3
// (of 8192, 128 experts, 8.7 to 9.1).
constexpr int kRowWaves = 8, kPair = 1;

// Experts lane, lane + 64, ... of the logits of PAIR tokens from t on (up to
// t1 - 1), all their loads in flight together; -inf past the end.  Partial logits are summed in their order.
template <int EPL, int PAIR>
__device__ __forceinline__ void load_rows(const RowArgs &a, int t, int t1, float (&l)[PAIR][EPL]) {
  const int lane = lane_id();
  const int64_t part = int64_t(a.tokens.T) * a.E;
  const float *src = a.parts ? a.parts : a.logits;
  const int nz = a.parts ? a.z : 1;
#pragma unroll
  for (int q = 0; q < PAIR; ++q)
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[q][i] = a.parts && a.bias ? a.bias[min(lane + kWave * i, a.E - 1)] : 0.f;
  // (the bias first: its place in the sum is free, its loads are not waited for)
#pragma unroll 2
  for (int z = 0; z < nz; ++z)
#pragma unroll
    for (int q = 0; q < PAIR; ++q)
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        l[q][i] += src[z * part + int64_t(min(t + q, t1 - 1)) * a.E + min(lane + kWave * i, a.E - 1)];
  if (a.parts) {
#pragma unroll
    for (int q = 0; q < PAIR; ++q)
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + kWave * i;
        if (t + q < t1 && e < a.E) a.logits[int64_t(t + q) * a.E + e] = l[q][i];
      }
  }
#pragma unroll
  for (int q = 0; q < PAIR; ++q)
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + kWave * i >= a.E) l[q][i] = -INFINITY;
}
template <int EPL>
__device__ __forceinline__ void softmax_row(float (&l)[EPL]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
  m = wave_max(m);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    l[i] = expf(l[i] - m);
    s += l[i];
  }
  const float r = 1.0f / wave_sum(s);
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] *= r;
}

// One counted token: its probabilities and its slots (slot j in lane j).
template <int EPL>
__device__ __forceinline__ void count_row(const RowArgs &a, float (&l)[EPL], int slot, float (&sum)[EPL],
                                          int32_t (&cnt)[EPL], int32_t &n) {
  softmax_row<EPL>(l);
  ++n;
#pragma unroll
  for (int i = 0; i < EPL; ++i) sum[i] += l[i];
  for (int j = 0; j < a.K; ++j) {
    const int e = read_lane_i(slot, j);
#pragma unroll
    for (int i = 0; i < EPL; ++i) cnt[i] += e == lane_id() + kWave * i;
  }
}

// Forward: a workgroup takes a chunk of consecutive tokens, 8 at a time, and
// leaves, for every sequence among them, the sums of its counted tokens'
// probabilities and the counts of their slots, at place chunk number +
// sequence number (which no other pair shares).  A wave's row is
// requested before the tokens' sequence is looked up.  2048 tokens and 512
// experts: 8.9 us for 8 MB of partial logits read and 4 MB written, a chain
// of three memory round trips (rows, the sequence table, records) and the
// exponentials; a 4-fold split of the logits' reduction made this kernel 40 us.
template <int EPL>
__global__ __launch_bounds__(kRowWaves * kWave) void balance_rows_kernel(RowArgs a) {
  __shared__ float ps[kRowWaves][EPL * kWave];
  __shared__ int32_t cs[kRowWaves][EPL * kWave], ns[kRowWaves];
  const int c0 = int(blockIdx.x) * a.chunk, c1 = min(c0 + a.chunk, a.tokens.T);
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  float sum[EPL];
  int32_t cnt[EPL], n;
  auto reset = [&] {
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum[i] = 0.f, cnt[i] = 0;
    n = 0;
  };
  auto flush = [&](int b) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) ps[wave][lane + kWave * i] = sum[i], cs[wave][lane + kWave * i] = cnt[i];
    if (lane == 0) ns[wave] = n;
    __syncthreads();
    const int64_t at = int64_t(blockIdx.x) + b;
    for (int e = threadIdx.x; e < a.E; e += kRowWaves * kWave) {
      float p = ps[0][e];
      int32_t c = cs[0][e];
#pragma unroll
      for (int w = 1; w < kRowWaves; ++w) p += ps[w][e], c += cs[w][e];
      a.psum[at * a.E + e] = p;
      a.count[at * a.E + e] = c;
    }
    if (threadIdx.x == 0) {
      int32_t all = ns[0];
#pragma unroll
      for (int w = 1; w < kRowWaves; ++w) all += ns[w];
      a.ntok[at] = all;
    }
    __syncthreads();
    reset();
  };
  reset();
  int b = -1, end = 0;  // the sequence of the tokens at hand, where it ends
  for (int c = c0; c < c1; c += kPair * kRowWaves) {
    const int tw = c + kPair * wave;
    float l[kPair][EPL];
    int slot[kPair];
    bool on[kPair];
#pragma unroll
    for (int q = 0; q < kPair; ++q) {
      const int t = min(tw + q, c1 - 1);
      slot[q] = a.idx[int64_t(t) * a.K + min(lane, a.K - 1)];  // slot j in lane j
      on[q] = !a.tokens.mask || a.tokens.mask[t];
    }
    load_rows<EPL, kPair>(a, tw, c1, l);
    int lo, hi;
    token_range(a.tokens, lo, hi);
    int t0 = max(c, lo);
    const int t2 = min(min(c + kPair * kRowWaves, c1), hi);
    while (t0 < t2) {  // the part of these tokens that lies in one sequence
      if (b < 0 || t0 >= end) {
        const int nb = __builtin_amdgcn_readfirstlane(sequence_of(a.tokens, t0));
        if (b >= 0 && nb != b) flush(b);
        b = nb;
        end = a.tokens.off ? max(a.tokens.off[b + 1], t0 + 1) : hi;
      }
      const int t1 = min(t2, end);
#pragma unroll
      for (int q = 0; q < kPair; ++q) {
        if (tw + q < t0 || tw + q >= t1 || !on[q]) continue;
        count_row<EPL>(a, l[q], slot[q], sum, cnt, n);
      }
      t0 = t1;
    }
  }
  if (b >= 0) flush(b);
}

struct FinishArgs {
  Tokens tokens;
  int E, K, chunk;
  const float *psum;
  const int32_t *count, *ntok;
  int32_t *counts, *seq_tokens;
  float *mean;
  float *terms;   // [n][blocks of 64 experts]: sum of count * mean
  int32_t *ticket;
  float *loss;
};

constexpr int kFinishThreads = 1024;
constexpr int kFinishRows = kFinishThreads / kWave;  // records summed side by side (16)

// One sequence and 64 experts: the records of its chunks, 16 side by side.
// The workgroup that is the last to finish adds up the loss, in a fixed order,
// without a launch of its own.  5.8 us at 4 sequences of 512 tokens
// and 512 experts: the records are 256 KB per 64 experts and sequence, read
// once.
__global__ __launch_bounds__(kFinishThreads) void balance_finish_kernel(FinishArgs a) {
  __shared__ float ps[kFinishRows][kWave];
  __shared__ int32_t cs[kFinishRows][kWave], ns[kFinishRows];
  const int b = blockIdx.y, lane = lane_id(), row = int(threadIdx.x) / kWave;
  const int e = blockIdx.x * kWave + lane;
  int lo = 0, hi = a.tokens.T;
  if (a.tokens.off) {
    lo = min(max(a.tokens.off[b], 0), a.tokens.T);
    hi = min(max(a.tokens.off[b + 1], lo), a.tokens.T);
  }
  const int c0 = lo / a.chunk, c1 = hi > lo ? (hi - 1) / a.chunk + 1 : c0;
  float p = 0.f;
  int32_t c = 0, n = 0;
#pragma unroll 8
  for (int q = c0 + row; q < c1; q += kFinishRows) {
    const int64_t at = int64_t(q + b) * a.E + min(e, a.E - 1);
    p += a.psum[at];
    c += a.count[at];
    n += a.ntok[q + b];
  }
  ps[row][lane] = p, cs[row][lane] = c;
  if (lane == 0) ns[row] = n;
  __syncthreads();
  if (row) return;
#pragma unroll
  for (int i = 1; i < kFinishRows; ++i) p += ps[i][lane], c += cs[i][lane], n += ns[i];
  const float m = n ? p / float(n) : 0.f;
  if (e < a.E) {
    a.mean[int64_t(b) * a.E + e] = m;
    a.counts[int64_t(b) * a.E + e] = c;
  }
  // this workgroup's part of sum_b E / (k n_b) sum_e c_be P_be
  const float term = wave_sum(e < a.E ? float(c) * m : 0.f) * (n ? float(a.E) / (float(a.K) * float(n)) : 0.f);
  const int blocks = gridDim.x, total = blocks * gridDim.y;
  int last = total == 1;
  if (lane == 0) {
    if (blockIdx.x == 0) __hip_atomic_store(a.seq_tokens + b, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(a.terms + b * blocks + blockIdx.x, term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (total > 1)
      last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
  }
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  float s = 0.f, f = 0.f;
  for (int i = lane; i < total; i += kWave)
    s += __hip_atomic_load(a.terms + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = lane; i < int(gridDim.y); i += kWave)
    f += __hip_atomic_load(a.seq_tokens + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0 ? 1.f : 0.f;
  s = wave_sum(s);
  f = wave_sum(f);
  if (lane == 0) a.loss[0] = f > 0.f ? s / f : 0.f;
}

// Backward of the rows: dl of a chunk of tokens, cut into its three planes
// (8192 tokens, 128 experts: 9.1 us for 4.2 MB read and 6.3 MB written).
template <int EPL>
__global__ __launch_bounds__(kRowWaves * kWave) void balance_dlogits_kernel(RowArgs a) {
  const int c0 = int(blockIdx.x) * a.chunk, c1 = min(c0 + a.chunk, a.tokens.T);
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int lo, hi;
  token_range(a.tokens, lo, hi);
  int filled = 0;
  for (int b = lane; b < a.tokens.n; b += kWave) filled += a.seq_tokens[b] > 0;
  const float nf = wave_sum(float(filled));
  const float up = a.dloss ? a.dloss[0] : 1.0f;
  float gb[EPL];  // d loss / d p of sequence `of`
  int of = -1;
#pragma unroll
  for (int i = 0; i < EPL; ++i) gb[i] = 0.f;
  for (int t = c0 + kPair * wave; t < c1; t += kPair * kRowWaves) {
    float l[kPair][EPL], dws[kPair], lsel[kPair];
    int slots[kPair];  // slot j in lane j
#pragma unroll
    for (int q = 0; q < kPair; ++q) {
      const int64_t tq = min(t + q, c1 - 1);
      const int64_t at = tq * a.K + min(lane, a.K - 1);
      slots[q] = a.dtopk ? a.idx[at] : -1;
      dws[q] = a.dtopk ? a.dtopk[at] : 0.f;
      if (lane >= a.K || unsigned(slots[q]) >= unsigned(a.E)) slots[q] = -1;
    }
    load_rows<EPL, kPair>(a, t, c1, l);
#pragma unroll
    for (int q = 0; q < kPair; ++q)
      lsel[q] = a.dtopk ? a.logits[int64_t(min(t + q, c1 - 1)) * a.E + max(slots[q], 0)] : 0.f;
#pragma unroll
    for (int q = 0; q < kPair; ++q) {
      if (t + q >= c1) continue;
      const bool on = t + q >= lo && t + q < hi && (!a.tokens.mask || a.tokens.mask[t + q]);
      float d[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) d[i] = 0.f;
      if (on) {
        const int b = __builtin_amdgcn_readfirstlane(sequence_of(a.tokens, t + q));
        if (b != of) {
          of = b;
          const int n = a.seq_tokens[b];
          const float fn = float(n);
          // (a zero n or nf: no token of the forward pass counted; nothing flows)
          const float coef = n > 0 && nf > 0.f ? up * float(a.E) / (float(a.K) * fn * fn * nf) : 0.f;
          const int mean = int(int64_t(n) * a.K / a.E);
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            gb[i] = coef * float(a.counts[int64_t(b) * a.E + min(lane + kWave * i, a.E - 1)] - mean);
        }
        float(&p)[EPL] = l[q];
        softmax_row<EPL>(p);
        float g[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) g[i] = gb[i];
        // the routing weights' part, slot j in lane j
        const int slot = slots[q];
        const float dw = slot >= 0 ? dws[q] : 0.f;
        float add = dw;
        if (a.dtopk && a.renorm) {
          const float ls = slot >= 0 ? lsel[q] : -INFINITY;
          const float m = wave_max(ls);
          const float ex = slot >= 0 ? expf(ls - m) : 0.f;
          const float w = ex * (1.0f / wave_sum(ex));
          const float s = wave_sum(slot >= 0 ? w * dw : 0.f);
          add = slot >= 0 ? w * (dw - s) : 0.f;
        }
        auto scatter = [&](float (&to)[EPL]) {
          for (int j = 0; j < a.K; ++j) {
            const int e = read_lane_i(slot, j);
            const float v = read_lane(add, j);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
              if (e == lane + kWave * i) to[i] += v;
          }
        };
        if (a.dtopk && !a.renorm) scatter(g);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s += p[i] * g[i];
        s = wave_sum(s);
#pragma unroll
        for (int i = 0; i < EPL; ++i) d[i] = p[i] * (g[i] - s);
        if (a.dtopk && a.renorm) scatter(d);
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + kWave * i;
        if (e < a.ld) {
          uint32_t w[kPieces];
          split<kPieces>(e < a.E ? d[i] : 0.f, w);
#pragma unroll
          for (int c = 0; c < kPieces; ++c)
            a.dl[(int64_t(c) * a.tokens.T + t + q) * a.ld + e] = uint16_t(w[c]);
        }
      }
    }
  }
}

// Partial sums of dW and of dbias, added in their order: p holds [parts]
// records of nw and then nb values, either of which may be unwanted.
__global__ __launch_bounds__(kThreads) void sum_parts_kernel(const float *p, int parts, int64_t nw, int nb, float *dw,
                                                             float *db) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= nw + nb) return;
  float s = 0.f;
#pragma unroll 8
  for (int z = 0; z < parts; ++z) s += p[int64_t(z) * (nw + nb) + i];
  if (i < nw) {
    if (dw) dw[i] = s;
  } else if (db) {
    db[i - nw] = s;
  }
}

// The whole reduction of a small call in one workgroup: rows, sums over each
// sequence's tokens and the loss, instead of further launches that cost more
// than their work (16 tokens, 8 experts: the call 8 us instead of 12.8).
constexpr int kSmallWaves = 8, kSmallPair = 2, kSmallTokens = 32, kSmallSeqs = 8;
template <int EPL>
__global__ __launch_bounds__(kSmallWaves *kWave) void balance_small_kernel(RowArgs a, FinishArgs f) {
  __shared__ float ps[kSmallWaves][EPL * kWave], ls[kSmallWaves];
  __shared__ int32_t cs[kSmallWaves][EPL * kWave], ns[kSmallWaves];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int T = a.tokens.T;
  int lo, hi;
  token_range(a.tokens, lo, hi);
  float l[kSmallPair][EPL];
  if (a.parts) {  // tokens of no sequence: their logits alone
    for (int t = kSmallPair * wave; t < lo; t += kSmallPair * kSmallWaves) load_rows<EPL, kSmallPair>(a, t, lo, l);
    for (int t = hi + kSmallPair * wave; t < T; t += kSmallPair * kSmallWaves) load_rows<EPL, kSmallPair>(a, t, T, l);
  }
  float loss = 0.f;
  int filled = 0;
  for (int b = 0; b < a.tokens.n; ++b) {
    int t0 = lo, t1 = hi;
    if (a.tokens.off) {
      t0 = min(max(a.tokens.off[b], 0), T);
      t1 = min(max(a.tokens.off[b + 1], t0), T);
    }
    float sum[EPL];
    int32_t cnt[EPL], n = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum[i] = 0.f, cnt[i] = 0;
    for (int t = t0 + kSmallPair * wave; t < t1; t += kSmallPair * kSmallWaves) {
      int slot[kSmallPair];
#pragma unroll
      for (int q = 0; q < kSmallPair; ++q) slot[q] = a.idx[int64_t(min(t + q, t1 - 1)) * a.K + min(lane, a.K - 1)];
      load_rows<EPL, kSmallPair>(a, t, t1, l);
#pragma unroll
      for (int q = 0; q < kSmallPair; ++q)
        if (t + q < t1 && (!a.tokens.mask || a.tokens.mask[t + q])) count_row<EPL>(a, l[q], slot[q], sum, cnt, n);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) ps[wave][lane + kWave * i] = sum[i], cs[wave][lane + kWave * i] = cnt[i];
    if (lane == 0) ns[wave] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) n += ns[w];
    const float weight = n ? float(a.E) / (float(a.K) * float(n)) : 0.f;
    for (int e = threadIdx.x; e < a.E; e += kSmallWaves * kWave) {
      float p = 0.f;
      int32_t c = 0;
#pragma unroll
      for (int w = 0; w < kSmallWaves; ++w) p += ps[w][e], c += cs[w][e];
      const float m = n ? p / float(n) : 0.f;
      f.mean[int64_t(b) * a.E + e] = m;
      f.counts[int64_t(b) * a.E + e] = c;
      loss += weight * float(c) * m;
    }
    if (threadIdx.x == 0) f.seq_tokens[b] = n;
    filled += n > 0;
    __syncthreads();
  }
  loss = wave_sum(loss);
  if (lane == 0) ls[wave] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) s += ls[w];
    f.loss[0] = filled ? s / float(filled) : 0.f;
  }
}

// Tokens per workgroup of the row kernels: 8 (one for each wave), more where
// the chunks would be many more than the GPU takes at once.
int chunk_tokens(int32_t T) { return T <= 8192 ? 8 : T <= 65536 ? 32 : 128; }
int chunks_of(int32_t T) { return (T + chunk_tokens(T) - 1) / chunk_tokens(T); }
int tiles_of(int64_t n, int tile = kTile) { return int((n + tile - 1) / tile); }

// Parts of a reduction of `steps` steps over `tiles` output tiles: enough
// workgroups to keep several on each of the GPU's 256 CUs, at least `least`
// steps each.
int parts_of(int64_t tiles, int steps, int want, int least) {
  int z = 1;
  while (tiles * z < want && steps >= 2 * z * least && z < 32) z *= 2;
  return z;
}
int logit_parts(const moe_layer_desc *d, int32_t T) {
  return parts_of(int64_t(tiles_of(T)) * tiles_of(d->n_experts), tiles_of(d->d_model, kStep), 512, 2);
}
int router_parts(const moe_layer_desc *d, int32_t T) {
  return parts_of(int64_t(tiles_of(d->d_model)) * tiles_of(d->n_experts), tiles_of(T, kStep), 512, 2);
}

// sums_only: bsum is wanted without the product (the first row of tiles makes it).
template <int DTA, bool KCA, int DTB, bool KCB, bool NATIVE, bool MASK>
void launch_gemm(GemmArgs g, int parts, hipStream_t s, bool sums_only = false) {
  const int steps = (g.K + kStep - 1) / kStep;
  g.per = (steps + parts - 1) / parts;
  if (!g.part) g.part = int64_t(g.a.rows) * g.b.rows;
  const dim3 grid(unsigned(tiles_of(g.b.rows)), sums_only ? 1u : unsigned(tiles_of(g.a.rows)), unsigned(parts));
  if constexpr (DTB == kDtPieces) {
    launch((split_gemm_kernel<DTA, KCA, DTB, KCB, NATIVE, MASK, true>), grid, dim3(kThreads), 0, s, g);
  } else {
    if (g.b.vec)
      launch((split_gemm_kernel<DTA, KCA, DTB, KCB, NATIVE, MASK, true>), grid, dim3(kThreads), 0, s, g);
    else
      launch((split_gemm_kernel<DTA, KCA, DTB, KCB, NATIVE, MASK, false>), grid, dim3(kThreads), 0, s, g);
  }
}

// Column tiles per workgroup: as many as leave two workgroups for each CU.
template <int DT, int KS>
void launch_dx(const GemmArgs &g, hipStream_t s) {
  const int64_t mt = tiles_of(g.a.rows);
  const int nt = tiles_of(g.b.rows), per = int(std::max<int64_t>(1, std::min<int64_t>(nt, mt * nt / 512)));
  const dim3 grid(unsigned((nt + per - 1) / per), unsigned(mt));
  if (g.b.vec) launch((balance_dx_kernel<DT, true, KS>), grid, dim3(kThreads), 0, s, g, per);
  else launch((balance_dx_kernel<DT, false, KS>), grid, dim3(kThreads), 0, s, g, per);
}

template <typename F>
void by_experts(int E, F &&f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}
template <typename F>
void by_dtype(int dt, F &&f) {
  if (dt == MOE_DT_BF16) f(std::integral_constant<int, kDtBF16>{});
  else if (dt == MOE_DT_F16) f(std::integral_constant<int, kDtF16>{});
  else f(std::integral_constant<int, kDtF32>{});
}

template <class T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}

Operand x_operand(const moe_layer_desc *d, int32_t T, const void *x, bool kc) {
  return Operand{x, d->d_model, kc ? T : d->d_model, 1};  // d_model is a multiple of 8
}

}  // namespace

BalanceWorkspace balance_workspace_layout(const moe_layer_desc *d, int32_t T, int32_t n_seqs) {
  BalanceWorkspace b{};
  const size_t E = d->n_experts, D = d->d_model, slots = size_t(chunks_of(T)) + n_seqs;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) & ~size_t(255);
    return at;
  };
  const int zl = logit_parts(d, T);
  b.parts = take(zl > 1 ? size_t(zl) * T * E * 4 : 0);
  b.psum = take(slots * E * 4);
  b.count = take(slots * E * 4);
  b.ntok = take(slots * 4);
  b.terms = take(size_t(n_seqs) * ((E + kWave - 1) / kWave) * 4);
  b.ticket = take(4);
  const size_t fwd = o;
  o = 0;
  const int zw = router_parts(d, T);
  b.ld = int((E + 7) / 8 * 8);
  b.dl = take(size_t(kPieces) * T * b.ld * 2);
  b.dwp = take(zw > 1 ? size_t(zw) * (D + 1) * E * 4 : 0);
  b.total = std::max(std::max(fwd, o), size_t(256));
  return b;
}

void launch_balance_loss(const moe_layer_desc *d, int32_t T, const void *x, const void *w_router, const float *bias,
                         const int32_t *topk_idx, const uint8_t *mask, int32_t n_seqs, const int32_t *seq_off,
                         float *logits, int32_t *counts, int32_t *seq_tokens, float *mean, float *loss, void *ws,
                         void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int E = d->n_experts, D = d->d_model;
  const BalanceWorkspace L = balance_workspace_layout(d, T, n_seqs);
  const Tokens tk{mask, seq_off, n_seqs, T};
  const int z = T > 0 ? logit_parts(d, T) : 1;
  if (T > 0) {
    GemmArgs g{};
    g.a = x_operand(d, T, x, true);
    g.b = Operand{w_router, E, E, E % 4 == 0};
    g.K = D;
    g.out = z > 1 ? at<float>(ws, L.parts) : logits;
    g.bias = z > 1 ? nullptr : bias;
    by_dtype(d->act_dtype, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      launch_gemm<DT, true, DT, false, DT == kDtF16, false>(g, z, s);
    });
  }
  RowArgs r{};
  r.tokens = tk, r.E = E, r.K = d->top_k, r.chunk = chunk_tokens(T);
  r.parts = z > 1 ? at<float>(ws, L.parts) : nullptr, r.z = z, r.bias = bias;
  r.logits = logits, r.idx = topk_idx;
  r.psum = at<float>(ws, L.psum), r.count = at<int32_t>(ws, L.count), r.ntok = at<int32_t>(ws, L.ntok);
  r.ticket = at<int32_t>(ws, L.ticket);
  if (T <= kSmallTokens && n_seqs <= kSmallSeqs && E <= 512) {
    FinishArgs f{};
    f.counts = counts, f.seq_tokens = seq_tokens, f.mean = mean, f.loss = loss;
    by_experts(E, [&](auto n) {
      constexpr int EPL = decltype(n)::value;
      if constexpr (EPL <= 8)
        launch((balance_small_kernel<EPL>), dim3(1), dim3(kSmallWaves * kWave), 0, s, r, f);
    });
    return;
  }
  by_experts(E, [&](auto n) {  // (without tokens: for the ticket alone)
    launch((balance_rows_kernel<decltype(n)::value>), dim3(std::max(1, chunks_of(T))), dim3(kRowWaves * kWave), 0, s, r);
  });
  FinishArgs f{tk, E, d->top_k, chunk_tokens(T), at<float>(ws, L.psum), at<int32_t>(ws, L.count), at<int32_t>(ws, L.ntok),
               counts, seq_tokens, mean, at<float>(ws, L.terms), at<int32_t>(ws, L.ticket), loss};
  const int blocks = (E + kWave - 1) / kWave;
  launch(balance_finish_kernel, dim3(blocks, n_seqs), dim3(kFinishThreads), 0, s, f);
}

void launch_balance_backward(const moe_layer_desc *d, int32_t T, const void *x, const void *w_router,
                             const int32_t *topk_idx, const uint8_t *mask, int32_t n_seqs, const int32_t *seq_off,
                             const float *logits, const int32_t *counts, const int32_t *seq_tokens,
                             const float *dloss, const float *dtopk_w, float *dx, float *dw, float *dbias, void *ws,
                             void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int E = d->n_experts, D = d->d_model;
  const BalanceWorkspace L = balance_workspace_layout(d, T, n_seqs);
  const Tokens tk{mask, seq_off, n_seqs, T};
  const Operand dl{at<void>(ws, L.dl), L.ld, T, 1, int64_t(T) * L.ld};
  if (T > 0) {
    RowArgs r{};
    r.tokens = tk, r.E = E, r.K = d->top_k, r.chunk = chunk_tokens(T);
    r.logits = const_cast<float *>(logits), r.idx = topk_idx;
    r.counts = counts, r.seq_tokens = seq_tokens, r.dloss = dloss, r.dtopk = dtopk_w, r.renorm = d->renormalize;
    r.dl = at<uint16_t>(ws, L.dl), r.ld = L.ld;
    by_experts(E, [&](auto n) {
      launch((balance_dlogits_kernel<decltype(n)::value>), dim3(chunks_of(T)), dim3(kRowWaves * kWave), 0, s, r);
    });
    if (dx) {
      GemmArgs g{};
      g.a = dl;
      const int esz = int(act_bytes(d));
      g.b = Operand{w_router, E, D, E % (16 / esz) == 0};
      g.K = E, g.out = dx;
      by_dtype(d->act_dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (E <= kStep) launch_dx<DT, 1>(g, s);
        else if (E <= 2 * kStep) launch_dx<DT, 2>(g, s);
        else launch_gemm<kDtPieces, true, DT, true, false, false>(g, 1, s);
      });
    }
  }
  if (dw || dbias) {
    const int z = router_parts(d, T);
    const int64_t nw = int64_t(D) * E;
    float *const parts = at<float>(ws, L.dwp);
    GemmArgs g{};
    g.a = x_operand(d, T, x, false);
    g.b = dl;
    g.b.rows = E;
    g.K = T, g.tokens = tk;
    g.out = z > 1 ? parts : dw;
    g.bsum = z > 1 ? parts + nw : dbias;
    g.part = g.bpart = nw + E;
    by_dtype(d->act_dtype, [&](auto dt) {
      launch_gemm<decltype(dt)::value, false, kDtPieces, false, false, true>(g, z, s, !dw);
    });
    if (z > 1)
      launch(sum_parts_kernel, dim3(unsigned((nw + E + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
             static_cast<const float *>(parts), z, nw, E, dw, dbias);
  }
}

}  // namespace moe
