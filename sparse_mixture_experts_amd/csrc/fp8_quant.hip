// fp8_quant.hip -- e4m3 quantisation in blocks of 128: rows (one scale for
// each 128 columns of a row, for activations) and matrices (one scale for
// each 128 x 128 block, for weights).
//
// Both kernels read their input once and hold it in registers between the
// maximum and the rounding, so they are bound by memory: an element costs its
// own bytes and one byte of code.  Matrices of 128 x 1536 x 2048 bf16 values
// (0.81 GB read, 0.40 GB written): 221 us, 5.45 TB/s (a large copy
// reaches 5.1).  32 rows of 2048: 5 us, a launch and one memory round trip.
#include "fp8_common.h"
#include "launch.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                       // elements per lane and row: one 16-byte store of codes
constexpr int kLanes = kFp8Block / kPer;       // lanes per row of a block (8)
constexpr int kRowsPass = kThreads / kLanes;   // rows per pass of the workgroup (32)

// 16 consecutive elements as fp32.
template <int DT>
__device__ __forceinline__ void load16(const void *p, int64_t i, float (&v)[kPer]) {
  if constexpr (DT == kDtF32) {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4 f = q[u];
      v[4 * u] = f.x, v[4 * u + 1] = f.y, v[4 * u + 2] = f.z, v[4 * u + 3] = f.w;
    }
  } else {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 w = q[u];
      const uint32_t s[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[8 * u + 2 * j] = half_lo<DT>(s[j]), v[8 * u + 2 * j + 1] = half_hi<DT>(s[j]);
    }
  }
}

__device__ __forceinline__ float absmax16(const float (&v)[kPer]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// PASSING: codes that nothing reads soon (a loaded layer's weights) do not
// displace what the L2 holds: 221 us instead of 230.
template <bool PASSING>
__device__ __forceinline__ void store16(uint8_t *p, const float (&v)[kPer], const Fp8Quant &q) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 w;
#pragma unroll
  for (int u = 0; u < 4; ++u) w[u] = fp8_pack4(q(v[4 * u]), q(v[4 * u + 1]), q(v[4 * u + 2]), q(v[4 * u + 3]));
  if constexpr (PASSING) __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(p));
  else *reinterpret_cast<u32x4 *>(p) = w;
}

// A workgroup takes 32 rows of one column block (their scales are then one
// 128-byte piece of the [block][row] table); 8 lanes hold a row's 128
// columns.  grid: column blocks fastest, then groups of 32 rows.
template <int DT>
__global__ __launch_bounds__(kThreads) void fp8_rows_kernel(const void *x, int rows, int cols, int nb, uint8_t *codes,
                                                            float *scales) {
  const int j = int(blockIdx.x % unsigned(nb));
  const int r = int(blockIdx.x / unsigned(nb)) * kRowsPass + int(threadIdx.x) / kLanes;
  const int c = j * kFp8Block + int(threadIdx.x) % kLanes * kPer;
  if (r >= rows) return;  // whole groups of 8 lanes
  float v[kPer] = {};
  const int64_t at = int64_t(r) * cols + c;
  if (c < cols) load16<DT>(x, at, v);  // cols is a multiple of 16
  const Fp8Quant q(max8_lanes(absmax16(v)));
  if (c < cols) store16<false>(codes + at, v, q);
  if (threadIdx.x % kLanes == 0) scales[int64_t(j) * rows + r] = q.scale;
}

// A workgroup takes one 128 x 128 block: four rows of 16 elements per lane.
template <int DT>
__global__ __launch_bounds__(kThreads) void fp8_blocks_kernel(const void *x, int rows, int cols, int nbr, int nbc,
                                                              uint8_t *codes, float *scales) {
  constexpr int kPass = kFp8Block / kRowsPass;  // 4
  __shared__ float wmax[kThreads / kWave];
  const int jc = int(blockIdx.x % unsigned(nbc));
  const int rest = int(blockIdx.x / unsigned(nbc));
  const int jr = rest % nbr;
  const int64_t base = int64_t(rest / nbr) * rows * cols;
  const int c = jc * kFp8Block + int(threadIdx.x) % kLanes * kPer;
  const int r0 = jr * kFp8Block + int(threadIdx.x) / kLanes;
  float v[kPass][kPer] = {};
  float m = 0.f;
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int r = r0 + p * kRowsPass;
    if (r < rows && c < cols) load16<DT>(x, base + int64_t(r) * cols + c, v[p]);
  }
#pragma unroll
  for (int p = 0; p < kPass; ++p) m = fmaxf(m, absmax16(v[p]));
  m = wave_max(m);
  if (lane_id() == 0) wmax[threadIdx.x / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / kWave; ++i) m = fmaxf(m, wmax[i]);
  const Fp8Quant q(m);
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int r = r0 + p * kRowsPass;
    if (r < rows && c < cols) store16<true>(codes + base + int64_t(r) * cols + c, v[p], q);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = q.scale;
}

// The transpose of one 128 x 128 block of codes through LDS, 16 codes a load
// and a store; its scale moves to the mirrored place.
__global__ __launch_bounds__(kThreads) void fp8_transpose_kernel(const uint8_t *w, const float *ws, int N, int K,
                                                                 int nbn, int nbk, uint8_t *wt, float *wts) {
  __shared__ uint8_t t[kFp8Block][kFp8Block + 4];
  const int jk = int(blockIdx.x % unsigned(nbk));
  const int rest = int(blockIdx.x / unsigned(nbk)), jn = rest % nbn, m = rest / nbn;
  const int64_t base = int64_t(m) * N * K;
  const int r = int(threadIdx.x) / kLanes, c = int(threadIdx.x) % kLanes * kPer;
#pragma unroll
  for (int p = 0; p < kFp8Block; p += kRowsPass) {
    const int n = jn * kFp8Block + p + r, k = jk * kFp8Block + c;
    if (n < N && k < K) {
      const uint4 v = *reinterpret_cast<const uint4 *>(w + base + int64_t(n) * K + k);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t *>(&t[p + r][c + 4 * i]) = u[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < kFp8Block; p += kRowsPass) {
    const int k = jk * kFp8Block + p + r, n = jn * kFp8Block + c;
    if (k < K && n < N) {  // N is a multiple of 16
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = t[c + 4 * i][p + r] | uint32_t(t[c + 4 * i + 1][p + r]) << 8 | uint32_t(t[c + 4 * i + 2][p + r]) << 16 |
               uint32_t(t[c + 4 * i + 3][p + r]) << 24;
      *reinterpret_cast<uint4 *>(wt + base + int64_t(k) * N + n) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  if (threadIdx.x == 0) wts[(int64_t(m) * nbk + jk) * nbn + jn] = ws[(int64_t(m) * nbn + jn) * nbk + jk];
}

}  // namespace

void launch_fp8_transpose(int32_t n_matrices, int32_t N, int32_t K, const uint8_t *w, const float *w_scales,
                          uint8_t *wt, float *wt_scales, void *stream) {
  const int nbn = (N + kFp8Block - 1) / kFp8Block, nbk = (K + kFp8Block - 1) / kFp8Block;
  launch(fp8_transpose_kernel, dim3(unsigned(n_matrices) * unsigned(nbn) * unsigned(nbk)), dim3(kThreads), 0,
         static_cast<hipStream_t>(stream), w, w_scales, N, K, nbn, nbk, wt, wt_scales);
}

void launch_fp8_rows(const void *x, int32_t dtype, int32_t rows, int32_t cols, uint8_t *codes, float *scales,
                     void *stream) {
  const int nb = (cols + kFp8Block - 1) / kFp8Block;
  const dim3 grid(unsigned(nb) * unsigned((rows + kRowsPass - 1) / kRowsPass));
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto kern) { launch(kern, grid, dim3(kThreads), 0, s, x, rows, cols, nb, codes, scales); };
  if (dtype == MOE_DT_BF16) go(fp8_rows_kernel<kDtBF16>);
  else if (dtype == MOE_DT_F16) go(fp8_rows_kernel<kDtF16>);
  else go(fp8_rows_kernel<kDtF32>);
}

void launch_fp8_blocks(const void *x, int32_t dtype, int32_t matrices, int32_t rows, int32_t cols, uint8_t *codes,
                       float *scales, void *stream) {
  const int nbr = (rows + kFp8Block - 1) / kFp8Block, nbc = (cols + kFp8Block - 1) / kFp8Block;
  const dim3 grid(unsigned(matrices) * unsigned(nbr) * unsigned(nbc));
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto kern) { launch(kern, grid, dim3(kThreads), 0, s, x, rows, cols, nbr, nbc, codes, scales); };
  if (dtype == MOE_DT_BF16) go(fp8_blocks_kernel<kDtBF16>);
  else if (dtype == MOE_DT_F16) go(fp8_blocks_kernel<kDtF16>);
  else go(fp8_blocks_kernel<kDtF32>);
}

}  // namespace moe
