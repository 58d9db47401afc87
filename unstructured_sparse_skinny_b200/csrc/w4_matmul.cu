// Skinny product with 4-bit weights: C[N][M] = B[N][K] x A[M][K]^T, N <= 256.
//
// A CTA owns R strips of 16 rows and NT tiles of 8 activation rows; its warps
// share the units of 128 columns and the CTA adds their sums in a fixed order.
#include "w4.cuh"

namespace flashspmm {
namespace {

constexpr int kWarps = 8;

template <typename T, int NG, int R, int NT>
__global__ void __launch_bounds__(kWarps * 32) w4_matmul_kernel(W4Dev A, const uint16_t* __restrict__ B, int64_t ldb,
                                                                void* C, int64_t ldc, bool c_f32, int32_t N) {
  constexpr int kRows = 16 * R, kPitch = kRows + 4;  // + 4: the lanes of a fragment store to 32 banks
  __shared__ float red[kWarps][NT * 8][kPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int32_t n0 = blockIdx.y * (NT * 8);
  const int32_t strip0 = blockIdx.x * R;
  const int tiles = min(NT, (N - n0 + 7) / 8);
  float acc[R][NT][4] = {};
  const auto act = [&](int nt, int32_t k) {
    const int32_t n = n0 + 8 * nt + g;
    return load_act8<true>(n < N ? B + n * ldb : nullptr, k + 8 * t, A.K);
  };
  for (int32_t u = warp; u < A.units; u += kWarps) {
    uint4 c[R][2];
    W4Groups<T, NG> grp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t unit = A.unit(0, min(strip0 + r, A.strips - 1), u);
      c[r][0] = ld_stream(A.codes + unit * 64 + lane);
      c[r][1] = ld_stream(A.codes + unit * 64 + 32 + lane);
      grp[r].load(A, unit, g);
    }
    w4_unit<T, NG, R, NT>(c, grp, u * kW4UnitCols, tiles, act, acc);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][nt * 8 + 2 * t + (i & 1)][r * 16 + g + 8 * (i >> 1)] = acc[r][nt][i];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 8 * kRows; i += kWarps * 32) {
    const int n = i / kRows, row = i - n * kRows;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += red[w][n][row];
    const int64_t m = static_cast<int64_t>(strip0) * 16 + row;
    if (n0 + n < N && m < A.M) {
      if (c_f32)
        static_cast<float*>(C)[(n0 + n) * ldc + m] = sum;
      else
        static_cast<T*>(C)[(n0 + n) * ldc + m] = from_float<T>(sum);
    }
  }
}

template <typename T, int NG>
void matmul_as(const W4Dev& A, const uint16_t* B, int64_t ldb, void* C, int64_t ldc, bool c_f32, int32_t N,
               cudaStream_t s) {
#define FLASHSPMM_MATMUL(R, NT)                                                                                     \
  w4_matmul_kernel<T, NG, R, NT><<<dim3((A.strips + R - 1) / R, (N + NT * 8 - 1) / (NT * 8)), kWarps * 32, 0, s>>>( \
      A, B, ldb, C, ldc, c_f32, N)
  if (N <= 8)
    FLASHSPMM_MATMUL(2, 1);
  else
    FLASHSPMM_MATMUL(2, 2);
#undef FLASHSPMM_MATMUL
}

__global__ void __launch_bounds__(256) align_rows_kernel(const uint16_t* __restrict__ X, int64_t ld, int32_t K,
                                                         int64_t pitch, uint16_t* __restrict__ out) {
  const uint16_t* row = X + blockIdx.y * ld;
  const int64_t k = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (k >= pitch) return;
  *reinterpret_cast<uint4*>(out + blockIdx.y * pitch + k) = load_act8<false>(row, static_cast<int32_t>(k), K);
}

}  // namespace

bool rows_aligned(const void* X, int64_t ld, int32_t K) {
  return (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && ld % 8 == 0 && K % 8 == 0;
}

cudaError_t launch_align_rows(const void* X, int64_t ld, int32_t rows, int32_t K, void* out, cudaStream_t s) {
  const int64_t pitch = aligned_k(K);
  align_rows_kernel<<<dim3(static_cast<unsigned>((pitch / 8 + 255) / 256), rows), 256, 0, s>>>(
      static_cast<const uint16_t*>(X), ld, K, pitch, static_cast<uint16_t*>(out));
  note_launch();
  return cudaGetLastError();
}

size_t w4_matmul_workspace(int32_t M, int32_t K, int32_t N, bool aligned) {
  if (N > kW4FragmentTokens) return w4_gemm_workspace(M, K, N);
  return aligned ? 0 : static_cast<size_t>(N) * aligned_k(K) * 2;
}

cudaError_t launch_w4_matmul(const flashspmm_w4* in, const void* B, int64_t ldb, void* C, int64_t ldc, bool c_f32,
                             int32_t N, void* workspace, cudaStream_t s) {
  if (N > kW4FragmentTokens) return launch_w4_gemm(in, B, ldb, C, ldc, c_f32, N, workspace, s);
  W4Dev A = w4_dev(in);
  if (!rows_aligned(B, ldb, A.K)) {
    const cudaError_t e = launch_align_rows(B, ldb, N, A.K, workspace, s);
    if (e != cudaSuccess) return e;
    B = workspace;
    ldb = aligned_k(A.K);
    A.K = static_cast<int32_t>(min64(ldb, INT32_MAX));
  }
  const uint16_t* b = static_cast<const uint16_t*>(B);
#define FLASHSPMM_BY_GROUP(T)                                \
  if (A.group == 128)                                        \
    matmul_as<T, 1>(A, b, ldb, C, ldc, c_f32, N, s);         \
  else if (A.group == 64)                                    \
    matmul_as<T, 2>(A, b, ldb, C, ldc, c_f32, N, s);         \
  else                                                       \
    matmul_as<T, 4>(A, b, ldb, C, ldc, c_f32, N, s)
  if (in->dtype == FLASHSPMM_F16) {
    FLASHSPMM_BY_GROUP(__half);
  } else {
    FLASHSPMM_BY_GROUP(__nv_bfloat16);
  }
#undef FLASHSPMM_BY_GROUP
  note_launch();
  return cudaGetLastError();
}

}  // namespace flashspmm
