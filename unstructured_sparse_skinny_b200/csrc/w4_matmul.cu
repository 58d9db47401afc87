// Skinny product with 4-bit weights: C[N][M] = B[N][K] x A[M][K]^T, N <= 256.
// Few tokens run on the strips' engine (w4_strips.cuh), more on tcgen05
// (w4_gemm.cu).
#include <atomic>

#include "w4_strips.cuh"

namespace flashspmm {
namespace {

struct MatmulParams {
  W4Dev A;
  const uint16_t* B;
  int64_t ldb;
  void* C;
  int64_t ldc;
  bool c_f32;
  int32_t N;
  int32_t pairs;  // of strips a CTA
  uint32_t shared;
};

template <typename T, int NG, int NT>
__global__ void __launch_bounds__(kStripThreads, 2) w4_matmul_kernel(const MatmulParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t pair0 = blockIdx.x * p.pairs;
  const int32_t strip = min(2 * (pair0 + warp % p.pairs), p.A.strips - 1);
  const StripAt at[2] = {StripAt(p.A, p.A.unit(0, strip, 0), lane),
                         StripAt(p.A, p.A.unit(0, min(strip + 1, p.A.strips - 1), 0), lane)};
  float acc[2][NT][4] = {};
  strip_product<T, NG, NT>(
      at, p.A.units, p.A.K, p.N, p.pairs, smem, p.shared, [&](int32_t n) { return p.B + n * p.ldb; }, acc);
  strip_reduce<NT, false>(acc, p.pairs, p.N, smem, [&](int pair, int32_t n, int32_t row, float sum, float) {
    const int64_t m = static_cast<int64_t>(pair0 + pair) * 32 + row;
    if (m >= p.A.M) return;
    if (p.c_f32)
      static_cast<float*>(p.C)[n * p.ldc + m] = sum;
    else
      static_cast<T*>(p.C)[n * p.ldc + m] = from_float<T>(sum);
  });
}

template <typename T, int NG, int NT>
cudaError_t launch_as(MatmulParams& p, cudaStream_t s) {
  auto kernel = w4_matmul_kernel<T, NG, NT>;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(allowed.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStripShared);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(uint64_t(1) << (dev & 63));
  }
  const int32_t pairs = (p.A.strips + 1) / 2;
  p.pairs = pairs_per_cta(1, pairs);
  p.shared = strip_shared(p.N, p.A.units, NT);
  kernel<<<(pairs + p.pairs - 1) / p.pairs, kStripThreads, p.shared, s>>>(p);
  return cudaGetLastError();
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
  MatmulParams p{};
  p.A = w4_dev(in);
  if (!rows_aligned(B, ldb, p.A.K)) {
    const cudaError_t e = launch_align_rows(B, ldb, N, p.A.K, workspace, s);
    if (e != cudaSuccess) return e;
    B = workspace;
    ldb = aligned_k(p.A.K);
    p.A.K = static_cast<int32_t>(ldb);
  }
  p.B = static_cast<const uint16_t*>(B);
  p.ldb = ldb;
  p.C = C;
  p.ldc = ldc;
  p.c_f32 = c_f32;
  p.N = N;
  cudaError_t e;
#define FLASHSPMM_BY_TILES(T, NG) (N <= 8 ? launch_as<T, NG, 1>(p, s) : launch_as<T, NG, 2>(p, s))
#define FLASHSPMM_BY_GROUP(T)                          \
  e = p.A.group == 128  ? FLASHSPMM_BY_TILES(T, 1)     \
      : p.A.group == 64 ? FLASHSPMM_BY_TILES(T, 2)     \
                        : FLASHSPMM_BY_TILES(T, 4)
  if (in->dtype == FLASHSPMM_F16)
    FLASHSPMM_BY_GROUP(__half);
  else
    FLASHSPMM_BY_GROUP(__nv_bfloat16);
#undef FLASHSPMM_BY_GROUP
#undef FLASHSPMM_BY_TILES
  note_launch();
  return e;
}

}  // namespace flashspmm
