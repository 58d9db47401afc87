// Skinny product with 4-bit weights: C[N][M] = B[N][K] x A[M][K]^T, N <= 256.
// Few tokens and small products run here, the others on tcgen05 (w4_gemm.cu).

#include "w4_strips.cuh"

namespace flashspmm {
namespace {

constexpr int kMatmulWarps = 12;

struct MatmulParams {
  W4Dev A;
  const uint16_t* B;
  int64_t ldb;
  void* C;
  int64_t ldc;
  bool c_f32;
  int32_t N;
};

// One strip of 16 rows and eight tokens a CTA: its warps have the units in
// turn and add up at the end.  Codes come two units ahead; the activations,
// which all CTAs read again, from L1 and L2 as the fragments need them.  What
// bounds it is turning codes into fragments, 174 instructions a record: one and
// eight tokens of 12288^2 take 23 and 25 us, one of 49152 x 12288 71, two thirds
// of what HBM allows.  (Activations staged in shared memory first delay the
// short-lived CTAs more than they save, 29 and 54 us; CTAs that stay and read on
// into the next strip, 84 for 49152 x 12288; codes through a ring in shared
// memory, 78.)
template <typename T, int NG>
__global__ void __launch_bounds__(kMatmulWarps * 32, 2) w4_matmul_kernel(const MatmulParams p) {
  constexpr int kAhead = 2;
  __shared__ float red[kMatmulWarps][8][20];  // 16 rows, and the fragments' stores meet all banks
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint8_t* strip = p.A.at(p.A.unit(0, blockIdx.x, 0));
  const int32_t pitch = 8 * p.A.record;  // from a strip's unit to its next
  const int32_t units = p.A.units;
  const int32_t n0 = blockIdx.y * 8;
  const uint16_t* row = n0 + g < p.N ? p.B + (n0 + g) * p.ldb + 8 * t : nullptr;
  StripUnit<T, NG> buf[kAhead][1];
#pragma unroll
  for (int d = 0; d < kAhead; ++d)
    if (warp + d * kMatmulWarps < units) buf[d][0].read(strip + static_cast<int64_t>(warp + d * kMatmulWarps) * pitch, lane, p.A.zeros);
  float acc[1][1][4] = {};
  for (int32_t base = warp; base < units; base += kAhead * kMatmulWarps) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int32_t u = base + d * kMatmulWarps;
      if (u >= units) break;
      uint4 x[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        x[b] = make_uint4(0, 0, 0, 0);
        if (row && u * 128 + 32 * b + 8 * t < p.A.K) x[b] = __ldg(reinterpret_cast<const uint4*>(row + u * 128 + 32 * b));
      }
      strip_unit<T, NG, 1, 1, 1>(buf[d], 1, [&](int, int b, int) { return x[b]; }, acc);
      const int32_t next = u + kAhead * kMatmulWarps;
      if (next < units) buf[d][0].read(strip + static_cast<int64_t>(next) * pitch, lane, p.A.zeros);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[warp][2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[0][0][i];
  __syncthreads();
  if (threadIdx.x < 128) {
    const int i = threadIdx.x >> 4, r = threadIdx.x & 15, n = n0 + i;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kMatmulWarps; ++w) sum += red[w][i][r];
    sum = w4_raise<T>(sum);
    const int64_t m = static_cast<int64_t>(blockIdx.x) * 16 + r;
    if (n < p.N && m < p.A.M) {
      if (p.c_f32)
        static_cast<float*>(p.C)[n * p.ldc + m] = sum;
      else
        static_cast<T*>(p.C)[n * p.ldc + m] = from_float<T>(sum);
    }
  }
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

// Eight tokens at a time here, or all at once by tcgen05?  Fitted, in us: here
// 3.5 and 0.24 per 1000 records for every eight tokens, 0.3 with groups of 32;
// there 8.5 (two kernels, the joining of blocks) and 0.27 per 1000 records, for
// fp32 output, whose records are two steps there, 0.7.  The two round differently,
// so the choice goes by the sizes alone and not by where the activations lie
// (those that have to be copied first cost 2.5 us more here).  Measured, here and
// there, codes from HBM: 4096^2, 24 tokens 16 and 17, 32 tokens 21 and 19; 12288^2,
// 16 tokens 53 and 34; fp32 output of 8192^2, 24 tokens 41 and 42, 32 tokens 47 and 42.
static bool by_fragments(const flashspmm_w4* A, int32_t N, bool c_f32) {
  if (N <= 8) return true;
  const double records = 8e-3 * w4_blocks(A->M) * w4_units(A->K);
  const double each = A->group == 32 ? 0.3 : 0.24;
  return 3.5 + each * ((N + 7) / 8) * records < 8.5 + (c_f32 ? 0.7 : 0.27) * records;
}

// Enough for either output: fp32 goes by fragments whenever 16 bits do, and the image that tcgen05 takes is larger
// than a copy of the activations.
size_t w4_matmul_workspace(const flashspmm_w4* A, int32_t N, bool aligned) {
  if (!by_fragments(A, N, false)) return w4_gemm_workspace(A->M, A->K, N);
  return aligned ? 0 : static_cast<size_t>(N) * aligned_k(A->K) * 2;
}

cudaError_t launch_w4_matmul(const flashspmm_w4* in, const void* B, int64_t ldb, void* C, int64_t ldc, bool c_f32,
                             int32_t N, void* workspace, cudaStream_t s) {
  if (!by_fragments(in, N, c_f32)) return launch_w4_gemm(in, B, ldb, C, ldc, c_f32, N, workspace, s);
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
  const dim3 grid(p.A.strips, (N + 7) / 8);
#define FLASHSPMM_BY_GROUP(T)                                                                \
  p.A.group == 128  ? w4_matmul_kernel<T, 1><<<grid, kMatmulWarps * 32, 0, s>>>(p)         \
  : p.A.group == 64 ? w4_matmul_kernel<T, 2><<<grid, kMatmulWarps * 32, 0, s>>>(p)         \
                    : w4_matmul_kernel<T, 4><<<grid, kMatmulWarps * 32, 0, s>>>(p)
  if (in->dtype == FLASHSPMM_F16)
    FLASHSPMM_BY_GROUP(__half);
  else
    FLASHSPMM_BY_GROUP(__nv_bfloat16);
#undef FLASHSPMM_BY_GROUP
  note_launch();
  return cudaGetLastError();
}

}  // namespace flashspmm
