// extern "C" entry points of the 4-bit weights: argument checks, then the
// kernel launchers.  Same conventions as flashspmm_api.cu.
#include "w4.cuh"

using namespace flashspmm;

namespace {

constexpr int32_t kMaxExtent = 1 << 30;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool have_device() {
  int n = 0;
  return cudaGetDeviceCount(&n) == cudaSuccess && n > 0;
}

flashspmm_status done(cudaError_t e) { return e == cudaSuccess ? FLASHSPMM_OK : FLASHSPMM_ERR_CUDA; }

flashspmm_status check_shape(int32_t M, int32_t K, int32_t count, int32_t group) {
  if (M < 0 || K < 0 || count < 1) return FLASHSPMM_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return FLASHSPMM_ERR_UNSUPPORTED;
  if (M > kMaxExtent || K > kMaxExtent) return FLASHSPMM_ERR_UNSUPPORTED;
  return FLASHSPMM_OK;
}

// -1 if 64 bits do not hold it.
int64_t data_bytes(int32_t M, int32_t K, int32_t count, int32_t group, bool zeros) {
  const int64_t one = static_cast<int64_t>(w4_blocks(M)) * 8 * w4_units(K) * w4_record_bytes(kW4UnitCols / group, zeros);
  int64_t all = 0;
  return __builtin_mul_overflow(one, static_cast<int64_t>(count), &all) ? -1 : all;
}

flashspmm_status check_w4(const flashspmm_w4* A) {
  if (!A || A->zeros < 0 || A->zeros > 1) return FLASHSPMM_ERR_INVALID_ARG;
  const flashspmm_status st = check_shape(A->M, A->K, A->count, A->group);
  if (st != FLASHSPMM_OK) return st;
  if (A->dtype != FLASHSPMM_F16 && A->dtype != FLASHSPMM_BF16) return FLASHSPMM_ERR_UNSUPPORTED;
  if (data_bytes(A->M, A->K, A->count, A->group, A->zeros != 0) < 0) return FLASHSPMM_ERR_UNSUPPORTED;
  if (A->M > 0 && A->K > 0 && !A->data) return FLASHSPMM_ERR_INVALID_ARG;
  if (!aligned16(A->data)) return FLASHSPMM_ERR_ALIGNMENT;
  return FLASHSPMM_OK;
}

bool on2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

int64_t flashspmm_w4_bytes(int32_t M, int32_t K, int32_t count, int32_t group, int32_t zeros) {
  if (check_shape(M, K, count, group) != FLASHSPMM_OK || zeros < 0 || zeros > 1) return -1;
  return data_bytes(M, K, count, group, zeros != 0);
}

flashspmm_status flashspmm_w4_encode(const void* W, int64_t ldw, int32_t symmetric, const flashspmm_w4* A,
                                     void* stream) {
  const flashspmm_status st = check_w4(A);
  if (st != FLASHSPMM_OK) return st;
  if (ldw < A->K || (symmetric != 0) != (A->zeros == 0)) return FLASHSPMM_ERR_INVALID_ARG;
  if (A->M == 0 || A->K == 0) return FLASHSPMM_OK;
  if (!W) return FLASHSPMM_ERR_INVALID_ARG;
  if (!on2(W)) return FLASHSPMM_ERR_ALIGNMENT;
  if (!have_device()) return FLASHSPMM_ERR_NO_DEVICE;
  return done(launch_w4_encode(W, ldw, A, symmetric, static_cast<cudaStream_t>(stream)));
}

flashspmm_status flashspmm_w4_pack(const uint8_t* codes, const void* scales, const uint8_t* zeros,
                                   const flashspmm_w4* A, void* stream) {
  const flashspmm_status st = check_w4(A);
  if (st != FLASHSPMM_OK) return st;
  if ((zeros == nullptr) != (A->zeros == 0)) return FLASHSPMM_ERR_INVALID_ARG;
  if (A->M == 0 || A->K == 0) return FLASHSPMM_OK;
  if (!codes || !scales) return FLASHSPMM_ERR_INVALID_ARG;
  if (!on2(scales)) return FLASHSPMM_ERR_ALIGNMENT;
  if (!have_device()) return FLASHSPMM_ERR_NO_DEVICE;
  return done(launch_w4_pack(codes, scales, zeros, A, static_cast<cudaStream_t>(stream)));
}

flashspmm_status flashspmm_w4_decode(const flashspmm_w4* A, void* W, int32_t w_dtype, void* stream) {
  const flashspmm_status st = check_w4(A);
  if (st != FLASHSPMM_OK) return st;
  if (w_dtype != A->dtype && w_dtype != FLASHSPMM_F32) return FLASHSPMM_ERR_UNSUPPORTED;
  if (A->M == 0 || A->K == 0) return FLASHSPMM_OK;
  if (!W) return FLASHSPMM_ERR_INVALID_ARG;
  if (w_dtype == FLASHSPMM_F32 ? !on4(W) : !on2(W)) return FLASHSPMM_ERR_ALIGNMENT;
  if (!have_device()) return FLASHSPMM_ERR_NO_DEVICE;
  return done(launch_w4_decode(A, W, w_dtype == FLASHSPMM_F32, static_cast<cudaStream_t>(stream)));
}

size_t flashspmm_w4_matmul_workspace_bytes(const flashspmm_w4* A, const void* B, int64_t ldb, int32_t N) {
  if (check_w4(A) != FLASHSPMM_OK || N <= 0 || N > 256 || A->M == 0 || A->K == 0) return 0;
  return w4_matmul_workspace(A, N, rows_aligned(B, ldb, A->K));
}

flashspmm_status flashspmm_w4_matmul(const flashspmm_w4* A, const void* B, int64_t ldb, void* C, int64_t ldc,
                                     int32_t c_dtype, int32_t N, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  const flashspmm_status st = check_w4(A);
  if (st != FLASHSPMM_OK) return st;
  if (N < 0 || A->count != 1 || ldb < A->K || ldc < A->M) return FLASHSPMM_ERR_INVALID_ARG;
  if (N > 256 || (c_dtype != A->dtype && c_dtype != FLASHSPMM_F32)) return FLASHSPMM_ERR_UNSUPPORTED;
  if (A->M == 0 || N == 0) return FLASHSPMM_OK;
  const bool f32 = c_dtype == FLASHSPMM_F32;
  if (!C) return FLASHSPMM_ERR_INVALID_ARG;
  if (f32 ? !on4(C) : !on2(C)) return FLASHSPMM_ERR_ALIGNMENT;
  if (!have_device()) return FLASHSPMM_ERR_NO_DEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t width = f32 ? 4 : 2;
  if (A->K == 0) return done(cudaMemset2DAsync(C, ldc * width, 0, A->M * width, N, s));
  if (!B) return FLASHSPMM_ERR_INVALID_ARG;
  if (!on2(B)) return FLASHSPMM_ERR_ALIGNMENT;
  const size_t need = w4_matmul_workspace(A, N, rows_aligned(B, ldb, A->K));
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return FLASHSPMM_ERR_CAPACITY;
    if (!aligned16(workspace)) return FLASHSPMM_ERR_ALIGNMENT;
  }
  return done(launch_w4_matmul(A, B, ldb, C, ldc, f32, N, workspace, s));
}

size_t flashspmm_moe_w4_workspace_bytes(const flashspmm_w4* gate, const void* X, int64_t ldx, int32_t tokens,
                                        int32_t top_k) {
  if (check_w4(gate) != FLASHSPMM_OK || tokens <= 0 || tokens > kMoeMaxTokens || top_k <= 0 ||
      top_k > kMoeMaxTopK || gate->count > kMoeMaxExperts)
    return 0;
  return moe_workspace(tokens, gate->count, top_k, gate->K, gate->M, rows_aligned(X, ldx, gate->K));
}

flashspmm_status flashspmm_moe_w4(const flashspmm_w4* gate, const flashspmm_w4* up, const flashspmm_w4* down,
                                  const void* X, int64_t ldx, const void* router, int32_t router_dtype, int32_t tokens,
                                  int32_t top_k, int32_t renormalize, int32_t activation, int32_t* ids, float* weights,
                                  void* out, int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
  flashspmm_status st = check_w4(gate);
  if (st == FLASHSPMM_OK) st = check_w4(down);
  if (st == FLASHSPMM_OK && up) st = check_w4(up);
  if (st != FLASHSPMM_OK) return st;
  const int32_t E = gate->count, H = gate->K, F = gate->M;
  if (down->count != E || down->M != H || down->K != F || down->group != gate->group || down->dtype != gate->dtype)
    return FLASHSPMM_ERR_INVALID_ARG;
  if (up && (up->count != E || up->M != F || up->K != H || up->group != gate->group || up->dtype != gate->dtype))
    return FLASHSPMM_ERR_INVALID_ARG;
  if (tokens < 0 || top_k < 1 || ldx < H || ldo < H) return FLASHSPMM_ERR_INVALID_ARG;
  if (router && top_k > E) return FLASHSPMM_ERR_INVALID_ARG;
  if (activation != FLASHSPMM_ACT_SILU && activation != FLASHSPMM_ACT_GELU && activation != FLASHSPMM_ACT_RELU)
    return FLASHSPMM_ERR_UNSUPPORTED;
  if (router && router_dtype != gate->dtype && router_dtype != FLASHSPMM_F32) return FLASHSPMM_ERR_UNSUPPORTED;
  if (tokens > kMoeMaxTokens || E > kMoeMaxExperts || top_k > kMoeMaxTopK || H == 0 || F == 0)
    return FLASHSPMM_ERR_UNSUPPORTED;
  if (tokens == 0) return FLASHSPMM_OK;
  if (!X || !out || !ids || !weights) return FLASHSPMM_ERR_INVALID_ARG;
  if (!on2(X) || !on2(out) || !on4(ids) || !on4(weights) ||
      (router && (router_dtype == FLASHSPMM_F32 ? !on4(router) : !on2(router))))
    return FLASHSPMM_ERR_ALIGNMENT;
  if (!have_device()) return FLASHSPMM_ERR_NO_DEVICE;
  if (!workspace || workspace_bytes < moe_workspace(tokens, E, top_k, H, F, rows_aligned(X, ldx, H)))
    return FLASHSPMM_ERR_CAPACITY;
  if (!aligned16(workspace)) return FLASHSPMM_ERR_ALIGNMENT;
  MoeCall p{};
  p.gate = *gate;
  if (up) p.up = *up;
  p.down = *down;
  p.X = X;
  p.ldx = ldx;
  p.router = router;
  p.router_dtype = router_dtype;
  p.tokens = tokens;
  p.top_k = top_k;
  p.renormalize = renormalize != 0;
  p.activation = activation;
  p.ids = ids;
  p.weights = weights;
  p.out = out;
  p.ldo = ldo;
  return done(launch_moe_w4(p, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
