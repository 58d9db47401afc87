// 4-bit weights with group scales: layout, fragments and launchers, shared by
// the skinny matrix product and the experts' products.
//
// Layout.  A matrix of M x K codes is cut into strips of 16 rows, eight strips
// to a block of 128, and units of 128 columns.  A unit of one strip is one
// record: 1024 bytes of codes, its scales and, if there are any, its zero
// points.  The records of a block's eight strips follow one another, then come
// the block's next 128 columns, so a block's unit, or some strips of it, is one
// bulk copy.  A warp reads a record's codes with two 16-byte loads per lane, and
// every lane then holds exactly the codes of its own mma.m16n8k16 A fragments, so
// nothing is shuffled.  Lane l = 4 * g + t owns rows g and g + 8 and, in each
// 32-column block b of the unit, the eight columns 32 * b + 8 * t .. + 7.  The
// order of K inside a product is free as long as both operands use the same
// one: step s of block b takes columns 8 * t + 4 * s + {0, 1} as the
// fragment's first column pair and + {2, 3} as its second, so the B fragments
// of a block are one 16-byte load of eight neighbouring activations.  A block
// is 32 columns of K in every lane, so groups of 32, 64 and 128 columns end on
// block boundaries.  Word (b, s) of a lane is the (2 * (b & 1) + s)-th of its
// 16-byte load b / 2; its nibble i holds the first and nibble i + 4 the second
// value of fragment register a_i (a0: row g, first pair; a1: row g + 8, first;
// a2: row g, second; a3: row g + 8, second).
//
// Scales (16 bits) and zero points (8 bits) of a record are [g][group][row g,
// row g + 8], so a lane reads all it needs of either in one load.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace flashspmm {

constexpr int kW4StripRows = 16;
constexpr int kW4UnitCols = 128;
constexpr int kW4CodeBytes = 1024;  // of a record

__host__ __device__ constexpr int32_t w4_record_bytes(int groups, bool zeros) {
  return kW4CodeBytes + 32 * groups + (zeros ? 16 * groups : 0);
}

// A stack of 4-bit matrices as the kernels see it.
struct W4Dev {
  const uint8_t* data;
  int32_t record;  // bytes
  bool zeros;      // without them every zero point is 8
  int32_t M, K;
  int32_t strips;  // of one matrix that hold rows (the layout pads them to whole blocks)
  int32_t blocks;  // of one matrix
  int32_t units;   // of one strip
  int32_t group;

  // Number of unit u of a strip; its next unit is 8 further on.
  __device__ __forceinline__ int64_t unit(int64_t matrix, int32_t strip, int32_t u) const {
    return ((matrix * blocks + (strip >> 3)) * units + u) * 8 + (strip & 7);
  }
  __device__ __forceinline__ const uint8_t* at(int64_t unit) const { return data + unit * record; }
};

__host__ __device__ inline int32_t w4_strips(int32_t M) {
  return static_cast<int32_t>((static_cast<int64_t>(M) + kW4StripRows - 1) / kW4StripRows);
}
__host__ __device__ inline int32_t w4_blocks(int32_t M) {
  return static_cast<int32_t>((static_cast<int64_t>(M) + 127) / 128);
}
__host__ __device__ inline int32_t w4_units(int32_t K) {
  return static_cast<int32_t>((static_cast<int64_t>(K) + kW4UnitCols - 1) / kW4UnitCols);
}

inline W4Dev w4_dev(const flashspmm_w4* A) {
  W4Dev d;
  d.data = static_cast<const uint8_t*>(A->data);
  d.record = w4_record_bytes(kW4UnitCols / A->group, A->zeros != 0);
  d.zeros = A->zeros != 0;
  d.M = A->M;
  d.K = A->K;
  d.strips = w4_strips(A->M);
  d.blocks = w4_blocks(A->M);
  d.units = w4_units(A->K);
  d.group = A->group;
  return d;
}

// ---------------------------------------------------------------- 16-bit types

__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T>
__device__ __forceinline__ float bits_to_float(uint16_t b);
template <>
__device__ __forceinline__ float bits_to_float<__half>(uint16_t b) { return __half2float(__ushort_as_half(b)); }
template <>
__device__ __forceinline__ float bits_to_float<__nv_bfloat16>(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}

// ---------------------------------------------------------------- codes to A fragments

// (a & b) | c in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Fragments for sums of whole numbers times activations hold q - z, in bf16
// (q - z) 2^-13, exact like it: |q - z| <= 63, so a group's sum of 128 products
// stays below the largest fp32 value whatever bf16 activations it has, and what
// is scaled and added up is infinite only if the result nearly is.  The finished
// sum is multiplied by w4_raise.  At the other end sums are kept to 2^-136
// instead of 2^-149.  (fp16 activations are below 2^16.)
template <typename T>
inline constexpr int kW4Down = 0;  // binary orders
template <>
inline constexpr int kW4Down<__nv_bfloat16> = 13;
template <typename T>
__device__ __forceinline__ float w4_raise(float sum) {
  return kW4Down<T> ? sum * static_cast<float>(1 << kW4Down<T>) : sum;
}

// The pair {z, z} (first row) and its like for the second row, in the form
// that w4_fragment subtracts.
template <typename T, int Down>
struct W4Zero;
template <>
struct W4Zero<__half, 0> {
  __half2 lo, hi;  // 1024 + z, -(64 + z'), put together as bits: steps there are 1 and 1/16, and z < 64
  __device__ __forceinline__ W4Zero(int z0, int z1)
      : lo(__half2half2(__ushort_as_half(static_cast<uint16_t>(0x6400 | z0)))),
        hi(__half2half2(__ushort_as_half(static_cast<uint16_t>(0xD400 | (z1 << 4))))) {}
};
template <int Down>
struct W4Zero<__nv_bfloat16, Down> {
  static constexpr uint32_t kBase = 0x4300 - (Down << 7);  // 128 * 2^-Down
  __nv_bfloat162 lo, hi;                                    // (128 + z) * 2^-Down, (128 + z') * 2^-Down
  __device__ __forceinline__ W4Zero(int z0, int z1)
      : lo(__bfloat162bfloat162(__ushort_as_bfloat16(static_cast<uint16_t>(kBase | z0)))),
        hi(__bfloat162bfloat162(__ushort_as_bfloat16(static_cast<uint16_t>(kBase | z1)))) {}
};

// Eight codes of one word to the fragment (q - z) 2^-Down, exact: a nibble put
// under the bits of 1024 is 1024 + q (fp16, nibbles 0 and 4) or 1024 + 16 q
// (nibbles 1 and 5), and the subtraction, or the fused multiply by 1/16 and
// subtraction, rounds nothing.  bf16 has 7 mantissa bits: a nibble under 128 is
// 128 + q, and likewise at every other power of two.
__device__ __forceinline__ void w4_fragment(uint32_t w, const W4Zero<__half, 0>& z, uint32_t (&a)[4]) {
  const uint32_t base = 0x64006400u;
  const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));
  const uint32_t v = w >> 8;
  union U {
    uint32_t u;
    __half2 h;
  } x;
  x.u = and_or(w, 0x000F000Fu, base);
  x.h = __hsub2(x.h, z.lo);
  a[0] = x.u;
  x.u = and_or(w, 0x00F000F0u, base);
  x.h = __hfma2(x.h, sixteenth, z.hi);
  a[1] = x.u;
  x.u = and_or(v, 0x000F000Fu, base);
  x.h = __hsub2(x.h, z.lo);
  a[2] = x.u;
  x.u = and_or(v, 0x00F000F0u, base);
  x.h = __hfma2(x.h, sixteenth, z.hi);
  a[3] = x.u;
}
template <int Down>
__device__ __forceinline__ void w4_fragment(uint32_t w, const W4Zero<__nv_bfloat16, Down>& z, uint32_t (&a)[4]) {
  const uint32_t base = z.kBase * 0x10001u;
  union U {
    uint32_t u;
    __nv_bfloat162 h;
  } x;
  x.u = and_or(w, 0x000F000Fu, base);
  x.h = __hsub2(x.h, z.lo);
  a[0] = x.u;
  x.u = and_or(w >> 4, 0x000F000Fu, base);
  x.h = __hsub2(x.h, z.hi);
  a[1] = x.u;
  x.u = and_or(w >> 8, 0x000F000Fu, base);
  x.h = __hsub2(x.h, z.lo);
  a[2] = x.u;
  x.u = and_or(w >> 12, 0x000F000Fu, base);
  x.h = __hsub2(x.h, z.hi);
  a[3] = x.u;
}

// c += a (16 x 16) * b (16 x 8), fp32 sums.
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c = a (16 x 16) * b (16 x 8)
template <typename T>
__device__ __forceinline__ void mma16816_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816_zero<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
template <>
__device__ __forceinline__ void mma16816_zero<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// ---------------------------------------------------------------- loads

// Codes are read once: keep them out of L1, where the activations live.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Eight activations k .. k + 7 of one row as four fragment words, zero past K.
// Vec: the row starts on 16 bytes and holds a multiple of 8 values.
template <bool Vec>
__device__ __forceinline__ uint4 load_act8(const uint16_t* row, int32_t k, int32_t K) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (Vec) {
    if (row && k < K) v = *reinterpret_cast<const uint4*>(row + k);
  } else if (row && k > 0 && k < K - 8) {
    // inside a row that starts on any value: the four or five words that hold it, which hold no other row's
    const uint32_t odd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + k) >> 1) & 1u;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row + k - odd);
    const uint32_t w[5] = {p[0], p[1], p[2], p[3], odd ? p[4] : 0u};
    v = make_uint4(__funnelshift_r(w[0], w[1], 16 * odd), __funnelshift_r(w[1], w[2], 16 * odd),
                   __funnelshift_r(w[2], w[3], 16 * odd), __funnelshift_r(w[3], w[4], 16 * odd));
  } else if (row) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) w[i >> 1] |= static_cast<uint32_t>(row[k + i]) << (16 * (i & 1));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

// Scales and zero points of one unit as a lane needs them (NG groups a unit).
template <typename T, int NG>
struct W4Groups {
  uint32_t s[NG];            // {row g, row g + 8} in 16 bits each
  uint32_t z[(NG + 1) / 2];  // {row g, row g + 8} in 8 bits each, two groups to a word

  __device__ __forceinline__ void load(const uint8_t* record, int g, bool zeros) {
    const uint8_t* sp = record + kW4CodeBytes + g * (4 * NG);
    const uint8_t* zp = record + kW4CodeBytes + 32 * NG + g * (2 * NG);
    if (NG == 1) {
      s[0] = *reinterpret_cast<const uint32_t*>(sp);
      z[0] = zeros ? *reinterpret_cast<const uint16_t*>(zp) : 0x0808u;
    } else if (NG == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(sp);
      s[0] = v.x;
      s[NG - 1] = v.y;
      z[0] = zeros ? *reinterpret_cast<const uint32_t*>(zp) : 0x08080808u;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(sp);
      s[0] = v.x;
      s[1 % NG] = v.y;
      s[2 % NG] = v.z;
      s[NG - 1] = v.w;
      const uint2 q = zeros ? *reinterpret_cast<const uint2*>(zp) : make_uint2(0x08080808u, 0x08080808u);
      z[0] = q.x;
      z[(NG - 1) / 2] = q.y;
    }
  }
  __device__ __forceinline__ float scale(int i, int row) const {
    return bits_to_float<T>(static_cast<uint16_t>(row ? s[i] >> 16 : s[i] & 0xFFFF));
  }
  __device__ __forceinline__ int zero_point(int i, int row) const {
    return static_cast<int>(z[i >> 1] >> (16 * (i & 1) + 8 * row) & 0xFF);
  }
  __device__ __forceinline__ W4Zero<T, kW4Down<T>> zero(int i) const { return {zero_point(i, 0), zero_point(i, 1)}; }
};

// ---------------------------------------------------------------- launchers

cudaError_t launch_w4_encode(const void* W, int64_t ldw, const flashspmm_w4* A, int symmetric, cudaStream_t s);
cudaError_t launch_w4_pack(const uint8_t* codes, const void* scales, const uint8_t* zeros, const flashspmm_w4* A,
                           cudaStream_t s);
cudaError_t launch_w4_decode(const flashspmm_w4* A, void* W, bool f32, cudaStream_t s);

// Activations whose rows do not start on 16 bytes, or whose length is not a
// multiple of 8, are copied first: rows x K values to rows of aligned_k(K)
// values, zero behind K.
inline int64_t aligned_k(int32_t K) { return (static_cast<int64_t>(K) + 7) / 8 * 8; }
bool rows_aligned(const void* X, int64_t ld, int32_t K);
cudaError_t launch_align_rows(const void* X, int64_t ld, int32_t rows, int32_t K, void* out, cudaStream_t s);

size_t w4_matmul_workspace(const flashspmm_w4* A, int32_t N, bool aligned);
cudaError_t launch_w4_matmul(const flashspmm_w4* A, const void* B, int64_t ldb, void* C, int64_t ldc, bool c_f32,
                             int32_t N, void* workspace, cudaStream_t s);

// The same product by tcgen05 (w4_gemm.cu).
size_t w4_gemm_workspace(int32_t M, int32_t K, int32_t N);
cudaError_t launch_w4_gemm(const flashspmm_w4* A, const void* B, int64_t ldb, void* C, int64_t ldc, bool c_f32,
                           int32_t N, void* workspace, cudaStream_t s);

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;

struct MoeCall {
  flashspmm_w4 gate, up, down;  // up.data null: no gate product
  const void* X;
  int64_t ldx;
  const void* router;  // null: ids and weights are inputs
  int32_t router_dtype;
  int32_t tokens, top_k;
  bool renormalize;
  int32_t activation;
  int32_t* ids;
  float* weights;
  void* out;
  int64_t ldo;
};
size_t moe_workspace(int32_t T, int32_t E, int32_t top_k, int32_t H, int32_t F, bool aligned);
cudaError_t launch_moe_w4(const MoeCall& p, void* workspace, cudaStream_t s);

}  // namespace flashspmm
