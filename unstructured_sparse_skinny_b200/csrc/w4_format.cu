// 4-bit weights: encoder (dense -> codes, scales, zero points), packing of
// codes that a caller already has, and decoder.
//
// All three walk the units (16 rows x 128 columns) of w4.cuh, one warp each:
// a lane holds two rows of 4 x 8 columns, which are whole 16-byte pieces of
// the dense rows and exactly its own two 16-byte pieces of the codes, so both
// sides are moved in full sectors and a group's extremes need two shuffles.
// HBM bounds them: 12288^2, groups of 128, take 90 us to encode (4.2 TB/s), 76 to
// decode (5.0) and 59 to pack (3.9).  Rows that do not start on 16 bytes are moved
// by words: 12288 x 12285 take 201, 305 and 133 us.
#include "w4.cuh"

namespace flashspmm {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The 16 codes q[row][8 columns of block b] of a lane to the block's two words.
__device__ __forceinline__ void pack_block(const uint32_t (&q)[2][8], uint32_t& w0, uint32_t& w1) {
  uint32_t w[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i & 1, col = 4 * s + 2 * (i >> 1);
      v |= q[row][col] << (4 * i);
      v |= q[row][col + 1] << (4 * (i + 4));
    }
    w[s] = v;
  }
  w0 = w[0];
  w1 = w[1];
}

// A lane's share of a record.
__device__ __forceinline__ void put_codes(uint8_t* record, int lane, const uint32_t (&w)[8]) {
  reinterpret_cast<uint4*>(record)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(record)[32 + lane] = make_uint4(w[4], w[5], w[6], w[7]);
}
// Scales and zero points of rows g and g + 8 for one group.
template <int NG>
__device__ __forceinline__ void put_group(uint8_t* record, int g, int group, uint32_t scales, uint32_t points,
                                          bool zeros) {
  const int o = g * (2 * NG) + 2 * group;
  *reinterpret_cast<uint32_t*>(record + kW4CodeBytes + 2 * o) = scales;
  if (zeros) *reinterpret_cast<uint16_t*>(record + kW4CodeBytes + 32 * NG + o) = static_cast<uint16_t>(points);
}

__device__ __forceinline__ uint32_t code_of(uint32_t w0, uint32_t w1, int row, int col) {
  const uint32_t w = col < 4 ? w0 : w1;
  const int c = col & 3;
  const int nibble = row + 2 * (c >> 1) + 4 * (c & 1);
  return (w >> (4 * nibble)) & 0xF;
}

// Position of a unit: its matrix and the rows and columns of a lane.
struct Place {
  int64_t row;      // row g of the lane's unit in the stack's dense rows (matrix * M + row)
  bool ok0, ok1;    // rows g and g + 8 exist
  int32_t col0;     // first column of block 0 for this lane
  __device__ __forceinline__ Place(const W4Dev& A, int64_t unit, int lane) {
    const int64_t part = unit >> 3, block = part / A.units;
    const int32_t u = static_cast<int32_t>(part - block * A.units);
    const int64_t mat = block / A.blocks;
    const int64_t r = ((block - mat * A.blocks) * 8 + (unit & 7)) * kW4StripRows + (lane >> 2);
    row = mat * A.M + r;
    ok0 = r < A.M;
    ok1 = r + 8 < A.M;
    col0 = u * kW4UnitCols + 8 * (lane & 3);
  }
};

// Encoder.  Symmetric: s = max|w| / 7, z = 8.  Else: s = (max(w, 0) - min(w, 0))
// / 15, z = round(-min / s).  s is rounded to 16 bits first, and then
// q = clamp(round(w / s) + z, 0, 15), ties to even.  A group of zeros (or whose
// s rounds to zero) has s = 0 and q = z.
//
// round(w / s) without a division per value: w and s have at most 11
// significant bits, so w / s is either exactly half way between two integers
// or at least 2^-13 away from that.  fma(w, 1 / s, 1536) is w / s with an
// absolute error below 2^-18 rounded to a multiple of 2^-13: the half-way
// cases land exactly on the half, no other case reaches one, and adding
// 1.5 * 2^23 - 1536 then rounds to the even integer.
template <typename T, int NG, bool Sym, bool Vec>
__global__ void __launch_bounds__(kWarps * 32) w4_encode_kernel(const uint16_t* __restrict__ W, int64_t ldw, W4Dev A,
                                                                uint8_t* data, int64_t total) {
  constexpr int kBlocks = 4 / NG;  // 32-column blocks of a group
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); unit < total; unit += step) {
    const Place at(A, unit, lane);
    const uint16_t* r0 = at.ok0 ? W + at.row * ldw : nullptr;
    const uint16_t* r1 = at.ok1 ? W + (at.row + 8) * ldw : nullptr;
    uint4 raw[2][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      raw[0][b] = load_act8<Vec>(r0, at.col0 + 32 * b, A.K);
      raw[1][b] = load_act8<Vec>(r1, at.col0 + 32 * b, A.K);
    }
    uint8_t* record = data + unit * A.record;
    uint32_t words[8];
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
      float s[2];
      uint32_t zp[2];
      uint32_t q[kBlocks][2][8];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float w[kBlocks][8];
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const uint4 v = raw[r][gi * kBlocks + b];
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            w[b][i] = bits_to_float<T>(static_cast<uint16_t>(i & 1 ? x[i >> 1] >> 16 : x[i >> 1] & 0xFFFF));
            if (Sym) {
              hi = max_nan(hi, fabsf(w[b][i]));
            } else {
              hi = max_nan(hi, w[b][i]);
              lo = min_nan(lo, w[b][i]);
            }
          }
        }
#pragma unroll
        for (int m = 1; m <= 2; m <<= 1) {  // the four lanes of a row
          hi = max_nan(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m));
          if (!Sym) lo = min_nan(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m));
        }
        const float span = hi - lo;  // of two bf16 values it can pass the largest fp32
        s[r] = to_float(from_float<T>(Sym ? hi / 7.0f
                                          : isinf(span) ? (0.5f * hi - 0.5f * lo) / 7.5f : span / 15.0f));
        const float div = s[r] == 0.0f ? 1.0f : s[r];
        const float z = Sym ? 8.0f : fminf(fmaxf(rintf(-lo / div), 0.0f), 15.0f);
        zp[r] = static_cast<uint32_t>(z);
        // a reciprocal that stays finite: far below every useful scale both sides are raised by 2^100
        const bool tiny = div < 7.9e-31f;
        const float raise = tiny ? 1.2676506e30f : 1.0f;
        const float inv = 1.0f / (div * raise);
        const float from = 1536.0f - z, to = 1551.0f - z;
        if (tiny) {
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[b][i] *= raise;
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = fminf(fmaxf(fmaf(w[b][i], inv, 1536.0f), from), to);
            q[b][r][i] = (__float_as_uint(y + 12581376.0f) + zp[r]) & 0xF;
          }
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        pack_block(q[b], words[2 * (gi * kBlocks + b)], words[2 * (gi * kBlocks + b) + 1]);
      if ((lane & 3) == 0) {
        union {
          T t[2];
          uint32_t u;
        } pair;
        pair.t[0] = from_float<T>(s[0]);
        pair.t[1] = from_float<T>(s[1]);
        put_group<NG>(record, lane >> 2, gi, pair.u, zp[0] | (zp[1] << 8), !Sym);
      }
    }
    put_codes(record, lane, words);
  }
}

// Codes of one byte each ([count * M][K]) with scales and zero points
// [count * M][ceil(K / group)] to the layout.  A group's columns behind K get the
// code nearest to its zero point: a zero weight, or where the point is above 15
// the smallest that the group can have, so they overflow 16 bits only if all of
// its weights do.  (The activations that meet them are zeros.)
template <int NG, bool Vec>
__global__ void __launch_bounds__(kWarps * 32) w4_pack_kernel(const uint8_t* __restrict__ in,
                                                              const uint16_t* __restrict__ in_scales,
                                                              const uint8_t* __restrict__ in_zeros, W4Dev A,
                                                              uint8_t* data, int64_t total) {
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t groups = (static_cast<int64_t>(A.K) + A.group - 1) / A.group;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); unit < total; unit += step) {
    const Place at(A, unit, lane);
    const int64_t g0 = static_cast<int64_t>(at.col0 / kW4UnitCols) * NG;
    uint32_t zp[2][NG], sc[2][NG];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool ok = r ? at.ok1 : at.ok0;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) {
        const bool have = ok && g0 + gi < groups;
        const int64_t src = (at.row + 8 * r) * groups + g0 + gi;
        sc[r][gi] = have ? in_scales[src] : 0u;
        zp[r][gi] = have && in_zeros ? in_zeros[src] & 0x3Fu : 8u;
      }
    }
    uint32_t words[8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int32_t k = at.col0 + 32 * b;
      uint32_t q[2][8];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool ok = r ? at.ok1 : at.ok0;
        const uint32_t pad = min(zp[r][b * NG / 4], 15u);
        const uint8_t* p = in + (at.row + 8 * r) * A.K + k;
        if (Vec) {
          uint2 v = make_uint2(pad * 0x01010101u, pad * 0x01010101u);
          if (ok && k < A.K) v = *reinterpret_cast<const uint2*>(p);
#pragma unroll
          for (int i = 0; i < 8; ++i) q[r][i] = ((i < 4 ? v.x : v.y) >> (8 * (i & 3))) & 0xF;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) q[r][i] = ok && k + i < A.K ? p[i] & 0xFu : pad;
        }
      }
      pack_block(q, words[2 * b], words[2 * b + 1]);
    }
    uint8_t* record = data + unit * A.record;
    put_codes(record, lane, words);
    if ((lane & 3) == 0) {
#pragma unroll
      for (int gi = 0; gi < NG; ++gi)
        put_group<NG>(record, lane >> 2, gi, sc[0][gi] | (sc[1][gi] << 16), zp[0][gi] | (zp[1][gi] << 8), A.zeros);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  union {
    T t[8];
    uint4 u;
  } o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.t[i] = from_float<T>(v[i]);
  *reinterpret_cast<uint4*>(p) = o.u;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// On any value's boundary: three words and a fourth, or a value before and one behind them.
template <typename T>
__device__ __forceinline__ void store8_any(T* p, const float (&v)[8]) {
  union {
    T t[8];
    uint32_t u[4];
  } o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.t[i] = from_float<T>(v[i]);
  const uint32_t odd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) >> 1) & 1u;
  uint32_t* to = reinterpret_cast<uint32_t*>(p + odd);
#pragma unroll
  for (int i = 0; i < 3; ++i) to[i] = __funnelshift_r(o.u[i], o.u[i + 1], 16 * odd);
  if (odd) {
    p[0] = o.t[0];
    p[7] = o.t[7];
  } else {
    to[3] = o.u[3];
  }
}
__device__ __forceinline__ void store8_any(float*, const float (&)[8]) {}  // four bytes a value: not called
__device__ __forceinline__ void store1(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// Decoder: s * (q - z), exact in fp32, rounded once to the output type.
template <typename T, typename O, int NG, bool Vec>
__global__ void __launch_bounds__(kWarps * 32) w4_decode_kernel(W4Dev A, O* __restrict__ W, int64_t total) {
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); unit < total; unit += step) {
    const Place at(A, unit, lane);
    W4Groups<T, NG> grp;
    const uint8_t* record = A.at(unit);
    grp.load(record, lane >> 2, A.zeros);
    const uint4 c0 = ld_stream(record + lane * 16), c1 = ld_stream(record + 512 + lane * 16);
    const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int gi = b * NG / 4;
      const int32_t k = at.col0 + 32 * b;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (!(r ? at.ok1 : at.ok0) || k >= A.K) continue;
        const float s = grp.scale(gi, r);
        const int z = grp.zero_point(gi, r);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = s * static_cast<float>(static_cast<int>(code_of(words[2 * b], words[2 * b + 1], r, i)) - z);
        O* p = W + (at.row + 8 * r) * A.K + k;
        if (Vec) {
          store8(p, v);
        } else if (sizeof(O) == 2 && k + 8 <= A.K) {
          store8_any(p, v);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (k + i < A.K) store1(p + i, v[i]);
        }
      }
    }
  }
}

int grid_for(int64_t units) {
  const int sms = device_sm_count();
  const int64_t most = static_cast<int64_t>(sms > 0 ? sms : 1) * 8;
  return static_cast<int>(max64(1, min64((units + kWarps - 1) / kWarps, most)));
}

template <typename T, int NG>
void encode_as(const uint16_t* W, int64_t ldw, const W4Dev& A, const flashspmm_w4* out, bool sym, bool vec,
               int64_t total, cudaStream_t s) {
  uint8_t* data = static_cast<uint8_t*>(out->data);
  const int grid = grid_for(total);
#define FLASHSPMM_ENCODE(SYM, VEC) w4_encode_kernel<T, NG, SYM, VEC><<<grid, kWarps * 32, 0, s>>>(W, ldw, A, data, total)
  if (sym)
    vec ? FLASHSPMM_ENCODE(true, true) : FLASHSPMM_ENCODE(true, false);
  else
    vec ? FLASHSPMM_ENCODE(false, true) : FLASHSPMM_ENCODE(false, false);
#undef FLASHSPMM_ENCODE
}

template <typename T, typename O>
void decode_as(const W4Dev& A, O* W, bool vec, int64_t total, cudaStream_t s) {
  const int grid = grid_for(total);
#define FLASHSPMM_DECODE_NG(NG)                                                    \
  vec ? w4_decode_kernel<T, O, NG, true><<<grid, kWarps * 32, 0, s>>>(A, W, total) \
      : w4_decode_kernel<T, O, NG, false><<<grid, kWarps * 32, 0, s>>>(A, W, total)
  if (A.group == 128) {
    FLASHSPMM_DECODE_NG(1);
  } else if (A.group == 64) {
    FLASHSPMM_DECODE_NG(2);
  } else {
    FLASHSPMM_DECODE_NG(4);
  }
#undef FLASHSPMM_DECODE_NG
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t all_units(const flashspmm_w4* A) {
  return static_cast<int64_t>(A->count) * w4_blocks(A->M) * 8 * w4_units(A->K);
}

}  // namespace

cudaError_t launch_w4_encode(const void* W, int64_t ldw, const flashspmm_w4* out, int symmetric, cudaStream_t s) {
  const W4Dev A = w4_dev(out);
  const int64_t total = all_units(out);
  const bool vec = on16(W) && ldw % 8 == 0 && A.K % 8 == 0;
  const uint16_t* w = static_cast<const uint16_t*>(W);
  const bool sym = symmetric != 0;
#define FLASHSPMM_BY_GROUP(T)                                             \
  if (A.group == 128)                                                     \
    encode_as<T, 1>(w, ldw, A, out, sym, vec, total, s);                  \
  else if (A.group == 64)                                                 \
    encode_as<T, 2>(w, ldw, A, out, sym, vec, total, s);                  \
  else                                                                    \
    encode_as<T, 4>(w, ldw, A, out, sym, vec, total, s)
  if (out->dtype == FLASHSPMM_F16) {
    FLASHSPMM_BY_GROUP(__half);
  } else {
    FLASHSPMM_BY_GROUP(__nv_bfloat16);
  }
#undef FLASHSPMM_BY_GROUP
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_w4_pack(const uint8_t* in, const void* in_scales, const uint8_t* in_zeros, const flashspmm_w4* out,
                           cudaStream_t s) {
  const W4Dev A = w4_dev(out);
  const int64_t total = all_units(out);
  const bool vec = (reinterpret_cast<uintptr_t>(in) & 7u) == 0 && A.K % 8 == 0;
  const uint16_t* sc = static_cast<const uint16_t*>(in_scales);
  uint8_t* data = static_cast<uint8_t*>(out->data);
  const int grid = grid_for(total);
#define FLASHSPMM_PACK(NG)                                                                          \
  vec ? w4_pack_kernel<NG, true><<<grid, kWarps * 32, 0, s>>>(in, sc, in_zeros, A, data, total)     \
      : w4_pack_kernel<NG, false><<<grid, kWarps * 32, 0, s>>>(in, sc, in_zeros, A, data, total)
  if (A.group == 128)
    FLASHSPMM_PACK(1);
  else if (A.group == 64)
    FLASHSPMM_PACK(2);
  else
    FLASHSPMM_PACK(4);
#undef FLASHSPMM_PACK
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_w4_decode(const flashspmm_w4* in, void* W, bool f32, cudaStream_t s) {
  const W4Dev A = w4_dev(in);
  const int64_t total = all_units(in);
  const bool vec = on16(W) && A.K % 8 == 0;
  if (in->dtype == FLASHSPMM_F16) {
    if (f32)
      decode_as<__half, float>(A, static_cast<float*>(W), vec, total, s);
    else
      decode_as<__half, __half>(A, static_cast<__half*>(W), vec, total, s);
  } else {
    if (f32)
      decode_as<__nv_bfloat16, float>(A, static_cast<float*>(W), vec, total, s);
    else
      decode_as<__nv_bfloat16, __nv_bfloat16>(A, static_cast<__nv_bfloat16*>(W), vec, total, s);
  }
  note_launch();
  return cudaGetLastError();
}

}  // namespace flashspmm
