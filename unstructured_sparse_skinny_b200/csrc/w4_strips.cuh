// The product of strips of 4-bit rows with a few activation rows, on the
// tensor cores through mma.sync: the engine of the skinny product for few
// tokens and of the experts' products.
//
// A CTA of eight warps takes `pairs` pairs of strips (a pair is two strips of
// one matrix, or the same strip of two) and splits K among the warps of a
// pair.  A warp reads its codes straight to registers, two or three units
// ahead; each lane finds its own fragments there.  The activations are staged
// in shared memory once and serve all strips of the CTA.  Warps meet only
// where the activations do not fit at once, and at the end, to add up K.
//
// A group's weights enter the product as whole numbers q - z, and the fp32 sum
// of the group is scaled: no weight is rounded.
#pragma once

#include "sm100_primitives.cuh"
#include "w4.cuh"

namespace flashspmm {

constexpr int kStripWarps = 8;
constexpr int kStripThreads = kStripWarps * 32;
constexpr int kStripShared = 100 * 1024;  // two CTAs on an SM

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

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Where a lane finds a strip's units.
struct StripAt {
  const uint4* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  __device__ __forceinline__ StripAt() {}
  __device__ __forceinline__ StripAt(const W4Dev& A, int64_t unit, int lane) {
    const int64_t at = (unit * 8 + (lane >> 2)) * (2 * (kW4UnitCols / A.group));
    codes = A.codes + unit * 64 + lane;
    scales = A.scales + at;
    zeros = A.zeros ? A.zeros + at : nullptr;
  }
};

template <typename T, int NG>
struct StripUnit {
  uint4 c[2];
  W4Groups<T, NG> g;
  __device__ __forceinline__ void load(const StripAt& at, int32_t u) {
    // a strip's units are eight units apart
    const uint4* p = at.codes + static_cast<int64_t>(u) * 512;
    c[0] = ld_stream(p);
    c[1] = ld_stream(p + 32);
    const int64_t o = static_cast<int64_t>(u) * (128 * NG);
    g.load(at.scales + o, at.zeros ? at.zeros + o : nullptr);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& v = c[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
};

// acc += the unit's product with the staged activations; x[nt] is the lane's
// shared-memory address of the unit's first column for its row of tile nt.
template <typename T, int NG, int NT>
__device__ __forceinline__ void strip_unit(const StripUnit<T, NG> (&unit)[2], const uint32_t (&x)[NT], uint32_t offset,
                                           int tiles, float (&acc)[2][NT][4]) {
  constexpr int kBlocks = 4 / NG;
#pragma unroll
  for (int gi = 0; gi < NG; ++gi) {
    const W4Zero<T> z[2] = {unit[0].g.zero(gi), unit[1].g.zero(gi)};
    float d[2][NT][4];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int blk = gi * kBlocks + b;
      uint32_t a[2][2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w4_fragment(unit[r].word(2 * blk), z[r], a[r][0]);
        w4_fragment(unit[r].word(2 * blk + 1), z[r], a[r][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt > 0 && nt >= tiles) break;
        const uint4 v = ld_shared16(x[nt] + offset + blk * 64);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (b == 0)
            mma16816_zero<T>(d[r][nt], a[r][0], v.x, v.y);
          else
            mma16816<T>(d[r][nt], a[r][0], v.x, v.y);
          mma16816<T>(d[r][nt], a[r][1], v.z, v.w);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float s0 = unit[r].g.scale(gi, 0), s1 = unit[r].g.scale(gi, 1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt > 0 && nt >= tiles) break;
        acc[r][nt][0] = fmaf(s0, d[r][nt][0], acc[r][nt][0]);
        acc[r][nt][1] = fmaf(s0, d[r][nt][1], acc[r][nt][1]);
        acc[r][nt][2] = fmaf(s1, d[r][nt][2], acc[r][nt][2]);
        acc[r][nt][3] = fmaf(s1, d[r][nt][3], acc[r][nt][3]);
      }
    }
  }
}

// The whole product of this CTA's pairs: acc of each warp holds its share of K.
// `row(n)` is the n-th activation row, first asked for behind a barrier of the
// CTA; columns behind K are not read, and count as zeros.
template <typename T, int NG, int NT, typename Row>
__device__ __forceinline__ void strip_product(const StripAt (&at)[2], int32_t units, int32_t K, int32_t rows,
                                              int pairs, uint8_t* smem, uint32_t smem_bytes, const Row& row,
                                              float (&acc)[2][NT][4]) {
  constexpr int kAhead = NT == 1 && NG == 1 ? 3 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ways = kStripWarps / pairs;
  StripUnit<T, NG> buf[kAhead][2];
  const int32_t begin = warp / pairs;
#pragma unroll
  for (int d = 0; d < kAhead; ++d)
    if (begin + d * ways < units) {
      buf[d][0].load(at[0], begin + d * ways);
      buf[d][1].load(at[1], begin + d * ways);
    }
  // A row's pitch leaves the rows 64 bytes apart modulo 128, so the eight lanes
  // of a shared-memory phase (two rows of 64 bytes) meet all banks once.
  const int32_t chunk = min(units, (static_cast<int32_t>(smem_bytes) / rows - 64) / 256);
  const uint32_t pitch = chunk * 256 + 64;
  const int tiles = (rows + 7) / 8;
  uint32_t x[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) x[nt] = smem_u32(smem) + min(8 * nt + g, rows - 1) * pitch + 16 * t;
  int32_t base = begin;
  int next = 0;  // place in buf of the unit at `base`
  for (int32_t from = 0; from < units; from += chunk) {
    const int32_t count = min(chunk, units - from);
    __syncthreads();  // what was in shared memory has been read
    for (int32_t i = threadIdx.x; i < rows * count * 16; i += kStripThreads) {
      const int32_t n = i / (count * 16), c = i - n * (count * 16);
      *reinterpret_cast<uint4*>(smem + n * pitch + c * 16) = load_act8<true>(row(n), from * 128 + c * 8, K);
    }
    __syncthreads();
    const int32_t end = from + count;
    while (base < end) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        if (d == next && base < end) {
          strip_unit<T, NG, NT>(buf[d], x, (base - from) * 256, tiles, acc);
          const int32_t u = base + kAhead * ways;
          if (u < units) {
            buf[d][0].load(at[0], u);
            buf[d][1].load(at[1], u);
          }
          base += ways;
          next = next + 1 == kAhead ? 0 : next + 1;
        }
      }
    }
  }
}

// Adds the warps' shares of K and calls out(pair, n, strip of the pair, row of
// the strip, sum) for every row and activation row.  Pairwise sums of two
// strips at once where Both: out(pair, n, row, sum of strip 0, sum of strip 1).
template <int NT, bool Both, typename Out>
__device__ __forceinline__ void strip_reduce(const float (&acc)[2][NT][4], int pairs, int32_t rows, uint8_t* smem,
                                             const Out& out) {
  constexpr int kPitch = 36;  // 32 rows, and the fragments' stores meet all banks
  float* red = reinterpret_cast<float*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ways = kStripWarps / pairs;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(warp * NT * 8 + nt * 8 + 2 * t + (i & 1)) * kPitch + r * 16 + g + 8 * (i >> 1)] = acc[r][nt][i];
  __syncthreads();
  constexpr int kOut = Both ? 16 : 32;
  for (int32_t i = threadIdx.x; i < pairs * rows * kOut; i += kStripThreads) {
    const int32_t m = i % kOut, n = i / kOut % rows, pair = i / (kOut * rows);
    float sum[2] = {0.0f, 0.0f};
    for (int w = 0; w < ways; ++w) {
      const float* p = red + ((w * pairs + pair) * NT * 8 + n) * kPitch + m;
      sum[0] += p[0];
      if (Both) sum[1] += p[16];
    }
    out(pair, n, m, sum[0], sum[1]);
  }
}

// Host: pairs of strips a CTA takes.  More of them read the activations from
// shared memory more often for each time they are staged, and need fewer
// additions at the end; fewer of them give more CTAs.  `groups` sets of
// `pairs` pairs are to be spread over two CTAs on each SM.
inline int32_t pairs_per_cta(int64_t groups, int32_t pairs) {
  const int sms = device_sm_count();
  const int64_t want = 2 * static_cast<int64_t>(sms > 0 ? sms : 1);
  for (int32_t take = kStripWarps; take > 1; take /= 2)
    if (groups * ((pairs + take - 1) / take) >= want) return take;
  return 1;
}

// Host: dynamic shared memory for up to `rows` activation rows of `units`
// units and for the sums of tiles of NT.
inline uint32_t strip_shared(int32_t rows, int32_t units, int NT) {
  const int64_t sums = static_cast<int64_t>(kStripWarps) * NT * 8 * 36 * 4;
  const int64_t staged = static_cast<int64_t>(rows) * (static_cast<int64_t>(units) * 256 + 64);
  return static_cast<uint32_t>(max64(sums, min64(staged, kStripShared)));
}

}  // namespace flashspmm
