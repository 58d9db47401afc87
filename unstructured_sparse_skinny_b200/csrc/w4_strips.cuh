// The product of strips of 4-bit rows with a few activation rows, on the
// tensor cores through mma.sync: the engine of the experts' products.
//
// Two CTAs of sixteen warps share an SM.  A CTA takes `slots` strips (2, 4, 8
// or 16) and splits K among the warps of a strip.  A warp reads its records
// straight to registers, two units ahead; each lane finds its own fragments
// there.  The activations are staged in shared memory once and serve all strips
// of the CTA.  Warps meet only where the activations do not fit at once, and at
// the end, to add up K.  What bounds it is the rate at which the warps turn
// codes into fragments (some 160 instructions a record), so it is built for
// many warps: one strip each, 64 registers.
//
// A group's weights enter the product as whole numbers q - z, and the fp32 sum
// of the group is scaled: no weight is rounded.
#pragma once

#include "sm100_primitives.cuh"
#include "w4.cuh"

namespace flashspmm {

constexpr int kStripWarps = 16;
constexpr int kStripThreads = kStripWarps * 32;
constexpr int kStripShared = 108 * 1024;  // two CTAs on an SM

// One unit of a strip in a lane's registers.
template <typename T, int NG>
struct StripUnit {
  uint4 c[2];
  W4Groups<T, NG> g;
  __device__ __forceinline__ void load(const uint8_t* record, int lane, bool zeros) {
    c[0] = ld_stream(record + lane * 16);
    c[1] = ld_stream(record + 512 + lane * 16);
    g.load(record, lane >> 2, zeros);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& v = c[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
};

// acc += the unit's product with activations; x(nt, b) gives the lane's 16
// bytes of its row of tile nt and the unit's 32-column block b.
template <typename T, int NG, int NT, typename Act>
__device__ __forceinline__ void strip_unit(const StripUnit<T, NG>& unit, int tiles, const Act& x,
                                           float (&acc)[NT][4]) {
  constexpr int kBlocks = 4 / NG;
#pragma unroll
  for (int gi = 0; gi < NG; ++gi) {
    const W4Zero<T> z = unit.g.zero(gi);
    float d[NT][4];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int blk = gi * kBlocks + b;
      uint32_t a[2][4];
      w4_fragment(unit.word(2 * blk), z, a[0]);
      w4_fragment(unit.word(2 * blk + 1), z, a[1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt > 0 && nt >= tiles) break;
        const uint4 v = x(nt, blk);
        if (b == 0)
          mma16816_zero<T>(d[nt], a[0], v.x, v.y);
        else
          mma16816<T>(d[nt], a[0], v.x, v.y);
        mma16816<T>(d[nt], a[1], v.z, v.w);
      }
    }
    const float s0 = unit.g.scale(gi, 0), s1 = unit.g.scale(gi, 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt > 0 && nt >= tiles) break;
      acc[nt][0] = fmaf(s0, d[nt][0], acc[nt][0]);
      acc[nt][1] = fmaf(s0, d[nt][1], acc[nt][1]);
      acc[nt][2] = fmaf(s1, d[nt][2], acc[nt][2]);
      acc[nt][3] = fmaf(s1, d[nt][3], acc[nt][3]);
    }
  }
}

// The whole product of this warp's strip, its share of K: `strip` is the
// strip's first record, `pitch` the distance of its units.  `row(n)` is the
// n-th activation row, first asked for behind a barrier of the CTA; columns
// behind K are not read, and count as zeros.
template <typename T, int NG, int NT, typename Row>
__device__ __forceinline__ void strip_product(const uint8_t* strip, int32_t pitch, bool zeros, int32_t units,
                                              int32_t K, int32_t rows, int slots, uint8_t* smem, uint32_t smem_bytes,
                                              const Row& row, float (&acc)[NT][4]) {
  constexpr int kAhead = 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ways = kStripWarps / slots;
  StripUnit<T, NG> buf[kAhead];
  const int32_t begin = warp / slots;
#pragma unroll
  for (int d = 0; d < kAhead; ++d)
    if (begin + d * ways < units) buf[d].load(strip + static_cast<int64_t>(begin + d * ways) * pitch, lane, zeros);
  // A row's pitch leaves the rows 64 bytes apart modulo 128, so the eight lanes
  // of a shared-memory phase (two rows of 64 bytes) meet all banks once.
  const int32_t chunk = min(units, (static_cast<int32_t>(smem_bytes) / rows - 64) / 256);
  const uint32_t row_pitch = chunk * 256 + 64;
  const int tiles = (rows + 7) / 8;
  uint32_t x[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) x[nt] = smem_u32(smem) + min(8 * nt + g, rows - 1) * row_pitch + 16 * t;
  int32_t u = begin;
  int next = 0;  // place in buf of unit u
  for (int32_t from = 0; from < units; from += chunk) {
    const int32_t pieces = min(chunk, units - from) * 16;
    __syncthreads();  // what was in shared memory has been read
    for (int32_t i = threadIdx.x; i < rows * pieces; i += kStripThreads) {
      const int32_t n = i / pieces, c = i - n * pieces;
      *reinterpret_cast<uint4*>(smem + n * row_pitch + c * 16) = load_act8<true>(row(n), from * kW4UnitCols + c * 8, K);
    }
    __syncthreads();
    const int32_t end = min(units, from + chunk);
    while (u < end) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        if (d == next && u < end) {
          const uint32_t offset = (u - from) * 256;
          strip_unit<T, NG, NT>(
              buf[d], tiles,
              [&](int nt, int b) {
                uint4 v;
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                             : "r"(x[nt] + offset + b * 64)
                             : "memory");
                return v;
              },
              acc);
          const int32_t ahead = u + kAhead * ways;
          if (ahead < units) buf[d].load(strip + static_cast<int64_t>(ahead) * pitch, lane, zeros);
          u += ways;
          next = next + 1 == kAhead ? 0 : next + 1;
        }
      }
    }
  }
}

// Adds the warps' shares of K.  out(slot, n, row, sum), or with Pairs
// out(pair, n, row, sum of slot 2 pair, sum of slot 2 pair + 1).
template <int NT, bool Pairs, typename Out>
__device__ __forceinline__ void strip_reduce(const float (&acc)[NT][4], int slots, int32_t rows, uint8_t* smem,
                                             const Out& out) {
  constexpr int kPitch = 20;  // 16 rows, and the fragments' stores meet all banks
  float* red = reinterpret_cast<float*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      red[(warp * NT * 8 + nt * 8 + 2 * t + (i & 1)) * kPitch + g + 8 * (i >> 1)] = acc[nt][i];
  __syncthreads();
  constexpr int kStep = Pairs ? 2 : 1;
  for (int32_t i = threadIdx.x; i < slots / kStep * rows * 16; i += kStripThreads) {
    const int32_t m = i & 15, n = (i >> 4) % rows, s = (i >> 4) / rows * kStep;
    float sum[2] = {0.0f, 0.0f};
    for (int w = s; w < kStripWarps; w += slots) {
      sum[0] += red[(w * NT * 8 + n) * kPitch + m];
      if (Pairs) sum[1] += red[((w + 1) * NT * 8 + n) * kPitch + m];
    }
    out(s / kStep, n, m, sum[0], sum[1]);
  }
}

// Host: strips a CTA takes.  More of them stage the activations more seldom
// and need fewer additions at the end; fewer of them give more CTAs.  `sets`
// sets of `strips` strips are to be spread over two CTAs on each SM.
inline int32_t strips_per_cta(int64_t sets, int32_t strips, int32_t least) {
  const int sms = device_sm_count();
  const int64_t want = 2 * static_cast<int64_t>(sms > 0 ? sms : 1);
  for (int32_t take = kStripWarps; take > least; take /= 2)
    if (sets * ((strips + take - 1) / take) >= want) return take;
  return least;
}

// Host: dynamic shared memory for up to `rows` activation rows of `units`
// units and for the sums of tiles of NT.
inline uint32_t strip_shared(int32_t rows, int32_t units, int NT) {
  const int64_t sums = static_cast<int64_t>(kStripWarps) * NT * 8 * 20 * 4;
  const int64_t staged = static_cast<int64_t>(rows) * (static_cast<int64_t>(units) * 256 + 64);
  return static_cast<uint32_t>(max64(sums, min64(staged, kStripShared)));
}

}  // namespace flashspmm
