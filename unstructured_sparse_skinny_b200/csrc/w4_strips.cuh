// The product of strips of 4-bit rows with a few activation rows, on the
// tensor cores through mma.sync: the engine of the experts' products.
//
// CTAs of eight warps share an SM.  A warp has a pair of strips (two of one
// matrix, or the same of two matrices), whose fragments use each 16 bytes of
// activations twice; a CTA takes `pairs` pairs (1, 2, 4 or 8) and splits K among
// the warps of a pair.  A warp's records arrive by asynchronous copies in a ring
// of its own in shared memory, two units ahead: no other warp waits for them,
// and the registers they would fill are free for fragments (64 tokens, 64 experts
// of 4096 x 2048: 271 us for the layer, with two units ahead in registers 312;
// four units ahead leave less room for activations, 283).  The activations are
// staged in shared memory, as many units as fit at a time, and serve all strips
// of the CTA.  Warps meet only there, and at the end, to add up K.  What bounds
// it is the rate at which the warps turn codes into fragments: 177 instructions
// a record, issued in 65 % of the cycles, at half the rate of HBM.  (Sixteen
// warps with one strip each read the activations twice as often: a fifth slower.)
//
// A group's weights enter the product as whole numbers q - z (in bf16 times a
// power of two), and the fp32 sum of the group is scaled: no weight is rounded.
#pragma once

#include <cmath>

#include "sm100_primitives.cuh"
#include "w4.cuh"

namespace flashspmm {

constexpr int kStripWarps = 8;
constexpr int kStripThreads = kStripWarps * 32;
constexpr int kStripRing = 2;  // units of a warp on their way to shared memory

// CTAs that an SM holds, by the tiles of eight activation rows of their warps,
// and the shared memory of one.  (One tile: three in 80 registers a thread, 130
// us instead of 134 for 4 tokens, 8 experts of 4096 x 11008.  Two tiles spill
// there, 271 -> 356 us for 64 tokens, 64 experts of 4096 x 2048.)
constexpr int strip_ctas(int NT) { return NT == 1 ? 3 : NT == 2 ? 2 : 1; }
constexpr int strip_limit(int NT) { return (NT == 1 ? 74 : NT == 2 ? 112 : 224) * 1024; }

// One unit of a strip in a lane's registers.
template <typename T, int NG>
struct StripUnit {
  uint4 c[2];
  W4Groups<T, NG> g;
  // from global memory
  __device__ __forceinline__ void read(const uint8_t* record, int lane, bool zeros) {
    c[0] = ld_stream(record + lane * 16);
    c[1] = ld_stream(record + 512 + lane * 16);
    g.load(record, lane >> 2, zeros);
  }
  // from shared memory
  __device__ __forceinline__ void load(const uint8_t* record, int lane, bool zeros) {
    c[0] = *reinterpret_cast<const uint4*>(record + lane * 16);
    c[1] = *reinterpret_cast<const uint4*>(record + 512 + lane * 16);
    g.load(record, lane >> 2, zeros);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& v = c[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
};

// acc += the unit's product with activations, of R strips (w4_raise of a finished
// acc is the product); x(nt, b, part) gives the lane's 16 bytes of its row of
// tile nt and the unit's 32-column block b.  Activations of several parts are
// their sum.
template <typename T, int NG, int R, int NT, int Tiles, int Parts = 1, typename Act>
__device__ __forceinline__ void strip_unit(const StripUnit<T, NG> (&unit)[R], int tiles, const Act& x,
                                           float (&acc)[R][Tiles][4]) {
  constexpr int kBlocks = 4 / NG;
#pragma unroll
  for (int gi = 0; gi < NG; ++gi) {
    float d[R][NT][4];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int blk = gi * kBlocks + b;
      uint32_t a[R][2][4];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const auto z = unit[r].g.zero(gi);
        w4_fragment(unit[r].word(2 * blk), z, a[r][0]);
        w4_fragment(unit[r].word(2 * blk + 1), z, a[r][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt > 0 && nt >= tiles) break;
#pragma unroll
        for (int part = 0; part < Parts; ++part) {
          const uint4 v = x(nt, blk, part);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (b == 0 && part == 0)
              mma16816_zero<T>(d[r][nt], a[r][0], v.x, v.y);
            else
              mma16816<T>(d[r][nt], a[r][0], v.x, v.y);
          }
#pragma unroll
          for (int r = 0; r < R; ++r) mma16816<T>(d[r][nt], a[r][1], v.z, v.w);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
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

// A strip's first record for a warp.
struct StripAt {
  const uint8_t* record;
  int32_t pitch;  // to the strip's next unit
  bool zeros;
  __device__ __forceinline__ StripAt(const W4Dev& A, int64_t unit)
      : record(A.at(unit)), pitch(8 * A.record), zeros(A.zeros) {}
};

// Copies 16 bytes to shared memory without waiting for them, or zeros.
__device__ __forceinline__ void copy_or_zero(uint32_t to, const void* from, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(copy ? 16 : 0) : "memory");
}

// The shared memory a warp's units arrive in: places of a pair of records.
template <int NG>
struct StripRing {
  static constexpr uint32_t kRecord = kW4CodeBytes + 48 * NG, kPlace = 2 * kRecord, kBytes = kStripRing * kPlace;
  uint8_t* base;  // this warp's
  // Starts the copies of one pair of records, one group of copies for wait().
  __device__ __forceinline__ void ask(int place, const uint8_t* const (&from)[2], const bool (&zeros)[2], int lane) const {
    const uint32_t to = smem_u32(base) + place * kPlace;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      cp_async_16(to + r * kRecord + lane * 16, from[r] + lane * 16);
      cp_async_16(to + r * kRecord + 512 + lane * 16, from[r] + 512 + lane * 16);
    }
    // scales and zero points: half a warp a record
    const int piece = lane & 15;
    const bool second = lane >= 16;
    if (piece < ((second ? zeros[1] : zeros[0]) ? 3 * NG : 2 * NG))
      cp_async_16(to + (second ? kRecord : 0) + kW4CodeBytes + piece * 16,
             (second ? from[1] : from[0]) + kW4CodeBytes + piece * 16);
  }
  // The oldest of kStripRing groups has arrived, for the whole warp.
  static __device__ __forceinline__ void wait() {
    cp_async_wait<kStripRing - 1>();
    __syncwarp();
  }
};

// The whole product of this warp's strips, its share of K.  `row(n)` is the
// n-th activation row, first asked for behind a barrier of the CTA; columns
// behind K are not read, and count as zeros.  With two parts the rows from
// `rows` on are the first ones' second parts.  `staged` is shared memory for
// activations, behind the rings.
template <typename T, int NG, int NT, int Parts, typename Row>
__device__ __forceinline__ void strip_product(const StripAt (&at)[2], int32_t units, int32_t K, int32_t rows,
                                              int pairs, uint8_t* rings, uint8_t* staged, uint32_t staged_bytes,
                                              const Row& row, float (&acc)[2][NT][4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ways = kStripWarps / pairs;
  const StripRing<NG> ring{rings + warp * StripRing<NG>::kBytes};
  int32_t u = warp / pairs, asked = u;
  const uint8_t* from[2] = {at[0].record + static_cast<int64_t>(u) * at[0].pitch,
                            at[1].record + static_cast<int64_t>(u) * at[1].pitch};
  const bool zeros[2] = {at[0].zeros, at[1].zeros};
  const auto ask = [&](int place) {
    if (asked < units) ring.ask(place, from, zeros, lane);
    cp_async_commit();
    asked += ways;
#pragma unroll
    for (int r = 0; r < 2; ++r) from[r] += static_cast<int64_t>(ways) * at[r].pitch;
  };
#pragma unroll
  for (int d = 0; d < kStripRing; ++d) ask(d);
  // A row's pitch leaves the rows 64 bytes apart modulo 128, so the eight lanes
  // of a shared-memory phase (two rows of 64 bytes) meet all banks once.
  const int32_t chunk = min(units, (static_cast<int32_t>(staged_bytes) / (rows * Parts) - 64) / 256);
  const uint32_t row_pitch = chunk * 256 + 64;
  const int tiles = (rows + 7) / 8;
  uint32_t x[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) x[nt] = smem_u32(staged) + min(8 * nt + g, rows - 1) * row_pitch + 16 * t;
  const uint32_t below = rows * row_pitch;  // from a row to its second part
  int place = 0;                            // of unit u
  for (int32_t first = 0; first < units; first += chunk) {
    const int32_t pieces = min(chunk, units - first) * 16;
    __syncthreads();  // what was in shared memory has been read
    for (int32_t i = threadIdx.x; i < rows * Parts * pieces; i += kStripThreads) {
      const int32_t n = i / pieces, c = i - n * pieces, k = first * kW4UnitCols + c * 8;
      copy_or_zero(smem_u32(staged) + n * row_pitch + c * 16, row(n) + (k < K ? k : 0), k < K);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    for (const int32_t end = min(units, first + chunk); u < end; u += ways) {
      const uint32_t offset = (u - first) * 256;
      const auto act = [&](int nt, int b, int part) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(x[nt] + offset + part * below + b * 64)
                     : "memory");
        return v;
      };
      ring.wait();
      StripUnit<T, NG> unit[2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
        unit[r].load(ring.base + place * ring.kPlace + r * ring.kRecord, lane, at[r].zeros);
      // (a branch for a single tile: predicates alone leave the products of the others in the pipe)
      if (NT > 1 && tiles == 1)
        strip_unit<T, NG, 2, 1, NT, Parts>(unit, 1, act, acc);
      else
        strip_unit<T, NG, 2, NT, NT, Parts>(unit, tiles, act, acc);
      __syncwarp();
      ask(place);
      place = place + 1 == kStripRing ? 0 : place + 1;
    }
  }
}

// Adds the warps' shares of K: out(pair, n, row, sum of the first strip, of the second).
template <typename T, int NT, typename Out>
__device__ __forceinline__ void strip_reduce(const float (&acc)[2][NT][4], int pairs, int32_t rows, uint8_t* smem,
                                             const Out& out) {
  constexpr int kPitch = 36;  // 32 rows, and the fragments' stores meet all banks
  float* red = reinterpret_cast<float*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(warp * NT * 8 + nt * 8 + 2 * t + (i & 1)) * kPitch + r * 16 + g + 8 * (i >> 1)] = acc[r][nt][i];
  __syncthreads();
  for (int32_t i = threadIdx.x; i < pairs * rows * 16; i += kStripThreads) {
    const int32_t m = i & 15, n = (i >> 4) % rows, pair = (i >> 4) / rows;
    float a = 0.0f, b = 0.0f;
    for (int w = pair; w < kStripWarps; w += pairs) {
      a += red[(w * NT * 8 + n) * kPitch + m];
      b += red[(w * NT * 8 + n) * kPitch + 16 + m];
    }
    out(pair, n, m, w4_raise<T>(a), w4_raise<T>(b));
  }
}

// Host: pairs of strips a CTA takes, for `sets` sets of `pairs` with `rows`
// activation rows each.  The CTAs run in waves of `resident` on each SM; a CTA's
// time is its records', the staging of the activations and a fixed part, in
// records, as fitted with two CTAs an SM (22 KB/us for each of 296 at the rate of
// HBM: a record is 0.05 us, the fixed part some 3 us; staging a row's unit is a
// tenth of a record).  With one and three an SM the constants are the same: the
// choice is within 3 % of the best of 1, 2, 4 and 8 in all (us by this rule, and
// by each: 4 tokens, 8 experts of 4096 x 11008, 120, 134 124 121 120; 8 tokens, 64
// of 4096 x 2048, 217, 235 214 212 216; 64 tokens, 288, 482 360 302 289; 64 tokens,
// 4 of 4096 x 4096, 243, 431 325 261 302).
inline int32_t pairs_per_cta(double sets, int32_t pairs, int32_t units, double rows, int resident) {
  const int sms = device_sm_count();
  const double wave = static_cast<double>(resident) * (sms > 0 ? sms : 1);
  int32_t best = 1;
  double least = 0.0;
  for (int32_t take = 1; take <= kStripWarps; take *= 2) {
    const double ctas = sets * ((pairs + take - 1) / take);
    const double cost = std::ceil(ctas / wave) * (2.0 * take * units + 64.0 + 0.1 * rows * units);
    if (take == 1 || cost < least) {
      least = cost;
      best = take;
    }
  }
  return best;
}

// Host: dynamic shared memory for the rings, up to `rows` activation rows of
// `units` units and the sums of tiles of NT.
template <int NG>
inline uint32_t strip_shared(int32_t rows, int32_t units, int NT) {
  constexpr int64_t rings = kStripWarps * StripRing<NG>::kBytes;
  const int64_t sums = static_cast<int64_t>(kStripWarps) * NT * 8 * 36 * 4;
  const int64_t staged = static_cast<int64_t>(rows) * (static_cast<int64_t>(units) * 256 + 64);
  return static_cast<uint32_t>(rings + max64(sums, min64(staged, strip_limit(NT) - rings)));
}

}  // namespace flashspmm
