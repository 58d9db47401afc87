// Skinny product with 4-bit weights on the fifth-generation tensor cores, for
// more tokens than a warp's own fragments serve well.
//
// The work is blocks of 128 rows times units of 128 columns; every SM runs one
// CTA over an equal run of these steps.  Bulk copies bring codes and
// activations into shared memory; sixteen warps turn codes into 16-bit weights
// in registers (s * (q - z), rounded once) and store them straight to
// tensor memory, where tcgen05.mma takes its A operand from: the weights never
// pass through shared memory, whose bandwidth the activations need.  The
// 16x128b store shape places a lane's fragment registers as the packed
// layout holds them (row g and g + 8, column pairs t), so no lane exchanges
// anything.  That fixes the order of K inside a 16-column step; the
// activations are put into the same order, swizzled and padded by a small
// kernel first, after which one bulk copy brings a unit of them into shared
// memory.
//
// A block that one CTA has whole is stored at once.  The sums of one that
// several CTAs share go to the workspace, and the last of them to arrive adds
// them in their order.  Four warps do this behind the products; at the end of
// its run the whole CTA joins in, since nothing is left to overlap with.
//
// The rounding of the weights is the price of an A operand of 16 bits that holds
// the scale: half a step of the type a weight, independent of one another, which
// with the output's own rounding makes an error 1.34 times that of the latter
// alone (64 tokens of 12288^2, bf16: 2.2e-3 of the result's norm, 1.7e-3).
//
// For fp32 output the weights are not rounded: each unit is two steps, of the
// weights rounded to 16 bits and of what that leaves, which 16 bits hold exactly.
// The second step has its own image of the activations, zeros in place of what is
// not finite: infinity times a rest of zero would be NaN.
//
// What bounds it: up to 128 tokens the warps that make the weights (12288^2, 64
// tokens: 35 us; HBM would allow 12); at 256 tokens the
// products, 1024 cycles a unit, and the clock under the power limit (9216 x 36864:
// 128 us, 1.36 PFLOP/s, alone at 1965 MHz; 172 us, 1.01 PFLOP/s, in a loop at the
// 1305 MHz that 1000 W leave).  Some 8 us a call are fixed: two kernels, the
// ends of the runs and the joining of shared blocks.
#include <atomic>
#include <type_traits>

#include "sm100_primitives.cuh"
#include "w4.cuh"

namespace flashspmm {
namespace {

constexpr int kDequantWarps = 16;
constexpr int kEpilogueWarp = 16;          // 16 .. 19
constexpr int kMmaWarp = 20;               // 20, 21
constexpr int kLoadWarp = 22;              // 22 the activations, 23 the codes
constexpr int kThreads = 24 * 32;
constexpr int kBlockRows = 128;
constexpr int kMaxSlots = 4;               // units between codes and product
constexpr int kMaxRing = 12;               // units of codes in shared memory
constexpr int kSharedBytes = 224 * 1024;   // for activations and codes
constexpr uint32_t kUnitTmemCols = 64;     // 128 values of 16 bits
constexpr uint32_t kAccCols = 256;         // accumulators: see Accumulators
constexpr uint64_t kWaitBudgetNs = 1000000000ull;

struct GemmParams {
  W4Dev A;
  const uint8_t* image;  // [units, or steps of a block][2][n_pad][128 bytes], swizzled
  float* partials;       // [CTA][first, last block of its run][n_pad][128]
  int32_t* arrived;      // [blocks]
  void* C;
  int64_t ldc;
  bool c_f32;
  int32_t N, n_pad;
  int32_t slots, ring;
  int32_t steps;         // blocks * units, twice that many for unrounded weights
  int* status;
};

// ---------------------------------------------------------------- activations in the product's order

// One thread per row and 32-column block: position 16 s + 8 h + 2 t + e of a
// block holds column 8 t + 4 s + 2 h + e.  A block is half a 128-byte row of
// the tile, whose 16-byte chunks are exchanged by row (128-byte swizzle).
// Split: two tiles a unit, the second without the values that are not finite;
// `exponent` is the bits of an exponent in both halves of a word.
template <bool Vec, bool Split>
__global__ void __launch_bounds__(256) w4_stage_kernel(const uint16_t* __restrict__ B, int64_t ldb, int32_t N,
                                                       int32_t K, int32_t n_pad, int64_t blocks,
                                                       uint8_t* __restrict__ image, int32_t* __restrict__ arrived,
                                                       int64_t row_blocks, uint32_t exponent) {
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t j = i; j < row_blocks; j += static_cast<int64_t>(gridDim.x) * 256) arrived[j] = 0;
  if (i >= blocks * n_pad) return;
  const int32_t n = static_cast<int32_t>(i / blocks);
  const int64_t blk = i - static_cast<int64_t>(n) * blocks;
  const uint16_t* row = n < N ? B + n * ldb : nullptr;
  uint32_t w[16];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint4 v = load_act8<Vec>(row, static_cast<int32_t>(blk * 32 + 8 * t), K);
    w[4 * t] = v.x;
    w[4 * t + 1] = v.y;
    w[4 * t + 2] = v.z;
    w[4 * t + 3] = v.w;
  }
#pragma unroll
  for (int part = 0; part < (Split ? 2 : 1); ++part) {
    const int64_t half = Split ? (blk >> 2) * 4 + part * 2 + (blk >> 1 & 1) : blk >> 1;
    uint8_t* tile = image + half * (static_cast<int64_t>(n_pad) * 128) + n * 128;
    if (part == 1) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t low = exponent & 0xFFFFu, high = exponent & 0xFFFF0000u;
        if ((w[j] & low) == low) w[j] &= 0xFFFF0000u;
        if ((w[j] & high) == high) w[j] &= 0xFFFFu;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // c = 2 s + h
      const int chunk = ((blk & 1) * 4 + c) ^ (n & 7);
      *reinterpret_cast<uint4*>(tile + chunk * 16) = make_uint4(w[c], w[4 + c], w[8 + c], w[12 + c]);
    }
  }
}

// ---------------------------------------------------------------- primitives

// Untiled bulk load; both addresses 16-byte aligned, the size a multiple of 16.
__device__ __forceinline__ void bulk_load(void* smem, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(smem)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(pred));
  return pred != 0;
}

// 16 TMEM lanes x 32 columns: register 2 i is row g, 2 i + 1 row g + 8 of column 4 i + t.
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 TMEM lanes x 64 columns, likewise.
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[32]) {
  uint32_t half[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 16; ++i) half[i] = r[16 * h + i];
    tmem_store(taddr + 32 * h, half);
  }
}
// 16 TMEM lanes x 16 columns, likewise.
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem desc]^T
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---------------------------------------------------------------- codes to 16-bit weights

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t s, __half) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(s));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t s, __nv_bfloat16) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(s));
  return r;
}

// A weight has at most 8 + 6 (bf16) or 11 + 6 (fp16) significant bits, multiples of the type's smallest step: its
// rounding's rest is exact in 16 bits too.  Up to twice the largest 16-bit value, that is: the rounding stops at the
// largest, and a weight that both parts together cannot hold is infinite.
template <typename T>
struct Pair;
template <>
struct Pair<__half> {
  using Type = __half2;
  static constexpr uint32_t kLargest = 0x7BFF7BFFu;
};
template <>
struct Pair<__nv_bfloat16> {
  using Type = __nv_bfloat162;
  static constexpr uint32_t kLargest = 0x7F7F7F7Fu;
};
template <typename T>
__device__ __forceinline__ uint32_t part2(uint32_t a, uint32_t s, bool rest) {
  union U {
    uint32_t u;
    typename Pair<T>::Type v;
  } x, y, product, most, least;
  x.u = a;
  y.u = s;
  product.u = mul2(a, s, T());
  most.u = Pair<T>::kLargest;
  least.u = Pair<T>::kLargest | 0x80008000u;
  product.v = __hmax2_nan(__hmin2_nan(product.v, most.v), least.v);
  if (rest) {
    product.u ^= 0x80008000u;
    product.v = __hfma2(x.v, y.v, product.v);
  }
  return product.u;
}

// The P-th part (128 / P columns) of one strip of it as a lane holds it: codes, then 16-bit weights.
template <typename T, int NG, int P>
struct Part {
  static constexpr int kWords = 8 / P;                   // of 8 codes
  static constexpr int kGroups = NG > P ? NG / P : 1;    // scales that touch the part
  uint32_t w[kWords];
  uint32_t s[kGroups], z[kGroups];                       // {row g, row g + 8}

  __device__ __forceinline__ void load(const uint8_t* record, int part, int lane, bool zeros) {
    if (P == 1) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(record + i * 512 + lane * 16);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[(4 * i + 2) % kWords] = v.z;
        w[(4 * i + 3) % kWords] = v.w;
      }
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(record + (part >> 1) * 512 + lane * 16 + (part & 1) * 8);
      w[0] = v.x;
      w[1] = v.y;
    }
    const int at = (lane >> 2) * (2 * NG) + 2 * (part * NG / P);
    const uint8_t* scales = record + kW4CodeBytes + at * 2;
    const uint8_t* points = record + kW4CodeBytes + 32 * NG + at;
    if (kGroups == 1) {
      s[0] = *reinterpret_cast<const uint32_t*>(scales);
      z[0] = zeros ? *reinterpret_cast<const uint16_t*>(points) : 0x0808u;
    } else if (kGroups == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(scales);
      s[0] = v.x;
      s[1 % kGroups] = v.y;
      s[2 % kGroups] = v.z;
      s[kGroups - 1] = v.w;
      const uint2 q = zeros ? *reinterpret_cast<const uint2*>(points) : make_uint2(0x08080808u, 0x08080808u);
      z[0] = q.x & 0xFFFF;
      z[1 % kGroups] = q.x >> 16;
      z[2 % kGroups] = q.y & 0xFFFF;
      z[kGroups - 1] = q.y >> 16;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(scales);
      s[0] = v.x;
      s[kGroups - 1] = v.y;
      const uint32_t q = zeros ? *reinterpret_cast<const uint32_t*>(points) : 0x08080808u;
      z[0] = q & 0xFFFF;
      z[kGroups - 1] = q >> 16;
    }
  }

  // Split: in two parts, `rest` the second one.
  template <bool Split>
  __device__ __forceinline__ void weights(uint32_t (&r)[4 * kWords], bool rest) const {
#pragma unroll
    for (int gi = 0; gi < kGroups; ++gi) {
      const W4Zero<T, 0> zero(static_cast<int>(z[gi] & 0xFF), static_cast<int>(z[gi] >> 8));
      const uint32_t s0 = __byte_perm(s[gi], 0, 0x1010), s1 = __byte_perm(s[gi], 0, 0x3232);
#pragma unroll
      for (int i = gi * kWords / kGroups; i < (gi + 1) * kWords / kGroups; ++i) {
        uint32_t a[4];
        w4_fragment(w[i], zero, a);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r[4 * i + j] = Split ? part2<T>(a[j], j & 1 ? s1 : s0, rest) : mul2(a[j], j & 1 ? s1 : s0, T());
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ uint32_t idesc_of(int n) {
  const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;  // of A and B
  return umma_idesc_f16_f32(kBlockRows, n) | (type << 7) | (type << 10);
}

template <typename T>
__device__ __forceinline__ void store_row(const GemmParams& p, int64_t m, int32_t n0, const float (&v)[16]) {
  // 16 tokens of one row; a warp's lanes hold neighbouring rows
  const int32_t count = p.N - n0;
  if (p.c_f32) {
    float* c = static_cast<float*>(p.C) + n0 * p.ldc + m;
#pragma unroll
    for (int j = 0; j < 16; ++j, c += p.ldc)
      if (j < count) *c = v[j];
  } else {
    T* c = static_cast<T*>(p.C) + n0 * p.ldc + m;
#pragma unroll
    for (int j = 0; j < 16; ++j, c += p.ldc)
      if (j < count) *c = from_float<T>(v[j]);
  }
}

template <typename T>
__device__ __forceinline__ void store_four(const GemmParams& p, int32_t n, int64_t m, const float4& v) {
  const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (m + j < p.A.M) {
      if (p.c_f32)
        static_cast<float*>(p.C)[n * p.ldc + m + j] = x[j];
      else
        static_cast<T*>(p.C)[n * p.ldc + m + j] = from_float<T>(x[j]);
    }
}

// Two warps issue products, for every other unit each and into an accumulator
// of its own, where one could not issue as fast as a unit of few tokens is
// done (N <= 128); up to 64 tokens there is room for two blocks' accumulators.
struct Accumulators {
  int issuers, buffers;
  uint32_t cols;  // of one
  __device__ __forceinline__ explicit Accumulators(int32_t n_pad)
      : issuers(n_pad <= 128 ? 2 : 1), buffers(n_pad <= 64 ? 2 : 1), cols(n_pad <= 64 ? 64 : n_pad <= 128 ? 128 : 256) {}
  __device__ __forceinline__ uint32_t at(int issuer, int buffer) const { return (buffer * issuers + issuer) * cols; }
};

// ---------------------------------------------------------------- kernel

// A run of steps cut into segments of one block each.
struct Segment {
  int32_t block;
  int32_t from, to;  // steps
  bool whole;
};
__device__ __forceinline__ Segment segment_of(int32_t block, int32_t q0, int32_t q1, int32_t units) {
  Segment s;
  s.block = block;
  s.from = max(q0, block * units);
  s.to = min(q1, (block + 1) * units);
  s.whole = s.to - s.from == units;
  return s;
}

// Runs differ by a step at most, the longer ones first.
struct Runs {
  int32_t base, longer;
  __device__ __forceinline__ Runs(int32_t steps, int32_t ctas) : base(steps / ctas), longer(steps % ctas) {}
  __device__ __forceinline__ int32_t begin(int32_t cta) const { return cta * base + min(cta, longer); }
  __device__ __forceinline__ int32_t owner(int32_t q) const {
    const int32_t head = longer * (base + 1);
    return q < head ? q / (base + 1) : longer + (q - head) / base;
  }
};

// The accumulators of a segment to C (a whole block) or to the CTA's slot of
// the workspace, by `groups` warps per 32 rows, this one the `group`-th.
template <typename T>
__device__ __forceinline__ void drain_segment(const GemmParams& p, const Segment& seg, const Accumulators& acc,
                                              uint32_t tmem, int buffer, int32_t q0, int group, int groups, int quad,
                                              int lane) {
  const int row = quad * 32 + lane;
  const int64_t m = static_cast<int64_t>(seg.block) * kBlockRows + row;
  const uint32_t from = tmem + acc.at(0, buffer) + (static_cast<uint32_t>(quad * 32) << 16);
  const int first = static_cast<int>((seg.from - q0) & 1);
  // with two issuers: a segment of one unit has one sum, in its issuer's accumulator
  const bool both = acc.issuers == 2 && seg.to - seg.from > 1;
  const uint32_t one = acc.issuers == 2 && !both ? first * acc.cols : 0;
  float* part = p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (seg.from > q0)) * p.n_pad * kBlockRows + row;
  for (int32_t n0 = group * 16; n0 < p.n_pad; n0 += groups * 16) {
    uint32_t a[16], b[16];
    tmem_load_16(from + one + n0, a);
    if (both) tmem_load_16(from + acc.cols + n0, b);
    tmem_load_wait();
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      v[j] = both ? __uint_as_float(a[j]) + __uint_as_float(b[j]) : __uint_as_float(a[j]);
    if (!seg.whole) {
      float* o = part + n0 * kBlockRows;
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j * kBlockRows] = v[j];
    } else if (m < p.A.M) {
      store_row<T>(p, m, n0, v);
    }
  }
}

// The CTAs that share a block.
struct Sharers {
  int32_t first, last;
  int32_t first_slot;  // the others hold the block first in their run
  __device__ __forceinline__ Sharers(const Runs& runs, int32_t block, int32_t units) {
    const int32_t from = block * units;
    first = runs.owner(from);
    last = runs.owner(from + units - 1);
    first_slot = first * 2 + (runs.begin(first) < from);
  }
};

// One thread's call after a barrier of the block's warps: whether this CTA is
// the last of the block's to have its sums in the workspace.  The fences cover
// what the barrier ordered before them, and what follows the next one.
__device__ __forceinline__ bool arrive_at(const GemmParams& p, int32_t block, const Sharers& who) {
  __threadfence();
  const bool last = atomicAdd(&p.arrived[block], 1) == who.last - who.first;
  __threadfence();
  return last;
}

// All sums of a shared block, in the order of its CTAs, by `threads` threads.
template <typename T>
__device__ __forceinline__ void join_block(const GemmParams& p, int32_t block, const Sharers& who, int tid,
                                           int threads) {
  constexpr int kBatch = 4;  // loads in flight a thread and CTA
  const int32_t total = p.N * (kBlockRows / 4);
  const float4* base = reinterpret_cast<const float4*>(p.partials);
  const int64_t slot = static_cast<int64_t>(p.n_pad) * (kBlockRows / 4);
  for (int32_t i0 = tid; i0 < total; i0 += threads * kBatch) {
    float4 sum[kBatch] = {};
    for (int32_t c = who.first; c <= who.last; c += 2) {
      const float4* s0 = base + (c == who.first ? who.first_slot : c * 2) * slot;
      const float4* s1 = base + static_cast<int64_t>(c + 1) * 2 * slot;
      const bool second = c < who.last;
      float4 v0[kBatch], v1[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int32_t i = i0 + threads * j;
        v0[j] = i < total ? __ldcg(s0 + i) : make_float4(0, 0, 0, 0);
        v1[j] = second && i < total ? __ldcg(s1 + i) : make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        sum[j].x = sum[j].x + v0[j].x + v1[j].x;
        sum[j].y = sum[j].y + v0[j].y + v1[j].y;
        sum[j].z = sum[j].z + v0[j].z + v1[j].z;
        sum[j].w = sum[j].w + v0[j].w + v1[j].w;
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int32_t i = i0 + threads * j;
      if (i < total) store_four<T>(p, i / (kBlockRows / 4), static_cast<int64_t>(block) * kBlockRows + (i % (kBlockRows / 4)) * 4, sum[j]);
    }
  }
}

// P (1 or 4): warps share the columns of 32 rows of a unit P ways, so 4 / P groups of 4 P warps have units in turn.
// Split: two steps a unit, see part2.
template <typename T, int NG, int P, bool Split>
__global__ void __launch_bounds__(kThreads, 1) w4_gemm_kernel(const GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t codes_full[kMaxRing], codes_used[kMaxRing], full[kMaxSlots], used[kMaxSlots], acc_full[2], acc_empty[2], mma_done[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word, last_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kSteps = Split ? 2 : 1;  // of a unit
  const int32_t units = p.A.units * kSteps;
  const Runs runs(p.steps, gridDim.x);
  const int32_t q0 = runs.begin(blockIdx.x), q1 = runs.begin(blockIdx.x + 1);
  const uint32_t stage_bytes = static_cast<uint32_t>(p.n_pad) * 256, unit_bytes = 8 * p.A.record;
  const Accumulators acc(p.n_pad);
  uint8_t* tiles = smem + ((1024 - (smem_u32(smem) & 1023)) & 1023);
  uint8_t* codes = tiles + p.slots * stage_bytes;

  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&full[i], 4 * P + 1);  // the warps' weights and the copy of the activations
      mbar_init(&used[i], 1);
    }
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&codes_full[i], 1);
      mbar_init(&codes_used[i], 4 * P);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], acc.issuers);
      mbar_init(&acc_empty[i], 4);
      mbar_init(&mma_done[i], 1);
    }
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp < kDequantWarps) {
    // ---- codes -> tensor memory.  A slot, and a place of the ring of codes, belongs to one group: taken in
    // turns it could be two phases away from a group's wait, which parity does not tell from none.
    constexpr int kGroups = 4 / P;
    const int quad = warp & 3, part = (warp >> 2) % P, group = (warp >> 2) / P;
    const uint32_t dst =
        tmem + kAccCols + part * (kUnitTmemCols / P) + (static_cast<uint32_t>(quad * 32) << 16);
    const bool zeros = p.A.zeros;
    const uint8_t* mine = codes + quad * 2 * p.A.record;
    uint32_t phase = 1, ring_phase = 0;
    int ring = group, slot = group;
    for (int32_t q = q0 + group; q < q1; q += kGroups) {
      if (!mbar_wait(&codes_full[ring], ring_phase, abort_flag, kWaitBudgetNs, p.status)) break;
      __syncwarp();
      const uint8_t* record = mine + ring * unit_bytes;
      // Both strips' weights wait in registers for the slot, or with all 128 columns a warp, where the other
      // groups fill the time, one strip's.
      constexpr int kHeld = P > 1 ? 2 : 1;
      uint32_t r[kHeld][32 / P];
      bool ready = true;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Part<T, NG, P> strip;
        strip.load(record + j * p.A.record, part, lane, zeros);
        strip.template weights<Split>(r[j % kHeld], q & 1);
        if (j == kHeld - 1) {
          ready = mbar_wait(&used[slot], phase, abort_flag, kWaitBudgetNs, p.status);
          if (!ready) break;
          __syncwarp();
          tc_fence_after_sync();
        }
        if (P == 1) tmem_store(dst + slot * kUnitTmemCols + (static_cast<uint32_t>(16 * j) << 16), r[0]);
      }
      if (P > 1 && ready) {
        tmem_store(dst + slot * kUnitTmemCols, r[0]);
        tmem_store(dst + slot * kUnitTmemCols + (16u << 16), r[kHeld - 1]);
      }
      if (!ready) break;
      if (lane == 0) mbar_arrive(&codes_used[ring]);  // all lanes have their weights: the stores are the warp's
      tmem_store_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[slot]);
      ring += kGroups;
      if (ring >= p.ring) {
        ring -= p.ring;
        ring_phase ^= 1;
      }
      slot += kGroups;
      if (slot >= p.slots) {
        slot -= p.slots;
        phase ^= 1;
      }
    }
  } else if (warp < kMmaWarp) {
    // ---- all blocks of the run but the last: accumulators -> C or the workspace, behind the products
    griddep_wait();
    int buffer = 0;
    uint32_t phase = 0;
    for (int32_t block = q0 / units; (block + 1) * units < q1; ++block) {
      const Segment seg = segment_of(block, q0, q1, units);
      const Sharers who(runs, block, units);
      // a wait that runs out leaves wrong values and an error, not a warp missing at the barriers below
      mbar_wait(&acc_full[buffer], phase, abort_flag, kWaitBudgetNs, p.status);
      __syncwarp();
      tc_fence_after_sync();
      drain_segment<T>(p, seg, acc, tmem, buffer, q0, 0, 1, warp & 3, lane);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buffer]);
      if (++buffer == acc.buffers) {
        buffer = 0;
        phase ^= 1;
      }
      if (seg.whole) continue;
      named_barrier(1, 128);
      if (warp == kEpilogueWarp && lane == 0) last_word = arrive_at(p, seg.block, who);
      named_barrier(1, 128);
      if (!last_word) continue;
      join_block<T>(p, seg.block, who, threadIdx.x - kEpilogueWarp * 32, 128);
    }
  } else if (warp < kLoadWarp) {
    // ---- products: the warp walks the units as one and an elected lane issues (a loop of one lane alone
    // cannot keep the descriptors in uniform registers and took twice as long a unit)
    const int me = warp - kMmaWarp;
    if (me < acc.issuers) {
      const uint32_t idesc = idesc_of<T>(p.n_pad);
      const uint64_t desc0 = smem_desc_k_sw128(smem_u32(tiles));
      const uint32_t half = stage_bytes / 2 / 16;  // descriptor addresses count 16 bytes
      int32_t left = min(q1 - q0, units - q0 % units);  // steps of the current segment
      int32_t rest = q1 - q0;
      int slot = me, buffer = 0, skip = me;  // steps until the next one of this warp
      uint32_t phase = 0, acc_phase = 1;
      bool dead = false;
      while (rest > 0 && !dead) {
        if (!mbar_wait(&acc_empty[buffer], acc_phase, abort_flag, kWaitBudgetNs, p.status)) break;
        tc_fence_after_sync();
        const uint32_t d = tmem + acc.at(me, buffer);
        uint32_t accumulate = 0;
        rest -= left;
        int32_t at = skip;
        for (; at < left; at += acc.issuers) {
          if (!mbar_wait(&full[slot], phase, abort_flag, kWaitBudgetNs, p.status)) {
            dead = true;
            break;
          }
          tc_fence_after_sync();
          const uint64_t desc = desc0 + static_cast<uint32_t>(slot) * (2 * half);
          const uint32_t a = tmem + kAccCols + slot * kUnitTmemCols;
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 8; ++s)
              umma_f16_ts(d, a + s * 8, desc + (s >> 2) * half + (s & 3) * 2, idesc, s == 0 ? accumulate : 1u);
            umma_commit(&used[slot]);
          }
          __syncwarp();
          accumulate = 1;
          slot += acc.issuers;
          if (slot >= p.slots) {
            slot -= p.slots;
            phase ^= 1;
          }
        }
        if (dead) break;
        skip = at - left;
        if (elect_one()) umma_commit(&acc_full[buffer]);
        __syncwarp();
        if (++buffer == acc.buffers) {
          buffer = 0;
          acc_phase ^= 1;
        }
        left = min(rest, units);
      }
      if (elect_one()) umma_commit(&mma_done[me]);
    }
  } else {
    // ---- bulk copies (a warp walks the units, an elected lane issues): the activations of a unit, and by
    // another warp, which nothing but the ring holds back, its codes
    const bool of_codes = warp > kLoadWarp;
    if (!of_codes) griddep_wait();
    const int slots = of_codes ? p.ring : p.slots;
    uint64_t* filled = of_codes ? codes_full : full;
    uint64_t* freed = of_codes ? codes_used : used;
    const uint32_t bytes = of_codes ? unit_bytes : stage_bytes;
    // a block's units are consecutive: step q is the matrix's q-th
    int32_t u = q0 % units;
    const uint8_t* from = of_codes ? p.A.data + static_cast<int64_t>(q0 / kSteps) * unit_bytes
                                   : p.image + static_cast<int64_t>(u) * stage_bytes;
    uint8_t* to = of_codes ? codes : tiles;
    int32_t left = q1 - q0;
    int slot = 0, issued = 0;
    uint32_t phase = 1;
    for (; left > 0; --left) {
      if (!mbar_wait(&freed[slot], phase, abort_flag, kWaitBudgetNs, p.status)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&filled[slot], bytes);
        bulk_load(to + slot * bytes, from, bytes, &filled[slot]);
      }
      __syncwarp();
      ++u;
      if (!Split || !of_codes || (u & 1) == 0) from += bytes;
      if (u == units) {
        u = 0;
        if (!of_codes) from = p.image;
      }
      if (issued < slots) ++issued;
      if (++slot == slots) {
        slot = 0;
        phase ^= 1;
      }
    }
    // Copies in flight land before the CTA leaves: a phase ends with its copy, and for the activations with
    // the unit's weights; when another role has given up only a bounded wait is left to do.
    for (; issued > 0; --issued) {
      if (--slot < 0) {
        slot = slots - 1;
        phase ^= 1;
      }
      mbar_wait_drain(&filled[slot], phase ^ 1, kWaitBudgetNs, p.status);
    }
  }

  // ---- the run's last block, by all warps.  (They wait for the end of all products: a phase of acc_full
  // could still be two ahead of a warp that comes here early, which parity does not tell from none.)
  __syncwarp();
  const int32_t last_block = (q1 - 1) / units, before = last_block - q0 / units;
  const Segment seg = segment_of(last_block, q0, q1, units);
  const Sharers who(runs, last_block, units);
  const int buffer = before % acc.buffers;
  griddep_wait();
  for (int i = 0; i < acc.issuers; ++i) mbar_wait_drain(&mma_done[i], 0, kWaitBudgetNs, p.status);
  __syncwarp();
  tc_fence_after_sync();
  if (warp < kMmaWarp) drain_segment<T>(p, seg, acc, tmem, buffer, q0, warp >> 2, kMmaWarp / 4, warp & 3, lane);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  if (seg.whole) return;
  if (threadIdx.x == 0) last_word = arrive_at(p, seg.block, who);
  __syncthreads();
  if (!last_word) return;
  join_block<T>(p, seg.block, who, threadIdx.x, kThreads);
}

int32_t pad_n(int32_t N) { return (N + 15) / 16 * 16; }

// CTAs of a product: one per SM, but no more than leave each at least four
// steps, nor more than sixteen to a block (the last of them adds all sums).
int64_t ctas_of(int64_t blocks, int32_t units) {
  const int sms = device_sm_count();
  const int64_t steps = blocks * units;
  return max64(1, min64(min64(sms > 0 ? sms : 1, steps / 4), blocks * 16));
}

struct GemmWorkspace {
  size_t image, partials, arrived, bytes;
};
GemmWorkspace layout(int32_t M, int32_t K, int32_t N) {
  const int64_t blocks = (static_cast<int64_t>(M) + kBlockRows - 1) / kBlockRows;
  const int32_t units = w4_units(K);
  GemmWorkspace w;
  w.image = 0;
  w.partials = static_cast<size_t>(units) * pad_n(N) * 256 * 2;  // fp32 output needs both tiles of a unit
  w.arrived = w.partials + static_cast<size_t>(ctas_of(blocks, units)) * 2 * pad_n(N) * kBlockRows * sizeof(float);
  w.bytes = w.arrived + (static_cast<size_t>(blocks) * sizeof(int32_t) + 15) / 16 * 16;
  return w;
}

template <typename T, int NG, int P, bool Split>
cudaError_t launch_as(GemmParams& p, int64_t ctas, cudaStream_t s) {
  // P = 1: four groups of warps have units in turn, each a slot of its own.  P = 4, for tiles of which only three
  // fit: all warps on each unit.  (Two groups of two ways with two slots each: 34 instead of 32 us for 64 tokens of
  // 12288^2, for the waits and hand-overs of twice as many warps a unit.)
  p.slots = P == 1 ? 4 : 3;
  p.ring = static_cast<int32_t>(min64(kMaxRing, (kSharedBytes - p.slots * p.n_pad * 256) / (8 * p.A.record))) / 4 *
           4 * (P == 1) + 3 * (P == 4);
  auto kernel = w4_gemm_kernel<T, NG, P, Split>;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(allowed.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes + 1024);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(uint64_t(1) << (dev & 63));
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.slots) * p.n_pad * 256 + p.ring * 8 * p.A.record + 1024;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

size_t w4_gemm_workspace(int32_t M, int32_t K, int32_t N) { return layout(M, K, N).bytes; }

cudaError_t launch_w4_gemm(const flashspmm_w4* in, const void* B, int64_t ldb, void* C, int64_t ldc, bool c_f32,
                           int32_t N, void* workspace, cudaStream_t s) {
  const GemmWorkspace w = layout(in->M, in->K, N);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  GemmParams p{};
  p.A = w4_dev(in);
  p.image = base + w.image;
  p.partials = reinterpret_cast<float*>(base + w.partials);
  p.arrived = reinterpret_cast<int32_t*>(base + w.arrived);
  p.C = C;
  p.ldc = ldc;
  p.c_f32 = c_f32;
  p.N = N;
  p.n_pad = pad_n(N);
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInitializationError;
  const int64_t blocks = (static_cast<int64_t>(p.A.M) + kBlockRows - 1) / kBlockRows;
  const int64_t steps = blocks * p.A.units * (c_f32 ? 2 : 1);
  if (steps > INT32_MAX) return cudaErrorInvalidValue;  // 8 TB of codes
  p.steps = static_cast<int32_t>(steps);

  const int64_t k_blocks = static_cast<int64_t>(p.A.units) * 4;
  const dim3 grid(static_cast<unsigned>((k_blocks * p.n_pad + 255) / 256));
  const uint16_t* b = static_cast<const uint16_t*>(B);
  const uint32_t exponent = in->dtype == FLASHSPMM_F16 ? 0x7C007C00u : 0x7F807F80u;
#define FLASHSPMM_STAGE(VEC, SPLIT) \
  w4_stage_kernel<VEC, SPLIT><<<grid, 256, 0, s>>>(b, ldb, N, p.A.K, p.n_pad, k_blocks, base + w.image, p.arrived, blocks, exponent)
  if (rows_aligned(B, ldb, p.A.K))
    c_f32 ? FLASHSPMM_STAGE(true, true) : FLASHSPMM_STAGE(true, false);
  else
    c_f32 ? FLASHSPMM_STAGE(false, true) : FLASHSPMM_STAGE(false, false);
#undef FLASHSPMM_STAGE
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  const int64_t ctas = ctas_of(blocks, p.A.units);
#define FLASHSPMM_BY_OUTPUT(T, NG, P) (c_f32 ? launch_as<T, NG, P, true>(p, ctas, s) : launch_as<T, NG, P, false>(p, ctas, s))
#define FLASHSPMM_BY_PARTS(T, NG) (p.n_pad <= 128 ? FLASHSPMM_BY_OUTPUT(T, NG, 1) : FLASHSPMM_BY_OUTPUT(T, NG, 4))
#define FLASHSPMM_BY_GROUP(T)                          \
  e = p.A.group == 128  ? FLASHSPMM_BY_PARTS(T, 1)     \
      : p.A.group == 64 ? FLASHSPMM_BY_PARTS(T, 2)     \
                        : FLASHSPMM_BY_PARTS(T, 4)
  if (in->dtype == FLASHSPMM_F16)
    FLASHSPMM_BY_GROUP(__half);
  else
    FLASHSPMM_BY_GROUP(__nv_bfloat16);
#undef FLASHSPMM_BY_GROUP
#undef FLASHSPMM_BY_PARTS
#undef FLASHSPMM_BY_OUTPUT
  note_launch();
  return e;
}

}  // namespace flashspmm
