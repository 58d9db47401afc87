// Skinny product with 4-bit weights on the fifth-generation tensor cores, for
// more tokens than a warp's own fragments serve well.
//
// The work is blocks of 128 rows times units of 128 columns; every SM runs one
// CTA over an equal run of these steps.  Sixteen warps turn codes into 16-bit
// weights in registers (s * (q - z), rounded once) and store them straight to
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
// them in their order.
#include <atomic>
#include <type_traits>

#include "sm100_primitives.cuh"
#include "w4.cuh"

namespace flashspmm {
namespace {

constexpr int kDequantWarps = 16;          // four groups of four
constexpr int kEpilogueWarp = 16;          // 16 .. 19
constexpr int kMmaWarp = 20;               // 21 loads the activations
constexpr int kThreads = 22 * 32;
constexpr int kBlockRows = 128;
constexpr int kMaxSlots = 4;               // units between codes and product; slot j is filled by group j alone
constexpr int kTileBytes = 200 * 1024;     // shared memory for the activations
constexpr uint32_t kUnitTmemCols = 64;     // 128 values of 16 bits
constexpr uint32_t kAccCols = 256;         // one accumulator, or two of up to 128 columns
constexpr uint64_t kWaitBudgetNs = 1000000000ull;

struct GemmParams {
  W4Dev A;
  const uint8_t* image;  // [units][2][n_pad][128 bytes], swizzled
  float* partials;       // [CTA][first, last block of its run][n_pad][128]
  int32_t* arrived;      // [blocks]
  void* C;
  int64_t ldc;
  bool c_f32;
  int32_t N, n_pad;
  int32_t slots;
  int64_t steps;         // blocks * units
  int* status;
};

// ---------------------------------------------------------------- activations in the product's order

// One thread per row and 32-column block: position 16 s + 8 h + 2 t + e of a
// block holds column 8 t + 4 s + 2 h + e.  A block is half a 128-byte row of
// the tile, whose 16-byte chunks are exchanged by row (128-byte swizzle).
template <bool Vec>
__global__ void __launch_bounds__(256) w4_stage_kernel(const uint16_t* __restrict__ B, int64_t ldb, int32_t N,
                                                       int32_t K, int32_t n_pad, int64_t blocks,
                                                       uint8_t* __restrict__ image, int32_t* __restrict__ arrived,
                                                       int64_t row_blocks) {
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
  uint8_t* tile = image + (blk >> 1) * (static_cast<int64_t>(n_pad) * 128) + n * 128;
#pragma unroll
  for (int c = 0; c < 4; ++c) {  // c = 2 s + h
    const int chunk = ((blk & 1) * 4 + c) ^ (n & 7);
    *reinterpret_cast<uint4*>(tile + chunk * 16) = make_uint4(w[c], w[4 + c], w[8 + c], w[12 + c]);
  }
}

// ---------------------------------------------------------------- primitives

__device__ __forceinline__ void bulk_load(void* smem, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(smem)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// 16 TMEM lanes x 32 columns: register 2 i is row g, 2 i + 1 row g + 8 of column 4 i + t.
__device__ __forceinline__ void tmem_store_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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

__device__ __forceinline__ uint32_t mul2(uint32_t a, __half2 s) {
  union {
    uint32_t u;
    __half2 h;
  } x;
  x.u = a;
  x.h = __hmul2(x.h, s);
  return x.u;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, __nv_bfloat162 s) {
  union {
    uint32_t u;
    __nv_bfloat162 h;
  } x;
  x.u = a;
  x.h = __hmul2(x.h, s);
  return x.u;
}
__device__ __forceinline__ __half2 pair_of(uint16_t b, __half) { return __half2half2(__ushort_as_half(b)); }
__device__ __forceinline__ __nv_bfloat162 pair_of(uint16_t b, __nv_bfloat16) {
  return __bfloat162bfloat162(__ushort_as_bfloat16(b));
}

// Codes, scales and zero points of one unit of one strip as a lane holds them.
template <typename T, int NG>
struct Unit {
  uint4 c[2];
  W4Groups<T, NG> g;

  __device__ __forceinline__ void load(const W4Dev& A, int64_t unit, int lane) {
    const uint4* p = A.codes + unit * 64 + lane;
    c[0] = ld_stream(p);
    c[1] = ld_stream(p + 32);
    g.load(A, unit, lane >> 2);
  }

  // Half a unit (64 columns) as 16 registers of 16-bit weights.
  __device__ __forceinline__ void weights(int half, uint32_t (&r)[16]) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int gi = (2 * half + b) * NG / 4;
      const W4Zero<T> zero = g.zero(gi);
      const auto s0 = pair_of(static_cast<uint16_t>(g.s[gi] & 0xFFFF), T());
      const auto s1 = pair_of(static_cast<uint16_t>(g.s[gi] >> 16), T());
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t a[4];
        w4_fragment(b == 0 ? (s == 0 ? c[half].x : c[half].y) : (s == 0 ? c[half].z : c[half].w), zero, a);
        r[8 * b + 4 * s + 0] = mul2(a[0], s0);
        r[8 * b + 4 * s + 1] = mul2(a[1], s1);
        r[8 * b + 4 * s + 2] = mul2(a[2], s0);
        r[8 * b + 4 * s + 3] = mul2(a[3], s1);
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ uint32_t idesc_of(int n) {
  const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;  // of A and B
  return umma_idesc_f16_f32(kBlockRows, n) | (type << 7) | (type << 10);
}

__device__ __forceinline__ void store_out(const GemmParams& p, int64_t n, int64_t m, float v, __half) {
  if (p.c_f32)
    static_cast<float*>(p.C)[n * p.ldc + m] = v;
  else
    static_cast<__half*>(p.C)[n * p.ldc + m] = __float2half_rn(v);
}
__device__ __forceinline__ void store_out(const GemmParams& p, int64_t n, int64_t m, float v, __nv_bfloat16) {
  if (p.c_f32)
    static_cast<float*>(p.C)[n * p.ldc + m] = v;
  else
    static_cast<__nv_bfloat16*>(p.C)[n * p.ldc + m] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------- kernel

// A run of steps cut into segments of one block each.
struct Segment {
  int64_t block;
  int64_t from, to;  // steps
  bool whole;
};
__device__ __forceinline__ Segment segment_at(int64_t q, int64_t end, int32_t units) {
  Segment s;
  s.block = q / units;
  s.from = q;
  s.to = min64(end, (s.block + 1) * units);
  s.whole = s.to - s.from == units;
  return s;
}
__host__ __device__ __forceinline__ int64_t run_begin(int64_t steps, int64_t cta, int64_t ctas) {
  return steps * cta / ctas;
}
// The CTA whose run holds step q.
__device__ __forceinline__ int64_t run_owner(int64_t steps, int64_t q, int64_t ctas) {
  int64_t c = q * ctas / steps;
  while (run_begin(steps, c + 1, ctas) <= q) ++c;
  while (run_begin(steps, c, ctas) > q) --c;
  return c;
}

template <typename T, int NG>
__global__ void __launch_bounds__(kThreads, 1) w4_gemm_kernel(const GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t full[kMaxSlots], used[kMaxSlots], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word, last_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t units = p.A.units;
  const int64_t q0 = run_begin(p.steps, blockIdx.x, gridDim.x), q1 = run_begin(p.steps, blockIdx.x + 1, gridDim.x);
  const uint32_t stage_bytes = static_cast<uint32_t>(p.n_pad) * 256;
  const int accs = p.n_pad <= 128 ? 2 : 1;
  uint8_t* tiles = smem + ((1024 - (smem_u32(smem) & 1023)) & 1023);

  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&full[i], 5);  // four warps' weights and the copy of the activations
      mbar_init(&used[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
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
    // ---- codes -> tensor memory: 32 rows of the units of one slot.  (A slot that groups took in turns could
    // be two phases ahead of a group's wait, which parity does not tell from none.)
    const int quad = warp & 3, group = warp >> 2;
    const uint32_t dst = tmem + kAccCols + group * kUnitTmemCols + (static_cast<uint32_t>(quad * 32) << 16);
    const int64_t end = group < p.slots ? q1 : q0;  // no work for a group without a slot
    int64_t block = (q0 + group) / units;
    int32_t u = static_cast<int32_t>(q0 + group - block * units);
    const auto load = [&](Unit<T, NG> (&x)[2]) {
      const int64_t strip = block * 8 + quad * 2;
      x[0].load(p.A, min64(strip, p.A.strips - 1) * units + u, lane);
      x[1].load(p.A, min64(strip + 1, p.A.strips - 1) * units + u, lane);
      u += p.slots;
      while (u >= units) {
        u -= units;
        ++block;
      }
    };
    Unit<T, NG> now[2];
    if (q0 + group < end) load(now);
    uint32_t phase = 1;
    for (int64_t q = q0 + group; q < end; q += p.slots, phase ^= 1) {
      Unit<T, NG> next[2];
      if (q + p.slots < end) load(next);
      if (!mbar_wait(&used[group], phase, abort_flag, kWaitBudgetNs, p.status)) break;
      __syncwarp();
      tc_fence_after_sync();
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t r[16];
          now[j].weights(half, r);
          tmem_store_16x32(dst + half * (kUnitTmemCols / 2) + (static_cast<uint32_t>(16 * j) << 16), r);
        }
      tmem_store_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[group]);
      now[0] = next[0];
      now[1] = next[1];
    }
  } else if (warp < kMmaWarp) {
    // ---- accumulators -> C or the workspace
    griddep_wait();
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    int count = 0;
    for (int64_t q = q0; q < q1; ++count) {
      const Segment seg = segment_at(q, q1, units);
      q = seg.to;
      const int ab = count % accs;
      // a wait that runs out leaves wrong values and an error, not a warp missing at the barriers below
      mbar_wait(&acc_full[ab], static_cast<uint32_t>((count / accs) & 1), abort_flag, kWaitBudgetNs, p.status);
      __syncwarp();
      tc_fence_after_sync();
      const int64_t m = seg.block * kBlockRows + row;
      const int64_t slot_size = static_cast<int64_t>(p.n_pad) * kBlockRows;
      float* part = p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (seg.from > q0)) * slot_size;
      for (int32_t n0 = 0; n0 < p.n_pad; n0 += 16) {
        uint32_t r[16];
        tmem_load_16(tmem + ab * 128 + (static_cast<uint32_t>(quad * 32) << 16) + n0, r);
        tmem_load_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (!seg.whole)
            part[(n0 + j) * kBlockRows + row] = __uint_as_float(r[j]);
          else if (n0 + j < p.N && m < p.A.M)
            store_out(p, n0 + j, m, __uint_as_float(r[j]), T());
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
      if (seg.whole) continue;
      // the last of the block's CTAs adds all their sums, in order
      const int64_t first = run_owner(p.steps, seg.block * units, gridDim.x);
      const int64_t last = run_owner(p.steps, (seg.block + 1) * units - 1, gridDim.x);
      __threadfence();
      named_barrier(1, 128);
      if (threadIdx.x == kEpilogueWarp * 32)
        last_word = atomicAdd(&p.arrived[seg.block], 1) == static_cast<int32_t>(last - first);
      named_barrier(1, 128);
      if (!last_word) continue;
      __threadfence();
      const int tid = threadIdx.x - kEpilogueWarp * 32;
      // the block is the last of its first contributor's run, unless that run begins with it, and the first
      // of the others' runs
      const int64_t first_slot = first * 2 + (run_begin(p.steps, first, gridDim.x) < seg.block * units);
      const float4* base = reinterpret_cast<const float4*>(p.partials);
      const int64_t step = slot_size / 4;
      constexpr int kBatch = 8;  // loads in flight a thread
      for (int32_t i0 = tid; i0 < p.N * (kBlockRows / 4); i0 += 128 * kBatch) {
        float4 sum[kBatch] = {};
        for (int64_t c = first; c <= last; ++c) {
          const float4* src = base + (c == first ? first_slot : c * 2) * step;
          float4 v[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            v[j] = i0 + 128 * j < p.N * (kBlockRows / 4) ? __ldcg(src + i0 + 128 * j) : make_float4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            sum[j].x += v[j].x;
            sum[j].y += v[j].y;
            sum[j].z += v[j].z;
            sum[j].w += v[j].w;
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int32_t i = i0 + 128 * j;
          if (i >= p.N * (kBlockRows / 4)) break;
          const int32_t n = i / (kBlockRows / 4);
          const int64_t r = seg.block * kBlockRows + (i % (kBlockRows / 4)) * 4;
          const float v[4] = {sum[j].x, sum[j].y, sum[j].z, sum[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (r + k < p.A.M) store_out(p, n, r + k, v[k], T());
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ---- all products: the warp walks the units as one, an elected lane issues.  (With only that lane in
    // the loop the descriptors cannot stay in uniform registers: 1275 instead of %s cycles a unit of 64 tokens.)
    const uint32_t idesc = idesc_of<T>(p.n_pad);
    const uint64_t desc0 = smem_desc_k_sw128(smem_u32(tiles));
    const uint32_t half = stage_bytes / 2 / 16;  // descriptor addresses count 16 bytes
    int32_t left = static_cast<int32_t>(min64(q1 - q0, units - q0 % units));  // steps of the current segment
    int64_t rest = q1 - q0;
    int slot = 0, ab = 0, done_ab = 0;
    uint32_t phase = 0, acc_phase = 1, done_phase = 0;
    bool dead = false, any = false;
    while (rest > 0 && !dead) {
      if (!mbar_wait(&acc_empty[ab], acc_phase, abort_flag, kWaitBudgetNs, p.status)) break;
      tc_fence_after_sync();
      const uint32_t acc = tmem + ab * 128;
      uint32_t accumulate = 0;
      rest -= left;
      for (; left > 0; --left) {
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
            umma_f16_ts(acc, a + s * 8, desc + (s >> 2) * half + (s & 3) * 2, idesc, s == 0 ? accumulate : 1u);
          umma_commit(&used[slot]);
          if (left == 1) umma_commit(&acc_full[ab]);
        }
        __syncwarp();
        accumulate = 1;
        if (++slot == p.slots) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (dead) break;
      any = true;
      done_ab = ab;
      done_phase = acc_phase ^ 1;
      if (++ab == accs) {
        ab = 0;
        acc_phase ^= 1;
      }
      left = static_cast<int32_t>(min64(rest, units));
    }
    // everything issued has completed before tensor memory is given back
    if (dead) {
      if (elect_one()) umma_commit(&acc_full[ab]);
      __syncwarp();
      mbar_wait_drain(&acc_full[ab], acc_phase ^ 1, kWaitBudgetNs, p.status);
    } else if (any) {
      mbar_wait_drain(&acc_full[done_ab], done_phase, kWaitBudgetNs, p.status);
    }
    __syncwarp();
  } else if (lane == 0) {
    // ---- activations: one bulk copy per unit
    griddep_wait();
    int32_t u = static_cast<int32_t>(q0 % units);
    int slot = 0, issued = 0;
    uint32_t phase = 1;
    for (int64_t q = q0; q < q1; ++q) {
      if (!mbar_wait(&used[slot], phase, abort_flag, kWaitBudgetNs, p.status)) break;
      mbar_arrive_expect_tx(&full[slot], stage_bytes);
      bulk_load(tiles + slot * stage_bytes, p.image + static_cast<int64_t>(u) * stage_bytes, stage_bytes, &full[slot]);
      if (++u == units) u = 0;
      if (issued < p.slots) ++issued;
      if (++slot == p.slots) {
        slot = 0;
        phase ^= 1;
      }
    }
    // Copies in flight land before the CTA leaves: a unit's phase ends with its copy and its weights, and
    // when another role has given up only a bounded wait is left to do.
    for (; issued > 0; --issued) {
      if (--slot < 0) {
        slot = p.slots - 1;
        phase ^= 1;
      }
      mbar_wait_drain(&full[slot], phase ^ 1, kWaitBudgetNs, p.status);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
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
  w.partials = static_cast<size_t>(units) * pad_n(N) * 256;
  w.arrived = w.partials + static_cast<size_t>(ctas_of(blocks, units)) * 2 * pad_n(N) * kBlockRows * sizeof(float);
  w.bytes = w.arrived + (static_cast<size_t>(blocks) * sizeof(int32_t) + 15) / 16 * 16;
  return w;
}

template <typename T, int NG>
cudaError_t launch_as(const GemmParams& p, int64_t ctas, cudaStream_t s) {
  auto kernel = w4_gemm_kernel<T, NG>;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(allowed.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileBytes + 1024);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(uint64_t(1) << (dev & 63));
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.slots) * p.n_pad * 256 + 1024;
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
  p.slots = static_cast<int32_t>(min64(kMaxSlots, kTileBytes / (p.n_pad * 256)));
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInitializationError;
  const int64_t blocks = (static_cast<int64_t>(p.A.M) + kBlockRows - 1) / kBlockRows;
  p.steps = blocks * p.A.units;

  const int64_t k_blocks = static_cast<int64_t>(p.A.units) * 4;
  const dim3 grid(static_cast<unsigned>((k_blocks * p.n_pad + 255) / 256));
  const uint16_t* b = static_cast<const uint16_t*>(B);
  if (rows_aligned(B, ldb, p.A.K))
    w4_stage_kernel<true><<<grid, 256, 0, s>>>(b, ldb, N, p.A.K, p.n_pad, k_blocks, base + w.image, p.arrived, blocks);
  else
    w4_stage_kernel<false><<<grid, 256, 0, s>>>(b, ldb, N, p.A.K, p.n_pad, k_blocks, base + w.image, p.arrived, blocks);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  const int64_t ctas = ctas_of(blocks, p.A.units);
#define FLASHSPMM_BY_GROUP(T)                                  \
  e = p.A.group == 128  ? launch_as<T, 1>(p, ctas, s)          \
      : p.A.group == 64 ? launch_as<T, 2>(p, ctas, s)          \
                        : launch_as<T, 4>(p, ctas, s)
  if (in->dtype == FLASHSPMM_F16)
    FLASHSPMM_BY_GROUP(__half);
  else
    FLASHSPMM_BY_GROUP(__nv_bfloat16);
#undef FLASHSPMM_BY_GROUP
  note_launch();
  return e;
}

}  // namespace flashspmm
