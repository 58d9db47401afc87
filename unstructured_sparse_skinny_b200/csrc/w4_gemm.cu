// Skinny product with 4-bit weights on the fifth-generation tensor cores, for
// more tokens than a warp's own fragments serve well.
//
// A CTA owns 128 rows and a run of 128-column units of K; the CTAs of a
// cluster share the rows and split K.  Eight warps turn codes into 16-bit
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
// Split sums are joined through distributed shared memory, each CTA of the
// cluster adding its share of the columns in rank order.
#include <atomic>
#include <type_traits>

#include "sm100_primitives.cuh"
#include "w4.cuh"

namespace flashspmm {
namespace {

constexpr int kDequantWarps = 8;
constexpr int kMmaWarp = 8;                // warp 9 loads the activations
constexpr int kThreads = 320;
constexpr int kBlockRows = 128;
constexpr int kMaxStages = 6;
constexpr int kAhead = 3;                  // units of codes in flight in registers
constexpr int kSharedOfTwo = 108 * 1024, kSharedOfOne = 200 * 1024;  // a CTA's tiles with two or one on an SM
constexpr uint32_t kUnitTmemCols = 64;     // 128 values of 16 bits
constexpr uint64_t kWaitBudgetNs = 2000000000ull;

struct GemmParams {
  W4Dev A;
  const uint8_t* image;  // [units][2][n_pad][128 bytes], swizzled
  void* C;
  int64_t ldc;
  bool c_f32;
  int32_t N, n_pad;
  int32_t split;
  int32_t stages;
  uint32_t acc_cols;
  uint32_t tmem_cols;
  int* status;
};

// ---------------------------------------------------------------- activations in the product's order

// One thread per row and 32-column block: position 16 s + 8 h + 2 t + e of a
// block holds column 8 t + 4 s + 2 h + e.  A block is half a 128-byte row of
// the tile, whose 16-byte chunks are exchanged by row (128-byte swizzle).
template <bool Vec>
__global__ void __launch_bounds__(256) w4_stage_kernel(const uint16_t* __restrict__ B, int64_t ldb, int32_t N,
                                                       int32_t K, int32_t n_pad, int64_t blocks,
                                                       uint8_t* __restrict__ image) {
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float4 ld_peer(uint32_t smem_addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
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

// What a lane holds of one half (64 columns) of a unit of one strip.
template <int NG>
struct HalfUnit {
  static constexpr int kGroups = NG == 4 ? 2 : 1;  // scales that touch 64 columns
  uint4 c;
  uint32_t s[kGroups];  // {row g, row g + 8}
  uint32_t z;           // 8 bits each, kGroups pairs

  __device__ __forceinline__ void load(const W4Dev& A, int64_t unit, int half, int lane) {
    c = ld_stream(A.codes + unit * 64 + half * 32 + lane);
    const int64_t at = (unit * 8 + (lane >> 2)) * (2 * NG) + (NG == 1 ? 0 : half * NG);
    if (NG == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(A.scales + at));
      s[0] = v.x;
      s[kGroups - 1] = v.y;
      z = A.zeros ? __ldg(reinterpret_cast<const uint32_t*>(A.zeros + at)) : 0x08080808u;
    } else {
      s[0] = __ldg(reinterpret_cast<const uint32_t*>(A.scales + at));
      z = A.zeros ? __ldg(reinterpret_cast<const uint16_t*>(A.zeros + at)) : 0x0808u;
    }
  }
};

template <typename T, int NG>
__device__ __forceinline__ void to_weights(const HalfUnit<NG>& h, uint32_t (&r)[16]) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int gi = HalfUnit<NG>::kGroups == 2 ? b : 0;
    const uint32_t z = h.z >> (16 * gi);
    const W4Zero<T> zero(static_cast<int>(z & 0xFF), static_cast<int>((z >> 8) & 0xFF));
    const auto s0 = pair_of(static_cast<uint16_t>(h.s[gi] & 0xFFFF), T());
    const auto s1 = pair_of(static_cast<uint16_t>(h.s[gi] >> 16), T());
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t a[4];
      w4_fragment(b == 0 ? (s == 0 ? h.c.x : h.c.y) : (s == 0 ? h.c.z : h.c.w), zero, a);
      r[8 * b + 4 * s + 0] = mul2(a[0], s0);
      r[8 * b + 4 * s + 1] = mul2(a[1], s1);
      r[8 * b + 4 * s + 2] = mul2(a[2], s0);
      r[8 * b + 4 * s + 3] = mul2(a[3], s1);
    }
  }
}

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

template <typename T, int NG, int kMinBlocks>
__global__ void __launch_bounds__(kThreads, kMinBlocks) w4_gemm_kernel(const GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t b_full[kMaxStages], b_empty[kMaxStages], a_full[2], a_empty[2], acc_full;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t rank = static_cast<int32_t>(blockIdx.x % p.split);
  const int64_t block = blockIdx.x / p.split;
  const int32_t u0 = static_cast<int32_t>(static_cast<int64_t>(p.A.units) * rank / p.split);
  const int32_t count = static_cast<int32_t>(static_cast<int64_t>(p.A.units) * (rank + 1) / p.split) - u0;
  const uint32_t stage_bytes = static_cast<uint32_t>(p.n_pad) * 256;
  uint8_t* tiles = smem + ((1024 - (smem_u32(smem) & 1023)) & 1023);

  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], kDequantWarps);
      mbar_init(&a_empty[i], 1);
    }
    mbar_init(&acc_full, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const uint32_t tmem_a = tmem + p.acc_cols;

  if (warp < kDequantWarps) {
    // ---- codes -> tensor memory: 32 rows and half a unit per warp
    const int quad = warp & 3, half = warp >> 2;
    int64_t strip[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      strip[j] = min64(block * 8 + quad * 2 + j, p.A.strips - 1) * p.A.units + u0;
    HalfUnit<NG> ring[kAhead][2];
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
      if (d < count) {
        ring[d][0].load(p.A, strip[0] + d, half, lane);
        ring[d][1].load(p.A, strip[1] + d, half, lane);
      }
    const uint32_t dst = tmem_a + (static_cast<uint32_t>(quad * 32) << 16) + half * (kUnitTmemCols / 2);
    bool dead = false;
    for (int32_t base = 0; base < count && !dead; base += kAhead) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        const int32_t i = base + d;
        if (i < count && !dead) {
          uint32_t r0[16], r1[16];
          to_weights<T, NG>(ring[d][0], r0);
          to_weights<T, NG>(ring[d][1], r1);
          if (i + kAhead < count) {
            ring[d][0].load(p.A, strip[0] + i + kAhead, half, lane);
            ring[d][1].load(p.A, strip[1] + i + kAhead, half, lane);
          }
          const int buf = i & 1;
          if (!mbar_wait(&a_empty[buf], static_cast<uint32_t>(((i >> 1) & 1) ^ 1), abort_flag, kWaitBudgetNs,
                         p.status))
            dead = true;
          __syncwarp();
          tc_fence_after_sync();
          tmem_store_16x32(dst + buf * kUnitTmemCols, r0);
          tmem_store_16x32(dst + buf * kUnitTmemCols + (16u << 16), r1);
          tmem_store_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&a_full[buf]);
        }
      }
    }
    // ---- accumulators -> C, or this CTA's share of the sum
    mbar_wait(&acc_full, 0, abort_flag, kWaitBudgetNs, p.status);
    __syncwarp();
    tc_fence_after_sync();
    float* part = reinterpret_cast<float*>(tiles);
    const int row = quad * 32 + lane;
    const int64_t m = block * kBlockRows + row;
    for (int32_t n0 = half * 16; n0 < p.n_pad; n0 += 32) {
      uint32_t r[16];
      tmem_load_16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + n0, r);
      tmem_load_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (p.split > 1)
          part[(n0 + j) * kBlockRows + row] = __uint_as_float(r[j]);
        else if (n0 + j < p.N && m < p.A.M)
          store_out(p, n0 + j, m, __uint_as_float(r[j]), T());
      }
    }
    tc_fence_before_sync();
  } else if (warp == kMmaWarp) {
    // ---- one thread issues all products
    if (lane == 0) {
      const uint32_t idesc = idesc_of<T>(p.n_pad);
      int32_t i = 0;
      for (; i < count; ++i) {
        const int stage = i % p.stages, buf = i & 1;
        if (!mbar_wait(&b_full[stage], static_cast<uint32_t>((i / p.stages) & 1), abort_flag, kWaitBudgetNs, p.status))
          break;
        if (!mbar_wait(&a_full[buf], static_cast<uint32_t>((i >> 1) & 1), abort_flag, kWaitBudgetNs, p.status)) break;
        tc_fence_after_sync();
        const uint32_t b0 = smem_u32(tiles) + stage * stage_bytes;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const uint32_t b = b0 + (s >> 2) * (stage_bytes / 2) + (s & 3) * 32;
          umma_f16_ts(tmem, tmem_a + buf * kUnitTmemCols + s * 8, smem_desc_k_sw128(b), idesc, i > 0 || s > 0);
        }
        umma_commit(&a_empty[buf]);
        umma_commit(&b_empty[stage]);
      }
      umma_commit(&acc_full);
      mbar_wait_drain(&acc_full, 0, kWaitBudgetNs, p.status);
    }
    __syncwarp();
  } else if (lane == 0) {
    // ---- activations: one bulk copy per unit
    griddep_wait();
    int32_t i = 0;
    for (; i < count; ++i) {
      const int stage = i % p.stages;
      if (!mbar_wait(&b_empty[stage], static_cast<uint32_t>(((i / p.stages) & 1) ^ 1), abort_flag, kWaitBudgetNs,
                     p.status))
        break;
      mbar_arrive_expect_tx(&b_full[stage], stage_bytes);
      bulk_load(tiles + stage * stage_bytes, p.image + static_cast<int64_t>(u0 + i) * stage_bytes, stage_bytes,
                &b_full[stage]);
    }
    for (int32_t j = i > p.stages ? i - p.stages : 0; j < i; ++j)  // copies in flight land before the CTA leaves
      mbar_wait_drain(&b_full[j % p.stages], static_cast<uint32_t>((j / p.stages) & 1), kWaitBudgetNs, p.status);
  }
  __syncthreads();
  // Tensor memory goes back before any wait for another CTA, so CTAs of two
  // kernels that share SMs can never wait for each other's.
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, p.tmem_cols);
  }
  if (p.split == 1) return;
  cluster_arrive();
  cluster_wait();
  const int32_t n_from = p.N * rank / p.split, n_to = p.N * (rank + 1) / p.split;
  const uint32_t part = smem_u32(tiles);
  for (int32_t i = threadIdx.x; i < (n_to - n_from) * (kBlockRows / 4); i += kThreads) {
    const int32_t n = n_from + i / (kBlockRows / 4), row = (i % (kBlockRows / 4)) * 4;
    float4 sum = make_float4(0, 0, 0, 0);
    for (int32_t r = 0; r < p.split; ++r) {
      const float4 v = ld_peer(part + static_cast<uint32_t>(n * kBlockRows + row) * 4, r);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
    const int64_t m = block * kBlockRows + row;
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (m + j < p.A.M) store_out(p, n, m + j, v[j], T());
  }
  cluster_arrive();  // this CTA's sums stay until its peers have read them
  cluster_wait();
}

// CTAs that share a row block.  More of them fill the SMs when there are few
// blocks; a CTA's fixed part (start, joining) is worth a few units.
int32_t choose_split(int64_t blocks, int32_t units, int slots) {
  int32_t best = 1;
  double least = 0;
  for (int32_t s = 1; s <= 8 && s <= units; ++s) {
    const int64_t waves = (blocks * s + slots - 1) / slots;
    const double cost = static_cast<double>(waves) * ((units + s - 1) / s + 4 + (s > 1 ? 2 : 0));
    if (s == 1 || cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

int32_t pad_n(int32_t N) { return (N + 15) / 16 * 16; }

template <typename T, int NG, int kMinBlocks>
cudaError_t launch_as(const GemmParams& p, int64_t blocks, size_t smem, cudaStream_t s) {
  auto kernel = w4_gemm_kernel<T, NG, kMinBlocks>;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(allowed.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kMinBlocks == 2 ? kSharedOfTwo : kSharedOfOne) + 1024);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(uint64_t(1) << (dev & 63));
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * p.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

size_t w4_gemm_workspace(int32_t K, int32_t N) { return static_cast<size_t>(w4_units(K)) * pad_n(N) * 256; }

cudaError_t launch_w4_gemm(const flashspmm_w4* in, const void* B, int64_t ldb, void* C, int64_t ldc, bool c_f32,
                           int32_t N, void* workspace, cudaStream_t s) {
  GemmParams p{};
  p.A = w4_dev(in);
  p.image = static_cast<const uint8_t*>(workspace);
  p.C = C;
  p.ldc = ldc;
  p.c_f32 = c_f32;
  p.N = N;
  p.n_pad = pad_n(N);
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInitializationError;

  const int64_t blocks32 = static_cast<int64_t>(p.A.units) * 4;
  const int64_t threads = blocks32 * p.n_pad;
  const dim3 grid(static_cast<unsigned>((threads + 255) / 256));
  const uint16_t* b = static_cast<const uint16_t*>(B);
  uint8_t* image = static_cast<uint8_t*>(workspace);
  if (rows_aligned(B, ldb, p.A.K))
    w4_stage_kernel<true><<<grid, 256, 0, s>>>(b, ldb, N, p.A.K, p.n_pad, blocks32, image);
  else
    w4_stage_kernel<false><<<grid, 256, 0, s>>>(b, ldb, N, p.A.K, p.n_pad, blocks32, image);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  // Up to 128 columns two CTAs share an SM (256 columns of tensor memory and
  // at most 110 KB of shared memory each, but more than a third of an SM's);
  // above that one has it all.
  const bool two = p.n_pad <= 128;
  const uint32_t stage_bytes = static_cast<uint32_t>(p.n_pad) * 256;
  p.stages = static_cast<int32_t>(min64(kMaxStages, (two ? kSharedOfTwo : kSharedOfOne) / stage_bytes));
  p.acc_cols = p.n_pad <= 32 ? 32 : p.n_pad <= 64 ? 64 : p.n_pad <= 128 ? 128 : 256;
  p.tmem_cols = two ? 256 : 512;
  const size_t smem = static_cast<size_t>(max64(80 * 1024, static_cast<int64_t>(p.stages) * stage_bytes)) + 1024;
  const int sms = device_sm_count();
  const int64_t blocks = (static_cast<int64_t>(p.A.M) + kBlockRows - 1) / kBlockRows;
  p.split = choose_split(blocks, p.A.units, (sms > 0 ? sms : 1) * (two ? 2 : 1));
#define FLASHSPMM_GEMM(T, NG) \
  e = two ? launch_as<T, NG, 2>(p, blocks, smem, s) : launch_as<T, NG, 1>(p, blocks, smem, s)
#define FLASHSPMM_BY_GROUP(T)          \
  if (p.A.group == 128) {              \
    FLASHSPMM_GEMM(T, 1);              \
  } else if (p.A.group == 64) {        \
    FLASHSPMM_GEMM(T, 2);              \
  } else {                             \
    FLASHSPMM_GEMM(T, 4);              \
  }
  if (in->dtype == FLASHSPMM_F16) {
    FLASHSPMM_BY_GROUP(__half)
  } else {
    FLASHSPMM_BY_GROUP(__nv_bfloat16)
  }
#undef FLASHSPMM_BY_GROUP
#undef FLASHSPMM_GEMM
  note_launch();
  return e;
}

}  // namespace flashspmm
