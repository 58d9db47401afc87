// A mixture-of-experts layer for a few tokens with 4-bit experts.
//
//   logits = router x            (sums of 46 bits: their order decides which experts run)
//   ids, p = top_k(logits)       (ties to the lower index), p = softmax over the chosen or over all
//   h_e    = act(gate_e x) * (up_e x), or act(gate_e x)
//   out    = sum over the token's experts of p * (down_e h_e)
//
// Three to five kernels, each started while the one before it ends: logits;
// routing, which turns the choice into one list of tokens per running expert
// (and makes a small layer's logits too); gate and up with the activation; down,
// weighted; and the sum over a token's experts, which up to eight tokens is part
// of down.  An expert's codes are read once for every 8, 16 or 32 of its tokens,
// and every sum has a fixed order: no atomics on values.
#include <atomic>
#include <type_traits>

#include "w4_strips.cuh"

namespace flashspmm {
namespace {

constexpr int kRouteWarps = 16;
constexpr int kRouteThreads = kRouteWarps * 32;
constexpr int kRouteCtas = 8;  // one cluster
constexpr int kDirectTokens = 8;  // see moe_down_direct_kernel

// An expert that runs: its tokens are pairs [first, first + count), and their
// bits among the first 32 tokens.
struct __align__(16) Slot {
  int32_t expert, first, count;
  uint32_t tokens;
};

struct Workspace {
  Slot* slots;           // [E], the first *running of them in use
  int32_t* running;
  int32_t* pair_token;   // [T * top_k], by expert, tokens ascending
  float* pair_weight;
  int32_t* place;        // [T][top_k]: the pair of a token's j-th expert, -1 where there is none
  double* logits;        // [T][E]
  uint16_t* h;           // [2][T * top_k][ldh]: rounded, and what the rounding left
  float* y;              // [T * top_k][H], weighted
  uint16_t* x;           // aligned copy of the activations, if one is needed
  int64_t ldh;
  size_t bytes;
};

size_t up16(size_t v) { return (v + 15) / 16 * 16; }

Workspace carve(void* base, int32_t T, int32_t E, int32_t top_k, int32_t H, int32_t F, bool aligned) {
  Workspace w;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(base) + o;
    o += up16(bytes);
    return at;
  };
  const size_t pairs = static_cast<size_t>(T) * top_k;
  w.ldh = aligned_k(F);
  w.slots = reinterpret_cast<Slot*>(take(sizeof(Slot) * E));
  w.running = reinterpret_cast<int32_t*>(take(4));
  w.pair_token = reinterpret_cast<int32_t*>(take(4 * pairs));
  w.pair_weight = reinterpret_cast<float*>(take(4 * pairs));
  w.place = reinterpret_cast<int32_t*>(take(4 * pairs));
  w.logits = reinterpret_cast<double*>(take(sizeof(double) * T * E));
  w.h = reinterpret_cast<uint16_t*>(take(2 * 2 * pairs * w.ldh));
  w.y = reinterpret_cast<float*>(take(sizeof(float) * pairs * H));
  w.x = reinterpret_cast<uint16_t*>(take(aligned ? 0 : static_cast<size_t>(T) * aligned_k(H) * 2));
  w.bytes = o;
  return w;
}

// ---------------------------------------------------------------- router

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = bits_to_float<T>(static_cast<uint16_t>(i & 1 ? x[i >> 1] >> 16 : x[i >> 1] & 0xFFFF));
}

// Eight router values k .. k + 7 of a row of H.
template <typename T>
struct RouterRow {
  template <bool Vec>
  static __device__ __forceinline__ void load(const void* base, int64_t row, int32_t k, int32_t H, float (&f)[8]) {
    unpack8<T>(load_act8<Vec>(static_cast<const uint16_t*>(base) + row * H, k, H), f);
  }
};
template <>
struct RouterRow<float> {
  template <bool Vec>
  static __device__ __forceinline__ void load(const void* base, int64_t row, int32_t k, int32_t H, float (&f)[8]) {
    const float* p = static_cast<const float*>(base) + row * H;
    if (Vec) {  // H is a multiple of 8 here
      float4 a = make_float4(0, 0, 0, 0), b = a;
      if (k < H) {
        a = *reinterpret_cast<const float4*>(p + k);
        b = *reinterpret_cast<const float4*>(p + k + 4);
      }
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = k + i < H ? p[k + i] : 0.0f;
    }
  }
};

// A sum of some 46 bits in two fp32 words: the rounding of every addition is
// computed (Knuth's two-sum) and added up beside.  64-bit arithmetic would do,
// but the conversions to it run at some 5 a cycle and SM: 17 us for one token
// and 128 experts of 2048 columns on a cluster, where this takes 3.
// (Every step is an intrinsic: an expression the compiler could turn into a fused
// multiply-add, which leaves no rounding to compute.)
struct Sum2 {
  float s = 0.0f, c = 0.0f;
  __device__ __forceinline__ void add(float p, float below) {
    const float t = __fadd_rn(s, p), z = __fsub_rn(t, s);
    const float left = __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(p, z));
    c = __fadd_rn(c, __fadd_rn(left, below));
    s = t;
  }
  // of an infinite sum the rounding is not a number, and not wanted
  __device__ __forceinline__ double value() const {
    return static_cast<double>(s) + static_cast<double>(c == c ? c : 0.0f);
  }
};
// w * x: a product of two 16-bit values is exact in fp32, of an fp32 router's its rounding is kept.
template <typename RT>
__device__ __forceinline__ void add_product(Sum2& sum, float w, float x) {
  const float p = __fmul_rn(w, x);
  sum.add(p, std::is_same<RT, float>::value ? __fmaf_rn(w, x, -p) : 0.0f);
}

// A CTA has EB experts and TB tokens; its threads share the columns, eight
// neighbours each.  Equal router rows give equal logits bit for bit: the order
// of a sum depends on H and the tile's shape alone.
template <typename T, typename RT, bool Vec, int EB, int TB>
__global__ void __launch_bounds__(256) moe_logits_kernel(const uint16_t* __restrict__ X, int64_t ldx,
                                                         const void* __restrict__ router, int32_t H, int32_t tokens,
                                                         int32_t E, double* __restrict__ logits) {
  __shared__ double part[8][EB * TB];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t e0 = blockIdx.x * EB, t0 = blockIdx.y * TB;
  Sum2 acc[EB][TB];
  for (int32_t k = 8 * threadIdx.x; k < H; k += 2048) {
    float w[EB][8];
    uint4 raw[TB];
#pragma unroll
    for (int i = 0; i < EB; ++i) RouterRow<RT>::template load<Vec>(router, min(e0 + i, E - 1), k, H, w[i]);
    // rows are padded to 8 values, and the router's values behind H are zeros
#pragma unroll
    for (int j = 0; j < TB; ++j) raw[j] = load_act8<true>(X + min(t0 + j, tokens - 1) * ldx, k, H);
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      float x[8];
      unpack8<T>(raw[j], x);
#pragma unroll
      for (int i = 0; i < EB; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) add_product<RT>(acc[i][j], w[i][c], x[c]);
    }
  }
#pragma unroll
  for (int i = 0; i < EB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      double v = acc[i][j].value();
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
      if (lane == 0) part[warp][i * TB + j] = v;
    }
  __syncthreads();
  if (threadIdx.x < EB * TB) {
    const int32_t e = e0 + threadIdx.x / TB, t = t0 + threadIdx.x % TB;
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += part[w][threadIdx.x];
    if (e < E && t < tokens) logits[static_cast<int64_t>(t) * E + e] = sum;
  }
}

// ---------------------------------------------------------------- routing

// Whole numbers in the order of the values.  A NaN counts as the lowest.
__device__ __forceinline__ unsigned long long sort_key(double v) {
  v += 0.0;  // -0 is 0
  const unsigned long long b = __double_as_longlong(v);
  return v != v ? 0ull : b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_value(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>(k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}

// The top_k of one token by one warp, 32 * Per experts at most.  The chosen
// experts are always top_k different ones; the weights of a token with a NaN
// among its logits are NaN.
template <int Per>
__device__ __forceinline__ void top_k_of(const double* logits, int32_t E, int32_t top_k, bool renormalize, int lane,
                                         int32_t* ids, float* weights) {
  // 0 marks what is behind E or taken; the lowest value (and NaN) counts as 1
  unsigned long long key[Per];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < Per; ++i) {
    const int32_t e = lane + 32 * i;
    const double v = e < E ? __ldcg(logits + e) : 0.0;
    nan |= v != v;
    key[i] = e < E ? max(sort_key(v), 1ull) : 0ull;
  }
  nan = __any_sync(0xFFFFFFFFu, nan);
  unsigned long long rest[Per];
#pragma unroll
  for (int i = 0; i < Per; ++i) rest[i] = key[i];
  double top = 0.0;
  int32_t my_id = 0;
  float my_e = 0.0f, sum = 0.0f;
  for (int32_t j = 0; j < top_k; ++j) {
    unsigned long long best = rest[0];
#pragma unroll
    for (int i = 1; i < Per; ++i) best = max(best, rest[i]);
    const uint32_t high = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(best >> 32));
    const uint32_t low = __reduce_max_sync(
        0xFFFFFFFFu, static_cast<uint32_t>(best >> 32) == high ? static_cast<uint32_t>(best) : 0u);
    const unsigned long long taken = (static_cast<unsigned long long>(high) << 32) | low;
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int i = Per - 1; i >= 0; --i)
      if (rest[i] == taken) at = lane + 32 * i;
    at = __reduce_min_sync(0xFFFFFFFFu, at);
#pragma unroll
    for (int i = 0; i < Per; ++i)
      if (lane + 32 * i == static_cast<int32_t>(at)) rest[i] = 0;
    const double value = key_value(taken);
    if (j == 0) top = value;
    const float e = expf(static_cast<float>(value - top));
    sum += e;
    if (lane == j) {
      my_id = static_cast<int32_t>(at);
      my_e = e;
    }
  }
  if (!renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < Per; ++i)
      if (lane + 32 * i < E) sum += expf(static_cast<float>(key_value(key[i]) - top));
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
  }
  if (lane < top_k) {
    ids[lane] = my_id;
    weights[lane] = nan ? __int_as_float(0x7FC00000) : my_e / sum;
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (The barrier before it brings a warp's lanes together: an .aligned arrival counts for the whole warp, also
// while one of its lanes is still in a branch.)
__device__ __forceinline__ void cluster_sync() {
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same shared-memory address in the cluster's first CTA.
__device__ __forceinline__ uint32_t in_first_cta(const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}

// The logits of a small layer by a cluster: CTA `rank` has every eighth expert,
// and `ways` of its warps share an expert's columns.
template <typename T, typename RT, bool Vec, int TB>
__device__ __forceinline__ void small_logits(const uint16_t* X, int64_t ldx, const void* router, int32_t H,
                                             int32_t tokens, int32_t E, int rank,
                                             double (&part)[kRouteWarps][kMoeMaxTokens], double* logits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t mine = (E - rank + kRouteCtas - 1) / kRouteCtas;
  int ways = kRouteWarps;
  while (ways > 1 && kRouteWarps / ways < mine) ways /= 2;
  const int at_once = kRouteWarps / ways;
  for (int32_t base = 0; base < mine; base += at_once) {
    const int32_t i = base + warp / ways, e = rank + kRouteCtas * i;
    for (int32_t t0 = 0; t0 < tokens && i < mine; t0 += TB) {
      Sum2 acc[TB];
#pragma unroll(TB == 1 ? 4 : 2)
      for (int32_t k = 8 * (lane + 32 * (warp % ways)); k < H; k += 256 * ways) {
        float w[8];
        uint4 raw[TB];
        RouterRow<RT>::template load<Vec>(router, e, k, H, w);
#pragma unroll
        for (int j = 0; j < TB; ++j) raw[j] = load_act8<true>(X + min(t0 + j, tokens - 1) * ldx, k, H);
#pragma unroll
        for (int j = 0; j < TB; ++j) {
          float x[8];
          unpack8<T>(raw[j], x);
#pragma unroll
          for (int c = 0; c < 8; ++c) add_product<RT>(acc[j], w[c], x[c]);
        }
      }
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        double v = acc[j].value();
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
        if (lane == 0) part[warp][min(t0 + j, tokens - 1)] = v;
      }
    }
    __syncthreads();
    for (int32_t o = threadIdx.x; o < at_once * tokens; o += kRouteThreads) {
      const int32_t j = o / tokens, t = o - j * tokens;
      if (base + j >= mine) continue;
      double sum = 0.0;
      for (int w = 0; w < ways; ++w) sum += part[j * ways + w][t];
      logits[static_cast<int64_t>(t) * E + rank + kRouteCtas * (base + j)] = sum;
    }
    __syncthreads();
  }
}

struct RouteParams {
  bool given;          // ids and weights are inputs
  const uint16_t* X;   // a small layer's activations, whose logits are made here; else nullptr
  int64_t ldx;
  const void* router;
  int32_t H, tokens, E, top_k;
  bool renormalize, router_f32, router_vec;
  int32_t* ids;
  float* weights;
};

// A cluster: a warp per token chooses (or takes the caller's choice) and sets
// the token's bit in its experts' sets, which the first CTA holds; then that
// CTA makes the running experts' lists: their sizes' running sum, and a pair's
// place in its list from the bits below its own.  An id outside 0 .. E - 1
// contributes nothing; one that a token names twice runs once with the sum of
// its weights.
template <typename T, int Per>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteParams p, Workspace ws) {
  __shared__ unsigned long long mask[kMoeMaxExperts];
  __shared__ int32_t start[kMoeMaxExperts];
  __shared__ int32_t part[kRouteWarps][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t tokens = p.tokens, E = p.E, top_k = p.top_k;
  int32_t* ids = p.ids;
  float* weights = p.weights;
  const uint32_t rank = cluster_rank();
  mask[tid] = 0;
  griddep_wait();
  griddep_launch_dependents();
  if (p.X) {
    __shared__ double sums[kRouteWarps][kMoeMaxTokens];
#define FLASHSPMM_SMALL(RT, VEC)                                                                                   \
  tokens == 1 ? small_logits<T, RT, VEC, 1>(p.X, p.ldx, p.router, p.H, tokens, E, rank, sums, ws.logits) \
              : small_logits<T, RT, VEC, 2>(p.X, p.ldx, p.router, p.H, tokens, E, rank, sums, ws.logits)
    if (p.router_f32)
      p.router_vec ? (FLASHSPMM_SMALL(float, true)) : (FLASHSPMM_SMALL(float, false));
    else
      p.router_vec ? (FLASHSPMM_SMALL(T, true)) : (FLASHSPMM_SMALL(T, false));
#undef FLASHSPMM_SMALL
    __threadfence();
  }
  cluster_sync();
  for (int32_t t = rank + kRouteCtas * warp; t < tokens; t += kRouteCtas * kRouteWarps) {
    if (!p.given)
      top_k_of<Per>(ws.logits + static_cast<int64_t>(t) * E, E, top_k, p.renormalize, lane, ids + t * top_k,
                    weights + t * top_k);
    __syncwarp();
    if (lane < top_k) {
      const int32_t e = ids[t * top_k + lane];
      if (e >= 0 && e < E)
        // in halves of 32 bits: the 64-bit form lost bits that two CTAs set at the same time
        asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(in_first_cta(&mask[e]) + (t >> 5) * 4),
                     "r"(1u << (t & 31))
                     : "memory");
    }
  }
  __threadfence();
  cluster_sync();
  if (rank != 0) return;
  const int32_t count = tid < E ? __popcll(mask[tid]) : 0, runs = count > 0;
  int32_t first = count, slot = runs;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int32_t a = __shfl_up_sync(0xFFFFFFFFu, first, m), b = __shfl_up_sync(0xFFFFFFFFu, slot, m);
    if (lane >= m) {
      first += a;
      slot += b;
    }
  }
  if (lane == 31) {
    part[warp][0] = first;
    part[warp][1] = slot;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    first += part[w][0];
    slot += part[w][1];
  }
  start[tid] = first - count;
  if (tid == kRouteThreads - 1) *ws.running = slot;
  if (runs) ws.slots[slot - 1] = Slot{tid, first - count, count, static_cast<uint32_t>(mask[tid])};
  __syncthreads();
  for (int32_t i = tid; i < tokens * top_k; i += kRouteThreads) {
    const int32_t t = i / top_k, e = __ldcg(ids + i);
    int32_t place = -1;
    if (e >= 0 && e < E) {
      const int32_t at = start[e] + __popcll(mask[e] & ((1ull << t) - 1));
      float w = 0.0f;
      bool again = false;  // a token's sum counts an expert's pair once
      for (int32_t j = 0; j < top_k; ++j)
        if (__ldcg(ids + t * top_k + j) == e) {
          w += __ldcg(weights + t * top_k + j);
          again |= t * top_k + j < i;
        }
      ws.pair_token[at] = t;
      ws.pair_weight[at] = w;
      if (!again) place = at;
    }
    ws.place[i] = place;
  }
}

// ---------------------------------------------------------------- experts

__device__ __forceinline__ float activate(int kind, float v) {
  if (kind == FLASHSPMM_ACT_SILU) return v / (1.0f + expf(-v));
  if (kind == FLASHSPMM_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678f));
  return v < 0.0f ? 0.0f : v;  // relu, NaN kept
}

struct ExpertParams {
  W4Dev gate, up;        // up.data null: no gate product
  W4Dev down;
  const uint16_t* X;
  int64_t ldx;
  int32_t H;             // columns of X that may be read
  int32_t tokens;
  int32_t activation;
  int64_t rest;          // from an h to what its rounding left, in values
  int32_t pairs;         // of strips a CTA takes
  uint32_t shared;
  Workspace ws;
};

// h[pair][f] for some strips of 16 rows f of a running expert.  As the next
// product's tensor-core operand h is rounded to the activations' type; what the
// rounding leaves is kept too, rounded likewise, and multiplied beside it.
// (Without that an output has 1.5 times the error that its own rounding makes: a
// few large h carry it.  The second products cost a tenth of the layer.)
template <typename T, int NG, int NT, bool Gated>
__global__ void __launch_bounds__(kStripThreads, strip_ctas(NT)) moe_gate_up_kernel(const ExpertParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr uint32_t rings = kStripWarps * StripRing<NG>::kBytes;
  uint8_t* staged = smem + rings;
  __shared__ int32_t token[kMoeMaxTokens];
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int32_t>(blockIdx.y) >= *p.ws.running) return;
  const Slot slot = p.ws.slots[blockIdx.y];
  const W4Dev& A = p.gate;
  const int32_t pair0 = blockIdx.x * p.pairs, pair = pair0 + (threadIdx.x >> 5) % p.pairs, last = A.strips - 1;
  // a warp's strips: the same of gate and up, or without a gate product neighbours
  const int64_t unit0 = A.unit(slot.expert, min(Gated ? pair : 2 * pair, last), 0);
  const int64_t unit1 = Gated ? unit0 : A.unit(slot.expert, min(2 * pair + 1, last), 0);
  const StripAt at[2] = {StripAt(A, unit0), StripAt(Gated ? p.up : A, unit1)};
  if (threadIdx.x < slot.count) token[threadIdx.x] = p.ws.pair_token[slot.first + threadIdx.x];
  for (int32_t n0 = 0; n0 < slot.count; n0 += NT * 8) {
    const int32_t rows = min(slot.count - n0, NT * 8);
    float acc[2][NT][4] = {};
    strip_product<T, NG, NT, 1>(
        at, A.units, p.H, rows, p.pairs, smem, staged, p.shared - rings, [&](int32_t n) { return p.X + token[n0 + n] * p.ldx; }, acc);
    const auto store = [&](int32_t n, int32_t f, float v) {
      // columns behind F pad h to 16 bytes: finite whatever x holds
      if (f >= p.ws.ldh) return;
      T* h = reinterpret_cast<T*>(p.ws.h) + (slot.first + n0 + n) * p.ws.ldh + f;
      const T rounded = from_float<T>(f < A.M ? v : 0.0f);
      const float left = f < A.M ? v - to_float(rounded) : 0.0f;
      *h = rounded;
      h[p.rest] = from_float<T>(isfinite(left) ? left : 0.0f);  // of an h that rounds to infinity: nothing
    };
    strip_reduce<T, NT>(acc, p.pairs, rows, staged, [&](int i, int32_t n, int32_t row, float a, float b) {
      const int32_t f = (pair0 + i) * (Gated ? 16 : 32) + row;
      a = activate(p.activation, a);
      store(n, f, Gated ? a * b : a);
      if (!Gated) store(n, f + 16, activate(p.activation, b));
    });
  }
}

// y[pair] = weight * down h for some pairs of strips of a running expert.
template <typename T, int NG, int NT>
__global__ void __launch_bounds__(kStripThreads, strip_ctas(NT)) moe_down_kernel(const ExpertParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr uint32_t rings = kStripWarps * StripRing<NG>::kBytes;
  uint8_t* staged = smem + rings;
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int32_t>(blockIdx.y) >= *p.ws.running) return;
  const Slot slot = p.ws.slots[blockIdx.y];
  const W4Dev& A = p.down;
  const int32_t pair0 = blockIdx.x * p.pairs, pair = pair0 + (threadIdx.x >> 5) % p.pairs, last = A.strips - 1;
  const StripAt at[2] = {StripAt(A, A.unit(slot.expert, min(2 * pair, last), 0)),
                         StripAt(A, A.unit(slot.expert, min(2 * pair + 1, last), 0))};
  for (int32_t n0 = 0; n0 < slot.count; n0 += NT * 8) {
    const int32_t rows = min(slot.count - n0, NT * 8), first = slot.first + n0;
    float acc[2][NT][4] = {};
    strip_product<T, NG, NT, 2>(
        at, A.units, static_cast<int32_t>(p.ws.ldh), rows, p.pairs, smem, staged, p.shared - rings,
        [&](int32_t n) { return p.ws.h + (n < rows ? first + n : first + n - rows) * p.ws.ldh + (n < rows ? 0 : p.rest); },
        acc);
    strip_reduce<T, NT>(acc, p.pairs, rows, staged, [&](int i, int32_t n, int32_t row, float a, float b) {
      const int32_t m = (pair0 + i) * 32 + row;
      const float w = p.ws.pair_weight[first + n];
      float* y = p.ws.y + static_cast<int64_t>(first + n) * A.M;
      if (m < A.M) y[m] = w * a;
      if (m + 16 < A.M) y[m + 16] = w * b;
    });
  }
}

// Up to eight tokens: a CTA has a pair of strips of the output and all running
// experts, whose units its warps share in runs.  A token is a column of the
// product, so a warp adds an expert's weighted sums in registers and the CTA its
// warps', and no partial result leaves the SM.  Where the expert is not a
// token's choice the column's activations are zeros and its sum is not added: a
// scale that is not finite makes it NaN.
constexpr int kDirectWarps = 16, kDirectSlots = kDirectTokens * kMoeMaxTopK;
constexpr uint32_t kNotChosen = 0x80000000u;  // -0 for a weight: a choice's own is made +0

template <typename T, int NG>
__global__ void __launch_bounds__(kDirectWarps * 32, 1) moe_down_direct_kernel(const ExpertParams p,
                                                                               T* __restrict__ out, int64_t ldo) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Slot slots[kDirectSlots];
  __shared__ float weight[kDirectSlots][kDirectTokens];
  __shared__ float red[kDirectWarps][kDirectTokens][36];  // 32 rows, and the fragments' stores meet all banks
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  const int32_t running = *p.ws.running, units = p.down.units;
  const int32_t strip[2] = {static_cast<int32_t>(2 * blockIdx.x),
                            min(static_cast<int32_t>(2 * blockIdx.x + 1), p.down.strips - 1)};
  for (int i = threadIdx.x; i < running * kDirectTokens; i += kDirectWarps * 32) {
    const Slot s = p.ws.slots[i >> 3];
    const int n = i & 7;
    if (n == 0) slots[i >> 3] = s;
    weight[i >> 3][n] = s.tokens >> n & 1 ? p.ws.pair_weight[s.first + __popc(s.tokens & ((1u << n) - 1))] + 0.0f
                                          : __uint_as_float(kNotChosen);
  }
  __syncthreads();
  const int64_t items = static_cast<int64_t>(running) * units;
  const int32_t from = static_cast<int32_t>(items * warp / kDirectWarps);
  const int32_t to = static_cast<int32_t>(items * (warp + 1) / kDirectWarps);
  const W4Dev& A = p.down;
  const StripRing<NG> ring{smem + warp * StripRing<NG>::kBytes};
  const int32_t s0 = from / units, u0 = from - s0 * units;
  // the next records to be asked for
  int32_t asked = from, s_ask = s0, u_ask = u0;
  const bool zeros[2] = {A.zeros, A.zeros};
  const uint8_t* record[2];
  const auto seek = [&](int32_t unit) {
#pragma unroll
    for (int r = 0; r < 2; ++r) record[r] = A.at(A.unit(slots[s_ask].expert, strip[r], unit));
  };
  const auto ask = [&](int place) {
    if (asked < to) {
      ring.ask(place, record, zeros, lane);
      ++asked;
#pragma unroll
      for (int r = 0; r < 2; ++r) record[r] += 8 * A.record;
      if (++u_ask == units) {
        u_ask = 0;
        ++s_ask;
        if (asked < to) seek(0);
      }
    }
    cp_async_commit();
  };
  if (from < to) seek(u0);
#pragma unroll
  for (int d = 0; d < kStripRing; ++d) ask(d);
  // the next activations: a lane's registers of a block are filled for the next unit as soon as they are free
  int32_t s_x = s0, u_x = u0;
  const uint16_t* row = nullptr;
  const auto seek_row = [&] {
    const uint32_t tokens = slots[s_x].tokens;
    row = tokens >> g & 1 ? p.ws.h + (slots[s_x].first + __popc(tokens & ((1u << g) - 1))) * p.ws.ldh + 8 * t : nullptr;
  };
  uint4 x[4][2];
  const auto load_x = [&](int b, int part) {
    x[b][part] = make_uint4(0, 0, 0, 0);
    if (row && u_x * kW4UnitCols + 32 * b + 8 * t < p.ws.ldh)
      x[b][part] = *reinterpret_cast<const uint4*>(row + (part ? p.rest : 0) + u_x * kW4UnitCols + 32 * b);
  };
  if (from < to) {
    seek_row();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      load_x(b, 0);
      load_x(b, 1);
    }
  }
  int32_t s = s0, u = u0;
  float total[2][4] = {}, acc[2][1][4] = {};
  int place = 0;
  for (int32_t i = from; i < to; ++i) {
    if (++u_x == units) {
      u_x = 0;
      ++s_x;
      if (i + 1 < to) seek_row();
    }
    if (i + 1 == to) row = nullptr;
    ring.wait();
    StripUnit<T, NG> unit[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) unit[r].load(ring.base + place * ring.kPlace + r * ring.kRecord, lane, A.zeros);
    strip_unit<T, NG, 2, 1, 1, 2>(unit, 1,
                                  [&](int, int b, int part) {
                                    const uint4 v = x[b][part];
                                    load_x(b, part);
                                    return v;
                                  },
                                  acc);
    __syncwarp();
    ask(place);
    place = place + 1 == kStripRing ? 0 : place + 1;
    if (++u == units || i + 1 == to) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float w = weight[s][2 * t + (k & 1)];
          if (__float_as_uint(w) != kNotChosen) total[r][k] = fmaf(w, acc[r][0][k], total[r][k]);
          acc[r][0][k] = 0.0f;
        }
      u = 0;
      ++s;
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int k = 0; k < 4; ++k) red[warp][2 * t + (k & 1)][16 * r + g + 8 * (k >> 1)] = total[r][k];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int n = threadIdx.x >> 5, r = threadIdx.x & 31;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kDirectWarps; ++w) sum += red[w][n][r];
    const int32_t m = blockIdx.x * 32 + r;
    if (n < p.tokens && m < A.M) out[n * ldo + m] = from_float<T>(w4_raise<T>(sum));
  }
}

// out[token] = the sum of its pairs' y, in the order of its choice.
template <typename T>
__global__ void __launch_bounds__(256) moe_join_kernel(const float* __restrict__ y, const int32_t* __restrict__ place,
                                                       int32_t top_k, int32_t H, T* __restrict__ out, int64_t ldo) {
  __shared__ int32_t at[kMoeMaxTopK];
  griddep_wait();
  if (threadIdx.x < top_k) at[threadIdx.x] = place[blockIdx.y * top_k + threadIdx.x];
  __syncthreads();
  const int32_t m = blockIdx.x * 256 + threadIdx.x;
  if (m >= H) return;
  float sum = 0.0f;
#pragma unroll 4
  for (int32_t j = 0; j < top_k; ++j)
    if (at[j] >= 0) sum += y[static_cast<int64_t>(at[j]) * H + m];
  out[blockIdx.y * ldo + m] = from_float<T>(sum);
}

// ---------------------------------------------------------------- host

// A kernel that may start while the one before it in the stream ends.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t shared, int cluster, cudaStream_t s,
                         Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Once per device: the kernel may use this much shared memory.
template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, std::atomic<uint64_t>& allowed, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (allowed.load() >> (dev & 63) & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) allowed.fetch_or(uint64_t(1) << (dev & 63));
  return e;
}

template <typename T, int NG, int NT, bool Gated>
cudaError_t experts_as(const MoeCall& c, ExpertParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> allowed[2];
  const int64_t most = min64(c.gate.count, static_cast<int64_t>(c.tokens) * c.top_k);
  const int32_t rows = c.tokens < NT * 8 ? c.tokens : NT * 8;
  // experts that run and their tokens, as even routing has them
  const double E = c.gate.count, pairs = static_cast<double>(c.tokens) * c.top_k;
  const double share = c.top_k < E ? c.top_k / E : 1.0, running = E * (1.0 - std::pow(1.0 - share, c.tokens));
  auto gate_up = moe_gate_up_kernel<T, NG, NT, Gated>;
  cudaError_t e = allow_shared(gate_up, allowed[0], strip_limit(NT));
  if (e != cudaSuccess) return e;
  int32_t all = Gated ? p.gate.strips : (p.gate.strips + 1) / 2;
  p.pairs = pairs_per_cta(running, all, p.gate.units, pairs / running, strip_ctas(NT));
  p.shared = strip_shared<NG>(rows, p.gate.units, NT);
  e = launch_after(gate_up, dim3((all + p.pairs - 1) / p.pairs, static_cast<unsigned>(most)), kStripThreads, p.shared,
                   1, s, p);
  if (e != cudaSuccess) return e;
  all = (p.down.strips + 1) / 2;
  if constexpr (NT == 1) {  // up to kDirectTokens tokens
    constexpr uint32_t rings = kDirectWarps * StripRing<NG>::kBytes;
    auto down = moe_down_direct_kernel<T, NG>;
    e = allow_shared(down, allowed[1], rings);
    if (e != cudaSuccess) return e;
    return launch_after(down, dim3(all), kDirectWarps * 32, rings, 1, s, p, static_cast<T*>(c.out), c.ldo);
  } else {
    auto down = moe_down_kernel<T, NG, NT>;
    e = allow_shared(down, allowed[1], strip_limit(NT));
    if (e != cudaSuccess) return e;
    p.pairs = pairs_per_cta(running, all, p.down.units, 2 * pairs / running, strip_ctas(NT));
    p.shared = strip_shared<NG>(2 * rows, p.down.units, NT);
    e = launch_after(down, dim3((all + p.pairs - 1) / p.pairs, static_cast<unsigned>(most)), kStripThreads, p.shared,
                     1, s, p);
    if (e != cudaSuccess) return e;
    return launch_after(moe_join_kernel<T>, dim3((p.down.M + 255) / 256, c.tokens), 256, 0, 1, s,
                        static_cast<const float*>(p.ws.y), static_cast<const int32_t*>(p.ws.place), c.top_k, p.down.M,
                        static_cast<T*>(c.out), c.ldo);
  }
}

template <typename T, typename RT>
cudaError_t logits_as(const MoeCall& c, const ExpertParams& p, cudaStream_t s) {
  const int32_t H = c.gate.K, E = c.gate.count;
  const bool vec = (reinterpret_cast<uintptr_t>(c.router) & 15u) == 0 && H % 8 == 0;
#define FLASHSPMM_LOGITS(VEC, EB, TB)                                                                       \
  moe_logits_kernel<T, RT, VEC, EB, TB><<<dim3((E + EB - 1) / EB, (c.tokens + TB - 1) / TB), 256, 0, s>>>( \
      p.X, p.ldx, c.router, H, c.tokens, E, p.ws.logits)
  if (c.tokens == 1)
    vec ? FLASHSPMM_LOGITS(true, 1, 1) : FLASHSPMM_LOGITS(false, 1, 1);
  else
    vec ? FLASHSPMM_LOGITS(true, 2, 4) : FLASHSPMM_LOGITS(false, 2, 4);
#undef FLASHSPMM_LOGITS
  note_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t layer_as(const MoeCall& c, ExpertParams& p, cudaStream_t s) {
  const int32_t E = c.gate.count, H = c.gate.K;
  // One cluster makes the logits of a small layer itself; a larger one has a kernel for them.  A layer of narrow
  // experts of 128 x 2048 logits takes, by cluster and with the kernel, 24 and 24 us for one token, 30 and 22 for two,
  // 34 and 22 for four, 46 and 26 for eight: above some 2^18 products the limit is too high.
  const bool small = static_cast<int64_t>(c.tokens) * E * H <= (2 << 20);
  RouteParams r{};
  r.given = c.router == nullptr;
  r.X = c.router && small ? p.X : nullptr;
  r.ldx = p.ldx;
  r.router = c.router;
  r.H = H;
  r.tokens = c.tokens;
  r.E = E;
  r.top_k = c.top_k;
  r.renormalize = c.renormalize;
  r.router_f32 = c.router_dtype == FLASHSPMM_F32;
  r.router_vec = (reinterpret_cast<uintptr_t>(c.router) & 15u) == 0 && H % 8 == 0;
  r.ids = c.ids;
  r.weights = c.weights;
  cudaError_t e = cudaSuccess;
  if (c.router && !small) e = r.router_f32 ? logits_as<T, float>(c, p, s) : logits_as<T, T>(c, p, s);
  if (e != cudaSuccess) return e;
  auto route = E <= 64 ? moe_route_kernel<T, 2> : E <= 128 ? moe_route_kernel<T, 4> : moe_route_kernel<T, 16>;
  e = launch_after(route, dim3(kRouteCtas), kRouteThreads, 0, kRouteCtas, s, r, p.ws);
  if (e != cudaSuccess) return e;
  // Tokens that an expert's codes serve at a time: 8, 16 or 32.  An expert with more reads its codes again; 32
  // leave an SM half as many warps, and are for experts that get more than 12 on average (8 experts of 4096 x
  // 2048, us with 16 and with 32: 8 tokens an expert 83 and 93, 12 98 and 105, 16 138 and 131, 32 186 and 180).
  const bool many = static_cast<int64_t>(c.tokens) * c.top_k > 12 * static_cast<int64_t>(E);
  const bool gated = c.up.data != nullptr;
#define FLASHSPMM_EXPERTS_OF(NG, NT) (gated ? experts_as<T, NG, NT, true>(c, p, s) : experts_as<T, NG, NT, false>(c, p, s))
#define FLASHSPMM_EXPERTS(NG)                                        \
  c.tokens <= kDirectTokens ? FLASHSPMM_EXPERTS_OF(NG, 1)            \
  : c.tokens <= 16 || !many ? FLASHSPMM_EXPERTS_OF(NG, 2)            \
                            : FLASHSPMM_EXPERTS_OF(NG, 4)
  return c.gate.group == 128  ? FLASHSPMM_EXPERTS(1)
         : c.gate.group == 64 ? FLASHSPMM_EXPERTS(2)
                              : FLASHSPMM_EXPERTS(4);
#undef FLASHSPMM_EXPERTS
#undef FLASHSPMM_EXPERTS_OF
}

}  // namespace

size_t moe_workspace(int32_t T, int32_t E, int32_t top_k, int32_t H, int32_t F, bool aligned) {
  return carve(nullptr, T, E, top_k, H, F, aligned).bytes;
}

cudaError_t launch_moe_w4(const MoeCall& c, void* workspace, cudaStream_t s) {
  const int32_t H = c.gate.K;
  const bool aligned = rows_aligned(c.X, c.ldx, H);
  ExpertParams p{};
  p.ws = carve(workspace, c.tokens, c.gate.count, c.top_k, H, c.gate.M, aligned);
  p.gate = w4_dev(&c.gate);
  if (c.up.data) p.up = w4_dev(&c.up);
  p.down = w4_dev(&c.down);
  p.X = static_cast<const uint16_t*>(c.X);
  p.ldx = c.ldx;
  p.H = static_cast<int32_t>(aligned_k(H));  // the aligned copy is padded with zeros
  p.tokens = c.tokens;
  p.rest = static_cast<int64_t>(c.tokens) * c.top_k * p.ws.ldh;
  p.activation = c.activation;
  if (!aligned) {
    const cudaError_t e = launch_align_rows(c.X, c.ldx, c.tokens, H, p.ws.x, s);
    if (e != cudaSuccess) return e;
    p.X = p.ws.x;
    p.ldx = aligned_k(H);
  }
  return c.gate.dtype == FLASHSPMM_F16 ? layer_as<__half>(c, p, s) : layer_as<__nv_bfloat16>(c, p, s);
}

}  // namespace flashspmm
