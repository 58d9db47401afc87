// A mixture-of-experts layer for a few tokens with 4-bit experts.
//
//   logits = router x            (64-bit sums: their order decides which experts run)
//   ids, p = top_k(logits)       (ties to the lower index), p = softmax over the chosen or over all
//   h_e    = act(gate_e x) * (up_e x), or act(gate_e x)
//   out    = sum over the token's experts of p * (down_e h_e)
//
// Four kernels: logits; routing, which turns the choice into one list of
// tokens per running expert; gate and up with the activation; down with the
// weighted sum.  Every expert's codes are read once however many of its tokens
// there are, and every sum has a fixed order: no atomics on values.
#include "w4.cuh"

namespace flashspmm {
namespace {

constexpr int kWarps = 8;
constexpr int kRouteThreads = 512;

// An expert that runs: its tokens are pairs [first, first + count).
struct __align__(16) Slot {
  int32_t expert, first, count, pad;
};

struct Workspace {
  Slot* slots;         // [E], the first *running of them in use
  int32_t* running;
  int32_t* pair_token; // [T * top_k], by expert, tokens ascending
  float* pair_weight;
  double* logits;      // [T][E]
  uint16_t* h;         // [T * top_k][ldh]
  uint16_t* x;         // aligned copy of the activations, if one is needed
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
  w.logits = reinterpret_cast<double*>(take(sizeof(double) * T * E));
  w.h = reinterpret_cast<uint16_t*>(take(2 * pairs * w.ldh));
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

// One warp per expert and four tokens.  Equal router rows give equal logits
// bit for bit: the order of a sum depends on H alone.
template <typename T, typename RT, bool Vec>
__global__ void __launch_bounds__(kWarps * 32) moe_logits_kernel(const uint16_t* __restrict__ X, int64_t ldx,
                                                                 const void* __restrict__ router, int32_t H,
                                                                 int32_t tokens, int32_t E,
                                                                 double* __restrict__ logits) {
  const int lane = threadIdx.x & 31;
  const int32_t e = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int32_t t0 = blockIdx.y * 4;
  if (e >= E) return;
  double acc[4] = {};
  for (int32_t k = 8 * lane; k < H; k += 256) {
    float w[8];
    RouterRow<RT>::template load<Vec>(router, e, k, H, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[8];
      // rows are padded to 8 values with zeros, so this load needs no check of H
      unpack8<T>(load_act8<true>(t0 + j < tokens ? X + (t0 + j) * ldx : nullptr, k, H), x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[j] = fma(static_cast<double>(w[i]), static_cast<double>(x[i]), acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], m);
    if (lane == 0 && t0 + j < tokens) logits[static_cast<int64_t>(t0 + j) * E + e] = acc[j];
  }
}

// ---------------------------------------------------------------- routing

// The top_k of one token by one warp.  A NaN counts as the lowest value, so
// the chosen experts are always top_k different ones; its token's weights are
// NaN.
__device__ __forceinline__ void top_k_of(const double* logits, int32_t E, int32_t top_k, bool renormalize, int lane,
                                         int32_t* ids, float* weights) {
  constexpr int kPer = kMoeMaxExperts / 32;
  const double lowest = -__longlong_as_double(0x7FF0000000000000ll);
  double v[kPer];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int32_t e = lane + 32 * i;
    v[i] = e < E ? logits[e] : lowest;
    if (v[i] != v[i]) {
      nan = true;
      v[i] = lowest;
    }
  }
  nan = __any_sync(0xFFFFFFFFu, nan);
  uint32_t used = 0;
  double top = 0.0;
  int32_t my_id = 0;
  float my_e = 0.0f, sum = 0.0f;
  for (int32_t j = 0; j < top_k; ++j) {
    double best = lowest;
    int32_t at = INT32_MAX;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int32_t e = lane + 32 * i;
      if (e < E && !(used >> i & 1) && (at == INT32_MAX || v[i] > best)) {
        best = v[i];
        at = e;
      }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      const double ov = __shfl_xor_sync(0xFFFFFFFFu, best, m);
      const int32_t oe = __shfl_xor_sync(0xFFFFFFFFu, at, m);
      if (ov > best || (ov == best && oe < at)) {
        best = ov;
        at = oe;
      }
    }
    if (j == 0) top = best;
    if ((at & 31) == lane) used |= 1u << (at >> 5);
    const float e = expf(static_cast<float>(best - top));
    sum += e;
    if (lane == j) {
      my_id = at;
      my_e = e;
    }
  }
  if (!renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < E) sum += expf(static_cast<float>(v[i] - top));
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
  }
  if (lane < top_k) {
    ids[lane] = my_id;
    weights[lane] = nan ? __int_as_float(0x7FC00000) : my_e / sum;
  }
}

// One CTA: the choice (or the caller's), then for every expert the set of its
// tokens as 64 bits, their counts' running sum, and the lists.  An id outside
// 0 .. E - 1 contributes nothing; one that a token names twice runs once with
// the sum of its weights.
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(bool given, int32_t tokens, int32_t E, int32_t top_k,
                                                                  bool renormalize, int32_t* ids, float* weights,
                                                                  Workspace ws) {
  __shared__ int32_t s_ids[kMoeMaxTokens * kMoeMaxTopK];
  __shared__ float s_weights[kMoeMaxTokens * kMoeMaxTopK];
  __shared__ unsigned long long mask[kMoeMaxExperts];
  __shared__ int32_t part[kRouteThreads / 32][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  mask[tid] = 0;
  const int32_t pairs = tokens * top_k;
  if (given) {
    for (int i = tid; i < pairs; i += kRouteThreads) {
      s_ids[i] = ids[i];
      s_weights[i] = weights[i];
    }
  } else {
    for (int32_t t = warp; t < tokens; t += kRouteThreads / 32)
      top_k_of(ws.logits + static_cast<int64_t>(t) * E, E, top_k, renormalize, lane, s_ids + t * top_k,
               s_weights + t * top_k);
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += kRouteThreads) {
    const int32_t e = s_ids[i];
    if (e >= 0 && e < E) atomicOr(&mask[e], 1ull << (i / top_k));
    if (!given) {
      ids[i] = e;
      weights[i] = s_weights[i];
    }
  }
  __syncthreads();
  unsigned long long mine = tid < E ? mask[tid] : 0;
  const int32_t count = __popcll(mine), runs = count > 0;
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
  int32_t before0 = 0, before1 = 0;
  for (int w = 0; w < warp; ++w) {
    before0 += part[w][0];
    before1 += part[w][1];
  }
  first += before0 - count;
  slot += before1 - runs;
  if (tid == kRouteThreads - 1) *ws.running = slot + runs;
  if (!runs) return;
  ws.slots[slot] = Slot{tid, first, count, 0};
  for (int32_t i = 0; i < count; ++i) {
    const int32_t t = __ffsll(static_cast<long long>(mine)) - 1;
    mine &= mine - 1;
    float w = 0.0f;
    for (int32_t j = 0; j < top_k; ++j)
      if (s_ids[t * top_k + j] == tid) w += s_weights[t * top_k + j];
    ws.pair_token[first + i] = t;
    ws.pair_weight[first + i] = w;
  }
}

// ---------------------------------------------------------------- gate and up

__device__ __forceinline__ float activate(int kind, float v) {
  if (kind == FLASHSPMM_ACT_SILU) return v / (1.0f + expf(-v));
  if (kind == FLASHSPMM_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678f));
  return fmaxf(v, 0.0f) + (v != v ? v : 0.0f);  // relu, NaN kept
}

// h[pair][f] for one strip of 16 rows f of one running expert.  h is rounded
// to the activations' type: it is the next product's tensor-core operand.
template <typename T, int NG, int R, int NT>
__global__ void __launch_bounds__(kWarps * 32) moe_gate_up_kernel(W4Dev gate, W4Dev up, const uint16_t* __restrict__ X,
                                                                  int64_t ldx, int32_t H, int activation,
                                                                  Workspace ws) {
  constexpr int kPass = NT < 2 ? NT : 2;  // tiles added up at a time, for the size of `red`
  constexpr int kRows = 16 * R, kPitch = kRows + 4;
  __shared__ float red[kWarps][kPass * 8][kPitch];
  __shared__ int32_t tok[kMoeMaxTokens];
  if (static_cast<int32_t>(blockIdx.y) >= *ws.running) return;
  const Slot slot = ws.slots[blockIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x < slot.count) tok[threadIdx.x] = ws.pair_token[slot.first + threadIdx.x];
  __syncthreads();
  const int tiles = (slot.count + 7) / 8;
  float acc[R][NT][4] = {};
  const auto act = [&](int nt, int32_t k) {
    const int n = 8 * nt + g;
    return load_act8<true>(n < slot.count ? X + tok[n] * ldx : nullptr, k + 8 * t, H);
  };
  for (int32_t u = warp; u < gate.units; u += kWarps) {
    uint4 c[R][2];
    W4Groups<T, NG> grp[R];
    const int64_t unit = gate.unit(slot.expert, blockIdx.x, u);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const W4Dev& A = r ? up : gate;
      c[r][0] = ld_stream(A.codes + unit * 64 + lane);
      c[r][1] = ld_stream(A.codes + unit * 64 + 32 + lane);
      grp[r].load(A, unit, g);
    }
    w4_unit<T, NG, R, NT>(c, grp, u * kW4UnitCols, tiles, act, acc);
  }
#pragma unroll
  for (int p = 0; p < NT / kPass; ++p) {
    if (p * kPass >= tiles) break;
    if (p > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int nt = 0; nt < kPass; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[warp][nt * 8 + 2 * t + (i & 1)][r * 16 + g + 8 * (i >> 1)] = acc[r][p * kPass + nt][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kPass * 8 * 16; i += kWarps * 32) {
      const int n = i >> 4, row = i & 15;
      const int32_t pair = p * kPass * 8 + n, f = blockIdx.x * 16 + row;
      if (pair >= slot.count || f >= ws.ldh) continue;
      float v = 0.0f, u = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        v += red[w][n][row];
        if (R == 2) u += red[w][n][16 * (R - 1) + row];
      }
      v = activate(activation, v);
      if (R == 2) v *= u;
      // columns behind F pad h to 16 bytes: finite whatever x holds
      reinterpret_cast<T*>(ws.h)[(slot.first + pair) * ws.ldh + f] = from_float<T>(f < gate.M ? v : 0.0f);
    }
  }
}

// ---------------------------------------------------------------- down

// out[.][strip of 16 rows]: the warps share all units of all running experts
// in runs; at an expert's end a warp adds its weighted sums to its own table
// of tokens, and the tables are added in a fixed order.
template <typename T, int NG, int NT>
__global__ void __launch_bounds__(kWarps * 32) moe_down_kernel(W4Dev A, int32_t tokens, T* __restrict__ out,
                                                               int64_t ldo, Workspace ws) {
  constexpr int kPitch = 16 + 4;
  __shared__ float sum[kWarps][NT * 8][kPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  for (int i = threadIdx.x; i < kWarps * NT * 8 * kPitch; i += kWarps * 32) (&sum[0][0][0])[i] = 0.0f;
  __syncthreads();
  const int32_t ldh = static_cast<int32_t>(ws.ldh);
  const int64_t items = static_cast<int64_t>(*ws.running) * A.units;
  int64_t i = items * warp / kWarps;
  const int64_t end = items * (warp + 1) / kWarps;
  while (i < end) {
    const int32_t s = static_cast<int32_t>(i / A.units);
    const Slot slot = ws.slots[s];
    const int64_t stop = min64(end, static_cast<int64_t>(s + 1) * A.units);
    const int tiles = (slot.count + 7) / 8;
    const int64_t unit0 = A.unit(slot.expert, blockIdx.x, 0);
    float acc[1][NT][4] = {};
    const auto act = [&](int nt, int32_t k) {
      const int n = 8 * nt + g;
      return load_act8<true>(n < slot.count ? ws.h + (slot.first + n) * ws.ldh : nullptr, k + 8 * t, ldh);
    };
    for (; i < stop; ++i) {
      const int32_t u = static_cast<int32_t>(i - static_cast<int64_t>(s) * A.units);
      uint4 c[1][2];
      W4Groups<T, NG> grp[1];
      const int64_t unit = unit0 + 8 * static_cast<int64_t>(u);
      c[0][0] = ld_stream(A.codes + unit * 64 + lane);
      c[0][1] = ld_stream(A.codes + unit * 64 + 32 + lane);
      grp[0].load(A, unit, g);
      w4_unit<T, NG, 1, NT>(c, grp, u * kW4UnitCols, tiles, act, acc);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = nt * 8 + 2 * t + j;
        if (n < slot.count) {
          const int32_t token = ws.pair_token[slot.first + n];
          const float w = ws.pair_weight[slot.first + n];
          sum[warp][token][g] = fmaf(w, acc[0][nt][j], sum[warp][token][g]);
          sum[warp][token][g + 8] = fmaf(w, acc[0][nt][2 + j], sum[warp][token][g + 8]);
        }
      }
    __syncwarp();  // the next expert's lanes hold other tokens
  }
  __syncthreads();
  for (int o = threadIdx.x; o < tokens * 16; o += kWarps * 32) {
    const int token = o >> 4, row = o & 15;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * 16 + row;
    if (m >= A.M) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sum[w][token][row];
    out[token * ldo + m] = from_float<T>(v);
  }
}

template <typename T, int NG, int NT>
void experts_as(const MoeCall& p, const uint16_t* X, int64_t ldx, int32_t H, const Workspace& ws,
                cudaStream_t s) {
  const W4Dev gate = w4_dev(&p.gate), down = w4_dev(&p.down);
  const int64_t most = min64(p.gate.count, static_cast<int64_t>(p.tokens) * p.top_k);
  const dim3 grid(gate.strips, static_cast<unsigned>(most));
  if (p.up.codes)
    moe_gate_up_kernel<T, NG, 2, NT>
        <<<grid, kWarps * 32, 0, s>>>(gate, w4_dev(&p.up), X, ldx, H, p.activation, ws);
  else
    moe_gate_up_kernel<T, NG, 1, NT><<<grid, kWarps * 32, 0, s>>>(gate, gate, X, ldx, H, p.activation, ws);
  note_launch();
  moe_down_kernel<T, NG, NT>
      <<<down.strips, kWarps * 32, 0, s>>>(down, p.tokens, static_cast<T*>(p.out), p.ldo, ws);
  note_launch();
}

template <typename T>
void layer_as(const MoeCall& p, const Workspace& ws, const uint16_t* X, int64_t ldx, cudaStream_t s) {
  const int32_t H = p.gate.K, E = p.gate.count;
  // X is aligned and padded here, so its rows can be read to a multiple of 8
  const int32_t Hp = static_cast<int32_t>(aligned_k(H));
  if (p.router) {
    const dim3 grid((E + kWarps - 1) / kWarps, (p.tokens + 3) / 4);
    const bool vec = (reinterpret_cast<uintptr_t>(p.router) & 15u) == 0 && H % 8 == 0;
#define FLASHSPMM_LOGITS(RT, VEC) \
  moe_logits_kernel<T, RT, VEC><<<grid, kWarps * 32, 0, s>>>(X, ldx, p.router, H, p.tokens, E, ws.logits)
    if (p.router_dtype == FLASHSPMM_F32)
      vec ? FLASHSPMM_LOGITS(float, true) : FLASHSPMM_LOGITS(float, false);
    else
      vec ? FLASHSPMM_LOGITS(T, true) : FLASHSPMM_LOGITS(T, false);
#undef FLASHSPMM_LOGITS
    note_launch();
  }
  moe_route_kernel<<<1, kRouteThreads, 0, s>>>(p.router == nullptr, p.tokens, E, p.top_k, p.renormalize,
                                               p.ids, p.weights, ws);
  note_launch();
#define FLASHSPMM_EXPERTS(NG)                       \
  if (p.tokens <= 8)                               \
    experts_as<T, NG, 1>(p, X, ldx, Hp, ws, s);     \
  else if (p.tokens <= 16)                         \
    experts_as<T, NG, 2>(p, X, ldx, Hp, ws, s);     \
  else if (p.tokens <= 32)                         \
    experts_as<T, NG, 4>(p, X, ldx, Hp, ws, s);     \
  else                                              \
    experts_as<T, NG, 8>(p, X, ldx, Hp, ws, s)
  if (p.gate.group == 128) {
    FLASHSPMM_EXPERTS(1);
  } else if (p.gate.group == 64) {
    FLASHSPMM_EXPERTS(2);
  } else {
    FLASHSPMM_EXPERTS(4);
  }
#undef FLASHSPMM_EXPERTS
}

}  // namespace

size_t moe_workspace(int32_t T, int32_t E, int32_t top_k, int32_t H, int32_t F, bool aligned) {
  return carve(nullptr, T, E, top_k, H, F, aligned).bytes;
}

cudaError_t launch_moe_w4(const MoeCall& p, void* workspace, cudaStream_t s) {
  const int32_t H = p.gate.K;
  const bool aligned = rows_aligned(p.X, p.ldx, H);
  const Workspace ws = carve(workspace, p.tokens, p.gate.count, p.top_k, H, p.gate.M, aligned);
  const uint16_t* X = static_cast<const uint16_t*>(p.X);
  int64_t ldx = p.ldx;
  if (!aligned) {
    const cudaError_t e = launch_align_rows(p.X, p.ldx, p.tokens, H, ws.x, s);
    if (e != cudaSuccess) return e;
    X = ws.x;
    ldx = aligned_k(H);
  }
  if (p.gate.dtype == FLASHSPMM_F16)
    layer_as<__half>(p, ws, X, ldx, s);
  else
    layer_as<__nv_bfloat16>(p, ws, X, ldx, s);
  return cudaGetLastError();
}

}  // namespace flashspmm
