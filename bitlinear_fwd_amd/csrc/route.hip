// The router of a layer with experts: each token's k largest logits, their weights, and the slots (a
// token at one of its experts) ordered by expert, then token.
//
// A counting sort whose order does not depend on timing.  Tokens are cut into chunks, one workgroup
// each.  k_route_top chooses and counts per chunk; k_route_place adds up the counts of the chunks before
// its own and of the experts before, and deals out the places in order: a wave takes 64 choices at a time
// and finds by ballots over the bits of the expert's number which lanes share one, so that a choice's
// place is its expert's next place plus the number of such lanes before it.  One chunk does both in one
// launch.
//
// Bound by latency where tokens are few (16 x 64, 4 choices: 4.6 us in one launch), else by operations: 65536 x 128
// bf16, 8 choices: 19 us for the choices, of which the logits' bytes are 3, and 10 us for the places.  A wave to a token,
// its lanes' largest searched for anew after each choice, took 46 us for the choices.
#include "experts.h"

#include <algorithm>

namespace bl {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;

// A logit as an integer of the same order; 0: never chosen (-inf, NaN).  +inf counts as the largest finite number, -0 as
// 0, so that numbers that are equal have equal keys.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > -__builtin_inff())) return 0;
  const uint32_t b = __float_as_uint(fminf(x, 3.402823466e38f) + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// A logit's key and, below it, its index turned round, so that of equal logits the one with the lowest index is the
// largest.  A bf16 logit's key has 16 bits: both fit 32.
template <typename T>
struct Entry {
  using Type = uint64_t;
  static __device__ __forceinline__ Type make(T x, bool there, int e) {
    return (uint64_t)(there ? key_of(x) : 0u) << 32 | (uint32_t)~e;
  }
  static __device__ __forceinline__ bool any(Type x) { return x >> 32; }
  static __device__ __forceinline__ float value(Type x) { return value_of((uint32_t)(x >> 32)); }
  static __device__ __forceinline__ int index(Type x) { return (int)~(uint32_t)x; }
};
template <>
struct Entry<uint16_t> {
  using Type = uint32_t;
  static __device__ __forceinline__ Type make(uint16_t x, bool there, int e) {
    return (there ? key_of(bf16_float(x)) & 0xffff0000u : 0u) | (0xffffu - (uint32_t)e);
  }
  static __device__ __forceinline__ bool any(Type x) { return x >> 16; }
  static __device__ __forceinline__ float value(Type x) {  // the key of a negative number ends in ones
    return value_of(x & 0x80000000u ? x & 0xffff0000u : x | 0xffffu);
  }
  static __device__ __forceinline__ int index(Type x) { return (int)(0xffffu - (x & 0xffffu)); }
};

// Over each row of 16 lanes, in every lane of it.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = quad_max(v);
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));         // row_half_mirror
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));      // row_mirror
}
__device__ __forceinline__ float row_sum(float v) {
  auto step = [&](auto c) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(c)::value, 0xf, 0xf, true));
  };
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  step(std::integral_constant<int, 0x141>{});
  step(std::integral_constant<int, 0x140>{});
  return v;
}
// Over G lanes (16, or the wave).
template <int G>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = row_max(v);
  if constexpr (G == 16) return v;
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return max(max(a, b), max(c, d));
}
template <int G>
__device__ __forceinline__ uint64_t lanes_max(uint64_t v) {
  const uint32_t high = (uint32_t)(v >> 32), top = lanes_max<G>(high);
  return (uint64_t)top << 32 | lanes_max<G>(high == top ? (uint32_t)v : 0u);
}
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
  v = row_sum(v);
  if constexpr (G == 16) return v;
  auto at = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
  return (at(0) + at(16)) + (at(32) + at(48));
}

// Descending order of a lane's V entries (Batcher's odd-even merge sort).
template <typename X, int V>
__device__ __forceinline__ void sort_entries(X (&x)[V]) {
  static_assert(V == 1 || V == 2 || V == 4 || V == 8, "a network of this size");
  auto order = [&](int i, int j) {
    const X a = x[i], b = x[j];
    x[i] = max(a, b);
    x[j] = min(a, b);
  };
  if constexpr (V == 2) order(0, 1);
  if constexpr (V >= 4) {
#pragma unroll
    for (int h = 0; h < V; h += 4) {
      order(h, h + 1), order(h + 2, h + 3);
      order(h, h + 2), order(h + 1, h + 3);
      order(h + 1, h + 2);
    }
  }
  if constexpr (V == 8) {
    order(0, 4), order(1, 5), order(2, 6), order(3, 7);
    order(2, 4), order(3, 5);
    order(1, 2), order(3, 4), order(5, 6);
  }
}

// The choices of a token, by G lanes with V consecutive logits each.  Lane j of them returns the j-th choice (-1: none)
// in `id` and its weight.  Each lane sorts its entries, and each choice is the largest of the lanes' first.
template <typename T, int G, int V>
__device__ __forceinline__ void choose(const RouteArgs& a, const T (&raw)[V], bool live, int& id, float& weight) {
  using E = Entry<T>;
  using X = typename E::Type;
  const int l = (threadIdx.x & 63) % G;
  X x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = E::make(raw[v], live && l * V + v < a.E, l * V + v);
  sort_entries(x);
  X top = lanes_max<G>(x[0]), mine = 0;  // mine: choice l
  const float peak = E::any(top) ? E::value(top) : 0.0f;
  float total = 0.0f;
  if (!a.renorm) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float w = exp_of(E::value(x[v]) - peak);  // (computed in any case: no branch)
      total += E::any(x[v]) ? w : 0.0f;
    }
    total = lanes_sum<G>(total);
  }
  for (int j = 0; j < a.k; ++j) {
    if (j) top = lanes_max<G>(x[0]);
    if (l == j) mine = top;
    // the lane that has it moves up its others (by masks: written as a choice between neighbours, the compiler makes
    // it an index into all of them, which took 75 more operations)
    const X taken = x[0] == top ? ~(X)0 : 0;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = (x[v] & ~taken) | (v + 1 < V ? x[v + 1 < V ? v + 1 : v] & taken : 0);
  }
  const bool have = E::any(mine);
  const float p = have ? exp_of(E::value(mine) - peak) : 0.0f;
  if (a.renorm) total = lanes_sum<G>(p);
  id = have ? E::index(mine) : -1;
  weight = have ? p / total : 0.0f;
}

// Choices and weights of the tokens [m0, m1), and how often each expert was chosen into `count` (LDS).
template <typename T, int G, int V>
__device__ __forceinline__ void choose_chunk(const RouteArgs& a, int64_t m0, int64_t m1, int32_t* count) {
  constexpr int kPer = 64 / G;  // tokens of a wave
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane % G;
  // the lane's logits of token m (past the last: the last again; past column E: anything)
  auto fetch = [&](int64_t m, T (&raw)[V]) {
    const T* p = static_cast<const T*>(a.logits) + min(m, m1 - 1) * a.E;
    if (l * V + V <= a.E) {
      __builtin_memcpy(raw, p + l * V, V * sizeof(T));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) raw[v] = p[min(l * V + v, a.E - 1)];
    }
  };
  T next[V];
  fetch(m0 + wave * kPer + lane / G, next);
  for (int64_t m = m0 + wave * kPer; m < m1; m += (blockDim.x >> 6) * kPer) {
    const int64_t mine = m + lane / G;
    T raw[V];
#pragma unroll
    for (int v = 0; v < V; ++v) raw[v] = next[v];
    fetch(mine + (blockDim.x >> 6) * kPer, next);
    int id;
    float w;
    choose<T, G, V>(a, raw, mine < m1, id, w);
    if (mine < m1 && l < a.k) {
      a.experts[mine * a.k + l] = id;
      a.weights[mine * a.k + l] = w;
      if (id >= 0) atomicAdd(&count[id], 1);
    }
  }
}

// Places of the choices [i0, i1) of chunk c.  LDS: base [waves][E], of which row 0 starts as the number
// of this chunk's choices per expert; total [E + 1].
__device__ __forceinline__ void place_chunk(const RouteArgs& a, int c, int chunks, int64_t i0, int64_t i1, int32_t* base,
                                            int32_t* total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int E = a.E, waves = blockDim.x >> 6;
  // each expert's choices in all chunks, and in those before this one
  int32_t* before = base;  // [E]
  if (chunks > 1) {
    for (int e = tid; e < E; e += blockDim.x) before[e] = total[e] = 0;
    __syncthreads();
    // groups of threads take the chunks in turn (integer sums: any order)
    const int width = 64 * ((E + 63) / 64), parts = max(1, (int)blockDim.x / width);
    for (int t = tid; t < width * parts; t += blockDim.x) {
      const int e = t % width, p = t / width;
      if (e >= E) continue;
      int all = 0, left = 0;
#pragma unroll 16
      for (int h = p; h < chunks; h += parts) {
        const int n = a.counts[(int64_t)h * E + e];
        all += n;
        left += h < c ? n : 0;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], left);
    }
  } else {
    for (int e = tid; e < E; e += blockDim.x) {
      total[e] = base[e];
      before[e] = 0;
    }
  }
  __syncthreads();
  // total: to the first place of each expert
  if (wave == 0) {
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int n = e0 + lane < E ? total[e0 + lane] : 0;
      int incl = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(incl, d, 64);
        if (lane >= d) incl += v;
      }
      if (e0 + lane < E) total[e0 + lane] = run + incl - n;
      run += __builtin_amdgcn_readlane(incl, 63);
    }
    if (lane == 0) total[E] = run;
  }
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {
    total[e] += before[e];  // this chunk's first place
    if (c == 0) a.offsets[e] = total[e];  // (before is 0 in chunk 0)
  }
  if (c == 0 && tid == 0) a.offsets[E] = total[E];
  const int64_t used = total[E], T = a.M * a.k;
  for (int64_t s = used + (int64_t)c * blockDim.x + tid; s < T; s += (int64_t)chunks * blockDim.x) a.rows[s] = -1;
  __syncthreads();
  // the waves share the choices in order; how often each expert comes up in each share
  for (int e = tid; e < E * waves; e += blockDim.x) base[e] = 0;
  __syncthreads();
  const int64_t share = ((i1 - i0 + waves - 1) / waves + 63) / 64 * 64;
  const int64_t lo = min(i0 + wave * share, i1), hi = min(lo + share, i1);
  int32_t* mine = base + wave * E;
  for (int64_t i = lo + lane; i < hi; i += 64) {
    const int e = a.experts[i];
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {
    int run = total[e];
    for (int w = 0; w < waves; ++w) {
      const int n = base[w * E + e];
      base[w * E + e] = run;
      run += n;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(max(E - 1, 1));
  for (int64_t i = lo; i < hi; i += 64) {
    const int64_t at = i + lane;
    const int e = at < hi ? a.experts[at] : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(e >> b & 1);
      same &= (e >> b & 1) ? set : ~set;
    }
    int place = -1;
    if (e >= 0) {
      const int next = mine[e];
      place = next + __popcll(same & ((1ull << lane) - 1));
      a.rows[place] = (int32_t)(at / a.k);
      if (lane == 63 - __builtin_clzll(same)) mine[e] = place + 1;
    }
    if (at < hi) a.slots[at] = place;
  }
}

template <typename T, int G, int V>
__global__ __launch_bounds__(kThreads) void k_route_one(RouteArgs a) {
  extern __shared__ int32_t lds[];  // [waves][E], [E + 1]
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) lds[e] = 0;
  __syncthreads();
  choose_chunk<T, G, V>(a, 0, a.M, lds);
  __threadfence_block();  // the choices are read again by other waves
  __syncthreads();
  place_chunk(a, 0, 1, 0, a.M * a.k, lds, lds + (blockDim.x >> 6) * a.E);
}

template <typename T, int G, int V>
__global__ __launch_bounds__(kThreads) void k_route_top(RouteArgs a, int chunk) {
  extern __shared__ int32_t lds[];  // [E]
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) lds[e] = 0;
  __syncthreads();
  const int64_t m0 = (int64_t)blockIdx.x * chunk;
  choose_chunk<T, G, V>(a, m0, min(m0 + chunk, a.M), lds);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[(int64_t)blockIdx.x * a.E + e] = lds[e];
}

__global__ __launch_bounds__(kThreads) void k_route_place(RouteArgs a, int chunk) {
  extern __shared__ int32_t lds[];  // [waves][E], [E + 1]
  const int64_t m0 = (int64_t)blockIdx.x * chunk;
  place_chunk(a, blockIdx.x, gridDim.x, m0 * a.k, min(m0 + chunk, a.M) * a.k, lds, lds + (blockDim.x >> 6) * a.E);
}

template <typename T, int G, int V>
hipError_t launch(const RouteArgs& a, const RoutePlan& p, hipStream_t s) {
  const size_t lds = (size_t)((kWaves + 1) * a.E + 1) * 4;
  if (p.chunks == 1) {
    k_route_one<T, G, V><<<1, kThreads, lds, s>>>(a);
    return hipGetLastError();
  }
  k_route_top<T, G, V><<<p.chunks, kThreads, (size_t)a.E * 4, s>>>(a, p.chunk);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_route_place<<<p.chunks, kThreads, lds, s>>>(a, p.chunk);
  return hipGetLastError();
}

}  // namespace

RoutePlan plan_route(int64_t M, int64_t E) {
  RoutePlan p;
  p.chunk = (int)M;
  if (M > 256) {
    p.chunk = (int)std::max<int64_t>(64, (M + 255) / 256);
    p.chunks = (int)((M + p.chunk - 1) / p.chunk);
    p.ws_bytes = (int64_t)p.chunks * E * 4;
  }
  return p;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const RoutePlan p = plan_route(a.M, a.E);
  auto go = [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    return a.bf16 ? launch<uint16_t, G, V>(a, p, s) : launch<float, G, V>(a, p, s);
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 4> four;
  const std::integral_constant<int, 8> eight;
  const std::integral_constant<int, 16> row;
  const std::integral_constant<int, 64> wave;
  if (a.E <= 16) return go(row, one);
  if (a.E <= 32) return go(row, two);
  if (a.E <= 64) return go(row, four);
  if (a.E <= 128) return go(row, eight);
  if (a.E <= 256) return go(wave, four);
  return go(wave, eight);
}

}  // namespace bl
