// Ternary products with an epilogue, for one matrix or for a matrix per expert, and the router in front
// of them: arguments, device helpers and launchers shared by the kernels.
//
// A product's rows are slots: slot s of group e (offsets[e] <= s < offsets[e + 1]) multiplies token row
// rows[s] of the int8 codes by matrix e.  One matrix is the case of one group that holds all rows.
#pragma once
#include "bl_internal.h"
#include "mxfp4.h"  // bf16_pair, load8, uniform_ptr, v4f

namespace bl {

// What happens to a product on its way out (a host struct of the C ABI, checked there).
struct Epilogue {
  const float* bias;     // [N], or [E][N] where there are experts; null: none
  const void* residual;  // null: none.  May be Y itself, so neither pointer is __restrict__
  void* Y;
  int64_t ldr, ldy;      // elements between rows
  int act;               // bl_activation
  int res_bf16, y_bf16;
  int stream;            // Y is written past the caches: its rows and their pieces of 16 bytes are aligned
};

// The matrices and which rows each of them takes.
struct Groups {
  const uint8_t* packed;  // [E][n_pad k_pad / 4]
  const float* gamma;     // [E]
  const int32_t* offsets; // [E + 1], null: one group with the slots 0 .. T - 1
  const int32_t* rows;    // [T], null: slot s takes row s
  int E;
  int64_t T, R;           // slots; rows of the codes
  int64_t N, K;
};

// Slots of group e, kept within 0 .. T whatever the offsets hold.
__device__ __forceinline__ int2 group_slots(const Groups& g, int e) {
  if (!g.offsets) return make_int2(0, (int)g.T);
  const int lo = max(0, min(g.offsets[e], (int)g.T));
  return make_int2(lo, max(lo, min(g.offsets[e + 1], (int)g.T)));
}

// Token row of slot s, -1 for a slot without one.
__device__ __forceinline__ int slot_row(const Groups& g, int s) {
  const int r = g.rows ? g.rows[s] : s;
  return (uint32_t)r < (uint32_t)g.R ? r : -1;
}

// Work is dealt in units of up to `height` consecutive slots of one group; the units of all groups are
// numbered in order.  Every lane of a wave calls these with the same arguments.  Offsets that break their
// rule may give units that overlap or are passed over, but never one outside 0 .. T.
struct Unit {
  int e, lo, hi;  // group and slots (lo >= hi: there is no such unit)
};
__device__ __forceinline__ int units_of(int2 s, int height) {
  return (int)(((uint32_t)(s.y - s.x) + height - 1) / height);
}
// Units of all groups, at most `most`.
__device__ __forceinline__ int count_units(const Groups& g, int height, int most) {
  if (!g.offsets) return (int)((g.T + height - 1) / height);
  int n = 0;
  for (int e = threadIdx.x & 63; e < g.E; e += 64) n = min(n + min(units_of(group_slots(g, e), height), most), most);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) n = min(n + __shfl_xor(n, d, 64), most);
  return __builtin_amdgcn_readfirstlane(n);
}
// Unit u; 64 groups are looked at together.
__device__ __forceinline__ Unit find_unit(const Groups& g, int height, int u) {
  if (!g.offsets) {
    const int64_t lo = (int64_t)u * height;
    if (lo >= g.T) return Unit{0, 0, 0};
    return Unit{0, (int)lo, (int)min(lo + height, g.T)};
  }
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int2 s = make_int2(0, 0);
    if (e0 + lane < g.E) s = group_slots(g, e0 + lane);
    const int mine = units_of(s, height);
    int incl = mine;  // units of this and the groups before it
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const uint64_t after = __ballot(incl > u);
    if (after) {
      const int l = __builtin_ctzll(after);
      const int at = u - __builtin_amdgcn_readlane(incl - mine, l);
      if ((uint32_t)at >= (uint32_t)__builtin_amdgcn_readlane(mine, l)) return Unit{0, 0, 0};
      const int lo = __builtin_amdgcn_readlane(s.x, l) + at * height, hi = __builtin_amdgcn_readlane(s.y, l);
      return Unit{e0 + l, lo, hi - lo < height ? hi : lo + height};
    }
    u -= __builtin_amdgcn_readlane(incl, 63);
  }
  return Unit{0, 0, 0};
}

// A launch cannot have more units than this (groups with slots have at most one unit that is not full).
inline int64_t most_units(int64_t E, int64_t T, int height) { return T / height + (E < T ? E : T); }

// e^x to a few units in the last place for x <= 0, which is all that the router's weights need: 2^(x log2 e) with the
// product's rounding error put back.  Below -104, where e^x is nothing in fp32, it gives 0.
constexpr float kLog2e = 1.44269502e+00f, kLog2eLow = 1.92596303e-08f, kLn2 = 6.93147182e-01f;
__device__ __forceinline__ float exp_of(float x) {
  x = fmaxf(x, -104.0f);
  const float t = x * kLog2e;
  const float low = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, low * kLn2, e);
}
// 1 / (1 + e^-x), which goes to 0 on the far left: e^-x reaches infinity, so its rounding error is put back as a factor
// (added, as above, it would be infinity less infinity).
__device__ __forceinline__ float sigmoid_of(float x) {
  x = __builtin_amdgcn_fmed3f(x, -104.0f, 104.0f);
  const float t = x * -kLog2e;
  const float low = __builtin_fmaf(x, -kLog2eLow, __builtin_fmaf(x, -kLog2e, -t));
  return __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_amdgcn_exp2f(t), __builtin_fmaf(low, kLn2, 1.0f), 1.0f));
}

// v (1 + erf(v / sqrt 2)) / 2 = v Phi(v), from the half h = |v| Phi(-|v|) that is missing on the right and all there is
// on the left.  Phi(-a) e^(a^2 / 2) is a polynomial in t = 1 / (1 + 0.35 a): coefficients fitted to the least relative
// error over 0 .. 16 (a linear programme), 0.6 half steps.  Behind 16, h is 0 in fp32, and a NaN stays one.
// That is off by up to 5 half steps of |v|, near 0, and on the left by 16 + a^2 of the result: kShort, for bf16
// results, whose half step is 65536 of these.  For fp32 results Phi(v) - 1/2 up to 1.25, where the errors of h would be
// the result's, is v times a polynomial in v^2 (fitted alike, 0.01 half steps): off by up to 2 half steps of |v|.
// (2048 x 6912 x 2560 to fp32 46.9 us, 41.2 if this too took the short form, and 16 more than that with erff.)
template <bool kShort>
__device__ __forceinline__ float gelu_of(float v) {
  const float a = fminf(fabsf(v), 16.0f), s = a * a;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, a, 1.0f));
  float q = __builtin_fmaf(-0.0291652922f, t, 0.1440676f);
  q = __builtin_fmaf(q, t, -0.255916238f);
  q = __builtin_fmaf(q, t, 0.159409747f);
  q = __builtin_fmaf(q, t, -0.0232757498f);
  q = __builtin_fmaf(q, t, 0.105579995f);
  q = __builtin_fmaf(q, t, 0.119814143f);
  q = __builtin_fmaf(q, t, 0.139864534f);
  q = __builtin_fmaf(q, t, 0.139621243f);
  const float e = __builtin_amdgcn_exp2f(-7.21347511e-01f * s);  // e^(-a^2 / 2)
  const float h = q * t * e * a, far = v < 0.0f ? -h : v - h;
  if constexpr (kShort) return far;
  float r = __builtin_fmaf(4.58148179e-07f, s, -8.96567417e-06f);
  r = __builtin_fmaf(r, s, 0.000114846669f);
  r = __builtin_fmaf(r, s, -0.00118693034f);
  r = __builtin_fmaf(r, s, 0.00997341517f);
  r = __builtin_fmaf(r, s, -0.0664903596f);
  r = __builtin_fmaf(r, s, 0.398942292f);
  return a < 1.25f ? v * __builtin_fmaf(v, r, 0.5f) : far;
}

__device__ __forceinline__ float relu_of(float v) { return v < 0.0f ? 0.0f : v; }  // (fmaxf would make a NaN 0)

// The activations of bl_activation, in fp32; kShort: for a result in bf16.
template <int kAct, bool kShort>
__device__ __forceinline__ float activate(float v) {
  if constexpr (kAct == 1) return relu_of(v);
  else if constexpr (kAct == 2) return relu_of(v) * relu_of(v);
  else if constexpr (kAct == 3) return v * sigmoid_of(v);
  else if constexpr (kAct == 4) return gelu_of<kShort>(v);
  // (1 + tanh u) / 2 = sigmoid(2 u)
  else if constexpr (kAct == 5) return v * sigmoid_of(1.59576912f * __builtin_fmaf(0.044715f * v * v, v, v));
  else return v;
}
template <bool kShort, int H>
__device__ __forceinline__ void activate_all(v4f (&v)[H], int act) {
  auto go = [&](auto a) {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[h][e] = activate<decltype(a)::value, kShort>(v[h][e]);
  };
  switch (act) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 3: return go(std::integral_constant<int, 3>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 5: return go(std::integral_constant<int, 5>{});
    default: return;
  }
}

__device__ __forceinline__ float bf16_float(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Four consecutive values of row p, those of columns before the end (left of them; the others 0).
__device__ __forceinline__ v4f load4(const void* base, int64_t at, int left, int bf16) {
  v4f r = {0, 0, 0, 0};
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    uint16_t h[4] = {0, 0, 0, 0};
    if (left >= 4) {
      __builtin_memcpy(h, p, 8);
    } else {
#pragma unroll
      for (int q = 0; q < 3; ++q)
        if (q < left) h[q] = p[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = bf16_float(h[q]);
  } else {
    const float* p = static_cast<const float*>(base) + at;
    if (left >= 4) {
      __builtin_memcpy(&r, p, 16);
    } else {
#pragma unroll
      for (int q = 0; q < 3; ++q)
        if (q < left) r[q] = p[q];
    }
  }
  return r;
}
__device__ __forceinline__ void store4(void* base, int64_t at, int left, int bf16, v4f v) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if (left >= 4) {
      const uint32_t w[2] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      __builtin_memcpy(p, w, 8);
    } else {
#pragma unroll
      for (int q = 0; q < 3; ++q)
        if (q < left) p[q] = bf16_bits(v[q]);
    }
  } else {
    float* p = static_cast<float*>(base) + at;
    if (left >= 4) {
      __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
      for (int q = 0; q < 3; ++q)
        if (q < left) p[q] = v[q];
    }
  }
}

// A token's scale: the exact products are multiplied by gamma a / 127.
__device__ __forceinline__ float token_scale(float gamma, float a) { return gamma * a / 127.0f; }

// 4 H consecutive values at element `at`; and the same to Y, past the caches where its pieces of 16 bytes are aligned
// (2048 x 6912 fp32 outputs of MXFP4 products: 30.3 us without, 26.4 so).
template <typename H>
__device__ __forceinline__ void load_row(const void* base, int64_t at, int bf16, v4f* v, H) {
  if (bf16) {
    uint16_t h[4 * H::value];
    __builtin_memcpy(h, static_cast<const uint16_t*>(base) + at, 8 * H::value);
#pragma unroll
    for (int i = 0; i < 4 * H::value; ++i) v[i / 4][i % 4] = bf16_float(h[i]);
  } else {
    __builtin_memcpy(v, static_cast<const float*>(base) + at, 16 * H::value);
  }
}
template <typename H>
__device__ __forceinline__ void store_row(const Epilogue& ep, int64_t at, const v4f* v, H) {
  v4u w = __builtin_bit_cast(v4u, v[0]);
  if constexpr (H::value == 2)
    w = v4u{bf16_pair(v[0][0], v[0][1]), bf16_pair(v[0][2], v[0][3]), bf16_pair(v[1][0], v[1][1]),
            bf16_pair(v[1][2], v[1][3])};
  char* y = static_cast<char*>(ep.Y) + at * (H::value == 2 ? 2 : 4);
  if (ep.stream) __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(y));
  else __builtin_memcpy(y, &w, 16);
}

// The end of the epilogue: residual, rounding and store of 4 H consecutive outputs n .. of row s (left of them before
// column N).
template <int H>
__device__ __forceinline__ void finish_row(const Epilogue& ep, int64_t s, int64_t n, int left, v4f (&v)[H]) {
  if (ep.residual) {
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (left > 4 * h) v[h] += load4(ep.residual, s * ep.ldr + n + 4 * h, min(left - 4 * h, 4), ep.res_bf16);
  }
  const int64_t at = s * ep.ldy + n;
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (left > 4 * h) store4(ep.Y, at + 4 * h, min(left - 4 * h, 4), ep.y_bf16, v[h]);
}

// The epilogue of four consecutive outputs n .. n + 3 of slot s (left of them before column N).
__device__ __forceinline__ void finish4(const Epilogue& ep, int64_t e, int64_t N, int64_t s, int64_t n, int left,
                                        v4i acc, float scale) {
  v4f b = {0, 0, 0, 0}, v[1];
  if (ep.bias) b = load4(ep.bias, e * N + n, left, 0);
#pragma unroll
  for (int q = 0; q < 4; ++q) v[0][q] = __builtin_fmaf((float)acc[q], scale, b[q]);
  if (ep.y_bf16) activate_all<true>(v, ep.act);
  else activate_all<false>(v, ep.act);
  finish_row(ep, s, n, left, v);
}

// How the products of T slots of E matrices (E = 0: one matrix, no tables) are computed.
enum { kFewKernel = 10, kGemmKernel = 11, kMidKernel = 12 };
struct ExpertsPlan {
  int kernel = kFewKernel;
  int threads = 256;
  int64_t groups = 0;         // workgroups
  int height = 16, width = 64;  // slots and outputs of a workgroup at a time
  int per = 1;                // mid: row blocks of a workgroup
  bool quantizes = false;     // takes x itself
};
// src: 0 codes, 1 bf16 x, 2 fp32 x
ExpertsPlan plan_experts(int64_t E, int64_t T, int64_t N, int64_t K, int src);
// The products of every slot by a plan for these sizes and src; sizes and pointers are validated by the C ABI.  X:
// where the plan says that the kernel quantises.
hipError_t launch_experts(const ExpertsPlan& p, const Groups& g, const void* X, int src, const int8_t* Xq,
                          const float* absmax, const Epilogue& ep, hipStream_t s);

constexpr int kFewChunks = 160;  // chunks of 256 codes in all rows that the kernel for few slots can take
hipError_t launch_experts_few(const ExpertsPlan& p, const Groups& g, const void* X, int src, const Epilogue& ep,
                              hipStream_t s);
hipError_t launch_experts_mid(const ExpertsPlan& p, const Groups& g, const int8_t* Xq, const float* absmax,
                              const Epilogue& ep, hipStream_t s);
hipError_t launch_experts_gemm(const ExpertsPlan& p, const Groups& g, const int8_t* Xq, const float* absmax,
                               const Epilogue& ep, hipStream_t s);

// Elements between the rows of H below.
inline int64_t combine_ld(int64_t N) { return (N + 3) / 4 * 4; }
// Y[m] = residual[m] + sum over j of weights[m][j] H[slots[m][j]], H fp32 [T][combine_ld(N)] the products of the
// slots.  Slots that no group holds or that have no token row are left out.
hipError_t launch_combine(const Groups& g, const float* H, const int32_t* slots, const float* weights, int64_t M, int k,
                          const Epilogue& ep, hipStream_t s);

// The router: chunks of tokens, one workgroup each; one chunk is one launch.
struct RoutePlan {
  int chunks = 1, chunk = 0;  // chunk: tokens of one
  int64_t ws_bytes = 0;       // [chunks][E] counts where there are several
};
RoutePlan plan_route(int64_t M, int64_t E);
constexpr int kMaxRouteExperts = 512;  // 8 logits to a lane; the waves' counts fit LDS
constexpr int kMaxRouteChoices = 16;
struct RouteArgs {
  const void* logits;
  int bf16, renorm;
  int64_t M;
  int E, k;
  int32_t* experts;  // [M][k]
  float* weights;    // [M][k]
  int32_t* offsets;  // [E + 1]
  int32_t* rows;     // [M k]
  int32_t* slots;    // [M][k]
  int32_t* counts;   // workspace
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

}  // namespace bl
