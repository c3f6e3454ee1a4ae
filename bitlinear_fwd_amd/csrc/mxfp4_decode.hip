// MXFP4 product for few tokens: Y[M][N] = sum_k Xv[m][k] Wv[n][k] with both matrices as codes
// and scales in the layout of mxfp4.h, fp32 accumulation in the matrix cores.
//
// Bound by the weights' bytes (17/32 byte each).  Up to 16 tokens (k_mx_few) the tokens' codes live in
// LDS and weights stream past: 1 x 28672 x 8192 21.9 us (5.7 TB/s of weights; a large copy moves 5.2),
// 1 x 8192 x 28672 from fp32 22.9, 1 x 6912 x 2560 4.1.  What took it there from 24 and 29 us: one
// launch instead of two, and workgroups that stay (16 waves to a unit) and keep the next group's
// loads in flight over the sums of this row block.  Loads past the caches, as the weights are read
// once.
// More tokens (k_mx_decode): a workgroup takes one 16-row block of the weights and TG groups of 16
// tokens; its waves split the columns in groups of four tiles and add their sums in LDS at the end, in
// wave order.  Each weight tile is loaded once (one coalesced 1 KiB wave load straight into operand
// registers) and serves TG matrix instructions; the tokens' tiles come from L2, which is what bounds
// it (0.1 us for a thousand products of a weight tile with 16 tokens).
#include "mxfp4.h"

#include <algorithm>

namespace bl {
namespace {

template <typename TY>
__device__ __forceinline__ void store_y(TY* y, float v) {
  if constexpr (sizeof(TY) == 4)
    *y = v;
  else
    *y = (TY)bf16_bits(v);
}

template <int TG, typename TY>
__global__ __launch_bounds__(512) void k_mx_decode(const uint8_t* __restrict__ codes,
                                                   const uint8_t* __restrict__ scales,
                                                   const uint8_t* __restrict__ xcodes,
                                                   const uint8_t* __restrict__ xscales, int64_t M, int64_t N,
                                                   int64_t tiles, int64_t groups, int64_t nblocks, int64_t xblocks,
                                                   TY* __restrict__ Y) {
  extern __shared__ v4f part[];  // [waves][TG][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t xb0 = (int64_t)blockIdx.y * TG;
  for (int64_t nb = blockIdx.x; nb < nblocks; nb += gridDim.x) {
    v4f acc[TG];
#pragma unroll
    for (int j = 0; j < TG; ++j) acc[j] = v4f{0, 0, 0, 0};
    for (int64_t g = wave; g < groups; g += waves) {
      const int sw = *reinterpret_cast<const int*>(scales + ((nb * groups + g) * 64 + lane) * 4);
      v4i w[4];
      static_for<4>([&](auto t) {
        w[t] = v4i{0, 0, 0, 0};
        if (4 * g + t < tiles)
          w[t] = *reinterpret_cast<const v4i*>(codes + (nb * tiles + 4 * g + t) * kMxTileBytes + 16 * lane);
      });
#pragma unroll
      for (int j = 0; j < TG; ++j) {
        const int64_t xb = min(xb0 + j, xblocks - 1);  // a group past the last repeats it; not stored
        const int sx = *reinterpret_cast<const int*>(xscales + ((xb * groups + g) * 64 + lane) * 4);
        static_for<4>([&](auto t) {
          v4i x = {0, 0, 0, 0};
          if (4 * g + t < tiles)
            x = *reinterpret_cast<const v4i*>(xcodes + (xb * tiles + 4 * g + t) * kMxTileBytes + 16 * lane);
          acc[j] = mx_mfma<t, t>(w[t], x, acc[j], sw, sx);
        });
      }
    }
#pragma unroll
    for (int j = 0; j < TG; ++j) part[(wave * TG + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int i = threadIdx.x; i < TG * 64; i += blockDim.x) {
      v4f s = part[i];
      for (int w = 1; w < waves; ++w) s += part[w * TG * 64 + i];
      const int64_t m = (xb0 + i / 64) * 16 + (i & 15), n = nb * 16 + 4 * ((i & 63) >> 4);
      if (m < M) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < N) store_y(Y + m * N + n + q, s[q]);
      }
    }
    __syncthreads();
  }
}

// Where k_mx_few takes the activations from.
enum { kFromCodes, kFromBf16, kFromF32 };

// Barrier between LDS writes and reads that leaves global loads in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Up to 16 tokens whose codes fit LDS.  The workgroup first fills LDS with the tokens' codes and
// scales (kFromCodes: copied; else quantised there from X[M][K], two lanes to a block), then walks
// over row blocks of the weights: its waves split the columns in groups of four tiles, the next
// group's loads in flight, and add their sums through LDS in wave order.
// LDS: sums, codes [4 groups tiles][4 blocks][M] x 16 bytes, scale bytes [4 groups tiles][4 blocks][M].
// magic: ceil(2^32 / M) (M > 1); i / M is the high word of i magic for the few thousand blocks that
// fit LDS.
template <int kSrc, typename TY>
__global__ __launch_bounds__(1024) void k_mx_few(const uint8_t* __restrict__ codes,
                                                 const uint8_t* __restrict__ scales, const void* __restrict__ X,
                                                 const uint8_t* __restrict__ xscales, int M, int64_t N, int64_t K,
                                                 int tiles, int groups, uint32_t magic, int64_t nblocks,
                                                 TY* __restrict__ Y) {
  extern __shared__ v4f part[];  // [2][workers][64], then the tokens
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6, workers = min(waves, groups);  // workers: waves with weights to read
  uint8_t* xc = reinterpret_cast<uint8_t*>(part + 2 * workers * 64);
  uint8_t* xs = xc + groups * 256 * M;

  v4i w[2][4];
  int sw[2];
  auto fetch = [&](int64_t nb, int g, v4i (&v)[4], int& sc) {
    const bool in = nb < nblocks;
    sc = in ? __builtin_nontemporal_load(reinterpret_cast<const int*>(scales + ((nb * groups + g) * 64 + lane) * 4)) : 0;
    static_for<4>([&](auto t) {
      v[t] = v4i{0, 0, 0, 0};
      if (in && 4 * g + t < tiles)
        v[t] = __builtin_nontemporal_load(
            reinterpret_cast<const v4i*>(codes + (nb * tiles + 4 * g + t) * kMxTileBytes + 16 * lane));
    });
  };
  int64_t nb = blockIdx.x;
  if constexpr (kSrc == kFromCodes) {
    const uint8_t* xcodes = static_cast<const uint8_t*>(X);
    for (int i = threadIdx.x; i < groups * 16 * M; i += blockDim.x) {
      const int cb = i / M, r = i - cb * M;  // tile and block, token
      v4i v = {0, 0, 0, 0};
      if (cb < 4 * tiles) v = *reinterpret_cast<const v4i*>(xcodes + (int64_t)cb * 256 + 16 * r);
      *reinterpret_cast<v4i*>(xc + 16 * i) = v;
    }
    for (int i = threadIdx.x; i < groups * 16 * M; i += blockDim.x) {
      const int cb = i / M, r = i - cb * M, c = cb >> 2, b = cb & 3;
      xs[i] = xscales[((c >> 2) * 64 + 16 * b + r) * 4 + (c & 3)];
    }
  } else {
    using T = std::conditional_t<kSrc == kFromBf16, uint16_t, float>;
    const T* x = static_cast<const T*>(X);
    const int p = threadIdx.x & 1, pairs = 32 * waves, items = M * 16 * groups;
    // item i: block i / M of token i % M, in the order of LDS, for two lanes; kBatch of a pair's items
    // are loaded before the first is used
    auto quantize = [&](auto batch) {
      constexpr int kBatch = decltype(batch)::value;
      for (int i0 = threadIdx.x >> 1; i0 < items; i0 += kBatch * pairs) {
        Raw8<T> v[kBatch][2];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int i = i0 + j * pairs, cb = M == 1 ? i : (int)__umulhi((uint32_t)i, magic), r = i - cb * M;
          const int col = 32 * cb + 16 * p, left = i < items ? (int)K - col : 0;
          const T* at = x + (r * (int)K + col);
          v[j][0] = load_raw8(at, left);
          v[j][1] = load_raw8(at + 8, left - 8);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const MxScale s = mx_scale(pair_max(max(top_bits(v[j][0]), top_bits(v[j][1]))));
          uint2 q;
          q.x = codes8(v[j][0], s);
          q.y = codes8(v[j][1], s);
          const int i = i0 + j * pairs;
          if (i < items) {
            *reinterpret_cast<uint2*>(xc + 16 * i + 8 * p) = q;
            if (p == 0) xs[i] = (uint8_t)s.e;
          }
        }
      }
    };
    if (items <= pairs)
      quantize(std::integral_constant<int, 1>{});
    else if (items <= 2 * pairs)
      quantize(std::integral_constant<int, 2>{});
    else
      quantize(std::integral_constant<int, 4>{});
  }
  if (wave >= workers) {  // more waves than groups of tiles: they have quantised, and keep the barriers
    lds_barrier();
    for (; nb < nblocks; nb += gridDim.x) lds_barrier();
    return;
  }
  fetch(nb, wave, w[0], sw[0]);
  lds_barrier();

  const int tok = min(lane & 15, M - 1);  // lanes of tokens past the last repeat it; not stored
  const uint8_t* xl = xc + 16 * ((lane >> 4) * M + tok);
  const uint8_t* sl = xs + (lane >> 4) * M + tok;
  v4f acc = {0, 0, 0, 0};
  int g = wave, turn = 0;
  while (nb < nblocks) {
    static_for<2>([&](auto u) {
      constexpr int cur = u;
      if (nb >= nblocks) return;
      const bool more = g + workers < groups;  // of this row block
      const int64_t nnb = more ? nb : nb + gridDim.x;
      const int ng = more ? g + workers : wave;
      fetch(nnb, ng, w[1 - cur], sw[1 - cur]);
      static_for<4>([&](auto t) {
        const v4i xv = *reinterpret_cast<const v4i*>(xl + (4 * g + t) * 64 * M);
        acc = mx_mfma<t, 0>(w[cur][t], xv, acc, sw[cur], sl[(4 * g + t) * 4 * M]);
      });
      if (!more) {
        v4f* mine = part + (turn & 1) * workers * 64;
        mine[wave * 64 + lane] = acc;
        acc = v4f{0, 0, 0, 0};
        lds_barrier();
        if (wave == turn % workers) {
          v4f s = mine[lane];
          for (int v = 1; v < workers; ++v) s += mine[v * 64 + lane];
          const int64_t n = nb * 16 + 4 * (lane >> 4);
          const int m = lane & 15;
          if (m < M) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + q < N) store_y(Y + m * N + n + q, s[q]);
          }
        }
        ++turn;
      }
      nb = nnb;
      g = ng;
    });
  }
}

template <int TG, typename TY>
void launch(const MxDecodePlan& p, const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
            const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, hipStream_t s) {
  k_mx_decode<TG, TY><<<dim3((unsigned)p.gx, (unsigned)p.gy), 64 * p.waves, p.waves * TG * 1024, s>>>(
      codes, scales, xcodes, xscales, M, N, mx_tiles(K), mx_groups(K), mx_row_blocks(N), mx_row_blocks(M),
      static_cast<TY*>(Y));
}

}  // namespace

// Blocks that a workgroup quantises by itself at most; beyond, the quantiser runs first.  Measured, one
// launch against two (graph replays; the issue of an eager call takes 9.3 and 14 us): 16 x 2560 x 2560
// 5.6 and 7.4 us, 16 x 2560 x 6912 (3584 blocks) 9.5 and 9.3, 4 x 8192 x 28672 (3584) 25.4 and 26.3.
constexpr int64_t kFewItems = 4096;

MxFewPlan plan_mx_few(int64_t M, int64_t N, int64_t K, int src) {
  MxFewPlan p;
  if (M > 16) return p;
  // Waves: one per group of four tiles, and enough that no pair of lanes quantises more than two
  // blocks; 16 at most.  Workgroups: what fits a compute unit with 16 waves, so that each fills its
  // LDS once and then streams weights.
  const int64_t groups = mx_groups(K), items = 16 * groups * M;
  if (src && items > kFewItems) return p;
  p.waves = (int)std::min<int64_t>(16, std::max(groups, src ? (items + 63) / 64 : 1));
  p.groups = std::min<int64_t>(mx_row_blocks(N), 256 * (16 / p.waves));
  p.lds = 2 * std::min<int64_t>(p.waves, groups) * 1024 + groups * 272 * M;
  p.ok = p.lds <= 160 * 1024;
  return p;
}

hipError_t launch_mx_few(const uint8_t* codes, const uint8_t* scales, const void* x, const uint8_t* xscales, int src,
                         int64_t M, int64_t N, int64_t K, void* Y, int ybf16, hipStream_t s) {
  const MxFewPlan p = plan_mx_few(M, N, K, src);
  if (!p.ok) return hipErrorInvalidConfiguration;
  auto go = [&](auto sc, auto yt) {
    using TY = decltype(yt);
    constexpr int kSrc = decltype(sc)::value;
    if (p.lds > 65536) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_mx_few<kSrc, TY>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)p.lds);
      if (e != hipSuccess) return e;
    }
    k_mx_few<kSrc, TY><<<dim3((unsigned)p.groups), 64 * p.waves, p.lds, s>>>(
        codes, scales, x, xscales, (int)M, N, K, (int)mx_tiles(K), (int)mx_groups(K),
        (uint32_t)(((uint64_t(1) << 32) + M - 1) / M), mx_row_blocks(N),
        static_cast<TY*>(Y));
    return hipGetLastError();
  };
  auto by_y = [&](auto sc) { return ybf16 ? go(sc, uint16_t{}) : go(sc, float{}); };
  switch (src) {
    case kFromCodes: return by_y(std::integral_constant<int, kFromCodes>{});
    case kFromBf16: return by_y(std::integral_constant<int, kFromBf16>{});
    default: return by_y(std::integral_constant<int, kFromF32>{});
  }
}

// Estimates in microseconds that fit both sides: the decode kernel by its products of a weight tile
// with 16 tokens (64 x 8192 x 8192: 131072 of them, 17.1 us; 128 x 2560 x 6912: 69120, 10.4; 256 x 6912
// x 2560: 138240, 14.7), the GEMM, while its 128 x 128 tiles fit the chip at once, by its steps of 128
// columns (20, 54, 64 and 224 steps: 11.8, 20.6, 25.2 and 73.6).  17 to 64 tokens of 8192 x 8192
// decode, 128 of them go through the GEMM (28.4 against 25.3), 128 of 2560 x 6912 decode (10.4
// against 20.6).
bool mx_decode_wins(int64_t M, int64_t N, int64_t K) {
  if (M <= 16) return true;
  if (M > 512) return false;
  const int64_t rounds = (((M + 127) / 128) * ((N + 127) / 128) + 511) / 512;
  const double decode = 3.0 + 1e-4 * (double)(mx_row_blocks(N) * mx_tiles(K)) * (double)mx_row_blocks(M);
  const double gemm = 5.0 + 0.31 * (double)(mx_tiles(K) * rounds);
  return decode <= gemm;
}

MxDecodePlan plan_mx_decode(int64_t M, int64_t N, int64_t K) {
  MxDecodePlan p;
  p.tg = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  p.waves = (int)std::min<int64_t>(8, std::max<int64_t>(1, mx_groups(K) / 2));
  p.gx = std::min<int64_t>(mx_row_blocks(N), 1 << 22);
  p.gy = (mx_row_blocks(M) + p.tg - 1) / p.tg;
  return p;
}

hipError_t launch_mx_decode(const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                            const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, int ybf16,
                            hipStream_t s) {
  const MxDecodePlan p = plan_mx_decode(M, N, K);
  auto go = [&](auto tg) {
    constexpr int TG = decltype(tg)::value;
    if (ybf16)
      launch<TG, uint16_t>(p, codes, scales, xcodes, xscales, M, N, K, Y, s);
    else
      launch<TG, float>(p, codes, scales, xcodes, xscales, M, N, K, Y, s);
  };
  if (p.tg == 1)
    go(std::integral_constant<int, 1>{});
  else if (p.tg == 2)
    go(std::integral_constant<int, 2>{});
  else
    go(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

}  // namespace bl
