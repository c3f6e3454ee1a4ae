// MXFP4 product for few tokens: Y[M][N] = sum_k Xv[m][k] Wv[n][k] with both matrices as codes
// and scales in the layout of mxfp4.h, fp32 accumulation in the matrix cores.
//
// Bound by the weights' bytes (17/32 byte each).  Up to 16 tokens (k_mx_few) the tokens' codes live in
// LDS and weights stream past: 1 x 28672 x 8192 21.9 us (5.7 TB/s of weights; a large copy moves 5.2),
// 1 x 8192 x 28672 from fp32 22.9, 1 x 6912 x 2560 4.1.  What took it there from 24 and 29 us: one
// launch instead of two, and workgroups that stay (16 waves to a unit) and keep the next group's
// loads in flight over the sums of this row block.  Loads past the caches, as the weights are read
// once.
// More tokens, or longer rows of up to 16 (k_mx_decode): a workgroup takes one or two 16-row blocks of
// the weights and TG groups of 16 tokens; its waves split the columns in groups of four tiles, and add
// their sums in LDS at the end, in wave order.  Each weight tile is one coalesced 1 KiB wave load
// straight into operand registers and serves TG matrix instructions; the tokens' tiles come from L2,
// which is what bounds it from some 32 tokens on (14 ns for a workgroup's product of a weight tile with
// 16 tokens).  The next group's weights are in flight over a whole group and the tokens' next tiles over
// most of one, without branches around the loads (those had every group wait for its own: 256 x 2560 x
// 6912 13.0 us, 11.8 so; 64 x 8192 x 28672 32.0 and 30.6).  16 x 8192 x 28672: 22.4 us, 5.6 TB/s of
// weights.  Groups of 16 tokens past the last are loaded and multiplied for nothing where their number is
// no multiple of TG: 33 to 48 tokens do the work of 64 (37 x 6909 x 2570 6.1 us), 65 to 80 that of 128.
#include "mxfp4.h"

#include <algorithm>
#include <atomic>

namespace bl {
namespace {

// Four consecutive outputs of a token, those before column N.
template <typename TY>
__device__ __forceinline__ void store_y(TY* y, int64_t left, v4f v) {
  if constexpr (sizeof(TY) == 4) {
    if (left >= 4) {
      __builtin_memcpy(y, &v, 16);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < left) y[q] = v[q];
    }
  } else {
    if (left >= 4) {
      const uint32_t w[2] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      __builtin_memcpy(y, w, 8);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < left) y[q] = bf16_bits(v[q]);
    }
  }
}

// Barrier between LDS writes and reads that leaves global loads in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// RB row blocks of the weights by TG groups of 16 tokens.  kOnce: each weight is read by one workgroup,
// and past the caches.
template <int TG, int RB, bool kOnce, typename TY>
__global__ __launch_bounds__(512) void k_mx_decode(const uint8_t* __restrict__ codes,
                                                   const uint8_t* __restrict__ scales,
                                                   const uint8_t* __restrict__ xcodes,
                                                   const uint8_t* __restrict__ xscales, int64_t M, int64_t N,
                                                   int tiles, int groups, int64_t nblocks, int64_t xblocks,
                                                   TY* __restrict__ Y) {
  extern __shared__ v4f part[];  // [waves][RB][TG][64]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int64_t xb0 = (int64_t)blockIdx.y * TG;
  const int last = tiles - 1;
  const uint32_t lane16 = 16 * lane, lane4 = 4 * lane;
  for (int64_t nb0 = (int64_t)blockIdx.x * RB; nb0 < nblocks; nb0 += (int64_t)gridDim.x * RB) {
    GlobalBytes wp[RB], xp[TG], sp[RB], xsp[TG];
#pragma unroll
    for (int i = 0; i < RB; ++i) {  // row blocks and token groups past the last repeat it; not stored
      const int64_t nb = min(nb0 + i, nblocks - 1);
      wp[i] = (GlobalBytes)uniform_ptr(codes + nb * tiles * kMxTileBytes);
      sp[i] = (GlobalBytes)uniform_ptr(scales + nb * groups * 256);
    }
#pragma unroll
    for (int j = 0; j < TG; ++j) {
      const int64_t xb = min(xb0 + j, xblocks - 1);
      xp[j] = (GlobalBytes)uniform_ptr(xcodes + xb * tiles * kMxTileBytes);
      xsp[j] = (GlobalBytes)uniform_ptr(xscales + xb * groups * 256);
    }
    v4f acc[RB][TG];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < TG; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    // The weights of this group of four tiles and, on their way from memory, of the wave's next; the
    // tokens' tiles come from L2, and their registers take the next group's once they have been used.
    // Past the last tile the last again, so that no load depends on a branch.
    v4i w[2][RB][4], x[TG][4];
    int sw[2][RB], sx[TG];
    auto tile_at = [&](int g, int t) { return (int64_t)min(4 * g + t, last) * kMxTileBytes; };
    auto fetch_w = [&](int g, v4i (&v)[RB][4], int (&sc)[RB]) {
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        sc[i] = *reinterpret_cast<GlobalInt>(sp[i] + (int64_t)g * 256 + lane4);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const GlobalV4i at = reinterpret_cast<GlobalV4i>(wp[i] + tile_at(g, t) + lane16);
          v[i][t] = kOnce ? __builtin_nontemporal_load(at) : *at;
        }
      }
    };
    auto fetch_x = [&](int g, int j) {
      sx[j] = *reinterpret_cast<GlobalInt>(xsp[j] + (int64_t)g * 256 + lane4);
#pragma unroll
      for (int t = 0; t < 4; ++t) x[j][t] = *reinterpret_cast<GlobalV4i>(xp[j] + tile_at(g, t) + lane16);
    };
    auto work = [&](int g, auto cur_c, auto more_c) {
      constexpr int cur = cur_c;
      constexpr bool more = decltype(more_c)::value;
      if constexpr (more) fetch_w(g + waves, w[1 - cur], sw[1 - cur]);
      __builtin_amdgcn_sched_barrier(0);
      // Tiles past the last take part with the last one's codes and both scales 2^-127: nothing is left
      // of their products in 32 bits.
      const int left = tiles - 4 * g;
      const uint32_t mask = left >= 4 ? ~0u : (1u << 8 * left) - 1;
      int s[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i) s[i] = sw[cur][i] & mask;
      static_for<TG>([&](auto jj) {
        constexpr int j = jj;
        const int sj = sx[j] & mask;
        static_for<4>([&](auto t) {
#pragma unroll
          for (int i = 0; i < RB; ++i) acc[i][j] = mx_mfma<t, t>(w[cur][i][t], x[j][t], acc[i][j], s[i], sj);
        });
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (more) fetch_x(g + waves, j);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;
    if (wave < groups) {
      int g = wave;
      fetch_w(g, w[0], sw[0]);
#pragma unroll
      for (int j = 0; j < TG; ++j) fetch_x(g, j);
      for (; g + 2 * waves < groups; g += 2 * waves) {
        work(g, even, std::true_type{});
        work(g + waves, odd, std::true_type{});
      }
      if (g + waves < groups) {
        work(g, even, std::true_type{});
        work(g + waves, odd, std::false_type{});
      } else {
        work(g, even, std::false_type{});
      }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < TG; ++j) part[((wave * RB + i) * TG + j) * 64 + lane] = acc[i][j];
    lds_barrier();
    for (int o = threadIdx.x; o < RB * TG * 64; o += blockDim.x) {
      v4f s = part[o];
      for (int v = 1; v < waves; ++v) s += part[v * RB * TG * 64 + o];
      const int i = o / (64 * TG), j = o / 64 % TG, l = o % 64;
      const int64_t m = (xb0 + j) * 16 + (l & 15), n = (nb0 + i) * 16 + 4 * (l >> 4);
      if (m < M) store_y(Y + m * N + n, N - n, s);
    }
    lds_barrier();
  }
}

// Where k_mx_few takes the activations from.
enum { kFromCodes, kFromBf16, kFromF32 };

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
    const int* sp = reinterpret_cast<const int*>(scales + ((nb * groups + g) * 64 + lane) * 4);
    sc = in ? __builtin_nontemporal_load(sp) : 0;
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
    else if (sizeof(T) == 4 || items <= 4 * pairs)
      quantize(std::integral_constant<int, 4>{});
    else
      quantize(std::integral_constant<int, sizeof(T) == 4 ? 4 : 8>{});
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
          if (m < M) store_y(Y + m * N + n, N - n, s);
        }
        ++turn;
      }
      nb = nnb;
      g = ng;
    });
  }
}

template <int TG, int RB, typename TY>
void launch(const MxDecodePlan& p, const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
            const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, hipStream_t s) {
  auto fn = &k_mx_decode<TG, RB, true, TY>;
  if constexpr (TG == 4) {  // more than 64 tokens read the weights more than once
    if (p.gy > 1) fn = &k_mx_decode<TG, RB, false, TY>;
  }
  fn<<<dim3((unsigned)p.gx, (unsigned)p.gy), 64 * p.waves, p.waves * RB * TG * 1024, s>>>(
      codes, scales, xcodes, xscales, M, N, (int)mx_tiles(K), (int)mx_groups(K), mx_row_blocks(N), mx_row_blocks(M),
      static_cast<TY*>(Y));
}

}  // namespace

// Blocks that a workgroup quantises by itself at most; beyond, the quantiser runs first.  Measured, one
// launch against two (graph replays; the issue of an eager call takes 8.5 and 14 us): 16 x 2560 x 2560
// 5.6 and 7.4 us, 16 x 2560 x 6912 (3584 blocks) 9.1 and 10.2, 4 x 8192 x 28672 (3584) 24.9 and 27.3; at
// the bound 16 x 2560 x 8192 9.6 and 10.4, 16 x 28672 x 8192 26.9 and 28.6, 4 x 2560 x 32768 15.3 and
// 16.7.  More blocks have not been measured.
constexpr int64_t kFewItems = 4096;
constexpr int64_t kFewLds = 160 * 1024;  // of a compute unit

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
  p.ok = p.lds <= kFewLds;
  return p;
}

hipError_t launch_mx_few(const uint8_t* codes, const uint8_t* scales, const void* x, const uint8_t* xscales, int src,
                         int64_t M, int64_t N, int64_t K, void* Y, int ybf16, hipStream_t s) {
  const MxFewPlan p = plan_mx_few(M, N, K, src);
  if (!p.ok) return hipErrorInvalidConfiguration;
  auto go = [&](auto sc, auto yt) {
    using TY = decltype(yt);
    constexpr int kSrc = decltype(sc)::value;
    // the LDS limit above 64 KiB is raised once per device for this kernel, to the most that a plan asks
    // for: host threads share it, and one with a smaller call must not lower it for another (a repeated
    // set from a concurrent first call is harmless)
    static std::atomic<uint64_t> raised{0};
    if (p.lds > 65536) {
      int dev = 0;
      hipError_t e = hipGetDevice(&dev);
      if (e != hipSuccess) return e;
      const uint64_t bit = uint64_t(1) << (dev & 63);
      if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_mx_few<kSrc, TY>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)kFewLds);
        if (e != hipSuccess) return e;
        raised.fetch_or(bit, std::memory_order_relaxed);
      }
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

constexpr int64_t kMxDecodeTokens = 4096;  // the most that the rule below was measured with

// Estimates in microseconds, fitted to 123 shapes of 20 to 4096 tokens measured both ways.  The decode
// kernel goes by rounds of one workgroup to a compute unit and their products of a weight tile with 16
// tokens; the GEMM by its steps of 128 columns, of one or two narrow tiles to a unit or of rounds of two
// wide ones; both by the weights' bytes.  Where the slower path is taken it is so by at most 5 % (200 x
// 8192 x 1024: 6.8 against 6.5 us).  Decode and GEMM in us: 64 x 8192 x 28672 30.6 and 72.2, 64 x 28672 x
// 8192 36.5 and 34.1, 256 x 8192 x 8192 37.7 and 24.5, 256 x 2560 x 6912 11.8 and 15.6, 512 x 2560 x 2560
// 11.4 and 8.5, 1500 x 128 x 8192 10.2 and 17.1.
bool mx_decode_wins(int64_t M, int64_t N, int64_t K) {
  if (M <= 16) return true;
  if (M > kMxDecodeTokens) return false;
  const auto rounds = [](int64_t groups, int64_t at_once) { return (double)((groups + at_once - 1) / at_once); };
  const double steps = (double)mx_tiles(K), stream = (double)mx_row_blocks(N) * steps * 1088.0 / 5e6;
  const MxDecodePlan d = plan_mx_decode(M, N, K);
  const double decode =
      std::max(2.8 + rounds(d.gx * d.gy, 256) * (0.4 + 0.0139 * steps * (double)(d.rb * d.tg)), 5.0 + stream);
  const MxGemmPlan g = plan_mx_gemm(M, N, K);
  const int64_t tiles = g.tiles_m * g.tiles_n;
  const double step = g.tile_n == 256 ? 0.8 * rounds(tiles, 512) : tiles <= 256 ? 0.22 : 0.36;
  const double gemm = std::max(4.8 + step * steps, 5.0 + stream) + 0.45e-6 * (double)M * (double)N;
  return decode <= gemm;
}

MxDecodePlan plan_mx_decode(int64_t M, int64_t N, int64_t K) {
  MxDecodePlan p;
  p.tg = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  p.gy = (mx_row_blocks(M) + p.tg - 1) / p.tg;
  // two row blocks share the tokens' tiles where the workgroups left fill the chip (64 x 8192 x 8192:
  // 12.5 us, 15.8 with one; 64 x 2560 x 6912, 160 row blocks: 9.3, 7.3 with one)
  p.rb = mx_row_blocks(N) * p.gy >= 256 ? 2 : 1;
  p.waves = (int)std::min<int64_t>(8, mx_groups(K));
  p.gx = std::min<int64_t>((mx_row_blocks(N) + p.rb - 1) / p.rb, 1 << 22);
  return p;
}

hipError_t launch_mx_decode(const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                            const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, int ybf16,
                            hipStream_t s) {
  const MxDecodePlan p = plan_mx_decode(M, N, K);
  auto go = [&](auto tg, auto rb) {
    constexpr int TG = decltype(tg)::value, RB = decltype(rb)::value;
    if (ybf16)
      launch<TG, RB, uint16_t>(p, codes, scales, xcodes, xscales, M, N, K, Y, s);
    else
      launch<TG, RB, float>(p, codes, scales, xcodes, xscales, M, N, K, Y, s);
  };
  auto by_rb = [&](auto tg) {
    if (p.rb == 2)
      go(tg, std::integral_constant<int, 2>{});
    else
      go(tg, std::integral_constant<int, 1>{});
  };
  if (p.tg == 1)
    by_rb(std::integral_constant<int, 1>{});
  else if (p.tg == 2)
    by_rb(std::integral_constant<int, 2>{});
  else
    by_rb(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

}  // namespace bl
