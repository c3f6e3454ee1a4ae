// MXFP4 product for few tokens: Y[M][N] = sum_k Xv[m][k] Wv[n][k] with both matrices as codes
// and scales in the layout of mxfp4.h, fp32 accumulation in the matrix cores.
//
// A workgroup takes one 16-row block of the weights and TG groups of 16 tokens; its waves split
// the columns in groups of four tiles and add their sums in LDS at the end, in wave order.  Each
// weight tile is loaded once (one coalesced 1 KiB wave load straight into operand registers) and
// serves TG matrix instructions.
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

template <int TG, typename TY>
void launch(const MxDecodePlan& p, const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
            const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, hipStream_t s) {
  k_mx_decode<TG, TY><<<dim3((unsigned)p.gx, (unsigned)p.gy), 64 * p.waves, p.waves * TG * 1024, s>>>(
      codes, scales, xcodes, xscales, M, N, mx_tiles(K), mx_groups(K), mx_row_blocks(N), mx_row_blocks(M),
      static_cast<TY*>(Y));
}

}  // namespace

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
