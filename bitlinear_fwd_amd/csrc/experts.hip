// Ternary products with an epilogue, for one matrix or by expert: which kernel takes them, and the sum over the
// slots of a token.
#include "experts.h"

#include <algorithm>
#include <cmath>

namespace bl {
namespace {

// One thread per four outputs of a token, and more where a launch cannot have so many.
constexpr int64_t kCombineGroups = int64_t(1) << 23;
__global__ __launch_bounds__(256) void k_combine(Groups g, const float* __restrict__ H,
                                                 const int32_t* __restrict__ slots,
                                                 const float* __restrict__ weights, int64_t M, int k, int64_t quads,
                                                 Epilogue ep) {
  const int first = max(0, min(g.offsets[0], (int)g.T)), last = max(0, min(g.offsets[g.E], (int)g.T));
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * quads; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / quads, n = 4 * (i - m * quads);
    const int left = (int)min(g.N - n, (int64_t)4);
    v4f v = {0, 0, 0, 0};
    for (int j = 0; j < k; ++j) {
      const int s = slots[m * k + j];
      if (s < first || s >= last || slot_row(g, s) < 0) continue;
      const v4f h = *reinterpret_cast<const v4f*>(H + (int64_t)s * (4 * quads) + n);  // (columns past N: not stored)
      const float w = weights[m * k + j];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf(w, h[q], v[q]);
    }
    if (ep.residual) v += load4(ep.residual, m * ep.ldr + n, left, ep.res_bf16);
    store4(ep.Y, m * ep.ldy + n, left, ep.y_bf16, v);
  }
}

}  // namespace

namespace {

// Estimates in us of each form of the kernels.  They are fitted to 10777 shapes that were measured in every form (5 to
// 2048 tokens of codes, 128 to 16384 outputs, 256 to 16384 columns, one matrix or 2 to 64 experts with up to four slots a
// token): the form that they choose takes 1.3 % longer than the fastest on average (one matrix 0.7 %, experts 1.9 %), and
// more than 10 % longer on 4 % of the shapes.
// The GEMM's tiles of `height` slots by `width` outputs: a stage of 128 columns takes `first` where each compute unit
// has at most one tile (its latency) and `more` a tile where several share it, `end` is what else a tile costs.
// 2048 x 6912 x 2560 in tiles of 128 x 256, 96 x 256, 64 x 256, 64 x 128: 37.7, 40.8, 39.2, 43.6 us; 2048 x 2560 x
// 6912: 43.7, 36.7, 43.4, 44.9; 512 x 2560 x 2560: 20.9, 17.4, 14.3, 10.8.
struct Tile {
  int height, width;
  double first, more, end;
};
constexpr Tile kTiles[] = {{128, 256, .796, .64, 3.17}, {96, 256, .597, .512, 2.32}, {64, 256, .549, .375, 1.52},
                           {64, 128, .367, .216, .993},  {32, 256, .373, .282, .956}, {32, 128, .266, .143, .82}};
constexpr double kGemmStart = 4.23;
// The decode kernel's workgroups of `height` slots by `per` row blocks: a chunk of 256 columns takes `first` on a
// compute unit that has one of them, `more` each where it has several (the rows' codes from L2 bound it); at the end
// each wave has its share of the blocks of 16 x 16 sums, kDecodeBlock apiece.  32 x 8192 x 8192 by 16 x 1, 2, 4 and
// 32 x 4: 19.7, 13.0, 9.0, 13.7 us, 16 x 2560 x 6912: 6.4, 6.5, 7.1, 8.2, 128 x 6912 x 2560: 20.0, 12.0, 10.4,
// 10.7; the GEMM 22.1, 19.1 and 9.6.
struct Decode {
  int height, per;
  double first, more;
};
constexpr Decode kDecodes[] = {{16, 1, .106, .0763}, {16, 2, .114, .103}, {16, 4, .147, .157}, {32, 4, .211, .328}};
constexpr double kDecodeStart = 3.52, kDecodeEnd = .131, kDecodeBlock = .433;

}  // namespace

ExpertsPlan plan_experts(int64_t E, int64_t T, int64_t N, int64_t K, int src) {
  ExpertsPlan p;
  const int64_t blocks = n_pad(N) / kTileRows, chunks = k_pad(K) / kTileCols;
  // groups that have slots, and units of them: the last unit of a group is about half full
  const double some = E ? (double)E * (1.0 - std::pow(1.0 - 1.0 / (double)E, (double)T)) : 1.0;
  auto units = [&](int height) {
    return E ? some * std::max(1.0, (double)T / some / height + 0.537) : (double)((T + height - 1) / height);
  };
  double best = 1e300;
  for (const Tile& t : kTiles) {
    const double stages = (double)(2 * chunks);
    const double rounds = std::ceil(units(t.height) * (double)((N + t.width - 1) / t.width) / 256.0);
    const double us = kGemmStart + (rounds > 1 ? rounds * (stages * t.more + t.end) : stages * t.first + t.end);
    if (us < best) best = us, p.kernel = kGemmKernel, p.height = t.height, p.width = t.width;
  }
  for (const Decode& d : kDecodes) {
    const double rounds = std::ceil(units(d.height) * (double)((blocks + d.per - 1) / d.per) / 256.0);
    // the waves of a workgroup split the columns; many workgroups keep a compute unit busy by themselves
    const int waves = (int)std::min<int64_t>(rounds > 5 ? 2 : rounds > 2 ? 4 : 8, chunks);
    const int shares = (d.per * (d.height / 16) + waves - 1) / waves;
    const double us =
        kDecodeStart + rounds * ((double)chunks * (rounds > 1 ? d.more : d.first) + kDecodeEnd) + kDecodeBlock * shares;
    if (us < best) best = us, p.kernel = kMidKernel, p.height = d.height, p.per = d.per, p.threads = 64 * waves;
  }
  // Up to four slots in one launch with the quantiser, which every workgroup (a row block) then does for itself: where
  // the rows times the matrices' tiles, the work that repeats, are few and so are the rows' codes.  294 shapes with 200
  // to 30000 tiles: the choice takes 0.5 % longer than the faster way on average.  bf16 x, one launch and two: 1 x 6912 x
  // 2560 4.9 and 5.9 us, 4 x 6912 x 2560 6.0 and 6.3, 1 x 2560 x 6912 5.0 and 6.8, 4 x 2560 x 6912 6.6 and 7.5, 4 x 4096 x
  // 4096 5.6 and 6.5, 2 of 16 experts 6912 x 2560 6.6 and 7.1; 4 x 14336 x 2560 12.1 and 7.1, 1 x 28672 x 8192 26 and 15.
  if (src && T <= 4 && K % 8 == 0 && T * blocks <= 18000 / chunks && T * chunks <= kFewChunks) {
    const double rows = E ? std::round((double)T / some) : (double)T;
    const int64_t wanted = (int64_t)std::ceil((double)chunks * rows / 3.5);
    const int waves = (int)std::min(std::min<int64_t>(16, chunks), wanted);
    p.kernel = kFewKernel, p.height = 16, p.per = 1, p.quantizes = true;
    p.threads = 64 * waves;
  }
  if (p.kernel != kGemmKernel) p.width = 16 * p.per;
  p.groups = (N + p.width - 1) / p.width * (E ? most_units(E, T, p.height) : (T + p.height - 1) / p.height);
  return p;
}

hipError_t launch_experts(const ExpertsPlan& p, const Groups& g, const void* X, int src, const int8_t* Xq,
                          const float* absmax, const Epilogue& ep, hipStream_t s) {
  if (p.kernel == kGemmKernel) return launch_experts_gemm(p, g, Xq, absmax, ep, s);
  if (p.kernel == kMidKernel) return launch_experts_mid(p, g, Xq, absmax, ep, s);
  return launch_experts_few(p, g, X, src, ep, s);
}

hipError_t launch_combine(const Groups& g, const float* H, const int32_t* slots, const float* weights, int64_t M, int k,
                          const Epilogue& ep, hipStream_t s) {
  const int64_t quads = (g.N + 3) / 4;
  const int64_t groups = std::min((M * quads + 255) / 256, kCombineGroups);
  k_combine<<<dim3((unsigned)groups), 256, 0, s>>>(g, H, slots, weights, M, k, quads, ep);
  return hipGetLastError();
}

}  // namespace bl
