// Ternary products with an epilogue, plainly: a wave per 16 slots x 16 outputs, operands from global memory.
#include "experts.h"

#include <algorithm>
#include <cmath>

namespace bl {
namespace {

__global__ __launch_bounds__(256) void k_experts(Groups g, const int8_t* __restrict__ Xq,
                                                 const float* __restrict__ absmax, Epilogue ep, int chunks,
                                                 int64_t nblocks, int columns) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t nb = (int64_t)(blockIdx.x % columns) * 4 + wave;
  const Unit u = find_unit(g, 16, blockIdx.x / columns);
  if (u.lo >= u.hi || nb >= nblocks) return;
  const int slot = u.lo + r, row = slot < u.hi ? slot_row(g, slot) : -1;
  const int8_t* x = Xq + (int64_t)max(row, 0) * chunks * kTileCols + 64 * q;
  const uint4* w = reinterpret_cast<const uint4*>(g.packed + ((int64_t)u.e * nblocks + nb) * chunks * kTileBytes) + lane;
  v4i acc = {0, 0, 0, 0};
  for (int c = 0; c < chunks; ++c) {
    const uint4 t = w[(int64_t)c * 64];
    const uint32_t word[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4i xv = *reinterpret_cast<const v4i*>(x + (int64_t)c * kTileCols + 16 * i);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(decode16(word[i]), xv, acc, 0, 0, 0);
    }
  }
  if (row < 0) return;
  const int64_t n = nb * 16 + 4 * q, left = g.N - n;
  if (left > 0) finish4(ep, u.e, g.N, slot, n, (int)min(left, (int64_t)4), acc, token_scale(g.gamma[u.e], absmax[row]));
}

// One thread per four outputs of a token.
__global__ __launch_bounds__(256) void k_combine(Groups g, const float* __restrict__ H,
                                                 const int32_t* __restrict__ slots,
                                                 const float* __restrict__ weights, int64_t M, int k, int64_t quads,
                                                 Epilogue ep) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / quads, n = 4 * (i - m * quads);
  if (m >= M) return;
  const int left = (int)min(g.N - n, (int64_t)4);
  const int first = max(0, min(g.offsets[0], (int)g.T)), last = max(0, min(g.offsets[g.E], (int)g.T));
  v4f v = {0, 0, 0, 0};
  for (int j = 0; j < k; ++j) {
    const int s = slots[m * k + j];
    if (s < first || s >= last || slot_row(g, s) < 0) continue;
    const v4f h = load4(H, (int64_t)s * g.N + n, left, 0);
    const float w = weights[m * k + j];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf(w, h[q], v[q]);
  }
  if (ep.residual) v += load4(ep.residual, m * ep.ldr + n, left, ep.res_bf16);
  store4(ep.Y, m * ep.ldy + n, left, ep.y_bf16, v);
}

}  // namespace

// The GEMM's tile.  A unit of `height` slots by `width` outputs takes `first` us where each compute unit has at
// most one tile (a stage of 128 columns has its latency) and `more` us where several share it; `end` is what else a
// tile costs.  Fitted to 37 shapes from 64 to 65536 rows, 128 to 8192 outputs and 900 to 8192 columns.
namespace {
struct Tile {
  int height, width;
  double first, more, end;
};
constexpr Tile kTiles[] = {{128, 256, .63, .66, 1.5}, {96, 256, .49, .475, 1.5}, {64, 256, .40, .365, 1.2},
                           {64, 128, .255, .218, 1.0}, {32, 256, .31, .25, .9}, {32, 128, .225, .137, .9}};
}  // namespace

ExpertsPlan plan_experts(int64_t E, int64_t T, int64_t N, int64_t K, int src) {
  ExpertsPlan p;
  const int64_t groups = E ? std::min(E, T) : 1;  // that have slots, at most
  if (T > 16 * groups) {
    const double stages = (double)(k_pad(K) / 128), each = (double)T / groups;
    double best = 1e300;
    for (const Tile& t : kTiles) {
      // units of groups of different sizes end half full
      const double units = E ? groups * std::max(1.0, each / t.height + 0.5) : (double)((T + t.height - 1) / t.height);
      const double rounds = std::ceil(units * ((N + t.width - 1) / t.width) / 256.0);
      const double us = rounds > 1 ? rounds * (stages * t.more + t.end) : stages * t.first + t.end;
      if (us < best) best = us, p.height = t.height, p.width = t.width;
    }
    p.kernel = kGemmKernel;
    p.groups = (N + p.width - 1) / p.width * (E ? most_units(E, T, p.height) : (T + p.height - 1) / p.height);
    return p;
  }
  p.groups = (n_pad(N) / kTileRows + 3) / 4 * (E ? most_units(E, T, 16) : (T + 15) / 16);
  return p;
}

hipError_t launch_experts(const Groups& g, const void* X, int src, const int8_t* Xq, const float* absmax,
                          const Epilogue& ep, hipStream_t s) {
  const int chunks = (int)(k_pad(g.K) / kTileCols);
  const int64_t nblocks = n_pad(g.N) / kTileRows;
  const ExpertsPlan p = plan_experts(g.offsets ? g.E : 0, g.T, g.N, g.K, src);
  if (p.kernel == kGemmKernel) return launch_experts_gemm(p, g, Xq, absmax, ep, s);
  k_experts<<<dim3((unsigned)p.groups), p.threads, 0, s>>>(g, Xq, absmax, ep, chunks, nblocks, (int)((nblocks + 3) / 4));
  return hipGetLastError();
}

hipError_t launch_combine(const Groups& g, const float* H, const int32_t* slots, const float* weights, int64_t M, int k,
                          const Epilogue& ep, hipStream_t s) {
  const int64_t quads = (g.N + 3) / 4;
  k_combine<<<dim3((unsigned)((M * quads + 255) / 256)), 256, 0, s>>>(g, H, slots, weights, M, k, quads, ep);
  return hipGetLastError();
}

}  // namespace bl
