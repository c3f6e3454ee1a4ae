// MXFP4 product for many tokens: Y[M][N] = sum_k Xv[m][k] Wv[n][k], both matrices as codes and
// scales in the layout of mxfp4.h, on the scaled matrix instructions (32x32x64, 4-bit operands).
//
// At 4 bits the matrix cores outrun the operands: a 32x32x64 step takes 32 cycles and eats 2 KiB, so
// what decides is how often a loaded byte is used and what else runs meanwhile.  Output tiles of 128
// tokens x 256 outputs by four waves of 64 x 128 (or 64 x 64, for 128 x 128, where the large tiles
// would leave compute units idle), sized so that two workgroups share a compute unit: one's first
// loads and output stores run under the other's matrix instructions.  Measured: tiles of 256 x 256
// with one workgroup to a unit use each byte more often, but load, compute and store in turn (2048 x
// 28672 x 8192 to bf16 with the quantiser 273 us, against 250; 8192^3 to bf16 283 us against 270,
// 4.08 PFLOP/s).  What bounds the large shapes now: with all-zero operands a 256 x 256 x 128 step of a
// compute unit took 0.71 us, with random ones 0.92 - 1.0 (0.43 at the nominal clock): power, then LDS
// (1150 of its cycles to 1024 of the matrix cores').  2048 x 6912 x 2560 to fp32, 27.2 us: 216 tiles of
// 256 x 256 worth of work on 256 compute units, and 57 MB of output.  Output rows are stored past the
// caches: 26.4 us against 30.3 there.
//   * 32x32x64 instructions: with the 16x16x128 form the waves cannot issue fast enough (5.4 against
//     9.6 PFLOP/s from registers, one wave per SIMD).  On random data power holds both back.
//   * The tile layout is the operand layout, so a 1 KiB tile goes from global memory straight into
//     LDS (direct loads, no registers) and a fragment is one conflict-free 16-byte LDS read per
//     lane.  Words of scales take the same way, once per four steps.
//   * Ring of three or four 128-column stages, worked on by halves of 64 columns: a half's matrix
//     instructions run on fragments already in registers, with the reads of the next half's spread
//     between them (in one go they fill the LDS queue, and the waves wait for one another).  In the
//     middle of a step the workgroup waits until the next stage has landed; by then every wave has
//     read the whole of this one, and the loads of the stage after the ring go into its slot.
//   * The direct loads are written in inline assembly (they have no output registers): for the
//     builtin the compiler would wait for every load in flight before any LDS read, as it cannot
//     tell which slot a load writes.  All ordering of loads against reads is by ring_wait below,
//     whose memory clobber keeps LDS reads on their side of it.
//   * Tile order: consecutive workgroups go to different XCDs, so each XCD gets a contiguous run of
//     tiles.  Where they do not all run at once, the run goes down bands of eight token tiles, so that
//     the 64 tiles at work on an XCD share eight tiles of each matrix rather than read all tokens
//     (8192^3 to bf16 271 us with tokens fastest, 263 so; 2048 x 8192 x 8192 71.8 and 69.0).
#include "mxfp4.h"

#include <algorithm>

namespace bl {
namespace {

// Wait until at most n direct loads of this wave are in flight and its LDS reads have returned,
// then for the other waves.
template <int n>
__device__ __forceinline__ void ring_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(n) : "memory");
}

// Two direct loads of 1 KiB (16 bytes per lane at `off`) from a and b to consecutive KiB of LDS from
// byte address `lds`.  The wait states: M0 and the bases may have been written just before.  Nothing else
// in these kernels uses M0 (which cannot be named as clobbered).
__device__ __forceinline__ void load2_lds(const uint8_t* a, const uint8_t* b, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_nop 4\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %2, %0\n\t"
      "s_add_u32 m0, m0, 0x400\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %2, %1"
      ::"s"(a), "s"(b), "v"(off), "s"(lds)
      : "memory", "scc");
}
// One direct load of 1 KiB, each lane's 16 bytes from its own address.
__device__ __forceinline__ void load1_lds(const uint8_t* p, uint32_t lds) {
  asm volatile(
      "s_nop 4\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, off"
      ::"v"(p), "s"(lds)
      : "memory");
}

template <typename T>
__device__ __forceinline__ T* uniform_ptr(T* p) {
  const uint64_t v = (uint64_t)p;
  return (T*)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
              (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

constexpr int kWN = 2, kWM = 2;  // waves of a workgroup along the outputs and along the tokens

// Each wave has kN x kM blocks of 16 weight rows and 16 tokens: output tiles of 16 kWM kM tokens x 16
// kWN kN outputs.  kR stages of 128 columns in the ring.  kKS 2: two groups of such waves, each with a
// ring of its own, take half of the columns each (in whole groups of four stages, the first group's no
// fewer) and add their sums through LDS; both go through the same number of barriers.
template <int kN, int kM, int kR, int kKS, typename TY>
__global__ __launch_bounds__(64 * kWN * kWM * kKS) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_mx_gemm(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, const uint8_t* __restrict__ xcodes,
    const uint8_t* __restrict__ xscales, int64_t M, int64_t N, int tiles, int groups, int nblocks, int xblocks,
    int tiles_m, int tiles_n, int band, TY* __restrict__ Y) {
  constexpr int W = kWN * kWM;
  constexpr int BN = kWN * kN, BM = kWM * kM;     // row blocks of a stage: weights, then tokens
  constexpr int kBlocks = BN + BM;
  constexpr int kStage = kBlocks * 1024;          // bytes
  constexpr int L = kBlocks / W;                  // direct loads per wave and stage
  constexpr int S = (kBlocks / 4 + W - 1) / W;    // and per wave and four stages, of scales
  constexpr int TN = kN / 2, TM = kM / 2;         // 32-row tiles of a wave
  constexpr int kGroupLds = kR * kStage + kBlocks * 256;  // a ring and its scales
  static_assert(L % 2 == 0, "direct loads come in pairs");
  static_assert(kKS == 1 || (kKS == 2 && TM == 2), "the two groups keep one of two token tiles each");
  extern __shared__ uint8_t lds_all[];            // per group a ring, then kBlocks x 256 bytes of scales
  const int lane = threadIdx.x & 63, wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = wave_all / W, wave = wave_all % W;
  const int wn = wave % kWN, wm = wave / kWN;
  uint8_t* lds = lds_all + kg * kGroupLds;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)lds;
  // this group's stages: `count` from stage `first`; `steps` for both
  const int steps = kKS == 1 ? tiles : min(tiles, (tiles + 7) / 8 * 4);
  const int first = kg * steps, count = kg == 0 ? steps : tiles - first;

  // tile of this workgroup: contiguous runs per XCD
  int id = blockIdx.x;
  {
    const int total = tiles_m * tiles_n;
    const int q = total / 8, r = total % 8, x = id % 8;
    id = x * q + min(x, r) + id / 8;
  }
  const int b = id / (band * tiles_n), in_band = id - b * band * tiles_n;
  const int high = min(band, tiles_m - b * band);  // token tiles of this band
  const int tn = in_band / high, tm = b * band + in_band - tn * high;

  // row block t of a stage (past the last: the last again, not stored)
  auto block = [&](int t, const uint8_t* w, const uint8_t* x, int64_t bytes) {
    return t < BN ? w + min(tn * BN + t, nblocks - 1) * bytes : x + min(tm * BM + t - BN, xblocks - 1) * bytes;
  };
  // this wave's direct loads: blocks L wave .. of the stage, and of the scales KiB S wave .. (four
  // blocks each; waves past the last repeat it, so that all have the same number in flight)
  const uint8_t* src[L];
#pragma unroll
  for (int j = 0; j < L; ++j)
    src[j] = uniform_ptr(block(L * wave + j, codes, xcodes, (int64_t)tiles * kMxTileBytes) +
                         (int64_t)first * kMxTileBytes);
  const uint8_t* ssrc[S];
  int sdst[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    sdst[j] = min(S * wave + j, kBlocks / 4 - 1);
    ssrc[j] = block(4 * sdst[j] + (lane >> 4), scales, xscales, (int64_t)groups * 256) + (int64_t)(first >> 2) * 256 +
              16 * (lane & 15);
  }
  auto issue = [&](int c, int slot, bool with_scales) {
#pragma unroll
    for (int j = 0; j < L; j += 2)
      load2_lds(src[j] + (int64_t)c * kMxTileBytes, src[j + 1] + (int64_t)c * kMxTileBytes, 16 * lane,
                lds0 + slot * kStage + (L * wave + j) * 1024);
    if (with_scales) {
#pragma unroll
      for (int j = 0; j < S; ++j)
        load1_lds(ssrc[j] + (int64_t)(c >> 2) * 256, lds0 + kR * kStage + sdst[j] * 1024);
    }
  };

  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  // fragments of 32 rows x 64 columns (two blocks' rows, half h of their columns) of this half step
  // and of the next, and the words of scales of this group of four steps and of the next
  v4i fa[2][TN], fb[2][TM];
  int sa[2][2][TN], sb[2][2][TM];
  const uint8_t* lane_codes = lds + ((lane >> 4) & 1) * 1024 + 16 * (16 * (lane >> 5) + (lane & 15));
  const uint8_t* lane_scales = lds + kR * kStage + ((lane >> 4) & 1) * 256 + 4 * (16 * (lane >> 5) + (lane & 15));
  // the reads of a half step, one at a time so that they can be spread over its matrix
  // instructions: TN + TM fragments of half h, and with scales the words of both halves
  auto read_one = [&](auto rr, int slot, auto hh, v4i (&a)[TN], v4i (&b)[TM], int (&wa)[2][TN], int (&wb)[2][TM]) {
    constexpr int r = rr, h = hh;
    if constexpr (r < TN)
      a[r] = *reinterpret_cast<const v4i*>(lane_codes + slot * kStage + (kN * wn + 2 * r) * 1024 + 512 * h);
    else if constexpr (r < TN + TM)
      b[r - TN] =
          *reinterpret_cast<const v4i*>(lane_codes + slot * kStage + (BN + kM * wm + 2 * (r - TN)) * 1024 + 512 * h);
    else if constexpr (r < 3 * TN + TM)
      wa[(r - TN - TM) / TN][(r - TN - TM) % TN] = *reinterpret_cast<const int*>(
          lane_scales + (kN * wn + 2 * ((r - TN - TM) % TN)) * 256 + 128 * ((r - TN - TM) / TN));
    else
      wb[(r - 3 * TN - TM) / TM][(r - 3 * TN - TM) % TM] = *reinterpret_cast<const int*>(
          lane_scales + (BN + kM * wm + 2 * ((r - 3 * TN - TM) % TM)) * 256 + 128 * ((r - 3 * TN - TM) / TM));
  };
  constexpr int kFrags = TN + TM, kAll = 3 * kFrags;
  const std::integral_constant<int, 0> half0;
  const std::integral_constant<int, 1> half1;

  const int last = count - 1;
#pragma unroll
  for (int c = 0; c < kR; ++c)
    if (c <= last) issue(c, c, c == 0);
  if (last >= kR - 1)
    ring_wait<(kR - 1) * L>();
  else
    ring_wait<0>();
  static_for<kAll>([&](auto r) { read_one(r, 0, half0, fa[0], fb[0], sa[0], sb[0]); });

  int slot = 0;
  for (int c0 = 0; c0 < steps; c0 += 8) {
    bool done = false;
    static_for<8>([&](auto tt) {
      constexpr int u = tt, t = u % 4, g = u / 4;  // step, its byte of the scales, buffer of their words
      const int c = c0 + u;
      if (done || c >= steps) {
        done = true;
        return;
      }
      const bool mine = kKS == 1 || c < count;
      // Half a step: TN batches of TM matrix instructions, with the reads of the next half in front
      // of all but the last, whose time (and the barrier's) covers the last read's latency.
      auto half = [&](auto hh, auto reads, int rslot) {
        constexpr int h = hh, kReads = decltype(reads)::value, kBatch = (kReads + TN - 2) / (TN - 1);
        static_for<TN>([&](auto bb) {
          constexpr int i = bb;
          static_for<kBatch>([&](auto rr) {
            if constexpr (i * kBatch + rr < kReads)
              read_one(std::integral_constant<int, i * kBatch + rr>{}, rslot, std::integral_constant<int, 1 - h>{},
                       fa[1 - h], fb[1 - h], sa[1 - g], sb[1 - g]);
          });
#pragma unroll
          for (int j = 0; j < TM; ++j)
            acc[i][j] = mx_mfma32<t, t>(fa[h][i], fb[h][j], acc[i][j], sa[g][h][i], sb[g][h][j]);
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      if (mine) half(half0, std::integral_constant<int, kFrags>{}, slot);
      // stage c + 1 has landed where at most the loads of c + 2 .. c + kR - 1 are in flight, and stage
      // c has been read by every wave: its slot takes stage c + kR
      if (c + kR - 1 <= last)
        ring_wait<(kR - 2) * L + ((t == 2 || (kR == 4 && t == 1)) ? S : 0)>();
      else
        ring_wait<0>();
      const int next = slot + 1 == kR ? 0 : slot + 1;
      if (c + kR <= last) issue(c + kR, slot, (t + kR) % 4 == 0);
      // (the reads of the step after the last fetch what is in LDS, for nothing)
      if (mine) half(half1, std::integral_constant<int, t == 3 ? kAll : kFrags>{}, next);
      slot = next;
    });
  }

  // Each wave turns its accumulators (lane l of a 32 x 32 tile: token l % 32, four times four
  // consecutive outputs) into whole rows through its share of the ring, 32 tokens at a time.  The
  // row stride puts the 32 tokens of a write on different banks.
  constexpr int kRow = 16 * kN * sizeof(TY) + (sizeof(TY) == 4 ? 16 : 8);  // bytes
  constexpr int kPer = 16 / sizeof(TY);                                    // outputs of a 16-byte piece
  constexpr int kPieces = 16 * kN / kPer;                                  // pieces of a row
  constexpr int kXchg = kKS == 1 ? 0 : 2 * W * TN * 4096;  // the two groups' exchanged tiles
  static_assert(kXchg + kKS * W * 32 * kRow <= kKS * kGroupLds, "exchange and slabs fit the rings");
  const bool stream = whole_pieces(N);
  ring_wait<0>();  // the other waves have read their last fragments
  if constexpr (kKS == 2) {  // group kg keeps token tile kg of each wave and sends the other
    auto send = [&](auto jj) {
      constexpr int j = jj;
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<v4f*>(lds_all + ((wave_all * TN + i) * 4 + q) * 1024 + 16 * lane) =
              v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    };
    auto add = [&](auto jj) {
      constexpr int j = jj;
      const int from = (1 - kg) * W + wave;
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f v = *reinterpret_cast<const v4f*>(lds_all + ((from * TN + i) * 4 + q) * 1024 + 16 * lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
        }
    };
    if (kg == 0)
      send(half1);
    else
      send(half0);
    ring_wait<0>();
    if (kg == 0)
      add(half0);
    else
      add(half1);
  }
  uint8_t* slab = lds_all + kXchg + wave_all * (32 * kRow);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    if (kKS == 2 && j != kg) continue;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint8_t* at = slab + (lane & 31) * kRow + (32 * i + 8 * q + 4 * (lane >> 5)) * sizeof(TY);
        const v4f v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if constexpr (sizeof(TY) == 4) {
          *reinterpret_cast<v4f*>(at) = v;
        } else {
          uint2 w;
          w.x = bf16_pair(v[0], v[1]);
          w.y = bf16_pair(v[2], v[3]);
          *reinterpret_cast<uint2*>(at) = w;
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // a wave's own writes, read by its other lanes
    const int64_t m0 = ((int64_t)tm * BM + kM * wm + 2 * j) * 16;
    const int64_t n0 = ((int64_t)tn * BN + kN * wn) * 16;
    if (stream && m0 + 32 <= M && n0 + 16 * kN <= N) {  // a whole slab, past the caches
#pragma unroll 8
      for (int t = 0; t < 32 * kPieces / 64; ++t) {
        const int piece = 64 * t + lane, r = piece / kPieces, c = piece % kPieces;
        v4u v;
        __builtin_memcpy(&v, slab + r * kRow + 16 * c, 8);
        __builtin_memcpy(reinterpret_cast<char*>(&v) + 8, slab + r * kRow + 16 * c + 8, 8);
        __builtin_nontemporal_store(v, reinterpret_cast<v4u_unaligned*>(Y + (m0 + r) * N + n0 + kPer * c));
      }
    } else {
#pragma unroll 8
      for (int t = 0; t < 32 * kPieces / 64; ++t) {
        const int piece = 64 * t + lane, r = piece / kPieces, c = piece % kPieces;
        const int64_t m = m0 + r, n = n0 + kPer * c, left = m < M ? N - n : 0;
        TY* y = Y + m * N + n;
        TY v[kPer];
        __builtin_memcpy(v, slab + r * kRow + 16 * c, 8);
        __builtin_memcpy(v + kPer / 2, slab + r * kRow + 16 * c + 8, 8);
        if (left >= kPer) {
          __builtin_memcpy(y, v, 16);
        } else {
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (e < left) y[e] = v[e];
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next slab is written
  }
}

template <int kN, int kM, int kR, int kKS, typename TY>
hipError_t launch(const MxGemmPlan& p, const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                  const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, hipStream_t s) {
  constexpr int lds = kKS * (kWN * kN + kWM * kM) * (kR * 1024 + 256);
  const auto fn = &k_mx_gemm<kN, kM, kR, kKS, TY>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  fn<<<dim3((unsigned)(p.tiles_m * p.tiles_n)), 64 * kWN * kWM * kKS, lds, s>>>(
      codes, scales, xcodes, xscales, M, N, (int)mx_tiles(K), (int)mx_groups(K), (int)mx_row_blocks(N),
      (int)mx_row_blocks(M), (int)p.tiles_m, (int)p.tiles_n, (int)p.band, static_cast<TY*>(Y));
  return hipGetLastError();
}

}  // namespace

MxGemmPlan plan_mx_gemm(int64_t M, int64_t N, int64_t K) {
  MxGemmPlan p;
  auto tiles = [&](int64_t tm, int64_t tn) { return ((M + tm - 1) / tm) * ((N + tn - 1) / tn); };
  // 2048 x 6912 x 2560: 30.1 us with 256 x 128 tiles, 34.4 with 128 x 128; 512 x 8192 x 8192, where the
  // large tiles are 128 on 256 compute units: 37.7 and 27.8
  p.tile_m = 128;
  p.tile_n = tiles(128, 256) >= 256 ? 256 : 128;
  p.tiles_m = (M + p.tile_m - 1) / p.tile_m;
  p.tiles_n = (N + p.tile_n - 1) / p.tile_n;
  p.band = p.tiles_m * p.tiles_n > 512 ? 8 : p.tiles_m;
  // Few tiles leave one workgroup to a compute unit, whose four waves then wait for each step's reads
  // and barrier with nothing else to run (0.3 us a step, 0.11 of it the matrix instructions): two groups
  // of waves halve the steps.  One group and two, us: 600 x 128 x 8192 23.6 and 19.6, 600 x 2560 x 6912
  // 22.1 and 19.0, 1024 x 4096 x 4096 (256 tiles, 32 steps) 16.2 and 15.8.  Of more tiles two share a
  // unit (600 x 6912 x 2560, 270 tiles, 15.3 and 19.9), and short sums do not pay for the exchange
  // (1024^3, 8 steps, 6.3 and 7.0).
  p.ks = p.tile_n == 128 && p.tiles_m * p.tiles_n <= 256 && mx_tiles(K) >= 16 ? 2 : 1;
  return p;
}

hipError_t launch_mx_gemm(const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                          const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, int ybf16,
                          hipStream_t s) {
  const MxGemmPlan p = plan_mx_gemm(M, N, K);
  auto go = [&](auto yt) {
    using TY = decltype(yt);
    if (p.tile_n == 256) return launch<8, 4, 3, 1, TY>(p, codes, scales, xcodes, xscales, M, N, K, Y, s);
    if (p.ks == 2) return launch<4, 4, 4, 2, TY>(p, codes, scales, xcodes, xscales, M, N, K, Y, s);
    return launch<4, 4, 4, 1, TY>(p, codes, scales, xcodes, xscales, M, N, K, Y, s);
  };
  return ybf16 ? go(uint16_t{}) : go(float{});
}

}  // namespace bl
