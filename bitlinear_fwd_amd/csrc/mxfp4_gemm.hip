// MXFP4 product for many tokens: Y[M][N] = sum_k Xv[m][k] Wv[n][k], both matrices as codes and
// scales in the layout of mxfp4.h, on the scaled matrix instructions (32x32x64, 4-bit operands).
//
// At 4 bits the matrix cores outrun the operands: a 32x32x64 step takes 32 cycles and eats 2 KiB, so
// what decides is how often a loaded byte is used, which way it takes, and what else runs meanwhile.
// Output tiles of 128 tokens x 256 outputs (or 128, where the large tiles would leave compute units
// idle) by four waves, each with all tokens and a quarter of the outputs; two or three workgroups share
// a compute unit, and one's first loads and output stores run under the other's matrix instructions.
// Per step of 128 columns of two wide tiles a compute unit spends 1024 cycles on matrix instructions,
// 820 on loads (60 bytes a cycle, to LDS or to registers) and 770 on LDS (the tokens' 64 bytes a cycle
// in, 128 out).  Measured before: both matrices through LDS, waves of 64 tokens x 128 outputs, which is
// 1540 cycles of LDS: 2048 x 6912 x 2560 to fp32 27.4 us, 24.4 so; 1024 x 4096 x 4096 16.1 and 13.4;
// 8192^3 to bf16 262 and 245, 4.5 PFLOP/s (from run to run 24.4 to 26.6 and 245 to 259 us); and tiles of
// 256 x 256 with one workgroup to a unit (load, compute and store in turn) 283.  What bounds the large
// shapes now is power: with all-zero operands 8192^3 takes 163 us.  2048 x 6912 x 2560: 432 tiles on 512
// places, 57 MB of output; zeros 20.5 us.
//   * 32x32x64 instructions: with the 16x16x128 form the waves cannot issue fast enough (5.4 against
//     9.6 PFLOP/s from registers, one wave per SIMD).
//   * The tile layout is the operand layout.  A wave loads its own weights' fragments straight from
//     global memory into registers, four steps ahead (with two, 512 x 8192 x 8192 took 40.8 us, not
//     26.2).  The tokens' tiles, which all four waves need, go from global memory straight into LDS
//     (direct loads, no registers), and a fragment is one conflict-free 16-byte LDS read per lane.
//     Words of scales take that way too, once per four steps.
//   * Ring of four 128-column stages, worked on by halves of 64 columns: a half's matrix instructions
//     run on fragments already in registers, with the reads of the next half's spread between them.  In
//     the middle of a step the workgroup waits until the next stage has landed; by then every wave has
//     read the whole of this one, and the loads of the stage after the ring go into its slot.  A step
//     has no branches: around a conditional load or wait the compiler moves the matrix instructions of
//     the first half behind the barrier.
//   * The direct loads are written in inline assembly (they have no output registers): for the
//     builtin the compiler would wait for every load in flight before any LDS read, as it cannot
//     tell which slot a load writes.  All ordering of those loads against reads is by ring_wait below,
//     whose memory clobber keeps LDS reads on their side of it.
//   * Tile order: consecutive workgroups go to different XCDs, so each XCD gets a contiguous run of
//     tiles.  Where they do not all run at once, the run goes down bands of eight token tiles, so that
//     the 64 tiles at work on an XCD share eight tiles of each matrix rather than read all tokens
//     (8192^3 to bf16 271 us with tokens fastest, 263 so; 2048 x 8192 x 8192 71.8 and 69.0).
//   * Output rows are stored past the caches where they are whole 16-byte pieces (2048 x 6912 x 2560
//     30.3 us without, 26.4 so).  A width that is no multiple of 128 is slower than the next one that is:
//     65536 x 520 x 640 to fp32 54 us, x 640 36; x 300 37, x 384 25; x 1100 103, x 1152 65; 16384 x 48 x 640
//     7.8, x 128 5.8.  Its rows start inside cache lines, which whole slabs then store in parts, and the
//     slabs at its edge store piece by piece (which of the two costs more has not been measured).
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

constexpr int kWaves = 4;  // of a workgroup: each has all tokens of the tile and a quarter of its outputs
constexpr int TM = 4;      // tiles of 32 tokens
constexpr int kR = 4;      // stages of 128 columns of the tokens in the ring
constexpr int kRW = 4;     // stages of a wave's weights in its registers

// Each wave has TN x TM tiles of 32 weight rows and 32 tokens: output tiles of 128 tokens x 128 TN
// outputs.
template <int TN, typename TY>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_mx_gemm(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, const uint8_t* __restrict__ xcodes,
    const uint8_t* __restrict__ xscales, int64_t M, int64_t N, int tiles, int groups, int nblocks, int xblocks,
    int tiles_m, int tiles_n, int band, TY* __restrict__ Y) {
  constexpr int W = kWaves;
  constexpr int BN = 2 * TN * W, BM = 2 * TM;     // row blocks of a stage: weights, then tokens
  constexpr int kBlocks = BN + BM;
  constexpr int kStage = BM * 1024;               // bytes: the tokens' tiles
  constexpr int L = BM / W;                       // direct loads per wave and stage
  constexpr int S = (kBlocks / 4 + W - 1) / W;    // and per wave and four stages, of scales
  static_assert(L == 2, "direct loads come in pairs");
  static_assert(kR == 4 && kRW == 4, "the loop is unrolled by four stages");
  extern __shared__ uint8_t lds[];                // the ring, then kBlocks x 256 bytes of scales
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)lds;
  const int last = tiles - 1;

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
  const int64_t row_bytes = (int64_t)tiles * kMxTileBytes;
  // this wave's direct loads: two of the tokens' blocks, and of the scales KiB S wave .. (four blocks
  // each; waves past the last repeat it, so that all have the same number in flight)
  const uint8_t* src[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) src[j] = uniform_ptr(block(BN + 2 * wave + j, codes, xcodes, row_bytes));
  const uint8_t* ssrc[S];
  int sdst[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    sdst[j] = min(S * wave + j, kBlocks / 4 - 1);
    ssrc[j] = block(4 * sdst[j] + (lane >> 4), scales, xscales, (int64_t)groups * 256) + 16 * (lane & 15);
  }
  // (stages past the last: the last again, so that the same number is in flight at every step)
  auto issue = [&](int stage, int slot, bool with_scales) {
    const int c = min(stage, last);
    load2_lds(src[0] + (int64_t)c * kMxTileBytes, src[1] + (int64_t)c * kMxTileBytes, 16 * lane,
              lds0 + slot * kStage + 2 * wave * 1024);
    if (with_scales) {
#pragma unroll
      for (int j = 0; j < S; ++j)
        load1_lds(ssrc[j] + (int64_t)(c >> 2) * 256, lds0 + kR * kStage + sdst[j] * 1024);
    }
  };
  // this wave's weights: tile i's rows, lane's 16 bytes of a half stage
  const int half_lane = 16 * (16 * (lane >> 5) + (lane & 15));
  const int wb0 = min(tn * BN + 2 * TN * wave, nblocks - 1);
  uint32_t woff[TN];
#pragma unroll
  for (int i = 0; i < TN; ++i)
    woff[i] = (uint32_t)((min(tn * BN + 2 * TN * wave + 2 * i + ((lane >> 4) & 1), nblocks - 1) - wb0) * row_bytes) +
              half_lane;
  GlobalBytes wsrc = (GlobalBytes)uniform_ptr(codes + wb0 * row_bytes);
  // From here on the compiler may not assume that nothing writes what wsrc points to, so that its loads
  // stay between the same two of the assembly statements, whose waits count them.
  asm volatile("" : "+s"(wsrc));

  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  // fragments of 32 rows x 64 columns (two blocks' rows, half h of their columns): of the weights for
  // kRW stages, of the tokens for this half step and the next; and the words of scales of this group of
  // four steps
  v4i fa[kRW][2][TN], fb[2][TM];
  int sa[2][TN], sb[2][TM];
  auto load_w = [&](int c, int h, v4i (&w)[TN]) {
    const GlobalBytes p = wsrc + (int64_t)min(c, last) * kMxTileBytes + 512 * h;
#pragma unroll
    for (int i = 0; i < TN; ++i) w[i] = *reinterpret_cast<GlobalV4i>(p + woff[i]);
  };
  const uint8_t* lane_codes = lds + ((lane >> 4) & 1) * 1024 + half_lane;
  const uint8_t* lane_scales = lds + kR * kStage + ((lane >> 4) & 1) * 256 + half_lane / 4;
  // the reads of a half step, one at a time so that they can be spread over matrix instructions: TM
  // fragments of half h of a slot, and the words of scales of half sh
  auto read_one = [&](auto rr, int slot, auto hh, auto ss, v4i (&bf)[TM]) {
    constexpr int r = rr, h = hh, sh = ss;
    if constexpr (r < TM)
      bf[r] = *reinterpret_cast<const v4i*>(lane_codes + slot * kStage + 2 * r * 1024 + 512 * h);
    else if constexpr (r < TM + TN)
      sa[sh][r - TM] =
          *reinterpret_cast<const int*>(lane_scales + (2 * TN * wave + 2 * (r - TM)) * 256 + 128 * sh);
    else
      sb[sh][r - TM - TN] = *reinterpret_cast<const int*>(lane_scales + (BN + 2 * (r - TM - TN)) * 256 + 128 * sh);
  };
  constexpr int kAll = 2 * TM + TN;
  const std::integral_constant<int, 0> half0;
  const std::integral_constant<int, 1> half1;

#pragma unroll
  for (int c = 0; c < kR; ++c) issue(c, c, c == 0);
#pragma unroll
  for (int c = 0; c < kRW; ++c) {
    load_w(c, 0, fa[c][0]);
    load_w(c, 1, fa[c][1]);
  }
  ring_wait<2 * TN * kRW>();
  static_for<kAll>([&](auto r) { read_one(r, 0, half0, half0, fb[0]); });

  auto step = [&](auto tt, int c, auto in_loop) {
    constexpr int t = tt;  // the step's byte of the scales and its slots
    // Half a step: TN x TM matrix instructions on what is in registers, between them the reads of the
    // next half.  The words of scales of half h of four steps are read in the half before their first
    // use, after the last use of those before.
    auto half = [&](auto hh, auto reads, int rslot) {
      constexpr int h = hh, kReads = decltype(reads)::value, kInst = TN * TM;
      static_for<kInst>([&](auto mm) {
        constexpr int m = mm, i = m / TM, j = m % TM;
        static_for<kReads>([&](auto rr) {
          if constexpr (decltype(rr)::value * (kInst - 1) / kReads == m)
            read_one(rr, rslot, std::integral_constant<int, 1 - h>{}, std::integral_constant<int, 1 - h>{},
                     fb[1 - h]);
        });
        acc[i][j] = mx_mfma32<t, t>(fa[t][h][i], fb[h][j], acc[i][j], sa[h][i], sb[h][j]);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    half(half0, std::integral_constant<int, t == 0 ? kAll : TM>{}, t);
    // Stage c + 1 has landed where at most the loads of weights of three steps and the direct loads of
    // two are in flight, and stage c has been read by every wave: its slot takes stage c + kR.
    ring_wait<in_loop ? 3 * 2 * TN + 2 * L + (t == 1 || t == 2 ? S : 0) : 2 * L>();
    issue(c + kR, t, t == 0);
    load_w(c + kRW, 0, fa[t][0]);
    __builtin_amdgcn_sched_barrier(0);
    // (the reads of the step after the last fetch what is in LDS, for nothing)
    half(half1, std::integral_constant<int, t == 3 ? kAll : TM>{}, (t + 1) % kR);
    load_w(c + kRW, 1, fa[t][1]);
    __builtin_amdgcn_sched_barrier(0);
  };
  const std::integral_constant<int, 2> third;
  const std::integral_constant<int, 3> fourth;
  int c = 0;
  for (; c + 4 <= tiles; c += 4) {
    step(half0, c, std::true_type{});
    step(half1, c + 1, std::true_type{});
    step(third, c + 2, std::true_type{});
    step(fourth, c + 3, std::true_type{});
  }
  if (c < tiles) {
    step(half0, c, std::false_type{});
    if (c + 1 < tiles) {
      step(half1, c + 1, std::false_type{});
      if (c + 2 < tiles) step(third, c + 2, std::false_type{});
    }
  }

  // Each wave turns its accumulators (lane l of a 32 x 32 tile: token l % 32, four times four
  // consecutive outputs) into whole rows through its share of the ring, 32 tokens at a time.  The
  // row stride puts the 32 tokens of a write on different banks.
  constexpr int kRow = 32 * TN * sizeof(TY) + (sizeof(TY) == 4 ? 16 : 8);  // bytes
  constexpr int kPer = 16 / sizeof(TY);                                    // outputs of a 16-byte piece
  constexpr int kPieces = 32 * TN / kPer;                                  // pieces of a row
  const bool stream = whole_pieces(N);
  ring_wait<0>();  // no load is in flight, and the other waves have read their last fragments
  uint8_t* slab = lds + wave * (32 * kRow);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
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
    const int64_t m0 = ((int64_t)tm * BM + 2 * j) * 16;
    const int64_t n0 = ((int64_t)tn * BN + 2 * TN * wave) * 16;
    if (stream && m0 + 32 <= M && n0 + 32 * TN <= N) {  // a whole slab, past the caches
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

template <int TN, typename TY>
hipError_t launch(const MxGemmPlan& p, const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                  const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, hipStream_t s) {
  // the ring with its scales, then a slab of 32 rows per wave
  constexpr int ring = kR * 2 * TM * 1024 + (2 * TN * kWaves + 2 * TM) * 256;
  constexpr int slab = 32 * (32 * TN * (int)sizeof(TY) + (sizeof(TY) == 4 ? 16 : 8));
  constexpr int lds = std::max(ring, kWaves * slab);
  static_assert(lds <= 65536, "no attribute needed");
  k_mx_gemm<TN, TY><<<dim3((unsigned)(p.tiles_m * p.tiles_n)), 64 * kWaves, lds, s>>>(
      codes, scales, xcodes, xscales, M, N, (int)mx_tiles(K), (int)mx_groups(K), (int)mx_row_blocks(N),
      (int)mx_row_blocks(M), (int)p.tiles_m, (int)p.tiles_n, (int)p.band, static_cast<TY*>(Y));
  return hipGetLastError();
}

}  // namespace

MxGemmPlan plan_mx_gemm(int64_t M, int64_t N, int64_t K) {
  MxGemmPlan p;
  // A tile of 256 outputs uses its tokens' tiles more often, two of them or three of 128 share a compute
  // unit.  128 and 256 wide, us: 512 x 8192 x 8192 (256 tiles of 128) 26.2 and 33.0, 1024 x 6912 x 2560
  // (432) 14.3 and 15.7, 1024 x 8192 x 8192 (512) 45.9 and 38.4, 700 x 8192 x 8192 (384) 41.4 and 34.3,
  // 2048 x 6912 x 2560 (864) 27.6 and 25.0.  Not where half a tile of fewer than four lies past the last
  // column: 16384 x 128 x 2560 12.1 and 16.7, 65536 x 640 x 2560 67.9 and 73.7 (65536 x 256 x 2560 40.4 and
  // 34.7, 65536 x 1100 x 2560 189.6 and 180.9).  That rule goes by the number of columns alone and takes the
  // slower side where the last one is nearly empty or the rows are long: 65536 x 520 x 640 53.4 and 50.4,
  // 16384 x 520 x 640 18.5 and 15.9, 65536 x 520 x 8192 224 and 214, 16384 x 384 x 8192 40.7 and 38.5.
  const int64_t columns = (N + 127) / 128, t128 = ((M + 127) / 128) * columns;
  const bool many = t128 > 512 || (t128 > 256 && mx_tiles(K) >= 48), waste = columns % 2 == 1 && columns < 7;
  p.tile_m = 128;
  p.tile_n = many && !waste ? 256 : 128;
  p.tiles_m = (M + p.tile_m - 1) / p.tile_m;
  p.tiles_n = (N + p.tile_n - 1) / p.tile_n;
  p.band = p.tiles_m * p.tiles_n > 512 ? 8 : p.tiles_m;
  return p;
}

hipError_t launch_mx_gemm(const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                          const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, int ybf16,
                          hipStream_t s) {
  const MxGemmPlan p = plan_mx_gemm(M, N, K);
  auto go = [&](auto yt) {
    using TY = decltype(yt);
    return p.tile_n == 256 ? launch<2, TY>(p, codes, scales, xcodes, xscales, M, N, K, Y, s)
                           : launch<1, TY>(p, codes, scales, xcodes, xscales, M, N, K, Y, s);
  };
  return ybf16 ? go(uint16_t{}) : go(float{});
}

}  // namespace bl
