// MXFP4 product for many tokens: Y[M][N] = sum_k Xv[m][k] Wv[n][k], both matrices as codes and
// scales in the layout of mxfp4.h, on the scaled matrix instructions (16x16x128, 4-bit operands).
//
// At 4 bits the matrix cores outrun the operands: a 16x16x128 step takes a wave 16 cycles and eats
// 2 KiB, so what decides is how often a loaded byte is used.  Hence output tiles of 256 x 256 by
// four waves of 128 x 128 each (64 matrix instructions per 16 KiB of fragments; 256 accumulator
// registers, one wave per SIMD), or 128 x 128 by four waves of 64 x 64 where the large tiles would
// leave compute units idle.
//   * The tile layout is the operand layout, so a 1 KiB tile goes from global memory straight into
//     LDS (direct loads, no registers) and a fragment is one conflict-free 16-byte LDS read per
//     lane.  Words of scales take the same way, once per four steps.
//   * The reads of a step's fragments are spread over the matrix instructions of the step before:
//     issued in one go they fill the LDS queue, and the four waves wait for one another.
//   * Ring of four 128-column stages.  Step s: wait until stage s + 1 has landed (everybody's, by a
//     barrier), issue the loads of stage s + 4 into the slot of stage s (its fragments were read in
//     step s - 1 and the barrier waits for them), read the fragments of step s + 1, and run the
//     matrix instructions of step s on fragments that are already there: with one wave per SIMD
//     nothing else hides the LDS latency.
//   * The direct loads are written in inline assembly (they have no output registers): for the
//     builtin the compiler would wait for every load in flight before any LDS read, as it cannot
//     tell which slot a load writes.  All ordering of loads against reads is by ring_wait below,
//     whose memory clobber keeps LDS reads on their side of it.
//   * Tile order: consecutive workgroups go to different XCDs, so each XCD gets a contiguous run of
//     tiles, tokens fastest, which shares weight rows in its L2.
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

// Direct loads of 1 KiB each from base[0 .. 3] (16 bytes per lane at `off`) to consecutive KiB of
// LDS from byte address `lds`.  The wait states: M0 and the bases may have been written just before.
__device__ __forceinline__ void load4_lds(const uint8_t* const (&base)[4], uint32_t off, uint32_t lds) {
  asm volatile(
      "s_nop 4\n\t"
      "s_mov_b32 m0, %5\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %4, %0\n\t"
      "s_add_u32 m0, m0, 0x400\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %4, %1\n\t"
      "s_add_u32 m0, m0, 0x400\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %4, %2\n\t"
      "s_add_u32 m0, m0, 0x400\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %4, %3"
      ::"s"(base[0]), "s"(base[1]), "s"(base[2]), "s"(base[3]), "v"(off), "s"(lds)
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

// Four waves in 2 x 2, each with kB x kB tiles of 16 x 16: output tiles of 32 kB x 32 kB.
template <int kB, typename TY>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(kB == 8 ? 1 : 2, kB == 8 ? 1 : 2))) void k_mx_gemm(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, const uint8_t* __restrict__ xcodes,
    const uint8_t* __restrict__ xscales, int64_t M, int64_t N, int tiles, int groups, int nblocks, int xblocks,
    int tiles_m, int total, TY* __restrict__ Y) {
  constexpr int kSide = 2 * kB;                  // row blocks of each matrix in a stage
  constexpr int kStage = 2 * kSide * 1024;       // bytes: weights, then tokens
  constexpr int kLoads = kSide / 2;              // direct loads per wave and stage
  constexpr int kScaleLoads = kSide * 512 / 4096;  // and per wave and four stages, of scales
  static_assert(kLoads % 4 == 0 && kScaleLoads >= 1, "whole batches of direct loads");
  extern __shared__ uint8_t lds[];               // four stages, then 2 kSide x 256 bytes of scales
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)lds;

  // tile of this workgroup: contiguous runs per XCD
  int id = blockIdx.x;
  {
    const int q = total / 8, r = total % 8, x = id % 8;
    id = x * q + min(x, r) + id / 8;
  }
  const int tm = id % tiles_m, tn = id / tiles_m;

  // this wave's direct loads: row blocks kLoads * wave .. of the stage (weights, then tokens)
  const uint8_t* src[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int t = kLoads * wave + j;
    const int64_t rb = t < kSide ? min(tn * kSide + t, nblocks - 1) : min(tm * kSide + t - kSide, xblocks - 1);
    src[j] = uniform_ptr((t < kSide ? codes : xcodes) + rb * tiles * kMxTileBytes);
  }
  const uint8_t* ssrc[kScaleLoads];
#pragma unroll
  for (int j = 0; j < kScaleLoads; ++j) {
    const int t = 4 * (kScaleLoads * wave + j) + (lane >> 4);  // four row blocks to a load
    const int64_t rb = t < kSide ? min(tn * kSide + t, nblocks - 1) : min(tm * kSide + t - kSide, xblocks - 1);
    ssrc[j] = (t < kSide ? scales : xscales) + rb * groups * 256 + 16 * (lane & 15);
  }
  auto issue = [&](int c, int slot, bool with_scales) {
#pragma unroll
    for (int j = 0; j < kLoads; j += 4) {
      const uint8_t* b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = src[j + i] + (int64_t)c * kMxTileBytes;
      load4_lds(b, 16 * lane, lds0 + slot * kStage + (kLoads * wave + j) * 1024);
    }
    if (with_scales) {
#pragma unroll
      for (int j = 0; j < kScaleLoads; ++j)
        load1_lds(ssrc[j] + (int64_t)(c >> 2) * 256, lds0 + 4 * kStage + (kScaleLoads * wave + j) * 1024);
    }
  };

  // fragments of 32 rows x 64 columns: two tiles' rows, half h of their columns
  constexpr int kT = kB / 2;
  v16f acc[kT][kT];
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  v4i fa[2][2][kT], fb[2][2][kT];
  int sa[2][2][kT], sb[2][2][kT];
  const int tile = (lane >> 4) & 1, slot = 16 * (lane >> 5) + (lane & 15);  // of a fragment, this lane's
  // The reads of a step, one at a time so that they can be spread over its matrix instructions:
  // 4 kT fragments, then (with scales) as many words of scales; both matrices in turn, first half
  // first.
  auto read_one = [&](auto rr, int ring, v4i (&a)[2][kT], v4i (&b)[2][kT], int (&wa)[2][kT], int (&wb)[2][kT]) {
    constexpr int r = rr, f = r % (4 * kT), h = f / (2 * kT), i = f % (2 * kT) / 2;
    constexpr int rb = 2 * i;
    const int base = f % 2 ? kSide + kB * wm : kB * wn;
    if constexpr (r < 4 * kT) {
      const v4i v = *reinterpret_cast<const v4i*>(lds + ring * kStage + (base + rb + tile) * 1024 + 16 * slot + 512 * h);
      if constexpr (f % 2)
        b[h][i] = v;
      else
        a[h][i] = v;
    } else {
      const int v = *reinterpret_cast<const int*>(lds + 4 * kStage + (base + rb + tile) * 256 + 4 * slot + 128 * h);
      if constexpr (f % 2)
        wb[h][i] = v;
      else
        wa[h][i] = v;
    }
  };

  // loads per stage: kLoads, and the scales' with every fourth (stage 0, 4, ...)
  constexpr int L = kLoads, S = kScaleLoads;
  const int last = tiles - 1;
  issue(0, 0, true);
  if (last >= 1) issue(1, 1, false);
  if (last >= 2) issue(2, 2, false);
  if (last >= 3) {
    issue(3, 3, false);
    ring_wait<3 * L>();
  } else {
    ring_wait<0>();
  }
  static_for<8 * kT>([&](auto r) { read_one(r, 0, fa[0], fb[0], sa[0], sb[0]); });

  for (int c0 = 0; c0 < tiles; c0 += 8) {
    bool done = false;
    static_for<8>([&](auto tt) {
      constexpr int u = tt, t = u % 4, cur = u % 2, g = u / 4;  // step, its byte of the scales, buffers
      const int c = c0 + u;
      if (done || c >= tiles) {
        done = true;
        return;
      }
      // stage c + 1 has landed where at most the loads of c + 2 and c + 3 are in flight
      if (c + 3 <= last)
        ring_wait<2 * L + ((t == 1 || t == 2) ? S : 0)>();
      else
        ring_wait<0>();
      // 2 kT batches of kT matrix instructions; the reads of the next step go in front of all but the
      // last two, whose time covers the latency of the last read, and the direct loads after the
      // first.  (The reads of the step after the last fetch what is in LDS, for nothing.)
      constexpr int kReads = t == 3 ? 8 * kT : 4 * kT, kBatch = (kReads + 2 * kT - 3) / (2 * kT - 2);
      static_for<2 * kT>([&](auto bb) {
        constexpr int h = bb / kT, i = bb % kT;
        static_for<kBatch>([&](auto rr) {
          if constexpr (bb * kBatch + rr < kReads)
            read_one(std::integral_constant<int, bb * kBatch + rr>{}, (t + 1) % 4, fa[1 - cur], fb[1 - cur], sa[1 - g],
                     sb[1 - g]);
        });
#pragma unroll
        for (int j = 0; j < kT; ++j)
          acc[i][j] = mx_mfma32<t, t>(fa[cur][h][i], fb[cur][h][j], acc[i][j], sa[g][h][i], sb[g][h][j]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (bb == 0) {
          if (c + 4 <= last) issue(c + 4, t, t == 0);
        }
      });
    });
  }

  // Each wave turns its accumulators (lane l of a 32 x 32 tile: token l % 32, four times four
  // consecutive outputs) into whole rows through its quarter of the ring, 32 tokens at a time.  The
  // row stride puts the 32 tokens of a write on different banks.
  constexpr int kRow = 16 * kB * sizeof(TY) + (sizeof(TY) == 4 ? 16 : 8);  // bytes
  constexpr int kPer = 16 / sizeof(TY);                                    // outputs of a 16-byte piece
  constexpr int kPieces = 16 * kB / kPer;                                  // pieces of a row
  static_assert(32 * kRow <= kStage, "a slab fits the wave's quarter");
  ring_wait<0>();  // the other waves have read their last fragments
  uint8_t* slab = lds + wave * kStage;
#pragma unroll
  for (int j = 0; j < kT; ++j) {
#pragma unroll
    for (int i = 0; i < kT; ++i) {
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
    const int64_t m0 = ((int64_t)tm * kSide + kB * wm + 2 * j) * 16;
    const int64_t n0 = ((int64_t)tn * kSide + kB * wn) * 16;
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
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next slab is written
  }
}

template <int kB, typename TY>
hipError_t launch(const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes, const uint8_t* xscales,
                  int64_t M, int64_t N, int64_t K, void* Y, hipStream_t s) {
  const MxGemmPlan p = plan_mx_gemm(M, N, K);
  constexpr int lds = 4 * 4 * kB * 1024 + 4 * kB * 256;
  const void* fn = reinterpret_cast<const void*>(&k_mx_gemm<kB, TY>);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  k_mx_gemm<kB, TY><<<dim3((unsigned)(p.tiles_m * p.tiles_n)), 256, lds, s>>>(
      codes, scales, xcodes, xscales, M, N, (int)mx_tiles(K), (int)mx_groups(K), (int)mx_row_blocks(N),
      (int)mx_row_blocks(M), (int)p.tiles_m, (int)(p.tiles_m * p.tiles_n), static_cast<TY*>(Y));
  return hipGetLastError();
}

}  // namespace

MxGemmPlan plan_mx_gemm(int64_t M, int64_t N, int64_t K) {
  MxGemmPlan p;
  auto tiles = [&](int64_t side) { return ((M + side - 1) / side) * ((N + side - 1) / side); };
  p.side = tiles(256) >= 128 ? 256 : 128;
  p.tiles_m = (M + p.side - 1) / p.side;
  p.tiles_n = (N + p.side - 1) / p.side;
  return p;
}

hipError_t launch_mx_gemm(const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                          const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, int ybf16,
                          hipStream_t s) {
  const bool big = plan_mx_gemm(M, N, K).side == 256;
  if (ybf16)
    return big ? launch<8, uint16_t>(codes, scales, xcodes, xscales, M, N, K, Y, s)
               : launch<4, uint16_t>(codes, scales, xcodes, xscales, M, N, K, Y, s);
  return big ? launch<8, float>(codes, scales, xcodes, xscales, M, N, K, Y, s)
             : launch<4, float>(codes, scales, xcodes, xscales, M, N, K, Y, s);
}

}  // namespace bl
