// Ternary products with an epilogue for many slots: int8 matrix instructions (16x16x64) on tiles of
// 32 TM slots x 128 TN outputs.
//
// A workgroup of four waves takes one tile; each wave has all its slots and a quarter of its outputs.
// A stage is 128 columns: the slots' codes (16 bytes a lane, rows gathered by address as they are loaded)
// and every wave's own packed weights go straight from global memory into a ring of stages in LDS.
//   * 16x16x64 instructions: with 32x32x32 the large shapes are bound by power (from registers alone, random
//     codes: 2770 against 4500 TOPS).
//   * The operands of a stage: in the packed layout lane (r, q) of 16 x 4 finds, in the 16-byte slot of row r
//     and columns 64 g .. 64 g + 63, the columns 16 i .. of its word i.  Half a chunk has two values of g, so
//     lanes q take slot g = q / 2 of them and words 2 (q % 2) and 2 (q % 2) + 1, one for each of two
//     instructions: 8 bytes of LDS a lane (any 32 lanes on all banks once), decoded with 9 operations for 16
//     weights.  The tokens' fragments take the same columns: 16-byte piece 2 q + i of the stage's row.
//   * A stage is worked on in four steps (instruction i, half of the slots).  A step's matrix instructions run on
//     operands that are in registers; between them the next step's fragments are read and weights decoded.
//   * Before a stage's last step the workgroup waits until the next stage has landed; by then every wave has
//     read the whole of this one, and the stage after the ring goes into its slot.
//   * The direct loads are written in inline assembly (they have no output registers): for the builtin
//     the compiler would wait for every load in flight before any LDS read, as it cannot tell which
//     slot a load writes.  ring_wait orders them against reads.
// Bound by power where sums are long (2048 x 8192 x 28672 to bf16 300 to 314 us, 3.1 POPS; 8192^3 352 us, and 289 us
// with all-zero operands); 2048 x 6912 x 2560 with SiLU 38.3 us, of which the first loads take 2, the sums 29 and the end
// 5: 432 tiles on 512 places, so that nothing runs under the end.  More than three stages in the ring made it slower (128
// x 256 tiles, one to a compute unit, 2560 columns: 13 us for the sums with three, 23 with four), and neither cache hints
// on the direct loads nor raised wave priority changed it.
#include "experts.h"

#include <algorithm>

namespace bl {
namespace {

// Wait until at most n direct loads of this wave are in flight and its LDS reads have returned, then for
// the other waves.
template <int n>
__device__ __forceinline__ void ring_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(n) : "memory");
}

// A direct load of 1 KiB: each lane's 16 bytes from its own address to LDS at byte address lds + 16 lane.
// Nothing else in this kernel uses M0 (which cannot be named as clobbered).
__device__ __forceinline__ void load_lds(const uint8_t* p, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, off"
      ::"v"(p), "s"(lds)
      : "memory");
}

// Four of the 16 codes of a packed word as bytes (decode16, one dword at a time).
template <int d>
__device__ __forceinline__ int decode4(uint32_t w) {
  if constexpr (d >= 2) w >>= 4;
  return (d & 1) == 0 ? (int)__builtin_amdgcn_perm(0u, 0x00FF0100u, w & 0x03030303u)
                      : (int)__builtin_amdgcn_perm(0x00000001u, 0x00008000u, w & 0x0C0C0C0Cu);
}

// Piece p (16 bytes) of row r lies in the row's slot p ^ row_swizzle(r).  A 16-byte read takes lanes 0-3, 12-15 and
// 20-27 (and so on) together: rows 0-3 and 12-15 at piece p with rows 4-11 at piece p ^ 2, which this puts on
// different banks.  With r / 2 % 8 itself half of them meet.
__device__ __forceinline__ int row_swizzle(int r) { return ((r >> 1) + 6) & 7; }


constexpr int kR = 3;  // stages in the ring

template <int TM, int TN>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_experts_gemm(
    Groups g, const int8_t* __restrict__ Xq, const float* __restrict__ absmax, Epilogue ep, int chunks, int nblocks,
    int tiles_n, int band) {
  constexpr int BM = 32 * TM, BN = 128 * TN;
  constexpr int kTokens = BM * 128;                 // bytes of a stage: the slots' codes,
  constexpr int kStage = kTokens + 4 * TN * 1024;   // then the waves' weights
  constexpr int kLoads = TM + TN;                   // direct loads of a wave and stage
  constexpr int kRow = 32 * TN * 4 + 16;            // bytes of a row of the output slab
  constexpr int kLds = std::max(kR * kStage, 4 * 32 * kRow);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)lds;

  // tile of this workgroup: a contiguous run of tiles for each XCD, in bands of `band` units that go down
  // the units first, so that the tiles at work share weights and slots in the XCD's cache
  int tn;
  Unit u;
  {
    const int units = count_units(g, BM, gridDim.x / tiles_n), total = units * tiles_n;
    if ((int)blockIdx.x >= total) return;
    const int q = total / 8, r = total % 8, x = blockIdx.x % 8;
    const int id = x * q + min(x, r) + blockIdx.x / 8;
    const int b = id / (band * tiles_n), in_band = id - b * band * tiles_n;
    const int high = min(band, units - b * band);
    tn = in_band / high;
    u = find_unit(g, BM, b * band + in_band - tn * high);
    if (u.lo >= u.hi) return;
  }
  const int stages = 2 * chunks;

  // This wave's loads.  Tokens: TM KiB of a stage, rows 8 (TM wave + j) + lane / 8.  Slots past the unit repeat its
  // last, slots without a row take row 0; neither is stored.
  const uint8_t* src[TM + TN];
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int r = 8 * (TM * wave + j) + (lane >> 3);
    const int row = max(slot_row(g, min(u.lo + r, u.hi - 1)), 0);
    src[j] = reinterpret_cast<const uint8_t*>(Xq) + (int64_t)row * chunks * kTileCols +
             16 * ((lane & 7) ^ row_swizzle(r));
  }
  // Weights: 32 rows (two row blocks) x 128 columns in a KiB; lane l has row l % 32, columns 64 (l / 32) ..
  // (blocks past the last repeat it; not stored)
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    const int nb = min((tn * BN + 32 * (TN * wave + i)) / 16 + ((lane >> 4) & 1), nblocks - 1);
    src[TM + i] = g.packed + ((int64_t)u.e * nblocks + nb) * chunks * kTileBytes + 16 * (16 * (lane >> 5) + (lane & 15));
  }
  // load l of the next stage into the slot at byte address `at` of the ring (stages past the last: the last again,
  // so that the same number is in flight)
  int next = 0;
  auto issue = [&](uint32_t at, auto ll) {
    constexpr int l = decltype(ll)::value;
    load_lds(src[l], lds0 + at + (l < TM ? (TM * wave + l) * 1024 : kTokens + (TN * wave + l - TM) * 1024));
    src[l] += next + 1 < stages ? (l < TM ? 128 : 512) : 0;
    if (l == kLoads - 1) ++next;
  };
  // the tokens' scales, and which of them there are, for the end
  float scale[TM];
  uint32_t live[TM];
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int slot = u.lo + 32 * j + (lane & 31), row = slot < u.hi ? slot_row(g, slot) : -1;
    live[j] = (uint32_t)__ballot(row >= 0);
    scale[j] = absmax[max(row, 0)];
  }

  constexpr int NB = 2 * TN, MB = 2 * TM;  // blocks of 16 outputs and of 16 slots of a wave
  v4i acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  // operands of a step and of the next (the weights': of an instruction), and this stage's packed weights
  v4i xf[2][TM], wf[2][NB];
  uint2 raw[NB];

  const int lr = lane & 15, lq = lane >> 4;
  uint32_t tok[2];  // this lane's token piece of either instruction
#pragma unroll
  for (int s = 0; s < 2; ++s) tok[s] = lr * 128 + 16 * ((2 * lq + s) ^ row_swizzle(lr));
  const uint32_t wlane = kTokens + TN * wave * 1024 + 16 * (32 * (lq >> 1) + lr) + 8 * (lq & 1);

  auto read_x = [&](uint32_t at, auto ss, auto jj, v4i (&x)[TM]) {  // fragment j of step s
    constexpr int s = decltype(ss)::value, j = decltype(jj)::value;
    x[j] = *reinterpret_cast<const v4i*>(lds + at + tok[s >> 1] + ((s & 1) * TM + j) * 2048);
  };
  auto read_w = [&](uint32_t at, auto ii) {
    constexpr int i = decltype(ii)::value;
    raw[i] = *reinterpret_cast<const uint2*>(lds + at + wlane + (i >> 1) * 1024 + (i & 1) * 256);
  };
  auto decode_part = [&](auto ss, auto part, v4i (&w)[NB]) {  // for instruction s
    constexpr int i = decltype(part)::value / 4, d = decltype(part)::value % 4;
    w[i][d] = decode4<d>(decltype(ss)::value == 0 ? raw[i].x : raw[i].y);
  };
  const std::integral_constant<int, 0> first;
  const std::integral_constant<int, 1> second;

#pragma unroll
  for (int c = 0; c < kR - 1; ++c) static_for<kLoads>([&](auto l) { issue(c * kStage, l); });
  ring_wait<(kR - 2) * kLoads>();
  static_for<NB>([&](auto i) { read_w(0, i); });
  static_for<TM>([&](auto j) { read_x(0, first, j, xf[0]); });
  static_for<4 * NB>([&](auto p) { decode_part(first, p, wf[0]); });

  // One stage, in slot t of the ring.  Step s: instruction s / 2 for half s % 2 of the slots.  Between the
  // instructions: the next step's token fragments, as early as can be; decoding (the second instruction's weights in
  // steps 0 and 1, the next stage's first ones in step 3); in step 0 the loads of the last stage of the ring, into
  // the slot that the stage before has left.
  uint32_t t = 0;
  for (int c = 0; c < stages; ++c) {
    const uint32_t nt = t == (kR - 1) * kStage ? 0 : t + kStage, last = t == 0 ? (kR - 1) * kStage : t - kStage;
    static_for<4>([&](auto ss) {
      constexpr int s = decltype(ss)::value, cur = s & 1, nxt = 1 - cur, ns = (s + 1) & 3;
      if constexpr (s == 3) ring_wait<(kR - 2) * kLoads>();
      constexpr int kInst = TM * NB, kL = s == 0 ? kLoads : 0, kW = s == 3 ? NB : 0;
      constexpr int kD = s == 3 ? 4 * NB : s < 2 ? 2 * NB : 0;
      constexpr int kReads = kW + TM, kD0 = s == 3 ? std::min(kReads, kInst / 3) : 0;  // decoding starts after kD0
      static_for<kInst>([&](auto mm) {
        // neighbours share an operand: fewer bits change
        constexpr int m = decltype(mm)::value, j = m / NB, i = j % 2 ? NB - 1 - m % NB : m % NB;
        acc[i][(s & 1) * TM + j] =
            __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[s >> 1][i], xf[cur][j], acc[i][(s & 1) * TM + j], 0, 0, 0);
        static_for<kReads>([&](auto rr) {
          constexpr int r = decltype(rr)::value;
          if constexpr (std::min(s == 3 ? r / 2 : r, kInst - 1) == m) {
            if constexpr (r < kW) read_w(nt, rr);
            else read_x(s == 3 ? nt : t, std::integral_constant<int, ns>{}, std::integral_constant<int, r - kW>{}, xf[nxt]);
          }
        });
        static_for<kL>([&](auto ll) {
          if constexpr (decltype(ll)::value * kInst / std::max(kL, 1) == m) issue(last, ll);
        });
        static_for<kD>([&](auto dd) {
          constexpr int d = decltype(dd)::value;
          if constexpr (kD0 + d * (kInst - kD0) / std::max(kD, 1) == m) {
            if constexpr (s == 3) decode_part(first, dd, wf[0]);
            else decode_part(second, std::integral_constant<int, d + 2 * NB * s>{}, wf[1]);
          }
        });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    t = nt;
  }

  // Epilogue.  Lane l of a 16 x 16 block has token l % 16 and outputs 4 (l / 16) ..; each wave turns its
  // accumulators into whole rows through its part of LDS, 32 tokens at a time, with the token's scale behind
  // its row.  The rest happens as the rows go out: a lane has the same columns of every row that it stores.
  ring_wait<0>();  // no load is in flight, and the other waves have read their last fragments
  uint8_t* slab = lds + wave * (32 * kRow);
  const float gamma = g.gamma[u.e];
  const int64_t n0 = (int64_t)tn * BN + 32 * TN * wave;
  auto rows_out = [&](auto kind) {
    constexpr bool bf16 = decltype(kind)::value;
    constexpr int per = bf16 ? 8 : 4, pieces = 32 * TN / per, rows = 64 / pieces;  // rows: of a wave's stores
    constexpr int H = per / 4;
    const bool whole = n0 + 32 * TN <= g.N;
    const int o = lane % pieces * per, left = (int)min(g.N - n0 - o, (int64_t)per);
    v4f b[per / 4];
#pragma unroll
    for (int h = 0; h < per / 4; ++h) {
      b[h] = v4f{0, 0, 0, 0};
      if (ep.bias && left > 4 * h) b[h] = load4(ep.bias, u.e * g.N + n0 + o + 4 * h, min(left - 4 * h, 4), 0);
    }
    // (a loop, of which only the writes to LDS are there TM times: code that runs once waits for its own
    // instructions, and with all of it TM times the end of a 128 x 256 tile took 6.7 us)
#pragma unroll 1
    for (int j = 0; j < TM; ++j) {
      const int slot0 = u.lo + 32 * j;
      if (slot0 >= u.hi) return;
      uint32_t there = 0;
      static_for<TM>([&](auto jj) {
        if (j != decltype(jj)::value) return;
        there = live[jj];
        if (lane < 32) *reinterpret_cast<float*>(slab + lane * kRow + 128 * TN) = token_scale(gamma, scale[jj]);
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<v4i*>(slab + (16 * h + lr) * kRow + 4 * (16 * i + 4 * lq)) =
                acc[i][2 * decltype(jj)::value + h];
      });
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // a wave's own writes, read by its other lanes
      if (whole) {  // no column is missing: rows at once, and no branch but for rows that are not there
        const Epilogue& e = ep;
        constexpr int kIt = 16 / rows;  // in two halves: registers
#pragma unroll 1
        for (int r0 = lane / pieces; r0 < 32; r0 += 16) {
          const int64_t s0 = slot0 + r0;
          v4f v[kIt * H], r4[kIt * H];
          if (e.residual) {
#pragma unroll
            for (int k = 0; k < kIt; ++k)
              if (there >> (r0 + k * rows) & 1)
                load_row(e.residual, (s0 + k * rows) * e.ldr + n0 + o, e.res_bf16, &r4[k * H],
                         std::integral_constant<int, H>{});
          }
#pragma unroll
          for (int k = 0; k < kIt; ++k) {
            const uint8_t* row = slab + (r0 + k * rows) * kRow;
            const float f = *reinterpret_cast<const float*>(row + 128 * TN);
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const v4i a = *reinterpret_cast<const v4i*>(row + 4 * o + 16 * h);
#pragma unroll
              for (int q = 0; q < 4; ++q) v[k * H + h][q] = __builtin_fmaf((float)a[q], f, b[h][q]);
            }
          }
          activate_all<bf16>(v, e.act);
          if (e.residual) {
#pragma unroll
            for (int k = 0; k < kIt * H; ++k) v[k] += r4[k];
          }
#pragma unroll
          for (int k = 0; k < kIt; ++k)
            if (there >> (r0 + k * rows) & 1)
              store_row(e, (s0 + k * rows) * e.ldy + n0 + o, &v[k * H], std::integral_constant<int, H>{});
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        continue;
      }
#pragma unroll 1
      for (int r = lane / pieces; r < 32; r += rows) {
        if (!(there >> r & 1) || left <= 0) continue;
        const float f = *reinterpret_cast<const float*>(slab + r * kRow + 128 * TN);
        const int64_t s = slot0 + r;
        v4f v[per / 4];
#pragma unroll
        for (int h = 0; h < per / 4; ++h) {
          const v4i a = *reinterpret_cast<const v4i*>(slab + r * kRow + 4 * o + 16 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[h][e] = __builtin_fmaf((float)a[e], f, b[h][e]);
        }
        activate_all<bf16>(v, ep.act);
        finish_row(ep, s, n0 + o, left, v);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next slab is written
    }
  };
  if (ep.y_bf16) rows_out(std::true_type{});
  else rows_out(std::false_type{});
}

}  // namespace

hipError_t launch_experts_gemm(const ExpertsPlan& p, const Groups& g, const int8_t* Xq, const float* absmax,
                               const Epilogue& ep, hipStream_t s) {
  const int chunks = (int)(k_pad(g.K) / kTileCols), nblocks = (int)(n_pad(g.N) / kTileRows);
  const int tiles_n = (int)((g.N + p.width - 1) / p.width);
  auto go = [&](auto tm, auto tn) {
    k_experts_gemm<decltype(tm)::value, decltype(tn)::value>
        <<<dim3((unsigned)p.groups), 256, 0, s>>>(g, Xq, absmax, ep, chunks, nblocks, tiles_n, 8);
    return hipGetLastError();
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 3> three;
  const std::integral_constant<int, 4> four;
  if (p.height == 128) return go(four, two);
  if (p.height == 96) return go(three, two);
  if (p.height == 64) return p.width == 256 ? go(two, two) : go(two, one);
  return p.width == 256 ? go(one, two) : go(one, one);
}

}  // namespace bl
