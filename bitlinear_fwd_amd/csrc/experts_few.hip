// Ternary products with an epilogue for few slots to a matrix: the packed weights stream past, a row block (16 outputs)
// at a time, straight into registers and through 16x16x64 int8 instructions; the waves of a workgroup split the
// columns and add their exact sums through LDS.
//
// k_few, a few slots in all: the workgroup first fills LDS with the codes of its unit's token rows, quantised there
// from fp32 or bf16 (which saves a launch), the rows' loads ahead of the first weights', then takes one row block.
// k_mid, units of 16 or 32 slots: token fragments come from the caches, up to four row blocks share them and up to
// two of them share a decoded weight fragment.
//
// Bound by latency (launch, one round trip for the rows and the weights, the sums) where the matrix is small: 1 x 6912 x
// 2560 4.9 us from bf16, 3.8 from codes.  k_mid with one slot reaches 4.8 TB/s of weights (8192 x 28672, 12.2 us); with
// 16 and more it is bound by the rows' codes, which every workgroup reads from L2 (8.6 TB/s): hence the row blocks that
// share them (32 x 8192 x 8192 by 1, 2, 4: 19.7, 13.0, 9.0 us).  Loads of 64 consecutive bytes of a row with the pieces
// exchanged between lanes afterwards (each load touches a quarter of the lines) were no faster.
#include "experts.h"


namespace bl {
namespace {

// Barrier between LDS writes and reads that leaves global loads in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Piece p (16 bytes) of a 256-column chunk of row r lies in its place p ^ few_swizzle(r), for reads of one piece of
// 16 rows: 16-byte reads take lanes 0-3, 12-15 and 20-27 together, rows 0-3 and 12-15 at piece p with rows 4-11
// at piece p ^ 4.
__device__ __forceinline__ int few_swizzle(int r) { return (r + 12) & 15; }

// The fp32 bits of the largest magnitude of eight elements, NaN passed over as the quantiser in a launch of its own does:
// an offset that makes the patterns of NaN, and only these, negative.
__device__ __forceinline__ uint32_t top_number(const Raw8<float>& r) {
  constexpr int kOff = 0x007fffff;
  int top = kOff;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, (int)((r.w[i] & 0x7fffffffu) + kOff));
  return (uint32_t)(top - kOff);
}
__device__ __forceinline__ uint32_t top_number(const Raw8<uint16_t>& r) {
  typedef unsigned short v2u __attribute__((ext_vector_type(2)));
  typedef short v2s __attribute__((ext_vector_type(2)));
  constexpr unsigned short kOff = 0x007f;
  v2s m = {kOff, kOff};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2u w = __builtin_bit_cast(v2u, r.w[i] & 0x7fff7fffu) + v2u{kOff, kOff};
    m = __builtin_elementwise_max(m, __builtin_bit_cast(v2s, w));
  }
  return (uint32_t)(max(m.x, m.y) - kOff) << 16;
}

constexpr int kKept = 4;    // pieces of 8 elements that a thread keeps between the two passes of the quantiser

// kSrc 1: bf16, 2: fp32 x[R][K], K a multiple of 8.  A workgroup takes one unit and one row block.
// kDepth: chunks of weights that a wave loads at a time.
template <int kSrc, int kDepth>
__global__ __launch_bounds__(1024) void k_few(Groups g, const void* __restrict__ X, Epilogue ep, int chunks,
                                               int nblocks) {
  extern __shared__ v4i part[];  // [waves][64], then scales [16], then the tokens
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  float* scales = reinterpret_cast<float*>(part + waves * 64);
  uint8_t* tok = reinterpret_cast<uint8_t*>(scales + 16);
  const Unit u = find_unit(g, 16, blockIdx.x / nblocks);
  if (u.lo >= u.hi) return;
  const int nb = (int)(blockIdx.x % nblocks);

  const int rows = u.hi - u.lo, K = (int)g.K, pitch = chunks * kTileCols;

  // The rows' loads go out before the weights', which they would wait behind.
  using T = std::conditional_t<kSrc == 2, float, uint16_t>;
  // wpr waves share a row; with fewer waves than rows a wave has several
  const int wpr = max(1, waves / rows), slice = wave % wpr, first_row = wave / wpr;
  const int pieces = chunks * 32, stride = 64 * wpr, piece0 = slice * 64 + lane;  // pieces of 8 elements
  auto row_of = [&](int r) {
    return static_cast<const T*>(X) + (int64_t)__builtin_amdgcn_readfirstlane(max(slot_row(g, u.lo + r), 0)) * K;
  };
  // piece p of a row (K is a multiple of 8), zeros past its end
  auto piece = [&](const T* x, int p) {
    Raw8<T> v;
    __builtin_memcpy(v.w, x + 8 * (int64_t)min(p, (K >> 3) - 1), 8 * sizeof(T));
    if (8 * p >= K) v = Raw8<T>{};
    return v;
  };
  Raw8<T> v[kKept];
  const bool kept = wpr > 1 && pieces <= kKept * stride && first_row < rows;
  const int nkept = kept ? (pieces + stride - 1) / stride : 0;
  {
    if (kept) {
      const T* x = row_of(first_row);
      v[0] = piece(x, piece0);
      if (nkept > 1) v[1] = piece(x, piece0 + stride);
      if (nkept > 2) {
        v[2] = piece(x, piece0 + 2 * stride);
        v[3] = piece(x, piece0 + 3 * stride);
      }
    }
  }

  // this wave's chunks of the row block: wave, wave + waves, .., kDepth at a time (past the last the last again, so that
  // no load of a batch depends on a branch)
  const int mine = (chunks - wave + waves - 1) / waves;
  const uint4* w0 = reinterpret_cast<const uint4*>(g.packed + ((int64_t)u.e * nblocks + nb) * chunks * kTileBytes) + lane;
  v4i w[kDepth];
  auto fetch = [&](int i) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      w[d] = __builtin_nontemporal_load(
          reinterpret_cast<const v4i*>(w0 + (int64_t)(wave + min(i + d, mine - 1) * waves) * 64));
  };
  fetch(0);

  {
    auto wave_max = [&](uint32_t m) {
      m = quad_max(m);
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xf, 0xf, true));
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xf, 0xf, true));
      return max(max((uint32_t)__builtin_amdgcn_readlane(m, 0), (uint32_t)__builtin_amdgcn_readlane(m, 16)),
                 max((uint32_t)__builtin_amdgcn_readlane(m, 32), (uint32_t)__builtin_amdgcn_readlane(m, 48)));
    };
    auto put = [&](int r, int p, const Raw8<T>& x, float s) {
      float f[8];
      widen8(x, f);
      uint2 q;
      q.x = quant_code4(f[0], f[1], f[2], f[3], s);
      q.y = quant_code4(f[4], f[5], f[6], f[7], s);
      const int at = 256 * (p >> 5) + 16 * (((p >> 1) & 15) ^ few_swizzle(r)) + 8 * (p & 1);
      *reinterpret_cast<uint2*>(tok + r * pitch + at) = q;
    };
    auto scale_of = [&](float a) { return a > 0.0f ? 127.0f / a : 0.0f; };
    auto row_max = [&](const T* x) {
      uint32_t m = 0;
#pragma unroll 2
      for (int p = piece0; p < pieces; p += stride) m = max(m, top_number(piece(x, p)));
      return wave_max(m);
    };
    auto row_put = [&](int r, const T* x, float s) {
#pragma unroll 2
      for (int p = piece0; p < pieces; p += stride) put(r, p, piece(x, p), s);
    };
    if (wpr > 1) {  // one row to a wave at most: its waves' maxima through LDS (the sums' place)
      uint32_t* top = reinterpret_cast<uint32_t*>(part);
      uint32_t m = 0;
      if (kept) {
        m = top_number(v[0]);
        if (nkept > 1) m = max(m, top_number(v[1]));
        if (nkept > 2) m = max(m, max(top_number(v[2]), top_number(v[3])));
        m = wave_max(m);
      } else if (first_row < rows) {
        m = row_max(row_of(first_row));
      }
      if (lane == 0) top[wave] = m;
      lds_barrier();
      if (first_row < rows) {
        m = 0;
        for (int i = 0; i < wpr; ++i) m = max(m, top[first_row * wpr + i]);
        const float a = __uint_as_float(m), s = scale_of(a);
        if (slice == 0 && lane == 0) scales[first_row] = a;
        if (kept) {
          if (piece0 < pieces) put(first_row, piece0, v[0], s);
          if (nkept > 1 && piece0 + stride < pieces) put(first_row, piece0 + stride, v[1], s);
          if (nkept > 2 && piece0 + 2 * stride < pieces) put(first_row, piece0 + 2 * stride, v[2], s);
          if (nkept > 3 && piece0 + 3 * stride < pieces) put(first_row, piece0 + 3 * stride, v[3], s);
        } else {
          row_put(first_row, row_of(first_row), s);
        }
      }
    } else {
      for (int r = wave; r < rows; r += waves) {
        const T* x = row_of(r);
        const float a = __uint_as_float(row_max(x));
        if (lane == 0) scales[r] = a;
        row_put(r, x, scale_of(a));
      }
    }
  }
  lds_barrier();

  // lane (r, q): token r (past the last: the last again, not stored), columns 64 q .. 64 q + 63 of a chunk
  const int lr = lane & 15, lq = lane >> 4, tr = min(lr, rows - 1);
  const uint8_t* xl = tok + tr * pitch;
  int place[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) place[i] = 16 * ((4 * lq + i) ^ few_swizzle(tr));
  const int row = slot_row(g, u.lo + tr);
  const float gamma = g.gamma[u.e], scale = token_scale(gamma, scales[tr]);
  v4i acc = {0, 0, 0, 0};
  for (int i = 0; i < mine; i += kDepth) {
    v4i t[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) t[d] = w[d];
    if (i + kDepth < mine) fetch(i + kDepth);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (i + d < mine) {
        const uint8_t* x = xl + (wave + (i + d) * waves) * kTileCols;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(decode16((uint32_t)t[d][k]),
                                                      *reinterpret_cast<const v4i*>(x + place[k]), acc, 0, 0, 0);
      }
    }
  }
  // the waves' sums
  part[wave * 64 + lane] = acc;
  lds_barrier();
  if (wave == 0) {
    v4i s = part[lane];
    for (int v = 1; v < waves; ++v) s += part[v * 64 + lane];
    const int64_t n = (int64_t)nb * 16 + 4 * lq, left = g.N - n;
    if (lr < rows && row >= 0 && left > 0) finish4(ep, u.e, g.N, u.lo + lr, n, (int)min(left, (int64_t)4), s, scale);
  }
}

// TG groups of 16 slots by RB row blocks; codes from global memory.
template <int TG, int RB>
__global__ __launch_bounds__(512) void k_mid(Groups g, const int8_t* __restrict__ Xq, const float* __restrict__ absmax,
                                             Epilogue ep, int chunks, int nblocks, int columns) {
  extern __shared__ v4i part[];  // [waves][RB][TG][64]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const Unit u = find_unit(g, 16 * TG, blockIdx.x / columns);
  if (u.lo >= u.hi) return;
  const int nb0 = (int)(blockIdx.x % columns) * RB;
  const int lr = lane & 15, lq = lane >> 4;
  const uint4* wp[RB];
  const int8_t* xp[TG];
#pragma unroll
  for (int i = 0; i < RB; ++i)  // row blocks and slots past the last repeat it; not stored
    wp[i] = reinterpret_cast<const uint4*>(
                g.packed + ((int64_t)u.e * nblocks + min(nb0 + i, nblocks - 1)) * chunks * kTileBytes) + lane;
#pragma unroll
  for (int j = 0; j < TG; ++j)
    xp[j] = Xq + (int64_t)max(slot_row(g, min(u.lo + 16 * j + lr, u.hi - 1)), 0) * chunks * kTileCols + 64 * lq;
  v4i acc[RB][TG];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < TG; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  uint4 w[2][RB];
  v4i x[TG][4];
  auto fetch_w = [&](int c, uint4 (&v)[RB]) {
#pragma unroll
    for (int i = 0; i < RB; ++i) v[i] = wp[i][(int64_t)c * 64];
  };
  auto fetch_x = [&](int c, auto j) {
#pragma unroll
    for (int s = 0; s < 4; ++s) x[j][s] = *reinterpret_cast<const v4i*>(xp[j] + (int64_t)c * kTileCols + 16 * s);
  };
  // past the wave's last chunk its last again, so that no load depends on a branch
  const int last = chunks - 1 - (chunks - 1 - wave) % waves;
  auto work = [&](int c, auto cur) {
    constexpr int k = decltype(cur)::value;
    const int next = min(c + waves, last);
    fetch_w(next, w[1 - k]);
    static_for<TG>([&](auto j) {
      static_for<4>([&](auto s) {
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const uint32_t word = s == 0 ? w[k][i].x : s == 1 ? w[k][i].y : s == 2 ? w[k][i].z : w[k][i].w;
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(decode16(word), x[j][s], acc[i][j], 0, 0, 0);
        }
      });
      fetch_x(next, j);
    });
  };
  fetch_w(wave, w[0]);
  static_for<TG>([&](auto j) { fetch_x(wave, j); });
  int c = wave;
  for (; c + waves < chunks; c += 2 * waves) {
    work(c, std::integral_constant<int, 0>{});
    work(c + waves, std::integral_constant<int, 1>{});
  }
  if (c < chunks) work(c, std::integral_constant<int, 0>{});
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < TG; ++j) part[((wave * RB + i) * TG + j) * 64 + lane] = acc[i][j];
  lds_barrier();
  for (int o = threadIdx.x; o < RB * TG * 64; o += blockDim.x) {
    v4i s = part[o];
    for (int v = 1; v < waves; ++v) s += part[v * RB * TG * 64 + o];
    const int l = o & 63, j = (o >> 6) % TG, i = (o >> 6) / TG, slot = u.lo + 16 * j + (l & 15);
    const int64_t n = (int64_t)(nb0 + i) * 16 + 4 * (l >> 4), left = g.N - n;
    if (slot >= u.hi || left <= 0) continue;
    const int row = slot_row(g, slot);
    if (row >= 0)
      finish4(ep, u.e, g.N, slot, n, (int)min(left, (int64_t)4), s, token_scale(g.gamma[u.e], absmax[row]));
  }
}

}  // namespace

hipError_t launch_experts_few(const ExpertsPlan& p, const Groups& g, const void* X, int src, const Epilogue& ep,
                              hipStream_t s) {
  const int chunks = (int)(k_pad(g.K) / kTileCols), nblocks = (int)(n_pad(g.N) / kTileRows), waves = p.threads / 64;
  static_assert(16 * 1024 + 64 + kFewChunks * kTileCols <= 64 * 1024, "LDS that a launch has without asking");
  const size_t lds = (size_t)waves * 1024 + 64 + (size_t)g.T * chunks * kTileCols;  // sums, scales, codes of all rows
  auto go = [&](auto sc, auto dd) {
    k_few<decltype(sc)::value, decltype(dd)::value>
        <<<dim3((unsigned)p.groups), p.threads, lds, s>>>(g, X, ep, chunks, nblocks);
    return hipGetLastError();
  };
  const int mine = (chunks + waves - 1) / waves;
  auto depth = [&](auto sc) {
    if (mine == 1) return go(sc, std::integral_constant<int, 1>{});
    if (mine == 2) return go(sc, std::integral_constant<int, 2>{});
    return go(sc, std::integral_constant<int, 4>{});
  };
  return src == 1 ? depth(std::integral_constant<int, 1>{}) : depth(std::integral_constant<int, 2>{});
}

hipError_t launch_experts_mid(const ExpertsPlan& p, const Groups& g, const int8_t* Xq, const float* absmax,
                              const Epilogue& ep, hipStream_t s) {
  const int chunks = (int)(k_pad(g.K) / kTileCols), nblocks = (int)(n_pad(g.N) / kTileRows);
  auto go = [&](auto tg, auto rb) {
    constexpr int TG = decltype(tg)::value, RB = decltype(rb)::value;
    k_mid<TG, RB><<<dim3((unsigned)p.groups), p.threads, (size_t)(p.threads / 64) * RB * TG * 1024, s>>>(
        g, Xq, absmax, ep, chunks, nblocks, (nblocks + RB - 1) / RB);
    return hipGetLastError();
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 4> four;
  if (p.height == 32) return go(two, four);
  return p.per == 4 ? go(one, four) : p.per == 2 ? go(one, two) : go(one, one);
}

}  // namespace bl
