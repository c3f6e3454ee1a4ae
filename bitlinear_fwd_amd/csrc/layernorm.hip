// Layer normalisation over the rows of x[M][K], and its gradients.
//
// Forward: mean = sum x / K, var = sum (x - mean)^2 / K, rstd = 1 / sqrt(var + eps),
// y = (x - mean) rstd w + b.  The row stays in registers between the two sums, so the variance is
// of centred values (no cancellation between a mean of squares and a squared mean) and x is read
// once.  The mean is taken of x less an element of the row, so its rounding goes by the spread of the
// row (below, at k_layernorm).
//
// Backward, with xhat = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),  dw = sum_m dy xhat,  db = sum_m dy.
// A workgroup walks over rows with the columns fixed to its threads, so the sums over the rows
// stay in registers until it ends and writes one partial row of dw and of db; a second launch
// adds the partial rows in order.  No atomics: results do not depend on timing.
//
// Both are bound by memory: x (and dy) in, y (dx) out.  A row is shared by a wave (up to 1024
// elements, forward) or by as many waves as hold it with one or two groups of 8 elements a thread;
// rows longer than 32768 (backward 12288) elements are read again for each sum, with the sums in
// fp64.  Measured (a large copy moves 5.2 TB/s): forward 8192 x 8192 bf16 47.8 us, 5.6 TB/s; 2048 x
// 8192 fp32 25.8 us, 5.2 TB/s; 16 x 2560 bf16 3.3 us, a launch and one round trip to memory.  Backward
// 8192 x 8192 bf16 91 us, 4.4 TB/s; 2048 x 2560 bf16 16.6 us, of which the second launch takes 4 and the
// first about 6 before and after its rows; 1003 x 7001 fp32 26.2 us.  The sums over a row cost most
// after the bytes: with lane exchanges through LDS and two barriers each, 8192 x 8192 took 53 us
// forward (50 so) and 112 backward; then the next row's loads, which the compiler had waited for before
// this row's sum (52.8 us with the mean as it is now, 47.8 since they stay in flight).
#include "layernorm.h"

#include <algorithm>

#include "mxfp4.h"

namespace bl {
namespace {

constexpr int64_t kMaxGrid = 1 << 20;    // workgroups of a launch; rows beyond are walked over
constexpr int64_t kCUs = 256;
// Rows per compute unit up to which a row is spread over as many threads as possible: the latency of
// one row counts (16 x 2560 bf16: 3.5 us, 4.9 with two groups a thread), beyond it the bytes in flight
// (8192 x 8192 bf16: 82 us with one group, 65 with two).
constexpr int kFewRows = 4;

// Sum over each 16 lanes, by lane moves; every lane gets its own 16's.
__device__ __forceinline__ float sum16(float v) {
  auto moved = [&](auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v += moved(std::integral_constant<int, 0xB1>{});   // quad_perm 1 0 3 2
  v += moved(std::integral_constant<int, 0x4E>{});   // quad_perm 2 3 0 1
  v += moved(std::integral_constant<int, 0x141>{});  // row_half_mirror
  v += moved(std::integral_constant<int, 0x140>{});  // row_mirror
  return v;
}
__device__ __forceinline__ double sum16(double v) {
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
// Sum over a wave; every lane gets it.
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  auto row = [&](int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}
__device__ __forceinline__ double wave_sum(double v) {
  v = sum16(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Sum of each v[] over the threads that share a row; every thread gets it.  kWave: a wave.  Else up to
// 16 waves, through LDS, with one barrier for all threads of the workgroup: `red` has kN values per
// wave of the row, this thread is in the row's wave-th of `waves`.  Two sums in a row take two
// different buffers, so that no thread writes what another still reads.
template <bool kWave, int kN, typename F>
__device__ __forceinline__ void row_sum(F (&v)[kN], F* red, int wave, int waves) {
#pragma unroll
  for (int j = 0; j < kN; ++j) v[j] = wave_sum(v[j]);
  if constexpr (!kWave) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int j = 0; j < kN; ++j) red[wave * kN + j] = v[j];
    }
    __syncthreads();
    const int l = threadIdx.x & 15;
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = sum16(l < waves ? red[l * kN + j] : F(0));
  }
}

// The eight columns of group g of a thread, as two runs of four.  A wave's 16-byte loads have to be
// consecutive: the runs are neighbours in a bf16 row and 4 `threads` columns apart in an fp32 one
// (2048 x 8192 fp32: 27.4 us, 32.0 with runs that are neighbours; backward 47.6 and 51.4).
struct Cols {
  int64_t a, b;
  __device__ __forceinline__ int64_t at(int i) const { return i < 4 ? a + i : b + i - 4; }
};
template <typename T>
__device__ __forceinline__ Cols cols(int i0, int g, int threads) {
  if constexpr (sizeof(T) == 4) return {4 * (int64_t)(i0 + 2 * g * threads), 4 * (int64_t)(i0 + (2 * g + 1) * threads)};
  const int64_t c = 8 * (int64_t)(i0 + g * threads);
  return {c, c + 4};
}
__device__ __forceinline__ void load4(const float* p, int64_t n, uint32_t* v) {
  if (n >= 4) {
    __builtin_memcpy(v, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? __float_as_uint(p[i]) : 0u;
  }
}
// A group of a row of K elements (0: none, all zeros).
__device__ __forceinline__ Raw8<uint16_t> load_group(const uint16_t* row, Cols c, int64_t K) {
  return load_raw8(row + c.a, K - c.a);
}
__device__ __forceinline__ Raw8<float> load_group(const float* row, Cols c, int64_t K) {
  Raw8<float> r;
  load4(row + c.a, K - c.a, r.w);
  load4(row + c.b, K - c.b, r.w + 4);
  return r;
}
__device__ __forceinline__ void load_params(const float* p, Cols c, int64_t K, float (&v)[8]) {
  Raw8<float> r;
  load4(p + c.a, K - c.a, r.w);
  load4(p + c.b, K - c.b, r.w + 4);
  widen8(r, v);
}
// stream: past the caches.
__device__ __forceinline__ void store_group(uint16_t* row, Cols c, int64_t K, const float (&v)[8], bool stream) {
  stream8(row + c.a, K - c.a, v, stream);
}
__device__ __forceinline__ void store_group(float* row, Cols c, int64_t K, const float (&v)[8], bool stream) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t col = h ? c.b : c.a;
    float* p = row + col;
    if (K - col >= 4) {
      v4u w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[4 * h + i]);
      if (stream)
        __builtin_nontemporal_store(w, reinterpret_cast<v4u_unaligned*>(p));
      else
        *reinterpret_cast<v4u_unaligned*>(p) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < K) p[i] = v[4 * h + i];
    }
  }
}

// How many elements of a row a wave has.
template <typename T, int kG>
__device__ __forceinline__ float wave_count(int wave, int threads, int K) {
  int n = 0;
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    const Cols c = cols<T>(64 * wave, g, threads);
    constexpr int kRun = sizeof(T) == 4 ? 256 : 512;  // fp32 has two runs of four columns a lane, bf16 one of eight
    n += min(max(K - (int)c.a, 0), kRun);
    if (sizeof(T) == 4) n += min(max(K - (int)c.b, 0), kRun);
  }
  return (float)n;
}

// One row per wave (kWave) or per workgroup, kG groups of 8 elements per thread (thread i of the T
// that share the row takes groups i, i + T, ...).  A workgroup walks over rows with the next row's
// loads in flight and (kHold) weight and bias in registers: read for every row they are four
// times a bf16 row's bytes.
// The mean is taken of x less a pivot, an element of the row (of three, the middle one, so that a single
// outlier is none; each wave has its own), and only what is returned is the sum of the two.  So what is
// rounded goes by the spread of a row and not by its mean, and a row of one value has exactly the
// variance 0: a sum of the elements themselves gave a constant 100000.3 a spread of 0.008, and rows of
// 1000 +- 0.01 outputs off by 4e-3.
// kQuads: K % 4 == 0, so that a run of four columns is of the row or behind it as a whole: its zeros
// then take no pivot, instead of a select for every element (8192 x 8192 bf16 47.8 us, 49.3 with selects;
// 2048 x 20000 fp32 81 and 92).
template <typename T, bool kWave, int kG, bool kHold, bool kQuads>
__global__ __launch_bounds__(kWave ? 256 : 1024) void k_layernorm(const T* __restrict__ X, int64_t M, int64_t K,
                                                                  const float* __restrict__ weight,
                                                                  const float* __restrict__ bias, float eps,
                                                                  T* __restrict__ Y, float* __restrict__ mean_out,
                                                                  float* __restrict__ rstd_out) {
  __shared__ float2 red_sum[16];
  __shared__ float red_sq[16];
  const int threads = kWave ? 64 : blockDim.x;
  const int i0 = kWave ? threadIdx.x & 63 : threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * (kWave ? 4 : 1);
  int64_t row = kWave ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  Raw8<T> raw[kG];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const Cols c8 = cols<T>(i0, g, threads);
      raw[g] = load_group(X + r * K, c8, r < M ? K : 0);
    }
  };
  // four groups of fp32 leave no registers for a row ahead (2048 x 20000: 77 us, 125 with one, which
  // spills; with the pivots 81, two registers spilled)
  constexpr bool kAhead = kG < 4 || sizeof(T) == 2;
  if constexpr (kAhead) fetch(row);
  float w[kG][8], b[kG][8];
  auto params = [&](int g) {
    const Cols c8 = cols<T>(i0, g, threads);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[g][i] = 1.0f;
      b[g][i] = 0.0f;
    }
    if (weight) load_params(weight, c8, K, w[g]);
    if (bias) load_params(bias, c8, K, b[g]);
  };
  if constexpr (kHold) {
#pragma unroll
    for (int g = 0; g < kG; ++g) params(g);
  }
  // the lanes of this wave whose first element is of the row, at least one
  const int wave = __builtin_amdgcn_readfirstlane(i0 >> 6);
  constexpr int kFirst = sizeof(T) == 4 ? 4 : 8;  // columns between the first elements of two lanes
  const int lanes = min(((int)K - wave * 64 * kFirst + kFirst - 1) / kFirst, 64);
  const float others = kWave ? 0.0f : wave_count<T, kG>(threadIdx.x & 15, threads, (int)K);
  float v[kG][8];
  // v -= p, and zeros stay zeros behind the row's end
  auto less = [&](float p) {
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const Cols c8 = cols<T>(i0, g, threads);
      const float pa = c8.a < K ? p : 0.0f, pb = c8.b < K ? p : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[g][i] = kQuads ? v[g][i] - (i < 4 ? pa : pb) : c8.at(i) < K ? v[g][i] - p : 0.0f;
    }
  };
  for (; row < M; row += step) {
    float sum[1] = {0.0f}, sq[1] = {0.0f};
    if constexpr (!kAhead) fetch(row);
    Raw8<T> cur[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      cur[g] = raw[g];
      // here, and not behind the next row's loads, the compiler waits for this row's
      if constexpr (kAhead) {
#pragma unroll
        for (uint32_t& word : cur[g].w) asm volatile("" : "+v"(word));
      }
    }
    if constexpr (kAhead) fetch(row + step);
#pragma unroll
    for (int g = 0; g < kG; ++g) widen8(cur[g], v[g]);
    auto of = [&](int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v[0][0]), lane)); };
    const float pivot = __builtin_amdgcn_fmed3f(of(0), of(lanes >> 1), of(lanes - 1));
    less(pivot);
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] += v[g][i];
    sum[0] = wave_sum(sum[0]);
    if constexpr (!kWave) {  // the waves' sums, of x less this wave's pivot
      if ((threadIdx.x & 63) == 0) red_sum[wave] = make_float2(sum[0], pivot);
      __syncthreads();
      const int l = threadIdx.x & 15;
      const float2 other = red_sum[l];
      sum[0] = sum16(l < threads >> 6 ? other.x + others * (other.y - pivot) : 0.0f);
    }
    const float off = sum[0] / (float)K;  // the mean less the pivot
    less(off);
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
      for (int i = 0; i < 8; ++i) sq[0] += v[g][i] * v[g][i];
    row_sum<kWave, 1>(sq, red_sq, i0 >> 6, threads >> 6);
    const float rstd = 1.0f / sqrtf(sq[0] / (float)K + eps);
    if (i0 == 0) {
      if (mean_out) mean_out[row] = pivot + off;
      if (rstd_out) rstd_out[row] = rstd;
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const Cols c8 = cols<T>(i0, g, threads);
      if constexpr (!kHold) params(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[g][i] = v[g][i] * rstd * w[g][i] + b[g][i];
      store_group(Y + row * K, c8, K, v[g], (kWave || kG > 1) && whole_pieces(K));
    }
  }
}

// Rows longer than the registers hold: read for the mean, for the variance and for the output.
template <typename T>
__global__ __launch_bounds__(1024) void k_layernorm_long(const T* __restrict__ X, int64_t M, int64_t K,
                                                         const float* __restrict__ weight,
                                                         const float* __restrict__ bias, float eps,
                                                         T* __restrict__ Y, float* __restrict__ mean_out,
                                                         float* __restrict__ rstd_out) {
  __shared__ double red[2][16];
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const T* x = X + row * K;
    double s[1] = {0.0};
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < K; col += 8 * 1024) {
      float v[8];
      load8(x + col, K - col, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += (double)v[i];
    }
    row_sum<false, 1>(s, red[0], threadIdx.x >> 6, 16);
    const double mean = s[0] / (double)K;
    double q[1] = {0.0};
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < K; col += 8 * 1024) {
      float v[8];
      load8(x + col, K - col, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double d = col + i < K ? (double)v[i] - mean : 0.0;
        q[0] += d * d;
      }
    }
    row_sum<false, 1>(q, red[1], threadIdx.x >> 6, 16);
    const float meanf = (float)mean, rstd = (float)(1.0 / sqrt(q[0] / (double)K + (double)eps));
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = meanf;
      if (rstd_out) rstd_out[row] = rstd;
    }
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < K; col += 8 * 1024) {
      float v[8], w[8], b[8];
      load8(x + col, K - col, v);
      if (weight) load8(weight + col, K - col, w);
      if (bias) load8(bias + col, K - col, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = (float)((double)v[i] - mean) * rstd;
        if (weight) v[i] *= w[i];
        if (bias) v[i] += b[i];
      }
      store8(Y + row * K + col, K - col, v);
    }
  }
}

// A workgroup's rows, `rows` at once by `threads` threads each (kWave: a wave each): dX, and
// (kSums) one partial row of dw at part[p][0][K] and of db at part[p][1][K], p the workgroup.
template <typename T, bool kWave, int kG, bool kSums>
__global__ __launch_bounds__(kG == 1 ? 1024 : 768) void k_layernorm_bwd(
    const T* __restrict__ dY, const T* __restrict__ X, int64_t M, int64_t K, int rows, int threads,
    const float* __restrict__ weight, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    T* __restrict__ dX, float* __restrict__ part) {
  __shared__ float red[2][32];     // two values per wave, in turns
  extern __shared__ float sums[];  // [2][8 kG][threads] where rows > 1
  const int sub = kWave ? threadIdx.x >> 6 : threadIdx.x / threads;
  const int i0 = kWave ? threadIdx.x & 63 : threadIdx.x - sub * threads;
  float dw[kG][8], db[kG][8], w[kG][8];
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    const Cols c8 = cols<T>(i0, g, threads);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[g][i] = 0.0f;
      db[g][i] = 0.0f;
      w[g][i] = 1.0f;
    }
    if (weight) load_params(weight, c8, K, w[g]);
  }
  Raw8<T> rx[kG], rd[kG];
  float rmean = 0.0f, rrstd = 0.0f;
  auto fetch = [&](int64_t row) {  // rows past the last count as zeros, which add nothing to a sum
    const bool in = row < M;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const Cols c8 = cols<T>(i0, g, threads);
      rx[g] = load_group(X + row * K, c8, in ? K : 0);
      rd[g] = load_group(dY + row * K, c8, in ? K : 0);
    }
    rmean = in ? mean_in[row] : 0.0f;
    rrstd = in ? rstd_in[row] : 0.0f;
  };
  const int64_t first = (int64_t)blockIdx.x * rows, step = (int64_t)gridDim.x * rows;
  int turn = 0;
  // two groups of fp32 leave no registers for a row ahead (2048 x 11000: 63.1 us, with nine registers
  // spilled once the sums are taken; 83.9 with a row ahead)
  constexpr bool kAhead = kG == 1 || sizeof(T) == 2;
  if constexpr (kAhead) fetch(first + sub);
  for (int64_t r0 = first; r0 < M; r0 += step) {  // the same trips for every thread: barriers inside
    float x[kG][8], d[kG][8];
    if constexpr (!kAhead) fetch(r0 + sub);
    const float mean = rmean, rstd = rrstd;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      widen8(rx[g], x[g]);
      widen8(rd[g], d[g]);
    }
    if constexpr (kAhead) fetch(r0 + step + sub);
    float c[2] = {0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const Cols c8 = cols<T>(i0, g, threads);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // past the row's end d is 0; x has to be finite there, which mean * rstd need not be
        x[g][i] = c8.at(i) < K ? (x[g][i] - mean) * rstd : 0.0f;
        if constexpr (kSums) {
          dw[g][i] += d[g][i] * x[g][i];
          db[g][i] += d[g][i];
        }
        d[g][i] *= w[g][i];
        c[0] += d[g][i];
        c[1] += d[g][i] * x[g][i];
      }
    }
    if (dX) {
      row_sum<kWave, 2>(c, red[turn] + 2 * sub * (threads >> 6), i0 >> 6, threads >> 6);
      turn ^= 1;
      c[0] /= (float)K;
      c[1] /= (float)K;
      const int64_t row = r0 + sub;
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const Cols c8 = cols<T>(i0, g, threads);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[g][i] = rstd * (d[g][i] - c[0] - x[g][i] * c[1]);
        store_group(dX + row * K, c8, row < M ? K : 0, d[g], whole_pieces(K));
      }
    }
  }
  if constexpr (kSums) {  // the rows' sums, added in order: one partial row per workgroup
    const int plane = 8 * kG * threads;
    for (int v = 0; v < (rows > 1 ? rows : 0); ++v) {
      if (sub == v) {
#pragma unroll
        for (int g = 0; g < kG; ++g) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int at = (8 * g + i) * threads + i0;
            if (v > 0) {
              dw[g][i] = sums[at] + dw[g][i];
              db[g][i] = sums[plane + at] + db[g][i];
            }
            if (v < rows - 1) {
              sums[at] = dw[g][i];
              sums[plane + at] = db[g][i];
            }
          }
        }
      }
      __syncthreads();
    }
    if (sub < rows - 1) return;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const Cols c8 = cols<T>(i0, g, threads);
      store_group(part + 2 * (int64_t)blockIdx.x * K, c8, K, dw[g], false);
      store_group(part + (2 * (int64_t)blockIdx.x + 1) * K, c8, K, db[g], false);
    }
  }
}

// dX of rows longer than the registers hold.
template <typename T>
__global__ __launch_bounds__(1024) void k_layernorm_bwd_long(const T* __restrict__ dY, const T* __restrict__ X,
                                                             int64_t M, int64_t K, const float* __restrict__ weight,
                                                             const float* __restrict__ mean_in,
                                                             const float* __restrict__ rstd_in, T* __restrict__ dX) {
  __shared__ double red[2][32];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const float mean = mean_in[row], rstd = rstd_in[row];
    double c[2] = {0.0, 0.0};
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < K; col += 8 * 1024) {
      float x[8], d[8], w[8];
      load8(X + row * K + col, K - col, x);
      load8(dY + row * K + col, K - col, d);
      if (weight) load8(weight + col, K - col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = weight ? d[i] * w[i] : d[i];
        c[0] += (double)g;
        // past the row's end g is 0, but mean * rstd need not be finite
        c[1] += (double)g * (double)(col + i < K ? (x[i] - mean) * rstd : 0.0f);
      }
    }
    row_sum<false, 2>(c, red[turn], threadIdx.x >> 6, 16);
    turn ^= 1;
    const float c0 = (float)(c[0] / (double)K), c1 = (float)(c[1] / (double)K);
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < K; col += 8 * 1024) {
      float x[8], d[8], w[8];
      load8(X + row * K + col, K - col, x);
      load8(dY + row * K + col, K - col, d);
      if (weight) load8(weight + col, K - col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = weight ? d[i] * w[i] : d[i];
        d[i] = rstd * (g - c0 - (x[i] - mean) * rstd * c1);
      }
      store8(dX + row * K + col, K - col, d);
    }
  }
}

// Partial rows of dw and db for long rows: a thread takes 8 columns of every gridDim.y-th row.
template <typename T>
__global__ __launch_bounds__(256) void k_layernorm_bwd_cols(const T* __restrict__ dY, const T* __restrict__ X,
                                                            int64_t M, int64_t K, const float* __restrict__ mean_in,
                                                            const float* __restrict__ rstd_in,
                                                            float* __restrict__ part) {
  const int64_t col = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (col >= K) return;
  float dw[8] = {}, db[8] = {};
  for (int64_t row = blockIdx.y; row < M; row += gridDim.y) {
    float x[8], d[8];
    load8(X + row * K + col, K - col, x);
    load8(dY + row * K + col, K - col, d);
    const float mean = mean_in[row], rstd = rstd_in[row];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] += d[i] * ((x[i] - mean) * rstd);
      db[i] += d[i];
    }
  }
  store8(part + 2 * (int64_t)blockIdx.y * K + col, K - col, dw);
  store8(part + (2 * (int64_t)blockIdx.y + 1) * K + col, K - col, db);
}

// dw and db: the sums of the partial rows.  A workgroup takes 32 columns of one of the two; its 32
// half waves take every 32nd partial row, all loads in flight, and are added in order.
__global__ __launch_bounds__(1024) void k_layernorm_bwd_sum(const float* __restrict__ part, int64_t parts, int64_t K,
                                                            float* __restrict__ dW, float* __restrict__ dB) {
  __shared__ float red[32][33];
  float* out = blockIdx.y ? dB : dW;
  if (!out) return;
  const int lane = threadIdx.x & 31, half = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (col < K) {
    const float* p = part + blockIdx.y * K + col;
#pragma unroll 8
    for (int64_t r = half; r < parts; r += 32) s += p[2 * r * K];
  }
  red[half][lane] = s;
  __syncthreads();
  if (half == 0 && col < K) {
    for (int h = 1; h < 32; ++h) s += red[h][lane];
    out[col] = s;
  }
}

template <typename T>
void launch_fwd(const void* X, int64_t M, int64_t K, const float* w, const float* b, float eps, void* Y, float* mean,
                float* rstd, hipStream_t s) {
  const T* x = static_cast<const T*>(X);
  T* y = static_cast<T*>(Y);
  auto go = [&](auto wave, auto gc, int waves, int resident) {  // resident: waves that a compute unit holds
    constexpr bool kWave = decltype(wave)::value;
    constexpr int kG = decltype(gc)::value, rows = kWave ? 4 : 1;
    const int64_t most = kCUs * std::max(1, resident / waves);
    const auto fn = K % 4 == 0 ? &k_layernorm<T, kWave, kG, kG <= 2, true> : &k_layernorm<T, kWave, kG, kG <= 2, false>;
    fn<<<dim3((unsigned)std::min<int64_t>((M + rows - 1) / rows, most)), 64 * waves, 0, s>>>(x, M, K, w, b, eps, y,
                                                                                            mean, rstd);
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 4> four;
  auto waves = [&](int groups) { return (int)((K + 512 * groups - 1) / (512 * groups)); };
  if (K <= 512)
    go(std::true_type{}, one, 4, 32);
  else if (K <= 1024)
    go(std::true_type{}, two, 4, 20);
  else if (K <= 8192 && M <= kCUs * kFewRows)
    go(std::false_type{}, one, waves(1), 32);
  else if (K <= 16384)
    go(std::false_type{}, two, waves(2), 20);
  else if (K <= 32768)
    go(std::false_type{}, four, waves(4), 16);
  else
    k_layernorm_long<T><<<dim3((unsigned)std::min(M, kMaxGrid)), 1024, 0, s>>>(x, M, K, w, b, eps, y, mean, rstd);
}

template <typename T>
void launch_bwd(const LnBwdPlan& p, const void* dY, const void* X, int64_t M, int64_t K, const float* w,
                const float* mean, const float* rstd, void* dX, float* part, hipStream_t s) {
  const T *dy = static_cast<const T*>(dY), *x = static_cast<const T*>(X);
  T* dx = static_cast<T*>(dX);
  if (p.rows == 0) {
    if (dx)
      k_layernorm_bwd_long<T><<<dim3((unsigned)std::min(M, kMaxGrid)), 1024, 0, s>>>(dy, x, M, K, w, mean, rstd, dx);
    if (part)
      k_layernorm_bwd_cols<T><<<dim3((unsigned)((K + 2047) / 2048), (unsigned)p.parts), 256, 0, s>>>(dy, x, M, K, mean,
                                                                                                  rstd, part);
    return;
  }
  auto go = [&](auto wave, auto gc) {
    constexpr bool kWave = decltype(wave)::value;
    constexpr int kG = decltype(gc)::value;
    const dim3 grid((unsigned)p.wgs), block((unsigned)(p.rows * p.threads));
    if (part) {
      const size_t lds = p.rows > 1 ? 2 * 8 * kG * p.threads * sizeof(float) : 0;
      k_layernorm_bwd<T, kWave, kG, true><<<grid, block, lds, s>>>(dy, x, M, K, p.rows, p.threads, w, mean, rstd, dx,
                                                                   part);
    } else {
      k_layernorm_bwd<T, kWave, kG, false><<<grid, block, 0, s>>>(dy, x, M, K, p.rows, p.threads, w, mean, rstd, dx,
                                                                  nullptr);
    }
  };
  if (p.threads == 64)
    go(std::true_type{}, std::integral_constant<int, 1>{});
  else if (p.groups == 1)
    go(std::false_type{}, std::integral_constant<int, 1>{});
  else
    go(std::false_type{}, std::integral_constant<int, 2>{});
}

}  // namespace

hipError_t launch_layernorm(const void* X, int bf16, int64_t M, int64_t K, const float* weight, const float* bias,
                            float eps, void* Y, float* mean, float* rstd, hipStream_t s) {
  if (bf16)
    launch_fwd<uint16_t>(X, M, K, weight, bias, eps, Y, mean, rstd, s);
  else
    launch_fwd<float>(X, M, K, weight, bias, eps, Y, mean, rstd, s);
  return hipGetLastError();
}

LnBwdPlan plan_layernorm_backward(int64_t M, int64_t K) {
  LnBwdPlan p;
  // one group of 8 elements per thread up to 16 waves a row, and as many rows as 16 waves hold (one
  // workgroup to a compute unit, so one partial row each); two groups and one row up to 12 waves.
  // Fewer workgroups write fewer partial rows, and lose more than that: 2048 x 2560 bf16 18.2 us, 20.6
  // with 192, 23.7 with 128.
  if (K <= 12288) {
    p.groups = K <= 8192 ? 1 : 2;
    const int waves = (int)((K + 512 * p.groups - 1) / (512 * p.groups));
    p.threads = 64 * waves;
    p.rows = p.groups == 1 ? (int)std::min<int64_t>(16 / waves, M) : 1;
    p.wgs = std::min<int64_t>((M + p.rows - 1) / p.rows, kCUs);
    p.parts = p.wgs;
  } else {
    p.parts = std::min<int64_t>(M, 64);
  }
  p.ws_bytes = p.parts * 2 * K * (int64_t)sizeof(float);
  return p;
}

hipError_t launch_layernorm_backward(const void* dY, const void* X, int bf16, int64_t M, int64_t K,
                                     const float* weight, const float* mean, const float* rstd, void* dX, float* dW,
                                     float* dB, float* workspace, hipStream_t s) {
  const LnBwdPlan p = plan_layernorm_backward(M, K);
  float* part = (dW || dB) ? workspace : nullptr;
  if (bf16)
    launch_bwd<uint16_t>(p, dY, X, M, K, weight, mean, rstd, dX, part, s);
  else
    launch_bwd<float>(p, dY, X, M, K, weight, mean, rstd, dX, part, s);
  if (part)
    k_layernorm_bwd_sum<<<dim3((unsigned)((K + 31) / 32), 2), 1024, 0, s>>>(part, p.parts, K, dW, dB);
  return hipGetLastError();
}

}  // namespace bl
