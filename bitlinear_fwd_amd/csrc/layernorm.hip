// Layer normalisation over the rows of x[M][K], and its gradients.
//
// Forward: mean = sum x / K, var = sum (x - mean)^2 / K, rstd = 1 / sqrt(var + eps),
// y = (x - mean) rstd w + b.  The row stays in registers between the two sums, so the variance is
// of centred values (no cancellation between a mean of squares and a squared mean) and x is read
// once.
//
// Backward, with xhat = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),  dw = sum_m dy xhat,  db = sum_m dy.
// A workgroup walks over rows with the columns fixed to its threads, so the sums over the rows
// stay in registers until it ends and writes one partial row of dw and of db; a second launch
// adds the partial rows in order.  No atomics: results do not depend on timing.
//
// Both are bound by memory: x (and dy) in, y (dx) out.  Rows are held by 64, 256 or 1024 threads
// with up to four groups of 8 elements each; longer rows are read again for each sum, with the
// sums in fp64.
#include "layernorm.h"

#include <algorithm>

#include "mxfp4.h"

namespace bl {
namespace {

constexpr int kMaxGroups = 4;          // groups of 8 elements a thread holds
constexpr int64_t kMaxGrid = 1 << 20;  // workgroups of a launch; rows beyond are walked over

// Sum of each v[] over the kTh threads that share a row; every thread gets it.  64 threads are a
// wave; more are the whole workgroup, through LDS (red: kN values per wave).
template <int kTh, int kN, typename F>
__device__ __forceinline__ void row_sum(F (&v)[kN], F* red) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] += __shfl_xor(v[j], off, 64);
  }
  if constexpr (kTh > 64) {
    __syncthreads();  // the values of the sum before have been read
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int j = 0; j < kN; ++j) red[(threadIdx.x >> 6) * kN + j] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      v[j] = red[j];
#pragma unroll
      for (int w = 1; w < kTh / 64; ++w) v[j] += red[w * kN + j];
    }
  }
}

// kTh threads per row, kG groups of 8 elements per thread (thread i takes group i, i + kTh, ...).
template <typename T, int kTh, int kG>
__global__ __launch_bounds__(kTh == 64 ? 256 : kTh) void k_layernorm(const T* __restrict__ X, int64_t M, int64_t K,
                                                                     const float* __restrict__ weight,
                                                                     const float* __restrict__ bias, float eps,
                                                                     T* __restrict__ Y, float* __restrict__ mean_out,
                                                                     float* __restrict__ rstd_out) {
  __shared__ float red[kTh / 64];
  constexpr int kRows = kTh == 64 ? 4 : 1;  // rows of a workgroup
  const int i0 = kTh == 64 ? (threadIdx.x & 63) : threadIdx.x;
  for (int64_t row = (int64_t)blockIdx.x * kRows + (kTh == 64 ? threadIdx.x >> 6 : 0); row < M;
       row += (int64_t)gridDim.x * kRows) {
    float v[kG][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int64_t col = 8 * (int64_t)(i0 + g * kTh);
      load8(X + row * K + col, K - col, v[g]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] += v[g][i];
    }
    row_sum<kTh, 1>(sum, red);
    const float mean = sum[0] / (float)K;
    float sq[1] = {0.0f};
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int64_t col = 8 * (int64_t)(i0 + g * kTh);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[g][i] = col + i < K ? v[g][i] - mean : 0.0f;
        sq[0] += v[g][i] * v[g][i];
      }
    }
    row_sum<kTh, 1>(sq, red);
    const float rstd = 1.0f / sqrtf(sq[0] / (float)K + eps);
    if (i0 == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int64_t col = 8 * (int64_t)(i0 + g * kTh);
      float w[8], b[8];
      if (weight) load8(weight + col, K - col, w);
      if (bias) load8(bias + col, K - col, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[g][i] *= rstd;
        if (weight) v[g][i] *= w[i];
        if (bias) v[g][i] += b[i];
      }
      store8(Y + row * K + col, K - col, v[g]);
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
  __shared__ double red[16];
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const T* x = X + row * K;
    double s[1] = {0.0};
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < K; col += 8 * 1024) {
      float v[8];
      load8(x + col, K - col, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += (double)v[i];
    }
    row_sum<1024, 1>(s, red);
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
    row_sum<1024, 1>(q, red);
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

// One workgroup's rows: dX, and (kSums) one partial row of dw at part[p][0][K] and of db at
// part[p][1][K], p the workgroup.
template <typename T, int kTh, int kG, bool kSums>
__global__ __launch_bounds__(256) void k_layernorm_bwd(const T* __restrict__ dY, const T* __restrict__ X, int64_t M,
                                                       int64_t K, const float* __restrict__ weight,
                                                       const float* __restrict__ mean_in,
                                                       const float* __restrict__ rstd_in, T* __restrict__ dX,
                                                       float* __restrict__ part) {
  __shared__ float red[2 * (kTh / 64)];
  constexpr int kRows = kTh == 64 ? 4 : 1;
  const int i0 = kTh == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t walker = (int64_t)blockIdx.x * kRows + (kTh == 64 ? threadIdx.x >> 6 : 0);
  float dw[kG][8], db[kG][8], w[kG][8];
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    const int64_t col = 8 * (int64_t)(i0 + g * kTh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[g][i] = 0.0f;
      db[g][i] = 0.0f;
      w[g][i] = 1.0f;
    }
    if (weight) load8(weight + col, K - col, w[g]);
  }
  for (int64_t row = walker; row < M; row += (int64_t)gridDim.x * kRows) {
    float x[kG][8], d[kG][8];
    const float mean = mean_in[row], rstd = rstd_in[row];
    float c[2] = {0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int64_t col = 8 * (int64_t)(i0 + g * kTh);
      load8(X + row * K + col, K - col, x[g]);
      load8(dY + row * K + col, K - col, d[g]);
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[g][i] = (x[g][i] - mean) * rstd;  // past the row's end d is 0, so the sums are not touched
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
      row_sum<kTh, 2>(c, red);
      c[0] /= (float)K;
      c[1] /= (float)K;
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const int64_t col = 8 * (int64_t)(i0 + g * kTh);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[g][i] = rstd * (d[g][i] - c[0] - x[g][i] * c[1]);
        store8(dX + row * K + col, K - col, d[g]);
      }
    }
  }
  if constexpr (kSums) {
    if constexpr (kTh == 64) {  // the four waves' sums, added in wave order: one partial row per workgroup
      __shared__ float sums[2][kG * 8][64];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if ((int)(threadIdx.x >> 6) == v) {
#pragma unroll
          for (int g = 0; g < kG; ++g) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (v > 0) {
                dw[g][i] = sums[0][8 * g + i][i0] + dw[g][i];
                db[g][i] = sums[1][8 * g + i][i0] + db[g][i];
              }
              if (v < 3) {
                sums[0][8 * g + i][i0] = dw[g][i];
                sums[1][8 * g + i][i0] = db[g][i];
              }
            }
          }
        }
        __syncthreads();
      }
      if (threadIdx.x < 192) return;
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int64_t col = 8 * (int64_t)(i0 + g * kTh);
      store8(part + 2 * (int64_t)blockIdx.x * K + col, K - col, dw[g]);
      store8(part + (2 * (int64_t)blockIdx.x + 1) * K + col, K - col, db[g]);
    }
  }
}

// dX of rows longer than the registers hold.
template <typename T>
__global__ __launch_bounds__(1024) void k_layernorm_bwd_long(const T* __restrict__ dY, const T* __restrict__ X,
                                                             int64_t M, int64_t K, const float* __restrict__ weight,
                                                             const float* __restrict__ mean_in,
                                                             const float* __restrict__ rstd_in, T* __restrict__ dX) {
  __shared__ double red[32];
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
        c[1] += (double)g * (double)((x[i] - mean) * rstd);
      }
    }
    row_sum<1024, 2>(c, red);
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

// dw and db: the sums of the partial rows.  A workgroup takes 64 columns of one of the two; its
// four waves take every fourth partial row and are added in order.
__global__ __launch_bounds__(256) void k_layernorm_bwd_sum(const float* __restrict__ part, int64_t parts, int64_t K,
                                                           float* __restrict__ dW, float* __restrict__ dB) {
  __shared__ float red[4][64];
  float* out = blockIdx.y ? dB : dW;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (col < K) {
    for (int64_t p = wave; p < parts; p += 4) s += part[(2 * p + blockIdx.y) * K + col];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < K) out[col] = red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane];
}

// Threads that share a row of K elements (0: the long-row form).
int row_threads(int64_t K, int64_t most) {
  for (int64_t th : {64, 256, 1024})
    if (th <= most && K <= th * 8 * kMaxGroups) return (int)th;
  return 0;
}

template <typename T, int kTh>
void launch_rows(int groups, int64_t M, int64_t K, const T* x, const float* w, const float* b, float eps, T* y,
                 float* mean, float* rstd, hipStream_t s) {
  const int64_t rows = kTh == 64 ? 4 : 1;
  const dim3 grid((unsigned)std::min<int64_t>((M + rows - 1) / rows, kMaxGrid)), block(kTh == 64 ? 256 : kTh);
  switch (groups) {
    case 1: k_layernorm<T, kTh, 1><<<grid, block, 0, s>>>(x, M, K, w, b, eps, y, mean, rstd); break;
    case 2: k_layernorm<T, kTh, 2><<<grid, block, 0, s>>>(x, M, K, w, b, eps, y, mean, rstd); break;
    case 3: k_layernorm<T, kTh, 3><<<grid, block, 0, s>>>(x, M, K, w, b, eps, y, mean, rstd); break;
    default: k_layernorm<T, kTh, 4><<<grid, block, 0, s>>>(x, M, K, w, b, eps, y, mean, rstd); break;
  }
}

template <typename T>
void launch_fwd(const void* X, int64_t M, int64_t K, const float* w, const float* b, float eps, void* Y, float* mean,
                float* rstd, hipStream_t s) {
  const T* x = static_cast<const T*>(X);
  T* y = static_cast<T*>(Y);
  const int th = row_threads(K, 1024);
  const int groups = th ? (int)((K + 8 * th - 1) / (8 * th)) : 0;
  if (th == 64)
    launch_rows<T, 64>(groups, M, K, x, w, b, eps, y, mean, rstd, s);
  else if (th == 256)
    launch_rows<T, 256>(groups, M, K, x, w, b, eps, y, mean, rstd, s);
  else if (th == 1024)
    launch_rows<T, 1024>(groups, M, K, x, w, b, eps, y, mean, rstd, s);
  else
    k_layernorm_long<T><<<dim3((unsigned)std::min(M, kMaxGrid)), 1024, 0, s>>>(x, M, K, w, b, eps, y, mean, rstd);
}

template <typename T, int kTh, int kG>
void launch_bwd_rows(const LnBwdPlan& p, int64_t M, int64_t K, const T* dy, const T* x, const float* w,
                     const float* mean, const float* rstd, T* dx, float* part, hipStream_t s) {
  if (part)
    k_layernorm_bwd<T, kTh, kG, true><<<dim3((unsigned)p.wgs), 256, 0, s>>>(dy, x, M, K, w, mean, rstd, dx, part);
  else
    k_layernorm_bwd<T, kTh, kG, false><<<dim3((unsigned)p.wgs), 256, 0, s>>>(dy, x, M, K, w, mean, rstd, dx, part);
}

template <typename T>
void launch_bwd(const LnBwdPlan& p, const void* dY, const void* X, int64_t M, int64_t K, const float* w,
                const float* mean, const float* rstd, void* dX, float* part, hipStream_t s) {
  const T *dy = static_cast<const T*>(dY), *x = static_cast<const T*>(X);
  T* dx = static_cast<T*>(dX);
  if (p.lanes == 0) {
    if (dx)
      k_layernorm_bwd_long<T><<<dim3((unsigned)std::min(M, kMaxGrid)), 1024, 0, s>>>(dy, x, M, K, w, mean, rstd, dx);
    if (part)
      k_layernorm_bwd_cols<T><<<dim3((unsigned)((K + 2047) / 2048), (unsigned)p.parts), 256, 0, s>>>(dy, x, M, K, mean,
                                                                                                  rstd, part);
    return;
  }
  auto go = [&](auto th, auto g) {
    launch_bwd_rows<T, decltype(th)::value, decltype(g)::value>(p, M, K, dy, x, w, mean, rstd, dx, part, s);
  };
  auto by_groups = [&](auto th) {
    switch (p.groups) {
      case 1: go(th, std::integral_constant<int, 1>{}); break;
      case 2: go(th, std::integral_constant<int, 2>{}); break;
      case 3: go(th, std::integral_constant<int, 3>{}); break;
      default: go(th, std::integral_constant<int, 4>{}); break;
    }
  };
  if (p.lanes == 64)
    by_groups(std::integral_constant<int, 64>{});
  else
    by_groups(std::integral_constant<int, 256>{});
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
  p.lanes = row_threads(K, 256);
  if (p.lanes) {
    const int64_t rows = p.lanes == 64 ? 4 : 1;
    p.groups = (int)((K + 8 * p.lanes - 1) / (8 * p.lanes));
    p.wgs = std::min<int64_t>((M + rows - 1) / rows, 512);
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
    k_layernorm_bwd_sum<<<dim3((unsigned)((K + 63) / 64), 2), 256, 0, s>>>(part, p.parts, K, dW, dB);
  return hipGetLastError();
}

}  // namespace bl
