// MXFP4 quantiser: x[R][K] to 4-bit codes and block scales in the layout of mxfp4.h, and
// optionally the values that the codes stand for.
//
// Per block of 32 columns: e = exponent field of the largest magnitude less 2 (0 at least), so
// that |x| / 2^(e - 127) < 8; code = the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even
// code, 6 from there on.  The division is by a power of two and the conversion instruction
// rounds once, so codes are exact functions of the inputs.  A block with a NaN or an infinity
// has the scale byte 255 (NaN) and zero codes.  Rows and columns of the padding are zeros.
//
// Bound by memory: x in, 17/32 byte an element out, and the values where they are asked for.  A
// workgroup takes 16 rows x 512 columns, each wave 4 of the rows: four lanes share a block (8
// elements, 16 or 32 bytes each), so a wave's load covers 256 or 512 consecutive bytes of each of
// its four rows, and a lane ends up with one 32-bit word of codes; the four tiles of the unit give
// each block's lane the four bytes of a word of scales.
#include "mxfp4.h"

#include <algorithm>

namespace bl {
namespace {

template <typename T, bool kValues>
__global__ __launch_bounds__(256) void k_mx_quant(const T* __restrict__ X, int64_t R, int64_t K, int64_t tiles,
                                                  int64_t groups, int64_t units, uint8_t* __restrict__ codes,
                                                  uint8_t* __restrict__ scales, T* __restrict__ values) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = 4 * wave + (lane >> 4), b = (lane >> 2) & 3, p = lane & 3;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t rb = u / groups, c4 = u % groups;
    const int64_t row = rb * kMxRows + r;
    const int64_t col = c4 * kMxGroupCols + 32 * b + 8 * p;
    Raw8<T> v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t left = row < R ? K - (col + kMxCols * t) : 0;
      v[t] = load_raw8(X + row * K + col + kMxCols * t, left);
    }
    uint32_t word = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const MxScale s = mx_scale(quad_max(top_bits(v[t])));
      const uint32_t q = codes8(v[t], s);
      word |= s.e << (8 * t);
      const int64_t c = 4 * c4 + t;
      if (c < tiles)
        *reinterpret_cast<uint32_t*>(codes + (rb * tiles + c) * kMxTileBytes + 16 * (16 * b + r) + 4 * p) = q;
      if constexpr (kValues) {
        const v2f f0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s.scale, 0);
        const v2f f1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s.scale, 1);
        const v2f f2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s.scale, 2);
        const v2f f3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s.scale, 3);
        float f[8] = {f0.x, f0.y, f1.x, f1.y, f2.x, f2.y, f3.x, f3.y};
        if (s.bad) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(0x7fc00000u);
        }
        const int64_t left = row < R ? K - (col + kMxCols * t) : 0;
        stream8(values + row * K + col + kMxCols * t, left, f, whole_pieces(K));
      }
    }
    if (p == 0) *reinterpret_cast<uint32_t*>(scales + ((rb * groups + c4) * 64 + 16 * b + r) * 4) = word;
  }
}

template <typename T>
void launch(const void* X, int64_t R, int64_t K, uint8_t* codes, uint8_t* scales, void* values, hipStream_t s) {
  const int64_t groups = mx_groups(K), units = mx_row_blocks(R) * groups;
  const dim3 grid((unsigned)std::min<int64_t>(units, 1 << 20));
  const T* x = static_cast<const T*>(X);
  if (values)
    k_mx_quant<T, true><<<grid, 256, 0, s>>>(x, R, K, mx_tiles(K), groups, units, codes, scales,
                                             static_cast<T*>(values));
  else
    k_mx_quant<T, false><<<grid, 256, 0, s>>>(x, R, K, mx_tiles(K), groups, units, codes, scales, nullptr);
}

}  // namespace

hipError_t launch_mx_quant(const void* X, int bf16, int64_t R, int64_t K, uint8_t* codes, uint8_t* scales,
                           void* values, hipStream_t s) {
  if (bf16)
    launch<uint16_t>(X, R, K, codes, scales, values, s);
  else
    launch<float>(X, R, K, codes, scales, values, s);
  return hipGetLastError();
}

}  // namespace bl
