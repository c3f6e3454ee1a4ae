// Microscaled 4-bit floating point (MXFP4): layout, conversions and launchers shared by the
// quantiser, the decode kernel and the GEMM.
//
// A block is 32 consecutive columns of a row.  Its scale byte e stands for 2^(e - 127) (255:
// NaN), its 32 codes for magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign bit.
//
// Layout of a matrix of R rows and K columns: 1024-byte tiles of 16 rows x 128 columns, tile
// (rb, c) at (rb * ceil(K / 128) + c) * 1024; in a tile, row r's block b (columns 32b ..
// 32b + 31) is the 16 bytes at 16 * (16 b + r), low nibble first.  So lane l of a wave that
// loads 16 bytes at 16 l holds row l % 16, block l / 16: exactly the operand of
// v_mfma_scale_f32_16x16x128_f8f6f4 (and, two tiles taken together, of the 32x32x64 form).
// The scales of four tiles 4 c4 .. 4 c4 + 3 sit in one 32-bit word per lane, tile 4 c4 + t in
// byte t, the words of (rb, c4) at ((rb * ceil(K / 512) + c4) * 64 + l) * 4: one wave load per
// four tiles, and the instruction's byte select picks the tile.
#pragma once
#include "bl_internal.h"

namespace bl {

constexpr int kMxRows = 16;        // rows of a tile
constexpr int kMxCols = 128;       // columns of a tile
constexpr int kMxTileBytes = 1024;
constexpr int kMxGroupCols = 512;  // columns that share a word of scales (four tiles)

inline int64_t mx_row_blocks(int64_t r) { return (r + kMxRows - 1) / kMxRows; }
inline int64_t mx_tiles(int64_t k) { return (k + kMxCols - 1) / kMxCols; }
inline int64_t mx_groups(int64_t k) { return (k + kMxGroupCols - 1) / kMxGroupCols; }
inline int64_t mx_codes_bytes(int64_t r, int64_t k) { return mx_row_blocks(r) * mx_tiles(k) * kMxTileBytes; }
inline int64_t mx_scales_bytes(int64_t r, int64_t k) { return mx_row_blocks(r) * mx_groups(k) * 256; }

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// acc += A B of one tile pair: A's 16 rows x 128 columns (lane l: row l % 16, block l / 16) by
// B's, the scales in bytes TA and TB of sa and sb.  acc[i] of lane l is the sum for A's row
// 4 (l / 16) + i and B's row l % 16.
template <int TA, int TB>
__device__ __forceinline__ v4f mx_mfma(v4i a, v4i b, v4f acc, int sa, int sb) {
  const v8i wa = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i wb = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, acc, 4, 4, TA, sa, TB, sb);
}

// The same of 32 rows x 64 columns by 32 rows: lane l holds row l % 32 (of two tiles: rows 0 .. 15
// of the first, then of the second), block l / 32 of the two in this half of the tiles' columns.
// acc[i] of lane l is the sum for A's row 8 (i / 4) + 4 (l / 32) + i % 4 and B's row l % 32.
typedef float v16f __attribute__((ext_vector_type(16)));
template <int TA, int TB>
__device__ __forceinline__ v16f mx_mfma32(v4i a, v4i b, v16f acc, int sa, int sb) {
  const v8i wa = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i wb = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wa, wb, acc, 4, 4, TA, sa, TB, sb);
}

// Scale of a block from the fp32 bits of its largest magnitude: e = max(exponent field - 2, 0), the
// power of two of that magnitude over 4, the grid's largest power; the number 2^(e - 127) (e = 0: a
// subnormal).  bad: the block holds a NaN or an infinity (e is 255 then, the scale any number).
struct MxScale {
  uint32_t e;
  float scale;
  bool bad;
};
__device__ __forceinline__ MxScale mx_scale(uint32_t top) {
  const uint32_t field = top >> 23, e = max(field, 2u) - 2;
  MxScale s;
  s.bad = field == 255;
  s.e = s.bad ? 255 : e;
  s.scale = __uint_as_float(max(e << 23, 0x00400000u));
  return s;
}

// Eight consecutive elements of a row as they are in memory (fp32, or bf16 as uint16_t); elements
// past n are 0.  Whole groups are read 16 bytes at a time at any alignment (the target's global loads
// need none).  widen8 makes fp32 of them, load8 does both.
template <typename T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p, int64_t n) {
  Raw8<T> r;
  if (n >= 8) {
    __builtin_memcpy(r.w, p, 8 * sizeof(T));
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = i < n ? __float_as_uint(p[i]) : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t n, float (&v)[8]) {
  widen8(load_raw8(p, n), v);
}

// The fp32 bits of the largest magnitude of eight elements (bf16: as 16-bit integers, two at a time).
__device__ __forceinline__ uint32_t top_bits(const Raw8<float>& r) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, r.w[i] & 0x7fffffffu);
  return top;
}
__device__ __forceinline__ uint32_t top_bits(const Raw8<uint16_t>& r) {
  typedef unsigned short v2u __attribute__((ext_vector_type(2)));
  v2u m = __builtin_bit_cast(v2u, r.w[0] & 0x7fff7fffu);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2u, r.w[i] & 0x7fff7fffu));
  return (uint32_t)max(m.x, m.y) << 16;
}
// The larger of two neighbouring lanes' values, and of the four lanes of a quad.
__device__ __forceinline__ uint32_t pair_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = pair_max(v);
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));
}
// The codes of eight elements, low nibble first (zeros where the block is bad).
__device__ __forceinline__ uint32_t codes8(const Raw8<float>& r, const MxScale& s) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(r.w[0]), __uint_as_float(r.w[1]), s.scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(r.w[2]), __uint_as_float(r.w[3]), s.scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(r.w[4]), __uint_as_float(r.w[5]), s.scale, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(r.w[6]), __uint_as_float(r.w[7]), s.scale, 3);
  return s.bad ? 0 : q;
}
__device__ __forceinline__ uint32_t codes8(const Raw8<uint16_t>& r, const MxScale& s) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, r.w[0]), s.scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, r.w[1]), s.scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, r.w[2]), s.scale, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, r.w[3]), s.scale, 3);
  return s.bad ? 0 : q;
}

// Two fp32 values to bf16 bits, to nearest with ties to even (one instruction; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const v2f f = {lo, hi};
  const v2bf b = __builtin_convertvector(f, v2bf);
  return __builtin_bit_cast(uint32_t, b);
}
__device__ __forceinline__ uint16_t bf16_bits(float f) { return (uint16_t)bf16_pair(f, 0.0f); }

// Eight fp32 values to a row; only the first n are written.
__device__ __forceinline__ void store8(float* p, int64_t n, const float (&v)[8]) {
  if (n >= 8) {
    __builtin_memcpy(p, v, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int64_t n, const float (&v)[8]) {
  if (n >= 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    __builtin_memcpy(p, w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = bf16_bits(v[i]);
  }
}

// store8 past the caches (quantiser with values, 6912 x 2560 fp32: 28.0 us, 35.2 with ordinary stores;
// layer norm 8192 x 8192 bf16 61 and 65 us).  Not for rows that start inside a 16-byte piece, whose
// partial lines it would write one by one (quantiser, 1003 x 7001 bf16: 9.8 against 9.1 us):
// whole_pieces tells.  The choice goes by the row length alone: outputs that the caches would hold are
// stored past them too, and what that costs a call that reads them at once has not been measured.
__host__ __device__ __forceinline__ bool whole_pieces(int64_t K) { return K % 8 == 0; }
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef v4u v4u_unaligned __attribute__((aligned(2)));
template <typename T>
__device__ __forceinline__ void stream8(T* p, int64_t n, const float (&v)[8], bool stream) {
  if (n < 8 || !stream) {
    store8(p, n, v);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4u w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[4 * h + i]);
      __builtin_nontemporal_store(w, reinterpret_cast<v4u_unaligned*>(p + 4 * h));
    }
  } else {
    v4u w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    __builtin_nontemporal_store(w, reinterpret_cast<v4u_unaligned*>(p));
  }
}

// Global memory, where the compiler cannot tell by itself.
using GlobalBytes = const __attribute__((address_space(1))) uint8_t*;
using GlobalV4i = const __attribute__((address_space(1))) v4i*;
using GlobalInt = const __attribute__((address_space(1))) int*;

// A pointer that is the same in every lane, into scalar registers.
template <typename T>
__device__ __forceinline__ T* uniform_ptr(T* p) {
  const uint64_t v = (uint64_t)p;
  return (T*)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
              (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// Launchers (sizes and pointers validated by the C ABI).
hipError_t launch_mx_quant(const void* X, int bf16, int64_t R, int64_t K, uint8_t* codes, uint8_t* scales,
                           void* values, hipStream_t s);
hipError_t launch_mx_decode(const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                            const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, int ybf16,
                            hipStream_t s);

// Few tokens (M <= 16) whose codes fit LDS, in one launch: src 0: x as codes and scales, 1: bf16, 2:
// fp32 x[M][K], quantised by every workgroup.
struct MxFewPlan {
  bool ok = false;
  int waves = 0;
  int64_t groups = 0;  // workgroups
  int64_t lds = 0;     // bytes
};
MxFewPlan plan_mx_few(int64_t M, int64_t N, int64_t K, int src);
hipError_t launch_mx_few(const uint8_t* codes, const uint8_t* scales, const void* x, const uint8_t* xscales, int src,
                         int64_t M, int64_t N, int64_t K, void* Y, int ybf16, hipStream_t s);

// Launch plan of the decode kernel.
struct MxDecodePlan {
  int waves = 4;       // waves per workgroup; they split the column groups
  int tg = 1;          // token groups of 16 per workgroup
  int rb = 1;          // row blocks per workgroup
  int64_t gx = 0, gy = 0;
};
MxDecodePlan plan_mx_decode(int64_t M, int64_t N, int64_t K);
// Whether the decode kernel is estimated to be faster than the GEMM.
bool mx_decode_wins(int64_t M, int64_t N, int64_t K);

// Launch plan of the GEMM: output tiles of tile_m tokens x tile_n outputs.
struct MxGemmPlan {
  int64_t tile_m = 128, tile_n = 128;
  int64_t tiles_m = 0, tiles_n = 0;
  int64_t band = 1;  // token tiles of a band of the tile order
};
MxGemmPlan plan_mx_gemm(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_gemm(const uint8_t* codes, const uint8_t* scales, const uint8_t* xcodes,
                          const uint8_t* xscales, int64_t M, int64_t N, int64_t K, void* Y, int ybf16,
                          hipStream_t s);

}  // namespace bl
