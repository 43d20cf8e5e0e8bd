// micro.hpp -- microscaled 8-bit (e4m3) and 4-bit (e2m1) numbers: 32 columns share a power of two
// (the format stands in embblock.h).
#pragma once

#include "embblock.h"
#include "tower_common.hpp"

namespace el {

constexpr int kMicroBlock = 32;
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight values as four words, two to a word in one conversion.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
template <class T>
__device__ inline u32x4 to_16bit(const float (&f)[8]) {
  u32x4 a;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 p = {f[2 * i], f[2 * i + 1]};
    uint32_t w;
    if constexpr (T::code == EL_BF16) w = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
    else w = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, f16x2));
    a[i] = w;
  }
  return a;
}

// 2^e of a scale byte e + 127 (1 .. 254); 255 (NaN) gives infinity.
__device__ inline float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// The scale byte of a block whose largest finite magnitude has the bits `amax`, for T = top: the
// smallest e with amax <= top 2^e.  With top = (1 + f) 2^t and amax = (1 + g) 2^E that is E - t,
// and one more where g > f.  (Subnormal magnitudes have the exponent bits 0, E = -127 or less.)
template <bool FP4>
__device__ inline uint32_t scale_byte(uint32_t amax) {
  constexpr uint32_t top_frac = FP4 ? 0x400000u : 0x600000u;  // 6 = 1.5 * 2^2, 448 = 1.75 * 2^8
  constexpr int top_exp = FP4 ? 2 : 8;
  const int e = static_cast<int>(amax >> 23) - top_exp + ((amax & 0x7fffffu) > top_frac);
  return static_cast<uint32_t>(max(e, 1));
}

// Largest magnitude over the four lanes that hold a block of 32 columns, eight each.
__device__ inline uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xf, 0xf, true)));  // lane ^ 1
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xf, 0xf, true)));  // lane ^ 2
}

// This lane's eight columns of a block held by four neighbouring lanes, as 8-bit codes; the block's
// scale byte to `byte`.
struct Codes8 { uint32_t lo, hi; };
__device__ inline Codes8 pack8(const float (&v)[8], uint32_t& byte) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = __float_as_uint(v[i]) & 0x7fffffffu;
    amax = max(amax, m < 0x7f800000u ? m : 0u);
  }
  byte = scale_byte<false>(quad_max(amax));
  const float inv = __uint_as_float((254u - byte) << 23);  // 2^-e, exact (e <= 120)
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // an infinity becomes NaN; the conversion keeps NaN
    const uint32_t m = __float_as_uint(v[i]) & 0x7fffffffu;
    q[i] = m == 0x7f800000u ? __uint_as_float(0x7fc00000u) : v[i] * inv;
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return Codes8{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}
__device__ inline void unpack8(uint32_t lo, uint32_t hi, float scale, float (&v)[8]) {
  // (the conversion multiplies by the scale)
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, scale, false), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, scale, true);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, scale, false), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, scale, true);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
}

// The same in 4 bits: eight codes in one word.
__device__ inline uint32_t pack4(const float (&v)[8], uint32_t& byte) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  amax = quad_max(amax);  // NaN and infinities compare as the largest
  if (amax >= 0x7f800000u) {
    byte = 255u;
    return 0u;
  }
  byte = scale_byte<true>(amax);
  const float inv = __uint_as_float((254u - byte) << 23);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0] * inv, v[1] * inv, 1.f, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2] * inv, v[3] * inv, 1.f, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4] * inv, v[5] * inv, 1.f, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6] * inv, v[7] * inv, 1.f, 3);
  return q;
}
__device__ inline void unpack4(uint32_t q, uint32_t byte, float (&v)[8]) {
  const float scale = scale_of(byte);
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 3);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
  if (byte == 255u)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(0x7fc00000u);
}

// Eight columns from c of a row of `cols` (at least eight), by whole loads without a branch: a vector
// that the row's end cuts is loaded from the row's last eight, and settle8 moves its columns to the front,
// zeros behind them (all zeros from c = cols on).  Apart, so that the load can be in flight meanwhile.
template <class T>
__device__ inline Raw8<T> load8_cut(const typename T::S* row, int c, int cols) {
  return load8_raw<T>(row + min(c, cols - 8));
}
template <class T>
__device__ inline void settle8(Raw8<T>& r, int c, int cols) {
  const int s = c + 8 - cols;
  if (s <= 0) return;
  if constexpr (Raw8<T>::W == 2) {
    uint32_t w[8] = {r.v[0][0], r.v[0][1], r.v[0][2], r.v[0][3], r.v[1][0], r.v[1][1], r.v[1][2], r.v[1][3]};
#pragma unroll
    for (int b = 4; b; b >>= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = s & b ? (e + b < 8 ? w[(e + b) & 7] : 0u) : w[e];
    r.v[0] = s < 8 ? u32x4{w[0], w[1], w[2], w[3]} : u32x4{0, 0, 0, 0};
    r.v[1] = s < 8 ? u32x4{w[4], w[5], w[6], w[7]} : u32x4{0, 0, 0, 0};
  } else {
    u32x4 v = r.v[0];
    if (s & 4) v = u32x4{v[2], v[3], 0, 0};
    if (s & 2) v = u32x4{v[1], v[2], v[3], 0};
    if (s & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    r.v[0] = s < 8 ? v : u32x4{0, 0, 0, 0};
  }
}
// The same at once, of a row of any width; c < cols.
template <class T>
__device__ inline Raw8<T> load8_row(const typename T::S* row, int c, int cols) {
  if (cols < 8) return load8_raw<T>(row + c, cols - c);
  Raw8<T> r = load8_cut<T>(row, c, cols);
  settle8<T>(r, c, cols);
  return r;
}

// The first n of eight values, a whole vector in 16-bit pairs.
template <class T>
__device__ inline void put_whole8(typename T::S* p, const float (&v)[8], int n) {
  if constexpr (sizeof(typename T::S) == 2) {
    if (n >= 8) {
      *reinterpret_cast<u32x4_any*>(p) = to_16bit<T>(v);
      return;
    }
  }
  store8<T>(p, v, n);
}

namespace tower {

constexpr int kMaxMicroCols = 1 << 20;
inline int64_t pad_to(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Sizes of a packed [M][K] array whose rows are padded to `pad` columns.  (2^34 elements are 2^31
// threads of eight.)
inline el_status check_packed_sizes(const char* fn, int64_t M, int64_t K, int pad, int pad_rows = 1) {
  if (M < 0) return bad(fn, "the number of rows must be >= 0");
  if (K < 1) return bad(fn, "K must be >= 1");
  if (K > kMaxMicroCols) return unsupported(fn, "K must be <= 2^20");
  if (pad_to(M, pad_rows) * pad_to(K, pad) > (int64_t{1} << 34)) return unsupported(fn, "padded rows times padded columns must be <= 2^34");
  return EL_OK;
}
inline el_status check_packed(const char* fn, const char* name, const void* codes, const void* scales, bool needed) {
  if (!codes || !scales) return needed ? bad(fn, std::string("the codes and scales of ") + name + " must not be null") : EL_OK;
  if (!al(codes, 16)) return bad(fn, std::string("the codes of ") + name + " must be 16-byte aligned");
  if (!al(scales, 4)) return bad(fn, std::string("the scales of ") + name + " must be 4-byte aligned");
  return EL_OK;
}

}  // namespace tower
}  // namespace el
