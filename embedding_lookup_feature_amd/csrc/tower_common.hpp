// tower_common.hpp -- what the dense-tower operators share: activations and their
// derivatives, the counter-based dropout mask, vectors of eight columns at any alignment, and
// the entry points' host-side checks.
#pragma once

#include <cmath>
#include <cstdio>
#include <exception>
#include <string>
#include <type_traits>

#include "el_internal.hpp"
#include "el_mfma.hpp"
#include "embtower.h"

namespace el {

// ---------------------------------------------------------------------------------------
// Eight consecutive columns as floats.  gfx950 takes 16-byte accesses at any element
// alignment, so one vector type serves aligned and unaligned rows; `n` < 8 (the last columns
// of a row that is no multiple of 8 wide) never touches memory past the row.
// ---------------------------------------------------------------------------------------
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x4 u32x4_f32 __attribute__((aligned(4)));

// The raw bits of eight columns: one 16-byte vector for 16-bit types, two for fp32.
template <class T>
struct Raw8 {
  static constexpr int W = sizeof(typename T::S) == 4 ? 2 : 1;
  u32x4 v[W];
};

template <class T>
__device__ inline Raw8<T> load8_raw(const typename T::S* p) {
  Raw8<T> r;
  if constexpr (Raw8<T>::W == 2) {
    r.v[0] = *reinterpret_cast<const u32x4_f32*>(p);
    r.v[1] = *reinterpret_cast<const u32x4_f32*>(p + 4);
  } else {
    r.v[0] = *reinterpret_cast<const u32x4_any*>(p);
  }
  return r;
}

typedef uint32_t u32_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x2 u32x2_f32 __attribute__((aligned(4)));

// The first n (1 .. 8) of the eight, zeros after them: a partial vector in pieces of 4, 2 and
// 1 elements.  Against one load per element: 23.4 against 24.4 us for a forward dense layer of
// odd sizes.  (Stores stay one per element: in pieces they cost the activation's backward at
// odd sizes 23.3 against 19.6 us.)
template <class T>
__device__ inline Raw8<T> load8_raw(const typename T::S* p, int n) {
  if (n >= 8) return load8_raw<T>(p);
  Raw8<T> r;
  if constexpr (Raw8<T>::W == 2) {
    uint32_t e[8] = {};
    if (n & 4) {
      const u32x4 q = *reinterpret_cast<const u32x4_f32*>(p);
      e[0] = q[0], e[1] = q[1], e[2] = q[2], e[3] = q[3];
    }
    if (n & 2) {
      const u32x2 q = *reinterpret_cast<const u32x2_f32*>(p + (n & 4));
      if (n & 4) e[4] = q[0], e[5] = q[1];
      else e[0] = q[0], e[1] = q[1];
    }
    if (n & 1) {
      const uint32_t q = __float_as_uint(p[n & 6]);
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        if ((n & 6) == i) e[i] = q;
    }
    r.v[0] = u32x4{e[0], e[1], e[2], e[3]};
    r.v[1] = u32x4{e[4], e[5], e[6], e[7]};
  } else {
    uint32_t w[4] = {};
    if (n & 4) {
      const u32x2 q = *reinterpret_cast<const u32x2_any*>(p);
      w[0] = q[0], w[1] = q[1];
    }
    if (n & 2) {
      const uint32_t q = *reinterpret_cast<const u32_any*>(p + (n & 4));
      if (n & 4) w[2] = q;
      else w[0] = q;
    }
    if (n & 1) {
      const uint32_t q = p[n & 6];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((n & 6) == 2 * i) w[i] = q;
    }
    r.v[0] = u32x4{w[0], w[1], w[2], w[3]};
  }
  return r;
}

template <class T>
__device__ inline void to_floats(const Raw8<T>& r, float* f) {
  if constexpr (Raw8<T>::W == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.v[i / 4][i % 4]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = T::to_f(static_cast<uint16_t>(r.v[0][i] & 0xffffu));
      f[2 * i + 1] = T::to_f(static_cast<uint16_t>(r.v[0][i] >> 16));
    }
  }
}

template <class T>
__device__ inline void store8(typename T::S* p, const float* f, int n) {
  if (n >= 8) {
    if constexpr (sizeof(typename T::S) == 4) {
      u32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(f[i]), b[i] = __float_as_uint(f[4 + i]);
      *reinterpret_cast<u32x4_f32*>(p) = a;
      *reinterpret_cast<u32x4_f32*>(p + 4) = b;
    } else {
      u32x4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i] = static_cast<uint32_t>(T::from_f(f[2 * i])) | (static_cast<uint32_t>(T::from_f(f[2 * i + 1])) << 16);
      *reinterpret_cast<u32x4_any*>(p) = a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = T::from_f(f[i]);
  }
}

// ---------------------------------------------------------------------------------------
// Activations: one function for the value and one for the derivative, the kind known at
// compile time.
// ---------------------------------------------------------------------------------------
// q = Phi(-|u|) and ex = exp(-u^2 / 2) = sqrt(2 pi) phi(u): the normal distribution function by
// the rational form 7.1.26 of Abramowitz and Stegun's Handbook (absolute error 1.5e-7 on erf,
// about one fp32 step of values near 1).  It shares its exponential with the derivative, and
// u Phi(u) = max(u, 0) - |u| q takes 13 plain instructions, one exp2 and one reciprocal.  In fp32
// u Phi(u) is off by at most 2.2e-7 for |u| <= 8; relative to itself that grows in the negative
// tail: 5e-5 at -3, 5e-4 at -4, 1.6e-3 at -5, 3.6e-3 at -6 (half a bf16 step is 3.9e-3).
__device__ inline float normal_tail(float u, float& ex) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.23164189f, fabsf(u), 1.f));
  ex = __builtin_amdgcn_exp2f(u * u * -0.72134752044448170f);
  float p = fmaf(0.5307027145f, t, -0.7265760135f);
  p = fmaf(p, t, 0.7107068705f);
  p = fmaf(p, t, -0.142248368f);
  p = fmaf(p, t, 0.127414796f);
  return p * t * ex;
}
__device__ inline float sigmoid(float u) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(u * -1.4426950408889634f));
}

template <int ACT>
__device__ inline float act_f(float u) {
  if constexpr (ACT == EL_ACT_RELU) return u > 0.f ? u : 0.f;
  if constexpr (ACT == EL_ACT_GELU) {
    float ex;
    // Phi(-64) is 0 in fp32, and no infinity meets it; minimum and maximum keep NaN
    const float a = __builtin_elementwise_minimum(fabsf(u), 64.f);
    return fmaf(-a, normal_tail(a, ex), __builtin_elementwise_maximum(u, 0.f));
  }
  if constexpr (ACT == EL_ACT_SILU) return u * sigmoid(u);
  return u;
}

template <int ACT>
__device__ inline float act_df(float u) {
  if constexpr (ACT == EL_ACT_RELU) return u > 0.f ? 1.f : 0.f;
  if constexpr (ACT == EL_ACT_GELU) {
    float ex;
    const float q = normal_tail(u, ex);
    return fmaf(u * ex, 0.39894228040143268f, u < 0.f ? q : 1.f - q);
  }
  if constexpr (ACT == EL_ACT_SILU) {
    const float s = sigmoid(u);
    return s * fmaf(u, 1.f - s, 1.f);
  }
  return 1.f;
}

// Eight values at once with the kind known at run time: one uniform branch per vector, for
// kernels whose other variants would be multiplied by the number of activations.
__device__ inline void act8(uint32_t act, float (&u)[8]) {
  switch (act) {
#define EL_ACT8_CASE(K)                                  \
  case K:                                                \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) u[i] = act_f<K>(u[i]); \
    break;
    EL_ACT8_CASE(EL_ACT_RELU)
    EL_ACT8_CASE(EL_ACT_GELU)
    EL_ACT8_CASE(EL_ACT_SILU)
#undef EL_ACT8_CASE
  }
}
// d[i] *= act'(u[i])
__device__ inline void act8_grad(uint32_t act, const float (&u)[8], float (&d)[8]) {
  switch (act) {
#define EL_ACT8_CASE(K)                                  \
  case K:                                                \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) d[i] *= act_df<K>(u[i]); \
    break;
    EL_ACT8_CASE(EL_ACT_RELU)
    EL_ACT8_CASE(EL_ACT_GELU)
    EL_ACT8_CASE(EL_ACT_SILU)
#undef EL_ACT8_CASE
  }
}

// ---------------------------------------------------------------------------------------
// The dropout mask (definition in embtower.h).
// ---------------------------------------------------------------------------------------
struct DropArgs {
  uint32_t top = 0;  // 2^16 T - 1 for T = 1 .. 65536; 0: nothing is dropped
  float scale = 1.f;
  uint32_t k0 = 0, k1 = 0;
  uint64_t offset = 0;
  const uint64_t* step = nullptr;
};

__device__ inline uint64_t drop_offset(const DropArgs& d) { return d.offset + (d.step ? d.step[0] : 0); }

// a ^ b ^ c in one instruction (a table of three bits; the compiler makes two).
__device__ inline uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) { return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96); }

// The eight 16-bit numbers of columns 8 group .. 8 group + 7 of row `row`, two per word.
__device__ inline u32x4 philox8(uint32_t group, uint32_t row, uint64_t offset, uint32_t k0, uint32_t k1) {
  uint32_t c0 = group, c1 = row, c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = xor3(static_cast<uint32_t>(b >> 32), c1, k0);
    c1 = static_cast<uint32_t>(b);
    c2 = xor3(static_cast<uint32_t>(a >> 32), c3, k1);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Number i (0 .. 7) of the eight is kept: number >= T, compared in the upper half of a word
// (`top` = 2^16 T - 1; T >= 1).
__device__ inline bool keep_of(const u32x4& bits, int i, uint32_t top) {
  return ((i & 1) ? bits[i >> 1] : bits[i >> 1] << 16) > top;
}

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
// Leaves the function with a status other than EL_OK.
#define EL_TRY(x)                    \
  do {                               \
    const el_status st_ = (x);       \
    if (st_ != EL_OK) return st_;    \
  } while (0)

namespace tower {

inline bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline el_status bad(const char* fn, const std::string& what) {
  return set_error(EL_ERR_INVALID_ARG, std::string(fn) + ": " + what);
}
inline el_status unsupported(const char* fn, const std::string& what) {
  return set_error(EL_ERR_UNSUPPORTED, std::string(fn) + ": " + what);
}

// Runs an entry point's body; no C++ exception leaves the C ABI.
template <class F>
el_status guarded(const char* fn, F&& body) noexcept {
  try {
    return body();
  } catch (const std::exception& e) {
    try {
      return set_error(EL_ERR_HIP, std::string(fn) + ": " + e.what());
    } catch (...) {
    }
  } catch (...) {
  }
  return EL_ERR_HIP;
}

// One [rows] x [cols] operand with row stride ld.
inline el_status check_rows(const char* fn, const char* name, const void* p, int64_t ld, int64_t cols,
                            bool needed, size_t elem) {
  if (!p) return needed ? bad(fn, std::string(name) + " is null") : EL_OK;
  if (!al(p, elem)) return bad(fn, std::string(name) + " must be aligned to its elements");
  if (ld < cols) return bad(fn, std::string("the row stride of ") + name + " must be >= its columns");
  if (ld >= (int64_t{1} << 40)) return bad(fn, std::string("the row stride of ") + name + " must be < 2^40");
  return EL_OK;
}

inline el_status check_act(const char* fn, uint32_t act) {
  return act <= EL_ACT_SILU ? EL_OK : bad(fn, "unknown activation");
}

// drop (or NULL) as the kernels take it.
inline el_status drop_args(const char* fn, const el_dropout* drop, DropArgs* out) {
  *out = DropArgs{};
  if (!drop) return EL_OK;
  if (!(drop->p >= 0.0 && drop->p <= 1.0)) return bad(fn, "the dropout probability must be in [0, 1]");
  if (!al(drop->step, 8)) return bad(fn, "dropout step must be 8-byte aligned");
  const uint64_t T = static_cast<uint64_t>(std::nearbyint(drop->p * 65536.0));
  out->top = T ? static_cast<uint32_t>((T << 16) - 1) : 0u;
  out->scale = T < 65536u ? static_cast<float>(65536.0 / (65536.0 - T)) : 0.f;
  out->k0 = static_cast<uint32_t>(drop->seed);
  out->k1 = static_cast<uint32_t>(drop->seed >> 32);
  out->offset = drop->offset;
  out->step = drop->step;
  return EL_OK;
}

inline el_status check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
  if (need == 0) return EL_OK;
  if (!ws || !al(ws, 256))
    return set_error(EL_ERR_WORKSPACE, std::string(fn) + ": workspace must be non-null and 256-byte aligned");
  if (have < need) {
    char buf[160];
    std::snprintf(buf, sizeof buf, "%s: workspace of %zu bytes, %zu needed", fn, have, need);
    return set_error(EL_ERR_WORKSPACE, buf);
  }
  return EL_OK;
}

// Calls f with the activation as a compile-time constant.
template <class F>
void with_act(uint32_t act, F&& f) {
  switch (act) {
    case EL_ACT_RELU: f(std::integral_constant<int, EL_ACT_RELU>{}); break;
    case EL_ACT_GELU: f(std::integral_constant<int, EL_ACT_GELU>{}); break;
    case EL_ACT_SILU: f(std::integral_constant<int, EL_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, EL_ACT_NONE>{}); break;
  }
}

}  // namespace tower
}  // namespace el
