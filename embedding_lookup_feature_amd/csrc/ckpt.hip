// ckpt.hip -- activations kept in 8 bits (microscaled e4m3): packing, and the activation with
// dropout and its gradient computed from them.
//
// Packing is bound by memory: 65536 x 1024 from bf16 41 us, 4.9 TB/s.  The activation is bound by
// instructions: with GELU and dropout the vector units are busy for 90 % of the forward's 61 us (3.3 TB/s)
// and 88 % of the backward's 75, some 260 and 310 issue slots of four cycles for eight values.  Twenty
// 64-bit products and twenty exclusive ors make the mask's number (the products, the reciprocals and the
// exponentials take four slots each); the conversions apply the scales, two values at a time.
// Two vectors a thread: no faster.
#include "micro.hpp"

namespace el {
namespace {

constexpr int kThreads = 256;

// One thread owns eight columns; four neighbouring lanes a block of 32, which never crosses a row.
struct PackArgs {
  const void* x;
  long ldx;
  int K, groups;  // columns, padded columns / 8
  int64_t items;  // M * groups
  uint8_t *codes, *scales;
};

template <class T>
__global__ __launch_bounds__(kThreads) void k_ckpt_pack(PackArgs a) {
  using S = typename T::S;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;
  const int64_t i = first + threadIdx.x;
  if (i >= a.items) return;
  const int64_t row0 = first / a.groups;  // uniform: one 64-bit division per workgroup
  const uint32_t local = static_cast<uint32_t>(first - row0 * a.groups) + threadIdx.x;
  const uint32_t dr = local / static_cast<uint32_t>(a.groups), grp = local - dr * a.groups;
  const int n = a.K - static_cast<int>(grp) * 8;
  float v[8] = {};
  if (n > 0) to_floats<T>(load8_row<T>(static_cast<const S*>(a.x) + (row0 + dr) * a.ldx, static_cast<int>(grp) * 8, a.K), v);
  uint32_t byte;
  const Codes8 q = pack8(v, byte);
  reinterpret_cast<uint2*>(a.codes)[i] = uint2{q.lo, q.hi};
  if ((threadIdx.x & 3) == 0) a.scales[i >> 2] = static_cast<uint8_t>(byte);
}

struct ActArgs {
  const uint8_t *codes, *scales;
  const void* dy;
  void* y;
  long lddy, ldy;
  int K, groups, vecs;  // columns, padded columns / 8, ceil(K / 8)
  int64_t items;        // M * vecs
  DropArgs drop;
};

// Outputs of 32 bits get GELU with an error relative to its value (0.5 u erfc(-u / sqrt 2)); for 16
// bits the tower's absolute 2.2e-7 is below half a step wherever the value counts.
template <class T, int ACT>
__device__ inline float value(float u) {
  if constexpr (ACT == EL_ACT_GELU && T::code == EL_F32) {
    // (erfc(64 / sqrt 2) is 0 in fp32, and no infinity meets it; the maximum keeps NaN)
    const float v = __builtin_elementwise_maximum(u, -64.f);
    return 0.5f * v * erfcf(-0.70710678118654752f * v);
  }
  return act_f<ACT>(u);
}
template <class T, int ACT>
__device__ inline float slope(float u) {
  if constexpr (ACT == EL_ACT_GELU && T::code == EL_F32)
    return fmaf(u * expf(-0.5f * u * u), 0.39894228040143268f, 0.5f * erfcf(-0.70710678118654752f * u));
  return act_df<ACT>(u);
}

template <class T, int ACT, bool BWD>
__global__ __launch_bounds__(kThreads) void k_ckpt_act(ActArgs a) {
  using S = typename T::S;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;
  if (first + threadIdx.x >= a.items) return;
  const int64_t row0 = first / a.vecs;
  const uint32_t local = static_cast<uint32_t>(first - row0 * a.vecs) + threadIdx.x;
  const uint32_t dr = local / static_cast<uint32_t>(a.vecs), grp = local - dr * a.vecs;
  const int64_t row = row0 + dr, i = row * a.groups + grp;
  const int n = a.K - static_cast<int>(grp) * 8;
  const uint2 q = reinterpret_cast<const uint2*>(a.codes)[i];
  const uint32_t byte = a.scales[i >> 2];
  float u[8], v[8];
  if (BWD) to_floats<T>(load8_row<T>(static_cast<const S*>(a.dy) + row * a.lddy, static_cast<int>(grp) * 8, a.K), v);
  unpack8(q.x, q.y, scale_of(byte), u);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = BWD ? v[e] * slope<T, ACT>(u[e]) : value<T, ACT>(u[e]);
  if (a.drop.top) {
    const u32x4 bits = philox8(grp, static_cast<uint32_t>(row), drop_offset(a.drop), a.drop.k0, a.drop.k1);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = keep_of(bits, e, a.drop.top) ? v[e] * a.drop.scale : 0.f;
  }
  put_whole8<T>(static_cast<S*>(a.y) + row * a.ldy + grp * 8l, v, n);
}

template <class F>
void with_type(el_dtype dtype, F&& f) {
  if (dtype == EL_F32) f(F32T{});
  else if (dtype == EL_F16) f(F16T{});
  else f(BF16T{});
}

unsigned blocks_of(int64_t items) { return static_cast<unsigned>((items + kThreads - 1) / kThreads); }

el_status run_act(const char* fn, const void* dy, int64_t lddy, const uint8_t* codes, const uint8_t* scales, int32_t M,
                  int32_t K, uint32_t act, const el_dropout* drop, void* y, int64_t ldy, const char* yname,
                  el_dtype dtype, bool bwd, hipStream_t stream) {
  if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
  EL_TRY(tower::check_packed_sizes(fn, M, K, kMicroBlock));
  EL_TRY(tower::check_act(fn, act));
  ActArgs a{};
  EL_TRY(tower::drop_args(fn, drop, &a.drop));
  EL_TRY(tower::check_packed(fn, "x", codes, scales, M > 0));
  const size_t e = dtype_size(dtype);
  if (bwd) EL_TRY(tower::check_rows(fn, "dy", dy, lddy, K, M > 0, e));
  EL_TRY(tower::check_rows(fn, yname, y, ldy, K, M > 0, e));
  if (M == 0) return EL_OK;
  a.codes = codes, a.scales = scales, a.dy = dy, a.lddy = lddy, a.y = y, a.ldy = ldy, a.K = K;
  a.groups = static_cast<int>(tower::pad_to(K, kMicroBlock) / 8), a.vecs = (K + 7) / 8;
  a.items = static_cast<int64_t>(M) * a.vecs;
  with_type(dtype, [&](auto t) {
    using T = decltype(t);
    tower::with_act(act, [&](auto A) {
      constexpr int ACT = decltype(A)::value;
      const dim3 grid(blocks_of(a.items));
      if (bwd) hipLaunchKernelGGL((k_ckpt_act<T, ACT, true>), grid, dim3(kThreads), 0, stream, a);
      else hipLaunchKernelGGL((k_ckpt_act<T, ACT, false>), grid, dim3(kThreads), 0, stream, a);
    });
  });
  return check_launch(fn);
}

}  // namespace
}  // namespace el

using namespace el;

extern "C" {

el_status el_ckpt_pack(const void* x, int64_t ldx, int32_t M, int32_t K, el_dtype dtype, uint8_t* codes,
                       uint8_t* scales, hipStream_t stream) {
  const char* fn = "el_ckpt_pack";
  return tower::guarded(fn, [&]() -> el_status {
    if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
    EL_TRY(tower::check_packed_sizes(fn, M, K, kMicroBlock));
    EL_TRY(tower::check_rows(fn, "x", x, ldx, K, M > 0, dtype_size(dtype)));
    EL_TRY(tower::check_packed(fn, "the output", codes, scales, M > 0));
    if (M == 0) return EL_OK;
    PackArgs a{x, ldx, K, static_cast<int>(tower::pad_to(K, kMicroBlock) / 8), 0, codes, scales};
    a.items = static_cast<int64_t>(M) * a.groups;
    with_type(dtype, [&](auto t) {
      hipLaunchKernelGGL((k_ckpt_pack<decltype(t)>), dim3(blocks_of(a.items)), dim3(kThreads), 0, stream, a);
    });
    return check_launch(fn);
  });
}

el_status el_ckpt_act_dropout_fwd(const uint8_t* codes, const uint8_t* scales, int32_t M, int32_t K, uint32_t act,
                                  const el_dropout* drop, void* y, int64_t ldy, el_dtype dtype, hipStream_t stream) {
  const char* fn = "el_ckpt_act_dropout_fwd";
  return tower::guarded(fn, [&]() -> el_status {
    return run_act(fn, nullptr, 0, codes, scales, M, K, act, drop, y, ldy, "y", dtype, false, stream);
  });
}

el_status el_ckpt_act_dropout_bwd(const void* dy, int64_t lddy, const uint8_t* codes, const uint8_t* scales, int32_t M,
                                  int32_t K, uint32_t act, const el_dropout* drop, void* dx, int64_t lddx,
                                  el_dtype dtype, hipStream_t stream) {
  const char* fn = "el_ckpt_act_dropout_bwd";
  return tower::guarded(fn, [&]() -> el_status {
    return run_act(fn, dy, lddy, codes, scales, M, K, act, drop, dx, lddx, "dx", dtype, true, stream);
  });
}

}  // extern "C"
