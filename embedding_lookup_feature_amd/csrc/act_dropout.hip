// act_dropout.hip -- activation, dropout from a counter-based generator and residual, forward
// and backward, as one pass over the data.
//
//   y  = residual + drop(act(x)),      dx = drop(dy * act'(x))
//
// One thread owns eight consecutive columns of a row, which share one Philox4x32-10 call (eight
// 16-bit numbers), so the mask costs ten rounds of two 32 x 32 -> 64 bit products per eight
// elements and is never read or written.
//
// Bound by memory: 65536 x 1024, bf16, GELU, dropout and residual (402 MB) 76.6 us, 5.3 TB/s, the
// rate of a copy; the gradient of 16411 x 479, fp32, SiLU and dropout (94 MB) 19.7 us, 4.8 TB/s.
// One vector per thread and no loop: the wavefronts of the next workgroups hide the loads, and
// the smallest calls, which are latency, stay one load, the arithmetic and one store (64 x 128:
// 2.1 us, the time of an empty kernel).
#include "tower_common.hpp"

namespace el {
namespace {

struct RowsArgs {
  const void *a, *b;  // forward: x, residual; backward: dy, x
  void* y;
  long lda, ldb, ldy;
  int N, groups;      // columns, ceil(N / 8)
  int64_t items;      // M * groups
  DropArgs drop;
};

constexpr int kThreads = 256;

template <class T, int ACT, bool BWD>
__global__ __launch_bounds__(kThreads) void k_act_dropout(RowsArgs p) {
  using S = typename T::S;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;
  if (first + threadIdx.x >= p.items) return;
  const int64_t row0 = first / p.groups;  // uniform: one 64-bit division per workgroup
  const uint32_t local = static_cast<uint32_t>(first - row0 * p.groups) + threadIdx.x;
  const uint32_t dr = local / static_cast<uint32_t>(p.groups), grp = local - dr * p.groups;
  const int64_t row = row0 + dr;
  const int n = p.N - static_cast<int>(grp) * 8;
  Raw8<T> ra = load8_raw<T>(static_cast<const S*>(p.a) + row * p.lda + grp * 8l, n), rb;
  if (p.b) rb = load8_raw<T>(static_cast<const S*>(p.b) + row * p.ldb + grp * 8l, n);
  float x[8], r[8];
  to_floats<T>(ra, x);
  if (p.b) to_floats<T>(rb, r);
  if constexpr (!BWD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = act_f<ACT>(x[i]);
  } else if constexpr (ACT != EL_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= act_df<ACT>(r[i]);
  }
  if (p.drop.top) {
    const u32x4 bits = philox8(grp, static_cast<uint32_t>(row), drop_offset(p.drop), p.drop.k0, p.drop.k1);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = keep_of(bits, i, p.drop.top) ? x[i] * p.drop.scale : 0.f;
  }
  if (!BWD && p.b)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] += r[i];
  store8<T>(static_cast<S*>(p.y) + row * p.ldy + grp * 8l, x, n);
}

template <class T, bool BWD>
void launch_typed(const RowsArgs& p, uint32_t act, hipStream_t st) {
  tower::with_act(act, [&](auto A) {
    const int64_t blocks = (p.items + kThreads - 1) / kThreads;
    hipLaunchKernelGGL((k_act_dropout<T, decltype(A)::value, BWD>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                       st, p);
  });
}

el_status launch_rows(const char* fn, RowsArgs p, int M, uint32_t act, el_dtype dtype, bool bwd, hipStream_t st) {
  p.groups = p.N / 8 + (p.N % 8 != 0);
  p.items = static_cast<int64_t>(M) * p.groups;
  if (p.items > 0xffffff00ll) return tower::unsupported(fn, "M * ceil(N / 8) must be < 2^32 - 255");  // threads of one launch
  const auto go = [&](auto t) {
    using T = decltype(t);
    bwd ? launch_typed<T, true>(p, act, st) : launch_typed<T, false>(p, act, st);
  };
  if (dtype == EL_F32) go(F32T{});
  else if (dtype == EL_F16) go(F16T{});
  else go(BF16T{});
  return check_launch(fn);
}

el_status check_common(const char* fn, int32_t M, int32_t N, uint32_t act, el_dtype dtype) {
  if (M < 0) return tower::bad(fn, "M must be >= 0");
  if (N < 1) return tower::bad(fn, "N must be >= 1");
  if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
  return tower::check_act(fn, act);
}

}  // namespace
}  // namespace el

using namespace el;

extern "C" {

el_status el_act_dropout_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t M,
                             int32_t N, uint32_t act, const el_dropout* drop, void* y, int64_t ldy,
                             el_dtype dtype, hipStream_t stream) {
  const char* fn = "el_act_dropout_fwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_common(fn, M, N, act, dtype));
    RowsArgs p{};
    EL_TRY(tower::drop_args(fn, drop, &p.drop));
    const size_t e = dtype_size(dtype);
    EL_TRY(tower::check_rows(fn, "x", x, ldx, N, M > 0, e));
    EL_TRY(tower::check_rows(fn, "residual", residual, ldr, N, false, e));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, N, M > 0, e));
    if (M == 0) return EL_OK;
    p.a = x, p.b = residual, p.y = y, p.lda = ldx, p.ldb = ldr, p.ldy = ldy, p.N = N;
    return launch_rows(fn, p, M, act, dtype, false, stream);
  });
}

el_status el_act_dropout_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, int32_t M, int32_t N,
                             uint32_t act, const el_dropout* drop, void* dx, int64_t lddx, el_dtype dtype,
                             hipStream_t stream) {
  const char* fn = "el_act_dropout_bwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_common(fn, M, N, act, dtype));
    RowsArgs p{};
    EL_TRY(tower::drop_args(fn, drop, &p.drop));
    const size_t e = dtype_size(dtype);
    EL_TRY(tower::check_rows(fn, "dy", dy, lddy, N, M > 0, e));
    EL_TRY(tower::check_rows(fn, "x", x, ldx, N, M > 0 && act != EL_ACT_NONE, e));
    EL_TRY(tower::check_rows(fn, "dx", dx, lddx, N, M > 0, e));
    if (M == 0) return EL_OK;
    p.a = dy, p.b = act == EL_ACT_NONE ? nullptr : x, p.y = dx, p.lda = lddy, p.ldb = ldx, p.ldy = lddx, p.N = N;
    return launch_rows(fn, p, M, act, dtype, true, stream);
  });
}

}  // extern "C"
