// dense_fp4.hip -- microscaled 4-bit numbers (e2m1): packing and unpacking, and the dense layer on
// them, y = residual + act(x4 w4^T + bias).
#include "micro.hpp"

namespace el {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kPad = 128;  // columns of a padded row: whole products of 128

struct PackArgs {
  const void* x;
  long ldx;
  int K, groups;  // columns, padded columns / 8
  int64_t items;  // M * groups
  uint8_t *codes, *scales;
};

// One thread owns eight columns; four neighbouring lanes a block of 32, which never crosses a row.
template <class T>
__global__ __launch_bounds__(kThreads) void k_fp4_pack(PackArgs a) {
  using S = typename T::S;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;
  const int64_t i = first + threadIdx.x;
  if (i >= a.items) return;
  const int64_t row0 = first / a.groups;  // uniform: one 64-bit division per workgroup
  const uint32_t local = static_cast<uint32_t>(first - row0 * a.groups) + threadIdx.x;
  const uint32_t dr = local / static_cast<uint32_t>(a.groups), grp = local - dr * a.groups;
  const int n = a.K - static_cast<int>(grp) * 8;
  float v[8] = {};
  if (n > 0) to_floats<T>(load8_raw<T>(static_cast<const S*>(a.x) + (row0 + dr) * a.ldx + grp * 8l, n), v);
  uint32_t byte;
  const uint32_t q = pack4(v, byte);
  reinterpret_cast<uint32_t*>(a.codes)[i] = q;
  if ((threadIdx.x & 3) == 0) a.scales[i >> 2] = static_cast<uint8_t>(byte);
}

struct UnpackArgs {
  const uint8_t *codes, *scales;
  void* y;
  long ldy;
  int K, groups, vecs;
  int64_t items;  // M * vecs
};
template <class T>
__global__ __launch_bounds__(kThreads) void k_fp4_unpack(UnpackArgs a) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;
  if (first + threadIdx.x >= a.items) return;
  const int64_t row0 = first / a.vecs;
  const uint32_t local = static_cast<uint32_t>(first - row0 * a.vecs) + threadIdx.x;
  const uint32_t dr = local / static_cast<uint32_t>(a.vecs), grp = local - dr * a.vecs;
  const int64_t row = row0 + dr, i = row * a.groups + grp;
  float v[8];
  unpack4(reinterpret_cast<const uint32_t*>(a.codes)[i], a.scales[i >> 2], v);
  store8<T>(static_cast<typename T::S*>(a.y) + row * a.ldy + grp * 8l, v, a.K - static_cast<int>(grp) * 8);
}

struct DenseArgs {
  const uint8_t *xc, *xs, *wc, *ws;
  int M, N, steps;  // steps of 128 columns
  const float* bias;
  const uint16_t* add;
  uint16_t* out;
  long ldadd, ldo;
  uint32_t act;
};

// 16 x 16 outputs from 128 columns: lane l holds row l % 16 of each operand, the block of 32 columns
// l / 16, and that block's scale byte; the accumulators of lane l are rows 4 (l / 16) .. +3 of the
// first operand and row l % 16 of the second.
__device__ inline f32x4 mfma_fp4(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb, const f32x4& c) {
  const i32x8 av = {static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]), 0, 0, 0, 0};
  const i32x8 bv = {static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3]), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, static_cast<int>(sa), 0, static_cast<int>(sb));
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_dense_fp4(DenseArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int tiles_c = (a.N + 63) / 64;
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int row0 = tr * 64 + (wave >> 1) * 32, col0 = tc * 64 + (wave & 1) * 32;
  f32x4 acc[2][2] = {};
  for (int k = 0; k < a.steps; ++k) {
    u32x4 x[2], w[2];
    uint32_t xs[2], ws[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long r = min(row0 + i * 16 + l16, a.M - 1), c = min(col0 + i * 16 + l16, a.N - 1);
      x[i] = *reinterpret_cast<const u32x4*>(a.xc + ((r * a.steps + k) * 4 + g) * 16);
      w[i] = *reinterpret_cast<const u32x4*>(a.wc + ((c * a.steps + k) * 4 + g) * 16);
      xs[i] = a.xs[(r * a.steps + k) * 4 + g];
      ws[i] = a.ws[(c * a.steps + k) * 4 + g];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma_fp4(w[i], ws[i], x[j], xs[j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = row0 + j * 16 + l16, c = col0 + i * 16 + g * 4;
      if (r >= a.M) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (c + e >= a.N) continue;
        float v[8] = {acc[i][j][e] + (a.bias ? a.bias[c + e] : 0.f)};
        act8(a.act, v);
        if (a.add) v[0] += T::to_f(a.add[r * a.ldadd + c + e]);
        a.out[r * a.ldo + c + e] = T::from_f(v[0]);
      }
    }
}

template <class F>
void with_type(el_dtype dtype, F&& f) {
  if (dtype == EL_F32) f(F32T{});
  else if (dtype == EL_F16) f(F16T{});
  else f(BF16T{});
}

long ceil_div(long a, long b) { return (a + b - 1) / b; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
long steps_of(long K) { return ceil_div(K, kPad); }
size_t code_bytes(long M, long K) { return round256(static_cast<size_t>(M) * steps_of(K) * kPad / 2); }
size_t scale_bytes(long M, long K) { return round256(static_cast<size_t>(M) * steps_of(K) * kPad / kMicroBlock); }

void launch_pack(const void* x, long ldx, int M, int K, el_dtype dtype, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  PackArgs a{x, ldx, K, static_cast<int>(steps_of(K) * kPad / 8), 0, codes, scales};
  a.items = static_cast<int64_t>(M) * a.groups;
  with_type(dtype, [&](auto t) {
    hipLaunchKernelGGL((k_fp4_pack<decltype(t)>), dim3(static_cast<unsigned>(ceil_div(a.items, kThreads))), dim3(kThreads), 0, st, a);
  });
}

bool dense_fp4_sizes_ok(int64_t M, int64_t K, int64_t N) {
  return M >= 1 && K >= 1 && N >= 1 && K <= tower::kMaxMicroCols && N <= tower::kMaxMicroCols && N * K < (int64_t{1} << 29) &&
         ceil_div(M, 256) * ceil_div(N, 256) < (1l << 21) && M * tower::pad_to(K, kPad) <= (int64_t{1} << 34);
}

}  // namespace
}  // namespace el

using namespace el;

extern "C" {

el_status el_fp4_pack(const void* x, int64_t ldx, int32_t M, int32_t K, el_dtype dtype, uint8_t* codes, uint8_t* scales,
                      hipStream_t stream) {
  const char* fn = "el_fp4_pack";
  return tower::guarded(fn, [&]() -> el_status {
    if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
    EL_TRY(tower::check_packed_sizes(fn, M, K, kPad));
    EL_TRY(tower::check_rows(fn, "x", x, ldx, K, M > 0, dtype_size(dtype)));
    EL_TRY(tower::check_packed(fn, "the output", codes, scales, M > 0));
    if (M == 0) return EL_OK;
    launch_pack(x, ldx, M, K, dtype, codes, scales, stream);
    return check_launch(fn);
  });
}

el_status el_fp4_unpack(const uint8_t* codes, const uint8_t* scales, int32_t M, int32_t K, void* y, int64_t ldy,
                        el_dtype dtype, hipStream_t stream) {
  const char* fn = "el_fp4_unpack";
  return tower::guarded(fn, [&]() -> el_status {
    if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
    EL_TRY(tower::check_packed_sizes(fn, M, K, kPad));
    EL_TRY(tower::check_packed(fn, "x", codes, scales, M > 0));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, K, M > 0, dtype_size(dtype)));
    if (M == 0) return EL_OK;
    UnpackArgs a{codes, scales, y, ldy, K, static_cast<int>(steps_of(K) * kPad / 8), (K + 7) / 8, 0};
    a.items = static_cast<int64_t>(M) * a.vecs;
    with_type(dtype, [&](auto t) {
      hipLaunchKernelGGL((k_fp4_unpack<decltype(t)>), dim3(static_cast<unsigned>(ceil_div(a.items, kThreads))), dim3(kThreads), 0, stream, a);
    });
    return check_launch(fn);
  });
}

size_t el_dense_fwd_fp4_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  return dense_fp4_sizes_ok(M, K, N) ? code_bytes(M, K) + scale_bytes(M, K) : 0;
}

el_status el_dense_fwd_fp4(const void* x, int64_t ldx, int32_t M, int32_t K, const uint8_t* w_codes,
                           const uint8_t* w_scales, const float* bias, int32_t N, uint32_t act, const void* residual,
                           int64_t ldr, void* y, int64_t ldy, el_dtype dtype, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  const char* fn = "el_dense_fwd_fp4";
  return tower::guarded(fn, [&]() -> el_status {
    if (dtype != EL_BF16 && dtype != EL_F16)
      return dtype_valid(dtype) ? tower::unsupported(fn, "dtype must be EL_BF16 or EL_F16") : tower::bad(fn, "unknown dtype");
    if (M < 0) return tower::bad(fn, "M must be >= 0");
    if (K < 1) return tower::bad(fn, "K must be >= 1");
    if (N < 1) return tower::bad(fn, "N must be >= 1");
    if (!dense_fp4_sizes_ok(std::max(M, 1), K, N))
      return tower::unsupported(fn, "K and N must be <= 2^20, N * K < 2^29, outputs below 2^21 tiles of 256 x 256 and M times padded K <= 2^34");
    EL_TRY(tower::check_act(fn, act));
    EL_TRY(tower::check_packed(fn, "w", w_codes, w_scales, true));
    if (!tower::al(bias, 4)) return tower::bad(fn, "bias must be aligned to its elements");
    EL_TRY(tower::check_rows(fn, "x", x, ldx, K, M > 0, 2));
    EL_TRY(tower::check_rows(fn, "residual", residual, ldr, N, false, 2));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, N, M > 0, 2));
    if (M == 0) return EL_OK;
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, el_dense_fwd_fp4_workspace_bytes(M, K, N)));
    DenseArgs a{};
    uint8_t* xc = static_cast<uint8_t*>(workspace);
    uint8_t* xs = xc + code_bytes(M, K);
    launch_pack(x, ldx, M, K, dtype, xc, xs, stream);
    EL_TRY(check_launch(fn));
    a.xc = xc, a.xs = xs, a.wc = w_codes, a.ws = w_scales, a.M = M, a.N = N, a.steps = static_cast<int>(steps_of(K));
    a.bias = bias, a.add = static_cast<const uint16_t*>(residual), a.ldadd = ldr;
    a.out = static_cast<uint16_t*>(y), a.ldo = ldy, a.act = act;
    const dim3 grid(static_cast<unsigned>(ceil_div(M, 64) * ceil_div(N, 64)));
    if (dtype == EL_BF16) hipLaunchKernelGGL((k_dense_fp4<BF16T>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((k_dense_fp4<F16T>), grid, dim3(kThreads), 0, stream, a);
    return check_launch(fn);
  });
}

}  // extern "C"
