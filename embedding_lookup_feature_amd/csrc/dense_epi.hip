// dense_epi.hip -- a dense layer with bias, activation, dropout and residual in its epilogue,
// and its backward.
//
//   forward      y  = residual + drop(act(x w^T + bias)),  pre = x w^T + bias
//   data grad    dx = dz w + dres,  dzb = drop(dx * act'(pre))
//   weight grad  dw = dz^T x,  db = column sums of dz
//
// The three products are one kernel over operands P (output rows) and Q (output columns),
// out[r][c] = sum_k P(r, k) Q(c, k), each operand either reduction-contiguous (element (i, k)
// at i * ld + k) or output-contiguous (at k * ld + i).
#include "tower_common.hpp"

namespace el {
namespace {

enum Product { FWD = 0, DGRAD = 1, WGRAD = 2 };

struct GemmArgs {
  const uint16_t *P, *Q;
  long ldp, ldq;
  int R, C;        // output rows, columns
  int red;         // reduction length
  int per_split;   // reduction per split (weight gradient)
  int tiles_c;     // column tiles
  int tiles;       // tiles of one split
  int total;       // tiles of all splits
  // forward: out = y, aux = pre (or null), add = residual (or null)
  // data gradient: out = dx, aux = dzb (or null), add = dres (or null), pre = the layer below's
  // weight gradient: part = fp32 [split][R][C]
  const uint16_t *add, *pre;
  uint16_t *out, *aux;
  long ldadd, ldpre, ldo, ldaux;
  const float* bias;
  float* part;
  DropArgs drop;
};

// The epilogue of one output group: columns c .. c+n-1 (c a multiple of 8, n <= 8) of row r.
template <class T, int PROD, int ACT>
__device__ inline void epilogue8(const GemmArgs& a, uint64_t offset, int r, int c, int n, float (&v)[8]) {
  float add[8], y[8];
  if (a.add) to_floats<T>(load8_raw<T>(a.add + r * a.ldadd + c, n), add);
  u32x4 bits = {};
  if (a.drop.threshold) bits = philox8(static_cast<uint32_t>(c) >> 3, static_cast<uint32_t>(r), offset, a.drop.k0, a.drop.k1);
  if constexpr (PROD == FWD) {
    if (a.bias)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) v[i] += a.bias[c + i];
    if (a.aux) store8<T>(a.aux + r * a.ldaux + c, v, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = act_f<ACT>(v[i]);
      if (a.drop.threshold) y[i] = keep_of(bits, i, a.drop.threshold) ? y[i] * a.drop.scale : 0.f;
      if (a.add) y[i] += add[i];
    }
    store8<T>(a.out + r * a.ldo + c, y, n);
  } else {
    if (a.add)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += add[i];
    store8<T>(a.out + r * a.ldo + c, v, n);
    if (a.aux) {
      float p[8];
      if (ACT != EL_ACT_NONE) to_floats<T>(load8_raw<T>(a.pre + r * a.ldpre + c, n), p);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = ACT == EL_ACT_NONE ? v[i] : v[i] * act_df<ACT>(p[i]);
        if (a.drop.threshold) y[i] = keep_of(bits, i, a.drop.threshold) ? y[i] * a.drop.scale : 0.f;
      }
      store8<T>(a.aux + r * a.ldaux + c, y, n);
    }
  }
}

// Eight consecutive reduction elements of operand row i, zeros outside.
template <bool RC>
__device__ inline u32x4 frag(const uint16_t* p, long ld, int i, int rows, int k, int kend) {
  u32x4 v = {};
  if (i < rows)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < kend) {
        const long at = RC ? i * ld + (k + e) : (k + e) * ld + i;
        v[e / 2] |= static_cast<uint32_t>(p[at]) << (16 * (e % 2));
      }
  return v;
}

// One 32 x 32 output tile per wavefront, fragments straight from global memory.
template <class T, bool P_RC, bool Q_RC, int PROD, int ACT>
__global__ __launch_bounds__(256) void k_dense_simple(GemmArgs a) {
  __shared__ float lds[4][32][36];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, l32 = lane & 31;
  const int tile = blockIdx.x * 4 + wave;  // the last workgroup's may lie past the end
  const int split = tile / a.tiles, t = tile - split * a.tiles;
  const int row0 = t / a.tiles_c * 32, col0 = t % a.tiles_c * 32;
  const int kbeg = split * a.per_split, kend = tile < a.total ? min(a.red, kbeg + a.per_split) : kbeg;
  f32x16 acc = {};
  for (int k = kbeg; k < kend; k += 16) {
    const u32x4 q = frag<Q_RC>(a.Q, a.ldq, col0 + l32, a.C, k + half * 8, kend);
    const u32x4 p = frag<P_RC>(a.P, a.ldp, row0 + l32, a.R, k + half * 8, kend);
    acc = mfma32<T>(q, p, acc);
  }
  // register r of the accumulator: column 8 (r / 4) + 4 half + r % 4, row l32
#pragma unroll
  for (int r = 0; r < 16; ++r) lds[wave][l32][acc_row(r, lane)] = acc[r];
  __syncthreads();
  if (tile >= a.total) return;
  if (PROD == WGRAD) {
    for (int i = lane; i < 1024; i += 64) {
      const int r = row0 + i / 32, c = col0 + i % 32;
      if (r < a.R && c < a.C) a.part[(static_cast<long>(split) * a.R + r) * a.C + c] = lds[wave][i / 32][i % 32];
    }
  } else {
    const uint64_t offset = a.drop.threshold ? drop_offset(a.drop) : 0;
    for (int i = lane; i < 128; i += 64) {
      const int r = row0 + i / 4, c = col0 + i % 4 * 8;
      if (r >= a.R || c >= a.C) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = lds[wave][i / 4][i % 4 * 8 + e];
      epilogue8<T, PROD, ACT>(a, offset, r, c, min(8, a.C - c), v);
    }
  }
}

// part[split][c] = sum over the split's rows of dz[m][c].
template <class T>
__global__ __launch_bounds__(256) void k_colsum(const uint16_t* dz, long ld, int M, int N, int per, float* part) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= N) return;
  const int m0 = blockIdx.y * per, m1 = min(M, m0 + per);
  float s = 0.f;
  for (int m = m0; m < m1; ++m) s += T::to_f(dz[m * ld + c]);
  part[static_cast<long>(blockIdx.y) * N + c] = s;
}

// out[i] = sum of the splits' part[split][i], in split order.
__global__ __launch_bounds__(256) void k_sum_parts(const float* part, long n, int splits, float* out) {
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int p = 0; p < splits; ++p) s += part[p * n + i];
  out[i] = s;
}

__global__ __launch_bounds__(256) void k_zero(float* p, long n) {
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

int ceil_div(long a, long b) { return static_cast<int>((a + b - 1) / b); }

// Batch slices of the weight gradient.
struct WgradPlan {
  int splits, per;
  size_t bytes;
};
WgradPlan plan_wgrad(int M, int K, int N) {
  const long tiles = static_cast<long>(ceil_div(N, 32)) * ceil_div(K, 32);
  long s = std::max<long>(1, 4096 / tiles);
  s = std::min<long>(s, ceil_div(M, 256));
  WgradPlan p;
  p.per = static_cast<int>((ceil_div(M, s) + 15l) / 16 * 16);
  p.splits = ceil_div(M, p.per);
  p.bytes = static_cast<size_t>(p.splits) * (static_cast<size_t>(N) * K + N) * 4;
  return p;
}

template <class T, bool P_RC, bool Q_RC, int PROD>
el_status launch_product(const char* fn, GemmArgs a, int splits, uint32_t act, hipStream_t st) {
  a.tiles_c = ceil_div(a.C, 32);
  const long tiles = static_cast<long>(ceil_div(a.R, 32)) * a.tiles_c;
  if (tiles * splits >= (1l << 25)) return tower::unsupported(fn, "the output has too many tiles for one launch");
  a.tiles = static_cast<int>(tiles);
  a.total = a.tiles * splits;
  const dim3 grid(ceil_div(tiles * splits, 4));
  if constexpr (PROD == WGRAD) {
    hipLaunchKernelGGL((k_dense_simple<T, P_RC, Q_RC, PROD, EL_ACT_NONE>), grid, dim3(256), 0, st, a);
  } else {
    tower::with_act(act, [&](auto A) {
      hipLaunchKernelGGL((k_dense_simple<T, P_RC, Q_RC, PROD, decltype(A)::value>), grid, dim3(256), 0, st, a);
    });
  }
  return check_launch(fn);
}

el_status check_dense_layer(const char* fn, const void* x, int64_t ldx, int32_t M, int32_t K, const void* w, int32_t N,
                            uint32_t act, el_dtype dtype) {
  if (dtype != EL_BF16 && dtype != EL_F16) {
    if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
    return tower::unsupported(fn, "dtype must be EL_BF16 or EL_F16");
  }
  if (M < 0) return tower::bad(fn, "M must be >= 0");
  if (K < 1) return tower::bad(fn, "K must be >= 1");
  if (N < 1) return tower::bad(fn, "N must be >= 1");
  // 2^31 elements of weights: partial sums and copies of them stay far inside 64-bit sizes
  if (static_cast<int64_t>(N) * K >= (int64_t{1} << 31)) return tower::unsupported(fn, "N * K must be < 2^31");
  if (!w) return tower::bad(fn, "w is null");
  if (!tower::al(w, 2)) return tower::bad(fn, "w must be aligned to its elements");
  const el_status s = tower::check_act(fn, act);
  if (s != EL_OK) return s;
  return tower::check_rows(fn, "x", x, ldx, K, M > 0, 2);
}

const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

}  // namespace
}  // namespace el

using namespace el;

#define EL_TRY(x)                    \
  do {                               \
    const el_status st_ = (x);       \
    if (st_ != EL_OK) return st_;    \
  } while (0)

extern "C" {

size_t el_dense_fwd_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  (void)M, (void)K, (void)N;
  return 0;
}

size_t el_dense_bwd_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  if (M < 1 || K < 1 || N < 1 || static_cast<int64_t>(N) * K >= (int64_t{1} << 31)) return 0;
  return plan_wgrad(M, K, N).bytes;
}

el_status el_dense_fwd(const void* x, int64_t ldx, int32_t M, int32_t K, const void* w, const float* bias, int32_t N,
                       uint32_t act, const el_dropout* drop, const void* residual, int64_t ldr, void* pre,
                       int64_t ldpre, void* y, int64_t ldy, el_dtype dtype, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  const char* fn = "el_dense_fwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_dense_layer(fn, x, ldx, M, K, w, N, act, dtype));
    GemmArgs a{};
    EL_TRY(tower::drop_args(fn, drop, &a.drop));
    if (!tower::al(bias, 4)) return tower::bad(fn, "bias must be aligned to its elements");
    EL_TRY(tower::check_rows(fn, "residual", residual, ldr, N, false, 2));
    EL_TRY(tower::check_rows(fn, "pre", pre, ldpre, N, false, 2));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, N, M > 0, 2));
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, el_dense_fwd_workspace_bytes(M, K, N)));
    if (M == 0) return EL_OK;
    a.P = u16(x), a.ldp = ldx, a.Q = u16(w), a.ldq = K, a.R = M, a.C = N, a.red = K, a.per_split = K;
    a.add = u16(residual), a.ldadd = ldr, a.aux = static_cast<uint16_t*>(pre), a.ldaux = ldpre;
    a.out = static_cast<uint16_t*>(y), a.ldo = ldy, a.bias = bias;
    return dtype == EL_BF16 ? launch_product<BF16T, true, true, FWD>(fn, a, 1, act, stream)
                            : launch_product<F16T, true, true, FWD>(fn, a, 1, act, stream);
  });
}

el_status el_dense_bwd(const void* x, int64_t ldx, int32_t M, int32_t K, const void* w, int32_t N, const void* dz,
                       int64_t lddz, const void* dres, int64_t lddres, void* dx, int64_t lddx, uint32_t act,
                       const el_dropout* drop, const void* pre, int64_t ldpre, void* dzb, int64_t lddzb, float* dw,
                       float* db, el_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "el_dense_bwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_dense_layer(fn, x, ldx, M, K, w, N, act, dtype));
    GemmArgs a{};
    EL_TRY(tower::drop_args(fn, drop, &a.drop));
    EL_TRY(tower::check_rows(fn, "dz", dz, lddz, N, M > 0, 2));
    EL_TRY(tower::check_rows(fn, "dres", dres, lddres, K, false, 2));
    EL_TRY(tower::check_rows(fn, "dx", dx, lddx, K, false, 2));
    EL_TRY(tower::check_rows(fn, "pre", pre, ldpre, K, dzb && act != EL_ACT_NONE && M > 0, 2));
    EL_TRY(tower::check_rows(fn, "dzb", dzb, lddzb, K, false, 2));
    if ((dzb || dres) && !dx) return tower::bad(fn, "dzb and dres need dx");
    if (!dw || !tower::al(dw, 4) || !tower::al(db, 4)) return tower::bad(fn, "dw must be non-null, dw and db aligned to their elements");
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, el_dense_bwd_workspace_bytes(M, K, N)));
    const long nk = static_cast<long>(N) * K;
    if (M == 0) {  // an empty batch: zero gradients, by a kernel (a captured fill stays a kernel node)
      hipLaunchKernelGGL(k_zero, dim3(ceil_div(nk, 256)), dim3(256), 0, stream, dw, nk);
      if (db) hipLaunchKernelGGL(k_zero, dim3(ceil_div(N, 256)), dim3(256), 0, stream, db, static_cast<long>(N));
      return check_launch(fn);
    }
    if (dx) {
      a.P = u16(dz), a.ldp = lddz, a.Q = u16(w), a.ldq = K, a.R = M, a.C = K, a.red = N, a.per_split = N;
      a.add = u16(dres), a.ldadd = lddres, a.out = static_cast<uint16_t*>(dx), a.ldo = lddx;
      a.aux = static_cast<uint16_t*>(dzb), a.ldaux = lddzb, a.pre = u16(pre), a.ldpre = ldpre;
      EL_TRY((dtype == EL_BF16 ? launch_product<BF16T, true, false, DGRAD>(fn, a, 1, act, stream)
                               : launch_product<F16T, true, false, DGRAD>(fn, a, 1, act, stream)));
    }
    const WgradPlan pl = plan_wgrad(M, K, N);
    float* part = static_cast<float*>(workspace);
    float* dbp = part + static_cast<size_t>(pl.splits) * nk;
    GemmArgs b{};
    b.P = u16(dz), b.ldp = lddz, b.Q = u16(x), b.ldq = ldx, b.R = N, b.C = K, b.red = M, b.per_split = pl.per;
    b.part = part;
    EL_TRY((dtype == EL_BF16 ? launch_product<BF16T, false, false, WGRAD>(fn, b, pl.splits, 0, stream)
                             : launch_product<F16T, false, false, WGRAD>(fn, b, pl.splits, 0, stream)));
    hipLaunchKernelGGL(k_sum_parts, dim3(ceil_div(nk, 256)), dim3(256), 0, stream, part, nk, pl.splits, dw);
    if (db) {
      const dim3 grid(ceil_div(N, 256), pl.splits);
      if (dtype == EL_BF16)
        hipLaunchKernelGGL((k_colsum<BF16T>), grid, dim3(256), 0, stream, u16(dz), lddz, M, N, pl.per, dbp);
      else
        hipLaunchKernelGGL((k_colsum<F16T>), grid, dim3(256), 0, stream, u16(dz), lddz, M, N, pl.per, dbp);
      hipLaunchKernelGGL(k_sum_parts, dim3(ceil_div(N, 256)), dim3(256), 0, stream, dbp, static_cast<long>(N), pl.splits, db);
    }
    return check_launch(fn);
  });
}

}  // extern "C"
