// dense_epi.hip -- a dense layer with bias, activation, dropout and residual in its epilogue,
// and its backward.
//
//   forward      y  = residual + drop(act(x w^T + bias)),  pre = x w^T + bias
//   data grad    dx = dz w + dres,  dzb = drop(dx * act'(pre))
//   weight grad  dw = dz^T x,  db = column sums of dz
//
// The three products are one kernel over operands P (output rows) and Q (output columns),
// out[r][c] = sum_k P(r, k) Q(c, k), each operand either reduction-contiguous (element (i, k)
// at i * ld + k: x, dz and w in the first two) or output-contiguous (at k * ld + i).
//
// Operands travel from global memory straight into LDS (no staging registers, no LDS store
// instructions), `ST` stages of BK reductions in a ring; a stage's slot is refilled as soon as
// every wavefront holds its last fragments in registers.  Reduction-contiguous fragments are
// plain 16-byte LDS reads, output-contiguous ones gfx950's transposing LDS reads, both from
// layouts whose 16-byte units are permuted so that the reads touch every bank once.
//
// What bounds it: the large products run at the matrix units' rate under the power limit (65536 x
// 1024 x 1024 bf16, y alone stored: 148 us, a library's product 115; with operands of zeros, the
// same work, 107 and 87), and behind each tile's products its epilogue moves residual, pre and y at
// the memory's rate with the matrix units idle, the generator and the activation beside it: 215 us
// forward with GELU, dropout, residual and pre, 363 us for both products of the backward, their
// partials' sums included (floors 121 and 242 of products, 105 and 158 of memory).
#include "dense_tile.hpp"

namespace el {
namespace {

// ---------------------------------------------------------------------------------------
// Few outputs (a forward of one to a few hundred rows): the weights' bytes and latency count.  A
// workgroup's wavefronts share out the reduction of one 16 x 16 tile, fragments straight from
// global memory (64 contiguous bytes of a row per read), and the partial tiles are added in
// wavefront order in LDS.  Any alignment.  1 x 1024 x 1024 takes 4.2 us and 77 x 512 x 1024 4.7
// (an empty kernel 2.1): a round of loads or two and a barrier, no longer the bytes.
// ---------------------------------------------------------------------------------------
constexpr int kFewWaves = 8;

template <class T>
__device__ inline f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  if constexpr (T::code == EL_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <class T>
__global__ __launch_bounds__(kFewWaves * 64) void k_dense_few(GemmArgs a) {
  constexpr int PITCH = 20, AHEAD = 4;
  __shared__ float lds[kFewWaves][16 * PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int tr = blockIdx.x / a.tiles_c, tc = blockIdx.x - tr * a.tiles_c;
  const int row0 = tr * 16, col0 = tc * 16;
  const int k0 = wave * a.per_split, kend = min(a.red, k0 + a.per_split);
  const uint16_t* q = a.Q + static_cast<long>(min(col0 + l16, a.C - 1)) * a.ldq;  // rows past the end: never stored
  const uint16_t* p = a.P + static_cast<long>(min(row0 + l16, a.R - 1)) * a.ldp;
  // the epilogue's operands are on their way while the products run
  const int r = row0 + threadIdx.x / 2, c = col0 + threadIdx.x % 2 * 8, n = min(8, a.C - c);
  const bool mine = threadIdx.x < 32 && r < a.R && n > 0;
  float v[8] = {};
  Raw8<T> add;
  if (mine) {
    if (a.add) add = load8_raw<T>(a.add + r * a.ldadd + c, n);
    if (a.bias)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = a.bias[min(c + e, a.C - 1)];
  }
  f32x4 acc = {};
  for (int k = k0; k < kend; k += 32 * AHEAD) {
    Raw8<T> fq[AHEAD], fp[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int at = k + u * 32 + g * 8;
      if (at < kend) {
        fq[u] = load8_raw<T>(q + at, kend - at);
        fp[u] = load8_raw<T>(p + at, kend - at);
      } else {
        fq[u].v[0] = fp[u].v[0] = u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) acc = mfma16<T>(fq[u].v[0], fp[u].v[0], acc);
  }
  // register e: column 4 g + e of row l16
  *reinterpret_cast<f32x4*>(&lds[wave][l16 * PITCH + g * 4]) = acc;
  __syncthreads();
  if (!mine) return;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += lds[w][threadIdx.x / 2 * PITCH + threadIdx.x % 2 * 8 + e];
  epilogue8<T, FWD, false>(a, a.drop.top ? drop_offset(a.drop) : 0, r, c, n, v, add, Pre8<T, false>{});
}

// A forward of few outputs: at most 64 tiles of 64 x 64 (512 x 512 x 512: 7.6 us against 9.1 in
// tiles; 300 x 1024 x 1024, 80 tiles: 14.7 against 13.8).
bool plan_few(long M, long N) { return ceil_div(M, 64) * ceil_div(N, 64) <= 64; }

template <class T>
el_status run_fwd(const char* fn, GemmArgs a, char* ws, hipStream_t st) {
  if (plan_few(a.R, a.C)) {
    a.tiles_c = static_cast<int>(ceil_div(a.C, 16));
    a.per_split = static_cast<int>(ceil_div(ceil_div(a.red, kFewWaves), 32) * 32);
    hipLaunchKernelGGL((k_dense_few<T>), dim3(static_cast<unsigned>(ceil_div(a.R, 16) * a.tiles_c)), dim3(kFewWaves * 64), 0,
                       st, a);
    return check_launch(fn);
  }
  Packs packs;
  packs.add(&a.P, &a.ldp, a.R, a.red, &ws);
  packs.add(&a.Q, &a.ldq, a.C, a.red, &ws);
  const el_status s = packs.run(fn, st);
  if (s != EL_OK) return s;
  a.red = static_cast<int>(pad8(a.red));  // the copies' padding is zero; whole rows need none
  a.red_q = a.per_split = a.red;
  return launch_product<T, FWD>(fn, a, plan_tiles(a.R, a.C), 1, st);
}

}  // namespace
}  // namespace el

using namespace el;

namespace {

template <class T>
el_status run_bwd(const char* fn, const uint16_t* x, long ldx, int M, int K, const uint16_t* w, int N, const uint16_t* dz,
                  long lddz, GemmArgs a, float* dw, float* db, char* ws, hipStream_t st) {
  Packs packs;
  packs.add(&dz, &lddz, M, N, &ws);
  packs.add(&x, &ldx, M, K, &ws);
  long ldw = K;
  if (a.out) packs.add(&w, &ldw, N, K, &ws);
  EL_TRY(packs.run(fn, st));
  const WgradPlan pl = plan_wgrad(M, K, N, wgrad_shares(M, K, a.out));
  GemmArgs b{};
  b.P = dz, b.ldp = lddz, b.Q = x, b.ldq = ldx, b.R = N, b.C = K, b.red = b.red_q = M, b.per_split = pl.per;
  b.part = pl.splits > 1 ? reinterpret_cast<float*>(ws) : dw;
  float* dbp = reinterpret_cast<float*>(ws + pl.dw_bytes);
  b.dbp = db ? dbp : nullptr;
  if (a.out) {
    // a copied dz has rows that end in zeros; the rows of w behind N read as zeros
    a.P = dz, a.ldp = lddz, a.Q = w, a.ldq = ldw, a.R = M, a.C = K;
    a.red = a.per_split = static_cast<int>(pad8(N));
    a.red_q = N;
    EL_TRY(launch_backward<T>(fn, a, plan_tiles(M, K), b, pl.shape, pl.splits, st));
  } else {
    EL_TRY((launch_product<T, WGRAD>(fn, b, pl.shape, pl.splits, st)));
  }
  launch_sums(Sums{b.part, dw, pl.splits > 1 ? static_cast<long>(N) * K : 0, pl.splits},
              Sums{dbp, db, db ? static_cast<long>(N) : 0, pl.db_rows}, st);
  return check_launch(fn);
}

}  // namespace

extern "C" {

size_t el_dense_fwd_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  if (!dense_sizes_ok(M, K, N) || plan_few(M, N) || !tiles_fit(M, N)) return 0;
  return packed_bytes(M, K) + packed_bytes(N, K);
}

size_t el_dense_bwd_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  if (!dense_sizes_ok(M, K, N)) return 0;
  return packed_bytes(M, N) + packed_bytes(M, K) + packed_bytes(N, K) +
         std::max(plan_wgrad(M, K, N, false).bytes, plan_wgrad(M, K, N, true).bytes);
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
    if (M == 0) return EL_OK;
    if (!tiles_fit(M, N)) return too_many_tiles(fn);
    const size_t need = plan_few(M, N) ? 0 : copy_bytes(x, ldx, M, K) + copy_bytes(w, K, N, K);
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, need));
    a.P = u16(x), a.ldp = ldx, a.Q = u16(w), a.ldq = K, a.R = M, a.C = N, a.red = K, a.act = act;
    a.add = u16(residual), a.ldadd = ldr, a.aux = static_cast<uint16_t*>(pre), a.ldaux = ldpre;
    a.out = static_cast<uint16_t*>(y), a.ldo = ldy, a.bias = bias;
    char* ws = static_cast<char*>(workspace);
    return dtype == EL_BF16 ? run_fwd<BF16T>(fn, a, ws, stream) : run_fwd<F16T>(fn, a, ws, stream);
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
    const long nk = static_cast<long>(N) * K;
    if (M == 0) {  // an empty batch: zero gradients, by a kernel (a captured fill stays a kernel node)
      launch_zero(dw, nk, stream);
      if (db) launch_zero(db, N, stream);
      return check_launch(fn);
    }
    if (dx && !tiles_fit(M, K)) return too_many_tiles(fn);
    const size_t need = copy_bytes(dz, lddz, M, N) + copy_bytes(x, ldx, M, K) + (dx ? copy_bytes(w, K, N, K) : 0) +
                        plan_wgrad(M, K, N, wgrad_shares(M, K, dx)).bytes;
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, need));
    a.add = u16(dres), a.ldadd = lddres, a.out = static_cast<uint16_t*>(dx), a.ldo = lddx, a.act = act;
    a.aux = static_cast<uint16_t*>(dzb), a.ldaux = lddzb, a.pre = dzb && act != EL_ACT_NONE ? u16(pre) : nullptr, a.ldpre = ldpre;
    char* ws = static_cast<char*>(workspace);
    return dtype == EL_BF16
               ? run_bwd<BF16T>(fn, u16(x), ldx, M, K, u16(w), N, u16(dz), lddz, a, dw, db, ws, stream)
               : run_bwd<F16T>(fn, u16(x), ldx, M, K, u16(w), N, u16(dz), lddz, a, dw, db, ws, stream);
  });
}

}  // extern "C"
