// dense_ckpt.hip -- a dense layer's backward with its input and the pre-activation of the layer
// below read from 8 bits:  dw = dz^T xq,  dx = dz w + dres,  dzb = drop(dx act'(preq)).
//
// The tiles of dense_tile.hpp, with two changes.  The data gradient's epilogue reads half the bytes
// for the pre-activation.  The weight gradient takes x's codes through registers, where the
// conversion to 16 bits applies the scale, to the LDS places that direct loads would fill.
//
// 65536 x 1024 x 1024 in bf16 with GELU, dropout and a skip: 355-369 us, what el_dense_bwd takes on 16-bit
// activations (352-356), for both products (242 at the rate of a large library product) are followed by
// their tiles' epilogues.  Unpacking both operands in front of the 16-bit kernels: 442 us.
#include "dense_tile.hpp"

namespace el {
namespace {

long padded(long K) { return tower::pad_to(K, kMicroBlock); }

template <class T>
el_status run(const char* fn, const uint8_t* xc, const uint8_t* xs, int M, int K, const uint16_t* w, int N,
              const uint16_t* dz, long lddz, GemmArgs a, const uint8_t* pc, const uint8_t* ps, float* dw, float* db,
              char* ws, hipStream_t st) {
  const WgradPlan pl = plan_wgrad(M, K, N, wgrad_shares(M, K, a.out));
  Packs packs;
  packs.add(&dz, &lddz, M, N, &ws);
  long ldw = K;
  if (a.out) packs.add(&w, &ldw, N, K, &ws);
  EL_TRY(packs.run(fn, st));
  GemmArgs b{};
  b.P = dz, b.ldp = lddz, b.codes = xc, b.scales = xs, b.kp = padded(K), b.R = N, b.C = K, b.red = b.red_q = M, b.per_split = pl.per;
  b.part = pl.splits > 1 ? reinterpret_cast<float*>(ws) : dw;
  float* dbp = reinterpret_cast<float*>(ws + pl.dw_bytes);
  b.dbp = db ? dbp : nullptr;
  if (a.out) {
    a.P = dz, a.ldp = lddz, a.Q = w, a.ldq = ldw, a.R = M, a.C = K;
    a.red = a.per_split = static_cast<int>(pad8(N));
    a.red_q = N;
    a.codes = pc, a.scales = ps, a.kp = padded(K);
    EL_TRY((launch_backward<T, true>(fn, a, plan_tiles(M, K), b, pl.shape, pl.splits, st)));
  } else {
    EL_TRY((launch_product<T, WGRAD, true>(fn, b, pl.shape, pl.splits, st)));
  }
  launch_sums(Sums{b.part, dw, pl.splits > 1 ? static_cast<long>(N) * K : 0, pl.splits},
              Sums{dbp, db, db ? static_cast<long>(N) : 0, pl.db_rows}, st);
  return check_launch(fn);
}

}  // namespace
}  // namespace el

using namespace el;

extern "C" {

size_t el_dense_bwd_ckpt_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  if (!dense_sizes_ok(M, K, N) || M * padded(K) > (int64_t{1} << 34)) return 0;
  return packed_bytes(M, N) + packed_bytes(N, K) + std::max(plan_wgrad(M, K, N, false).bytes, plan_wgrad(M, K, N, true).bytes);
}

el_status el_dense_bwd_ckpt(const uint8_t* x_codes, const uint8_t* x_scales, int32_t M, int32_t K, const void* w,
                            int32_t N, const void* dz, int64_t lddz, const void* dres, int64_t lddres, void* dx,
                            int64_t lddx, uint32_t act, const el_dropout* drop, const uint8_t* pre_codes,
                            const uint8_t* pre_scales, void* dzb, int64_t lddzb, float* dw, float* db, el_dtype dtype,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "el_dense_bwd_ckpt";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_dense_sizes(fn, M, K, N, dtype));
    EL_TRY(tower::check_packed_sizes(fn, M, K, kMicroBlock));
    EL_TRY(tower::check_act(fn, act));
    if (!w) return tower::bad(fn, "w is null");
    if (!tower::al(w, 2)) return tower::bad(fn, "w must be aligned to its elements");
    GemmArgs a{};
    EL_TRY(tower::drop_args(fn, drop, &a.drop));
    EL_TRY(tower::check_packed(fn, "x", x_codes, x_scales, M > 0));
    EL_TRY(tower::check_rows(fn, "dz", dz, lddz, N, M > 0, 2));
    EL_TRY(tower::check_rows(fn, "dres", dres, lddres, K, false, 2));
    EL_TRY(tower::check_rows(fn, "dx", dx, lddx, K, false, 2));
    const bool use_pre = dzb && act != EL_ACT_NONE;
    EL_TRY(tower::check_packed(fn, "pre", pre_codes, pre_scales, use_pre && M > 0));
    EL_TRY(tower::check_rows(fn, "dzb", dzb, lddzb, K, false, 2));
    if ((dzb || dres) && !dx) return tower::bad(fn, "dzb and dres need dx");
    if (!dw || !tower::al(dw, 4) || !tower::al(db, 4)) return tower::bad(fn, "dw must be non-null, dw and db aligned to their elements");
    if (M == 0) {
      launch_zero(dw, static_cast<long>(N) * K, stream);
      if (db) launch_zero(db, N, stream);
      return check_launch(fn);
    }
    if (dx && !tiles_fit(M, K)) return too_many_tiles(fn);
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, el_dense_bwd_ckpt_workspace_bytes(M, K, N)));
    a.add = u16(dres), a.ldadd = lddres, a.out = static_cast<uint16_t*>(dx), a.ldo = lddx, a.act = act;
    a.aux = static_cast<uint16_t*>(dzb), a.ldaux = lddzb;
    char* ws = static_cast<char*>(workspace);
    const uint8_t* pc = use_pre ? pre_codes : nullptr;
    return dtype == EL_BF16 ? run<BF16T>(fn, x_codes, x_scales, M, K, u16(w), N, u16(dz), lddz, a, pc, pre_scales, dw, db, ws, stream)
                            : run<F16T>(fn, x_codes, x_scales, M, K, u16(w), N, u16(dz), lddz, a, pc, pre_scales, dw, db, ws, stream);
  });
}

}  // extern "C"
