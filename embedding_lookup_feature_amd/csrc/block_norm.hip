// block_norm.hip -- the block norm's entry points: checks and the backward's plan.
#include "block_norm.hpp"

namespace el {
namespace {

__global__ __launch_bounds__(256) void k_zero4(JoinArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c < a.C && a.out[blockIdx.y]) a.out[blockIdx.y][c] = 0.f;
}

// The backward's grid (its partial sums are laid out by it) is a function of the sizes and of the form,
// aligned 16-bit rows without betas, other rows, loose rows with shared gates: as
// many workgroups as the registers let run at once.
enum Form { LEAN = 0, PLAIN = 1, FULL = 2 };
struct BwdPlan {
  int grid;
  int64_t span;  // rows of a workgroup where gate rows are shared
  size_t gate_bytes, bytes;
};
BwdPlan plan_bwd(int M, int C, int gate_rows, Form form) {
  BwdPlan p{};
  with_bwd_slot<true>(C, form == LEAN, [&](auto s) {
    using SL = decltype(s);
    const int most = kCus * ((form == FULL ? kBwdWaves<SL, true> : kBwdWaves<SL, false>) * 4 / SL::WAVES);
    p.grid = static_cast<int>(std::min<long>(most, ceil_div(M, SL::PER_WG)));
    const int64_t slots = static_cast<int64_t>(p.grid) * SL::PER_WG;
    p.span = SL::PER_WG * (M / slots + 1) + 1;
    if (gate_rows > 1) p.gate_bytes = round256(static_cast<size_t>(slots) * 2 * C * 4);
  });
  p.bytes = p.gate_bytes + round256(static_cast<size_t>(p.grid) * 4 * C * 4);
  return p;
}

constexpr int kMaxPerWg = 128;  // rows that a workgroup's slots hold at once

}  // namespace
}  // namespace el

using namespace el;

extern "C" {

el_status el_block_norm_fwd(const el_block_norm* p, const void* x, int64_t ldx, const void* f, int64_t ldf,
                            const void* gate, int64_t ldg, int32_t M, int32_t C, void* y, int64_t ldy, void* h,
                            int64_t ldh, float* post_stats, float* pre_stats, el_dtype dtype, hipStream_t stream) {
  const char* fn = "el_block_norm_fwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_norm(fn, p, M, C, dtype));
    const size_t e = dtype_size(dtype);
    EL_TRY(tower::check_rows(fn, "x", x, ldx, C, M > 0 && !f, e));
    EL_TRY(tower::check_rows(fn, "f", f, ldf, C, false, e));
    EL_TRY(tower::check_rows(fn, "gate", gate, ldg, C, false, e));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, C, false, e));
    EL_TRY(tower::check_rows(fn, "h", h, ldh, C, M > 0 && !y, e));
    if (M > 0 && !f && (gate || y || post_stats)) return tower::bad(fn, "gate, y and post_stats need f");
    if (post_stats && p->post == EL_NORM_NONE) return tower::bad(fn, "post_stats without a post norm");
    if (pre_stats && M > 0 && !h) return tower::bad(fn, "pre_stats need h");
    if (!tower::al(post_stats, 8) || !tower::al(pre_stats, 8)) return tower::bad(fn, "statistics must be 8-byte aligned");
    if (M == 0) return EL_OK;
    NormArgs a = common(p, M, C);
    a.x = x, a.ldx = ldx, a.f = f, a.ldf = ldf, a.gate = gate, a.ldg = ldg, a.y = y, a.ldy = ldy, a.h = h, a.ldh = ldh;
    a.post_stats = post_stats, a.pre_stats = pre_stats;
    bool aligned = C <= kMaxAlignedCols && C % 8 == 0;
    const auto ok = [&](const void* q, int64_t ld) { return aligned_rows(q, ld, e, kMaxPerWg); };
    aligned = aligned && ok(x, ldx) && ok(f, ldf) && ok(gate, ldg) && ok(y, ldy) && ok(h, ldh);
    with_type(dtype, [&](auto t) { launch_norm_fwd<decltype(t)>(a, aligned, stream); });
    return check_launch(fn);
  });
}

size_t el_block_norm_bwd_workspace_bytes(int32_t M, int32_t C, int32_t gate_rows) {
  if (M < 1 || C < 1 || C > kMaxCols || gate_rows < 1) return 0;
  size_t bytes = 0;
  for (const Form form : {LEAN, PLAIN, FULL}) bytes = std::max(bytes, plan_bwd(M, C, gate_rows, form).bytes);
  return bytes;
}

el_status el_block_norm_bwd(const el_block_norm* p, const void* dy, int64_t lddy, const void* dh, int64_t lddh,
                            const void* y, int64_t ldy, const void* f, int64_t ldf, const void* gate, int64_t ldg,
                            int32_t M, int32_t C, const float* post_stats, const float* pre_stats, void* dx,
                            int64_t lddx, void* df, int64_t lddf, void* dgate, int64_t lddg, float* dpost_gamma,
                            float* dpost_beta, float* dpre_gamma, float* dpre_beta, el_dtype dtype, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "el_block_norm_bwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_norm(fn, p, M, C, dtype));
    const size_t e = dtype_size(dtype);
    EL_TRY(tower::check_rows(fn, "dy", dy, lddy, C, false, e));
    EL_TRY(tower::check_rows(fn, "dh", dh, lddh, C, M > 0 && !dy, e));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, C, M > 0 && dh, e));
    EL_TRY(tower::check_rows(fn, "f", f, ldf, C, false, e));
    EL_TRY(tower::check_rows(fn, "gate", gate, ldg, C, false, e));
    EL_TRY(tower::check_rows(fn, "dx", dx, lddx, C, false, e));
    EL_TRY(tower::check_rows(fn, "df", df, lddf, C, false, e));
    EL_TRY(tower::check_rows(fn, "dgate", dgate, lddg, C, false, e));
    if (!tower::al(post_stats, 8) || !tower::al(pre_stats, 8)) return tower::bad(fn, "statistics must be 8-byte aligned");
    if (!tower::al(dpost_gamma, 4) || !tower::al(dpost_beta, 4) || !tower::al(dpre_gamma, 4) || !tower::al(dpre_beta, 4))
      return tower::bad(fn, "parameter gradients must be aligned to their elements");
    if (M > 0) {
      if (!f && (gate || df || dgate || dpost_gamma || dpost_beta)) return tower::bad(fn, "gate, df, dgate, dpost_gamma and dpost_beta need f");
      if (dgate && !gate) return tower::bad(fn, "dgate needs the gate");
      if (!dh && (dpre_gamma || dpre_beta)) return tower::bad(fn, "dpre_gamma and dpre_beta need dh");
      if (dh && !pre_stats) return tower::bad(fn, "pre_stats is null");
      if (f && p->post != EL_NORM_NONE && !post_stats) return tower::bad(fn, "post_stats is null");
    }
    JoinArgs j{nullptr, {dpost_gamma, dpost_beta, dpre_gamma, dpre_beta}, 0, C};
    const bool params = dpost_gamma || dpost_beta || dpre_gamma || dpre_beta;
    if (M == 0) {
      if (params) hipLaunchKernelGGL(k_zero4, dim3(static_cast<unsigned>(ceil_div(C, 256)), 4), dim3(256), 0, stream, j);
      return check_launch(fn);
    }
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, el_block_norm_bwd_workspace_bytes(M, C, p->gate_rows)));
    NormArgs a = common(p, M, C);
    a.gate_rows = std::min(p->gate_rows, M);
    a.dy = dy, a.lddy = lddy, a.dh = dh, a.lddh = lddh, a.y_in = y, a.ldy = ldy, a.f = f, a.ldf = ldf, a.gate = gate, a.ldg = ldg;
    a.dx = dx, a.lddx = lddx, a.df = df, a.lddf = lddf, a.dgate = dgate, a.lddg = lddg;
    a.post_stats = const_cast<float*>(post_stats), a.pre_stats = const_cast<float*>(pre_stats);
    for (int k = 0; k < 4; ++k) a.want |= j.out[k] ? 1u << k : 0u;
    const bool shared = gate && a.gate_rows > 1;
    // (rows of a workgroup with shared gates: aligned in one form must be aligned in the other)
    const int64_t span = std::max(plan_bwd(M, C, p->gate_rows, LEAN).span, plan_bwd(M, C, p->gate_rows, PLAIN).span);
    const auto ok = [&](const void* q, int64_t ld) { return aligned_rows(q, ld, e, shared ? span : kMaxPerWg); };
    const bool aligned = C <= kMaxAlignedCols && C % 8 == 0 && ok(dy, lddy) && ok(dh, lddh) && ok(y, ldy) && ok(f, ldf) &&
                         ok(gate, ldg) && ok(dx, lddx) && ok(df, lddf) && ok(dgate, lddg);
    const bool lean = aligned && !a.bp && !dpost_beta && !dpre_beta;
    const BwdPlan pl = plan_bwd(M, C, p->gate_rows, lean && e == 2 ? LEAN : !aligned && shared ? FULL : PLAIN);
    a.gate_part = static_cast<float*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.gate_bytes);
    j.part = a.part, j.parts = pl.grid;
    with_type(dtype, [&](auto t) { launch_norm_bwd<decltype(t)>(a, j, aligned, lean, shared, pl.grid, stream); });
    return check_launch(fn);
  });
}

}  // extern "C"
