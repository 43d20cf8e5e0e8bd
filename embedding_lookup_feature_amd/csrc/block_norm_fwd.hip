// block_norm_fwd.hip -- the norms behind one residual block and before the next, with the block's
// gate and residual scale (formulas in embblock.h).
#include "block_norm.hpp"

namespace el {
namespace {

// Aligned form: a workgroup's slots take consecutive rows; the next ones are on their way while
// these are worked on.  BETA: any shift is given.
template <class T, class SL, bool BETA>
__global__ __launch_bounds__(SL::THREADS) void k_norm_fwd_aligned(NormArgs a) {
  __shared__ float lds[2][SL::W][2];
  int turn = 0;
  constexpr int NV = SL::NV, PER = SL::PER_WG;
  const int in_slot = threadIdx.x % (SL::L * SL::W), c0 = in_slot * 8, sl = threadIdx.x / (SL::L * SL::W);
  View<T, SL> vx, vf, vg, vy, vh;
  vx.init(a.x, a.ldx, sl, c0, a.C), vf.init(a.f, a.ldf, sl, c0, a.C), vg.init(a.gate, a.ldg, sl, c0, a.C);
  vy.init(a.y, a.ldy, sl, c0, a.C), vh.init(a.h, a.ldh, sl, c0, a.C);
  const uint32_t vstat = in_slot == 0 ? sl * 8u : kNowhere;
  float gp[NV][8], gq[NV][8], bp[BETA ? NV : 1][8], bq[BETA ? NV : 1][8];
  load_param<SL>(a.gp, 1.f, c0, a.C, gp);
  load_param<SL>(a.gq, 1.f, c0, a.C, gq);
  if constexpr (BETA) load_param<SL>(a.bp, 0.f, c0, a.C, bp), load_param<SL>(a.bq, 0.f, c0, a.C, bq);
  const long stride = static_cast<long>(gridDim.x) * PER;
  Raw8<T> rx[NV], rf[NV], rg[NV];
  const auto fetch = [&](long r0) {
    const int rows = static_cast<int>(max(0l, min(static_cast<long>(PER), a.M - r0)));
    vx.load(vx.rsrc(r0, rows, a.C), rx);
    vf.load(vf.rsrc(r0, rows, a.C), rf);
    if (a.gate_rows == 1) {
      vg.load(vg.rsrc(r0, rows, a.C), rg);
    } else {  // the view begins at the first row's gate row
      const uint32_t S = a.gate_rows, g0 = static_cast<uint32_t>(r0) / S;  // (r0 < 2^32)
      const uint32_t gl = static_cast<uint32_t>(min(r0 + sl, a.M - 1l)) / S - g0;
      vg.at(gl, c0, a.C);
      vg.load(vg.rsrc(g0, rows, a.C), rg);
    }
  };
  long r0 = static_cast<long>(blockIdx.x) * PER;
  fetch(r0);
  for (; r0 < a.M; r0 += stride) {
    const int rows = static_cast<int>(min(static_cast<long>(PER), a.M - r0));
    float y[NV][8], f[NV][8], g[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) to_floats<T>(rx[j], y[j]), to_floats<T>(rf[j], f[j]), to_floats<T>(rg[j], g[j]);
    fetch(r0 + stride);
    if (a.f) {
      float mean = 0.f, rstd = 1.f;
      if (a.post != EL_NORM_NONE) row_stats<SL>(f, a.post, a, c0, lds, turn, mean, rstd);
      const auto rs = __builtin_amdgcn_make_buffer_rsrc(a.post_stats + r0 * 2, 0, a.post_stats ? rows * 8 : 0, 0x00027000);
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(mean), __float_as_uint(rstd)}, rs, vstat, 0, 0);
      const float scale = a.scale;
      if (a.gate && a.gate_act == EL_GATE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) g[j][e] = sigmoid(g[j][e]) * scale;
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) g[j][e] = a.gate ? g[j][e] * scale : scale;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float t = (f[j][e] - mean) * rstd;
          if constexpr (BETA) t = fmaf(t, gp[j][e], bp[j][e]);
          else t *= gp[j][e];
          y[j][e] = fmaf(g[j][e], t, y[j][e]);
        }
    }
    vy.store(vy.rsrc(r0, rows, a.C), y);
    float mean = 0.f, rstd = 1.f;
    if (a.h) {
      row_stats<SL>(y, a.pre, a, c0, lds, turn, mean, rstd);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float t = (y[j][e] - mean) * rstd;
          if constexpr (BETA) y[j][e] = fmaf(t, gq[j][e], bq[j][e]);
          else y[j][e] = t * gq[j][e];
        }
    }
    const auto rs = __builtin_amdgcn_make_buffer_rsrc(a.pre_stats + r0 * 2, 0, a.pre_stats ? rows * 8 : 0, 0x00027000);
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(mean), __float_as_uint(rstd)}, rs, vstat, 0, 0);
    vh.store(vh.rsrc(r0, rows, a.C), y);
  }
}

// General form.
template <class T, class SL>
__global__ __launch_bounds__(SL::THREADS) void k_block_norm_fwd(NormArgs a) {
  __shared__ float lds[2][SL::W][2];
  int turn = 0;
  const int in_slot = threadIdx.x % (SL::L * SL::W), c0 = in_slot * 8;
  const int slot = blockIdx.x * SL::PER_WG + threadIdx.x / (SL::L * SL::W), slots = gridDim.x * SL::PER_WG;
  for (long row = slot; row < a.M; row += slots) {
    RowRaw<T, SL> rx, rf, rg;
    if (a.x) rx.load(a.x, a.ldx, row, c0, a.C);
    if (a.f) rf.load(a.f, a.ldf, row, c0, a.C);
    if (a.gate) rg.load(a.gate, a.ldg, row / a.gate_rows, c0, a.C);
    float y[SL::NV][8];
#pragma unroll
    for (int j = 0; j < SL::NV; ++j) {
      if (a.x) to_floats<T>(rx.v[j], y[j]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) y[j][e] = 0.f;
    }
    if (a.f) {
      float f[SL::NV][8], mean = 0.f, rstd = 1.f;
#pragma unroll
      for (int j = 0; j < SL::NV; ++j) to_floats<T>(rf.v[j], f[j]);
      if (a.post != EL_NORM_NONE) {
        row_stats<SL>(f, a.post, a, c0, lds, turn, mean, rstd);
        if (a.post_stats && in_slot == 0) reinterpret_cast<float2*>(a.post_stats)[row] = make_float2(mean, rstd);
      }
#pragma unroll
      for (int j = 0; j < SL::NV; ++j) {
        const int c = c0 + j * SL::L * SL::W * 8, n = a.C - c;
        float ga[8], be[8], g[8];
        load_vec(a.gp, 1.f, c, n, ga);
        load_vec(a.bp, 0.f, c, n, be);
        if (a.gate) to_floats<T>(rg.v[j], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float t = fmaf((f[j][e] - mean) * rstd, ga[e], be[e]);
          y[j][e] = fmaf(a.gate ? gate_value(a.gate_act, g[e]) * a.scale : a.scale, t, y[j][e]);
        }
      }
      if (a.y) store_row<T, SL>(a.y, a.ldy, row, c0, a.C, y);
    }
    if (a.h) {
      float mean, rstd;
      row_stats<SL>(y, a.pre, a, c0, lds, turn, mean, rstd);
      if (a.pre_stats && in_slot == 0) reinterpret_cast<float2*>(a.pre_stats)[row] = make_float2(mean, rstd);
#pragma unroll
      for (int j = 0; j < SL::NV; ++j) {
        const int c = c0 + j * SL::L * SL::W * 8, n = a.C - c;
        float ga[8], be[8];
        load_vec(a.gq, 1.f, c, n, ga);
        load_vec(a.bq, 0.f, c, n, be);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[j][e] = fmaf((y[j][e] - mean) * rstd, ga[e], be[e]);
      }
      store_row<T, SL>(a.h, a.ldh, row, c0, a.C, y);
    }
  }
}

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
    with_type(dtype, [&](auto t) {
      with_slot(C, [&](auto s) {
        using SL = decltype(s);
        const long wgs = ceil_div(M, SL::PER_WG);
        if constexpr (SL::COLS <= kMaxAlignedCols) {
          const auto ok = [&](const void* q, int64_t ld) { return aligned_rows(q, ld, e, SL::PER_WG); };
          if (C % 8 == 0 && ok(x, ldx) && ok(f, ldf) && ok(gate, ldg) && ok(y, ldy) && ok(h, ldh)) {
            const auto go = [&](auto kernel) {
              const int grid = resident_grid(reinterpret_cast<const void*>(kernel), static_cast<int>(wgs), 0, SL::THREADS);
              hipLaunchKernelGGL(kernel, dim3(grid), dim3(SL::THREADS), 0, stream, a);
            };
            if (a.bp || a.bq) go(k_norm_fwd_aligned<decltype(t), SL, true>);
            else go(k_norm_fwd_aligned<decltype(t), SL, false>);
            return;
          }
        }
        const dim3 grid(static_cast<unsigned>(std::min<long>(wgs, 16l * kCus)));
        hipLaunchKernelGGL((k_block_norm_fwd<decltype(t), SL>), grid, dim3(SL::THREADS), 0, stream, a);
      });
    });
    return check_launch(fn);
  });
}

}  // extern "C"
