// block_norm_fwd.hpp -- the norms behind one residual block and before the next, with the block's
// gate and residual scale (formulas in embblock.h): one pass over the rows.
//
// Memory bounds it: x, f and the gate are read, y and h written.  65536 x 1024 in bf16: 120 us, 5.6 TB/s,
// a little above a copy's rate (215 us before the next rows' loads were in flight behind this row's
// arithmetic and stores).  One row: 3.5 us on the GPU, five dependent steps of latency.
#pragma once

#include "block_norm.hpp"

namespace el {
namespace {

// A workgroup's slots take consecutive rows; the next ones are on their way while these are worked
// on.  BETA: any shift is given.
template <class T, class SL, template <class, class> class View, bool BETA>
__global__ __launch_bounds__(SL::THREADS) void k_norm_fwd(NormArgs a) {
  __shared__ float lds[2][SL::WAVES][2];
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
    vx.load(vx.span(r0, rows, a.C), rx);
    vf.load(vf.span(r0, rows, a.C), rf);
    if (a.gate_rows == 1) {
      vg.load(vg.span(r0, rows, a.C), rg);
    } else {  // the view begins at the first row's gate row
      const uint32_t S = a.gate_rows, g0 = static_cast<uint32_t>(r0) / S;  // (r0 < 2^32)
      const uint32_t gl = static_cast<uint32_t>(min(r0 + sl, a.M - 1l)) / S - g0;
      vg.at(gl, c0, a.C);
      vg.load(vg.span(g0, rows, a.C), rg);
    }
  };
  long r0 = static_cast<long>(blockIdx.x) * PER;
  fetch(r0);
  for (; r0 < a.M; r0 += stride) {
    const int rows = static_cast<int>(min(static_cast<long>(PER), a.M - r0));
    float y[NV][8], f[NV][8], g[NV][8];
    vx.settle(rx), vf.settle(rf), vg.settle(rg);
#pragma unroll
    for (int j = 0; j < NV; ++j) to_floats<T>(rx[j], y[j]), to_floats<T>(rf[j], f[j]), to_floats<T>(rg[j], g[j]);
    fetch(r0 + stride);
    if (a.f) {
      float mean = 0.f, rstd = 1.f;
      if (a.post != EL_NORM_NONE) row_stats<SL>(f, a.post, a, c0, lds, turn, mean, rstd);
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(mean), __float_as_uint(rstd)}, stats_span(a.post_stats, r0, rows), vstat, 0, 0);
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
    vy.store(vy.span(r0, rows, a.C), y);
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
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(mean), __float_as_uint(rstd)}, stats_span(a.pre_stats, r0, rows), vstat, 0, 0);
    vh.store(vh.span(r0, rows, a.C), y);
  }
}

template <class T, class SL, template <class, class> class View, bool BETA>
void launch_one_fwd(const NormArgs& a, hipStream_t st) {
  const auto kernel = k_norm_fwd<T, SL, View, BETA>;
  const int grid = resident_grid(reinterpret_cast<const void*>(kernel), static_cast<int>(ceil_div(a.M, SL::PER_WG)), 0, SL::THREADS);
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(SL::THREADS), 0, st, a);
}

}  // namespace

template <class T>
void launch_norm_fwd(const NormArgs& a, bool aligned, hipStream_t st) {
  with_slot(a.C, [&](auto s) {
    using SL = decltype(s);
    if constexpr (SL::COLS <= kMaxAlignedCols) {
      if (aligned) {
        if (a.bp || a.bq) launch_one_fwd<T, SL, Aligned, true>(a, st);
        else launch_one_fwd<T, SL, Aligned, false>(a, st);
        return;
      }
    }
    launch_one_fwd<T, SL, Loose, true>(a, st);
  });
}

}  // namespace el
