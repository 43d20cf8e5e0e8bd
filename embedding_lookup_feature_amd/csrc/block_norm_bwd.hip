// block_norm_bwd.hip -- the block norm's backward: gradients of both norms' inputs, of the gate and
// of the parameters in one pass over the rows (formulas in embblock.h).
#include "block_norm.hpp"

namespace el {
namespace {

// Gradient at a norm's input from g, the one at its output (gamma in it), and the normalised row.
template <class SL>
__device__ inline void norm_grad(float (&g)[SL::NV][8], const float (&vh)[SL::NV][8], uint32_t kind, float rstd,
                                 const NormArgs& a, float (*lds)[SL::W][2], int& turn) {
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < SL::NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = fmaf(g[j][e], vh[j][e], s[0]), s[1] += g[j][e];
  slot_sums<SL>(s, lds, turn);
  const float m2 = s[0] * a.inv_c, m1 = kind == EL_NORM_LAYER ? s[1] * a.inv_c : 0.f;
#pragma unroll
  for (int j = 0; j < SL::NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) g[j][e] = (fmaf(-vh[j][e], m2, g[j][e]) - m1) * rstd;
}

template <class T, class SL>
__global__ __launch_bounds__(SL::THREADS) void k_block_norm_bwd(NormArgs a) {
  __shared__ float lds[2][SL::W][2];
  __shared__ float join[SL::PER_WG > 1 ? SL::THREADS * SL::NV * 8 : 1];
  int turn = 0;
  const int in_slot = threadIdx.x % (SL::L * SL::W), c0 = in_slot * 8;
  const int slot = blockIdx.x * SL::PER_WG + threadIdx.x / (SL::L * SL::W), slots = gridDim.x * SL::PER_WG;
  float acc[4][SL::NV][8] = {};  // dpost_gamma, dpost_beta, dpre_gamma, dpre_beta
  for (long at = slot; at < a.units; at += slots) {
    const int unit = static_cast<int>(at), grow = unit / a.per_gate;
    const long first = static_cast<long>(grow) * a.gate_rows + static_cast<long>(unit - grow * a.per_gate) * a.chunk;
    const long last = min(min(first + a.chunk, (grow + 1l) * a.gate_rows), static_cast<long>(a.M));
    float gsum[SL::NV][8] = {};
    for (long row = first; row < last; ++row) {
      RowRaw<T, SL> rdy, rdh, ry, rf, rg;
      if (a.dy) rdy.load(a.dy, a.lddy, row, c0, a.C);
      if (a.dh) rdh.load(a.dh, a.lddh, row, c0, a.C), ry.load(a.y_in, a.ldy, row, c0, a.C);
      if (a.f) rf.load(a.f, a.ldf, row, c0, a.C);
      if (a.gate) rg.load(a.gate, a.ldg, grow, c0, a.C);
      float D[SL::NV][8] = {}, v[SL::NV][8], g[SL::NV][8];
      if (a.dh) {
        const float2 st = reinterpret_cast<const float2*>(a.pre_stats)[row];
#pragma unroll
        for (int j = 0; j < SL::NV; ++j) {
          const int c = c0 + j * SL::L * SL::W * 8;
          float ga[8], dh[8];
          load_vec(a.gq, 1.f, c, a.C - c, ga);
          to_floats<T>(ry.v[j], v[j]);
          to_floats<T>(rdh.v[j], dh);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[j][e] = (v[j][e] - st.x) * st.y;
            acc[2][j][e] = fmaf(dh[e], v[j][e], acc[2][j][e]);
            acc[3][j][e] += dh[e];
            D[j][e] = dh[e] * ga[e];
          }
        }
        norm_grad<SL>(D, v, a.pre, st.y, a, lds, turn);
      }
      if (a.dy)
#pragma unroll
        for (int j = 0; j < SL::NV; ++j) {
          float dy[8];
          to_floats<T>(rdy.v[j], dy);
#pragma unroll
          for (int e = 0; e < 8; ++e) D[j][e] += dy[e];
        }
      if (a.dx) store_row<T, SL>(a.dx, a.lddx, row, c0, a.C, D);
      if (a.f) {
        float2 st = make_float2(0.f, 1.f);
        if (a.post != EL_NORM_NONE) st = reinterpret_cast<const float2*>(a.post_stats)[row];
#pragma unroll
        for (int j = 0; j < SL::NV; ++j) {
          const int c = c0 + j * SL::L * SL::W * 8;
          float ga[8], be[8], gt[8];
          load_vec(a.gp, 1.f, c, a.C - c, ga);
          load_vec(a.bp, 0.f, c, a.C - c, be);
          to_floats<T>(rf.v[j], v[j]);
          if (a.gate) to_floats<T>(rg.v[j], gt);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[j][e] = (v[j][e] - st.x) * st.y;
            const float sD = a.scale * D[j][e];
            gsum[j][e] = fmaf(sD, fmaf(v[j][e], ga[e], be[e]), gsum[j][e]);
            const float u = a.gate ? gate_value(a.gate_act, gt[e]) * sD : sD;
            acc[0][j][e] = fmaf(u, v[j][e], acc[0][j][e]);
            acc[1][j][e] += u;
            g[j][e] = u * ga[e];
          }
        }
        if (a.df) {
          if (a.post != EL_NORM_NONE) norm_grad<SL>(g, v, a.post, st.y, a, lds, turn);
          store_row<T, SL>(a.df, a.lddf, row, c0, a.C, g);
        }
      }
    }
    if (a.dgate) {
      if (a.per_gate > 1) {
        store_row<F32T, SL>(a.gate_part, a.C, unit, c0, a.C, gsum);
      } else {
        RowRaw<T, SL> rg;
        rg.load(a.gate, a.ldg, grow, c0, a.C);
#pragma unroll
        for (int j = 0; j < SL::NV; ++j) {
          float gt[8];
          to_floats<T>(rg.v[j], gt);
          if (a.gate_act == EL_GATE_SIGMOID)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float s = sigmoid(gt[e]);
              gsum[j][e] *= s * (1.f - s);
            }
        }
        store_row<T, SL>(a.dgate, a.lddg, grow, c0, a.C, gsum);
      }
    }
  }
  // The workgroup's sums of each asked parameter: its slots' added in slot order.
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!(a.want >> k & 1)) continue;
    float* out = a.part + (static_cast<long>(blockIdx.x) * 4 + k) * a.C;
    if constexpr (SL::PER_WG == 1) {
      store_row<F32T, SL>(out, 0, 0, c0, a.C, acc[k]);
    } else {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < SL::NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          join[(threadIdx.x / SL::L) * (SL::COLS) + c0 + j * SL::L * 8 + e] = acc[k][j][e];
      __syncthreads();
      for (int c = threadIdx.x; c < SL::COLS && c < a.C; c += SL::THREADS) {
        float s = join[c];
        for (int p = 1; p < SL::PER_WG; ++p) s += join[p * SL::COLS + c];
        out[c] = s;
      }
    }
  }
}

// out[c] = sum over p < parts of part[p * stride + c], up to four of them: 16 threads share a
// column's parts (thread s: parts s, s + 16, ...), their sums are added in thread order.
struct JoinArgs {
  const float* part;
  float* out[4];
  int parts, C;
};
__global__ __launch_bounds__(256) void k_join_params(JoinArgs a) {
  __shared__ float red[16][17];
  const int col = threadIdx.x & 15, s = threadIdx.x >> 4, k = blockIdx.y;
  if (!a.out[k]) return;
  const int c = blockIdx.x * 16 + col;
  float v = 0.f;
  if (c < a.C)
#pragma unroll 4
    for (int p = s; p < a.parts; p += 16) v += a.part[(static_cast<long>(p) * 4 + k) * a.C + c];
  red[s][col] = v;
  __syncthreads();
  if (s == 0 && c < a.C) {
    for (int i = 1; i < 16; ++i) v += red[i][col];
    a.out[k][c] = v;
  }
}

// dgate of a shared row: its units' partial sums in order, times the gate's derivative.
template <class T>
__global__ __launch_bounds__(256) void k_join_gate(NormArgs a, int rows) {
  const int vecs = (a.C + 7) / 8;
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  const long r = i / vecs;
  if (r >= rows) return;
  const int c = static_cast<int>(i - r * vecs) * 8, n = a.C - c;
  float v[8] = {}, g[8];
  for (int q = 0; q < a.per_gate; ++q) {
    float p[8];
    to_floats<F32T>(load8_raw<F32T>(a.gate_part + (r * a.per_gate + q) * a.C + c, n), p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += p[e];
  }
  if (a.gate_act == EL_GATE_SIGMOID) {
    to_floats<T>(load8_raw<T>(static_cast<const typename T::S*>(a.gate) + r * a.ldg + c, n), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = sigmoid(g[e]);
      v[e] *= s * (1.f - s);
    }
  }
  store8<T>(static_cast<typename T::S*>(a.dgate) + r * a.lddg + c, v, n);
}

__global__ __launch_bounds__(256) void k_zero4(JoinArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c < a.C && a.out[blockIdx.y]) a.out[blockIdx.y][c] = 0.f;
}

// ---------------------------------------------------------------------------------------
// Plan.
// ---------------------------------------------------------------------------------------
constexpr int kBwdGroups = 2 * kCus;  // workgroups of the backward at most

struct BwdPlan {
  int per_wg, grid, chunk, per_gate, units;
  size_t gate_bytes, bytes;
};
BwdPlan plan_bwd(int M, int C, int gate_rows) {
  BwdPlan p{};
  with_slot(C, [&](auto s) { p.per_wg = decltype(s)::PER_WG; });
  const long slots = static_cast<long>(kBwdGroups) * p.per_wg;
  const int rows = std::min(gate_rows, M);
  const long gates = ceil_div(M, rows);
  // a gate row is split over as many slots as would be idle otherwise
  const long split = std::min<long>(rows, std::max<long>(1, slots / gates));
  p.chunk = static_cast<int>(ceil_div(rows, split));
  p.per_gate = static_cast<int>(ceil_div(rows, p.chunk));
  p.units = static_cast<int>(gates * p.per_gate);
  p.grid = static_cast<int>(std::min<long>(kBwdGroups, ceil_div(p.units, p.per_wg)));
  p.gate_bytes = p.per_gate > 1 ? round256(static_cast<size_t>(p.units) * C * 4) : 0;
  p.bytes = p.gate_bytes + round256(static_cast<size_t>(p.grid) * 4 * C * 4);
  return p;
}

}  // namespace
}  // namespace el

using namespace el;

extern "C" {

size_t el_block_norm_bwd_workspace_bytes(int32_t M, int32_t C, int32_t gate_rows) {
  if (M < 1 || C < 1 || C > kMaxCols || gate_rows < 1) return 0;
  return plan_bwd(M, C, gate_rows).bytes;
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
    const BwdPlan pl = plan_bwd(M, C, p->gate_rows);
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, pl.bytes));
    NormArgs a = common(p, M, C);
    a.gate_rows = std::min(p->gate_rows, M);
    a.dy = dy, a.lddy = lddy, a.dh = dh, a.lddh = lddh, a.y_in = y, a.ldy = ldy, a.f = f, a.ldf = ldf, a.gate = gate, a.ldg = ldg;
    a.dx = dx, a.lddx = lddx, a.df = df, a.lddf = lddf, a.dgate = dgate, a.lddg = lddg;
    a.post_stats = const_cast<float*>(post_stats), a.pre_stats = const_cast<float*>(pre_stats);
    a.chunk = pl.chunk, a.per_gate = pl.per_gate, a.units = pl.units;
    a.gate_part = static_cast<float*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.gate_bytes);
    for (int k = 0; k < 4; ++k) a.want |= j.out[k] ? 1u << k : 0u;
    j.part = a.part, j.parts = pl.grid;
    with_type(dtype, [&](auto t) {
      using T = decltype(t);
      with_slot(C, [&](auto s) {
        using SL = decltype(s);
        hipLaunchKernelGGL((k_block_norm_bwd<T, SL>), dim3(pl.grid), dim3(SL::THREADS), 0, stream, a);
      });
      if (dgate && pl.per_gate > 1) {
        const int rows = static_cast<int>(ceil_div(M, a.gate_rows));
        hipLaunchKernelGGL((k_join_gate<T>), dim3(static_cast<unsigned>(ceil_div(static_cast<long>(rows) * ((C + 7) / 8), 256))),
                           dim3(256), 0, stream, a, rows);
      }
    });
    if (params) hipLaunchKernelGGL(k_join_params, dim3(static_cast<unsigned>(ceil_div(C, 16)), 4), dim3(256), 0, stream, j);
    return check_launch(fn);
  });
}

}  // extern "C"
