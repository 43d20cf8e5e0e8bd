// block_norm.hip -- the norms behind one residual block and before the next, with the block's gate
// and residual scale, forward and backward (formulas in embblock.h).
//
// Rows are independent but for the sums of the parameters' and the shared gates' gradients.  A slot
// (L lanes of a wavefront, or W whole wavefronts) owns a row: its columns stay in registers, eight
// to a vector, NV vectors a lane, between the one read of the row and the one write.
#include "tower_common.hpp"
#include "embblock.h"

namespace el {
namespace {

constexpr int kMaxCols = 32768;

struct NormArgs {
  uint32_t post, pre, gate_act;
  int gate_rows;
  float scale, eps, inv_c;
  const float *gp, *bp, *gq, *bq;  // post and pre gamma, beta
  const void *x, *f, *gate;        // forward
  const void *dy, *dh, *y_in;      // backward
  void *y, *h;                     // forward
  void *dx, *df, *dgate;           // backward
  long ldx, ldf, ldg, ldy, ldh, lddy, lddh, lddx, lddf, lddg;
  float *post_stats, *pre_stats;
  int M, C;
  // backward: units of rows that share a gate row
  int chunk;        // rows of a unit
  int per_gate;     // units of a gate row
  int units;
  float* gate_part;  // [units][C] where a gate row has several units
  float* part;       // [grid][4][C]: the parameters' partial sums
  uint32_t want;     // bit k: parameter sum k is asked for
};

// A slot: L lanes of one wavefront (W = 1), or W whole wavefronts (L = 64), NV vectors a lane.
template <int L_, int W_, int NV_>
struct Slot {
  static constexpr int L = L_, W = W_, NV = NV_;
  static constexpr int COLS = L * W * NV * 8;
  static constexpr int THREADS = W > 4 ? W * 64 : 256;
  static constexpr int PER_WG = THREADS / (L * W);
  static_assert(W == 1 || PER_WG == 1, "a slot of several wavefronts is a workgroup");
};

// Sums of N values over a slot; the same in all its lanes.
template <class SL, int N>
__device__ inline void slot_sums(float (&v)[N], float (*lds)[SL::W][2], int& turn) {
#pragma unroll
  for (int o = 1; o < SL::L; o <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], o);
  if constexpr (SL::W > 1) {
    // two buffers in turn: a wavefront that writes one has passed the barrier behind which nobody
    // reads it any more
    float(*b)[2] = lds[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) b[threadIdx.x >> 6][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = b[0][k];
#pragma unroll
      for (int w = 1; w < SL::W; ++w) s += b[w][k];
      v[k] = s;
    }
  }
}

// Columns c .. c+7 of a parameter (`fill` where there is none), zeros from the n-th on.
__device__ inline void load_vec(const float* p, float fill, int c, int n, float (&v)[8]) {
  if (p && n > 0) {
    to_floats<F32T>(load8_raw<F32T>(p + c, n), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? fill : 0.f;
  }
}

template <class T, class SL>
struct RowRaw {
  Raw8<T> v[SL::NV];
  __device__ inline void load(const void* base, long ld, long row, int c0, int C) {
    const typename T::S* p = static_cast<const typename T::S*>(base) + row * ld;
#pragma unroll
    for (int j = 0; j < SL::NV; ++j) {
      const int c = c0 + j * SL::L * SL::W * 8, n = C - c;
      if (n > 0) v[j] = load8_raw<T>(p + c, n);
      else
#pragma unroll
        for (int w = 0; w < Raw8<T>::W; ++w) v[j].v[w] = u32x4{0, 0, 0, 0};
    }
  }
};

template <class T, class SL>
__device__ inline void store_row(void* base, long ld, long row, int c0, int C, const float (&v)[SL::NV][8]) {
  typename T::S* p = static_cast<typename T::S*>(base) + row * ld;
#pragma unroll
  for (int j = 0; j < SL::NV; ++j) {
    const int c = c0 + j * SL::L * SL::W * 8, n = C - c;
    if (n > 0) store8<T>(p + c, v[j], n);
  }
}

// Mean and rstd of a slot's row (values past its end are zero).
template <class SL>
__device__ inline void row_stats(const float (&v)[SL::NV][8], uint32_t kind, const NormArgs& a, int c0,
                                 float (*lds)[SL::W][2], int& turn, float& mean, float& rstd) {
  float s[1] = {0.f};
  mean = 0.f;
  if (kind == EL_NORM_LAYER) {
#pragma unroll
    for (int j = 0; j < SL::NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[j][e];
    slot_sums<SL>(s, lds, turn);
    mean = s[0] * a.inv_c;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < SL::NV; ++j) {
      const int n = a.C - (c0 + j * SL::L * SL::W * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < n ? v[j][e] - mean : 0.f;
        s[0] = fmaf(d, d, s[0]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < SL::NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] = fmaf(v[j][e], v[j][e], s[0]);
  }
  slot_sums<SL>(s, lds, turn);
  rstd = 1.f / sqrtf(s[0] * a.inv_c + a.eps);
}

__device__ inline float gate_value(uint32_t act, float u) { return act == EL_GATE_SIGMOID ? sigmoid(u) : u; }

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
// Plans and launches.
// ---------------------------------------------------------------------------------------
constexpr int kCus = 256;
constexpr int kBwdGroups = 2 * kCus;  // workgroups of the backward at most

long ceil_div(long a, long b) { return (a + b - 1) / b; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Calls f with the narrowest slot that holds C columns.
template <class F>
void with_slot(int C, F&& f) {
  const int v = (C + 7) / 8;
  if (v <= 2) f(Slot<2, 1, 1>{});
  else if (v <= 4) f(Slot<4, 1, 1>{});
  else if (v <= 8) f(Slot<8, 1, 1>{});
  else if (v <= 16) f(Slot<16, 1, 1>{});
  else if (v <= 32) f(Slot<32, 1, 1>{});
  else if (v <= 64) f(Slot<64, 1, 1>{});
  else if (v <= 128) f(Slot<64, 1, 2>{});
  else if (v <= 256) f(Slot<64, 4, 1>{});
  else if (v <= 512) f(Slot<64, 4, 2>{});
  else if (v <= 1024) f(Slot<64, 16, 1>{});
  else if (v <= 2048) f(Slot<64, 16, 2>{});
  else f(Slot<64, 16, 4>{});
}

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

template <class F>
void with_type(el_dtype dtype, F&& f) {
  if (dtype == EL_F32) f(F32T{});
  else if (dtype == EL_F16) f(F16T{});
  else f(BF16T{});
}

el_status check_norm(const char* fn, const el_block_norm* p, int32_t M, int32_t C, el_dtype dtype) {
  if (!p) return tower::bad(fn, "the parameters are null");
  if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
  if (M < 0) return tower::bad(fn, "M must be >= 0");
  if (C < 1) return tower::bad(fn, "C must be >= 1");
  if (C > kMaxCols) return tower::unsupported(fn, "C must be <= 32768");
  if (p->post > EL_NORM_LAYER) return tower::bad(fn, "post must be EL_NORM_NONE, _RMS or _LAYER");
  if (p->pre != EL_NORM_RMS && p->pre != EL_NORM_LAYER) return tower::bad(fn, "pre must be EL_NORM_RMS or EL_NORM_LAYER");
  if (p->gate_act > EL_GATE_SIGMOID) return tower::bad(fn, "gate_act must be EL_GATE_NONE or EL_GATE_SIGMOID");
  if (p->gate_rows < 1) return tower::bad(fn, "gate_rows must be >= 1");
  if (!std::isfinite(p->scale)) return tower::bad(fn, "scale must be finite");
  if (!std::isfinite(p->eps) || p->eps < 0.f) return tower::bad(fn, "eps must be finite and >= 0");
  if (!tower::al(p->post_gamma, 4) || !tower::al(p->post_beta, 4) || !tower::al(p->pre_gamma, 4) || !tower::al(p->pre_beta, 4))
    return tower::bad(fn, "gammas and betas must be aligned to their elements");
  return EL_OK;
}

NormArgs common(const el_block_norm* p, int M, int C) {
  NormArgs a{};
  a.post = p->post, a.pre = p->pre, a.gate_act = p->gate_act, a.gate_rows = p->gate_rows;
  a.scale = p->scale, a.eps = p->eps, a.inv_c = 1.f / static_cast<float>(C);
  a.gp = p->post_gamma, a.bp = p->post_beta, a.gq = p->pre_gamma, a.bq = p->pre_beta;
  a.M = M, a.C = C;
  return a;
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
        const dim3 grid(static_cast<unsigned>(std::min<long>(wgs, 16l * kCus)));
        hipLaunchKernelGGL((k_block_norm_fwd<decltype(t), SL>), grid, dim3(SL::THREADS), 0, stream, a);
      });
    });
    return check_launch(fn);
  });
}

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
