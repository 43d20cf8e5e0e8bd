// block_norm_bwd.hpp -- the block norm's backward: gradients of both norms' inputs, of the gate and
// of the parameters in one pass over the rows (formulas in embblock.h).
//
// Memory bounds it: five rows are read (dy, dh, y, f, gate) and three written (dx, df, dgate) for some 90
// operations a value, so every row is in registers between its one read and its one write, and the
// parameters' sums stay there over all rows of a slot.  65536 x 1024 in bf16 with a gate: 201 us, 5.3
// TB/s, at the rate of a copy; gate rows shared by 26 rows of 128 (426062 rows, fp16, layer norms with
// betas): 141 us, 4.75 TB/s, 1.08 of the copy's time.  Before the views, the runs of rows and the lane sums it took
// 450 and 328 us.
#pragma once

#include "block_norm.hpp"
#include "block_rows.hpp"

namespace el {
namespace {

// Gradient at a norm's input from g, the one at its output (gamma in it), and the normalised row.
template <class SL>
__device__ inline void norm_grad(float (&g)[SL::NV][8], const float (&vh)[SL::NV][8], uint32_t kind, float rstd,
                                 const NormArgs& a, float (*lds)[SL::WAVES][2], int& turn) {
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

// The slope s (1 - s) of a sigmoid gate s comes from the smaller of s and 1 - s, its tail: of an s near 1
// the other cannot be formed again (in fp32 s (1 - s) is off by 0.9 % at u = 12 and 0 from 17 on).  A
// tail carries u's sign, which says which of the two it is.
__device__ inline float gate_tail(float u) { return copysignf(sigmoid(-fabsf(u)), u); }
__device__ inline float gate_of_tail(float t) { return (__float_as_int(t) < 0 ? 0.f : 1.f) - t; }
__device__ inline float slope_of_tail(float t) { return fmaf(-t, t, fabsf(t)); }

// SHARED: rows share gate rows, so a slot takes a run of consecutive rows (all slots the same number
// within one, whatever the number of rows that share) and adds up the gate's gradient over the gate
// rows in it: one that lies in the run is finished here, the others are left as partial sums
// (gate_part[slot][0] where the gate row began before this slot, [1] where it begins here).  Not
// SHARED: a workgroup's slots take consecutive rows, and every row has its own gate row, if any.
template <class T, class SL, template <class, class> class View, bool SHARED, bool BETA, int WAVES>
__global__ __launch_bounds__(SL::THREADS, WAVES) void k_norm_bwd(NormArgs a) {
  __shared__ float lds[2][SL::WAVES][2];
  __shared__ float join[SL::PER_WG > 1 ? SL::THREADS * SL::NV * 8 : 1];
  int turn = 0;
  constexpr int NV = SL::NV, PER = SL::PER_WG;
  const int in_slot = threadIdx.x % (SL::L * SL::W), c0 = in_slot * 8, sl = threadIdx.x / (SL::L * SL::W);
  const int slots = gridDim.x * PER, slot = blockIdx.x * PER + sl;
  // the rows of this workgroup's first slot and of this slot
  const RowRange wg = rows_of_slot(blockIdx.x * PER, slots, a.M), mine = rows_of_slot(slot, slots, a.M);
  const int local = SHARED ? mine.first - wg.first : sl;
  const int steps = SHARED ? wg.n : static_cast<int>(max(0l, (static_cast<long>(a.M) - blockIdx.x * PER + slots - 1) / slots));
  View<T, SL> vdy, vdh, vy, vf, vg, vdx, vdf, vdg;
  vdy.init(a.dy, a.lddy, local, c0, a.C), vdh.init(a.dh, a.lddh, local, c0, a.C), vy.init(a.y_in, a.ldy, local, c0, a.C);
  vf.init(a.f, a.ldf, local, c0, a.C), vdx.init(a.dx, a.lddx, local, c0, a.C), vdf.init(a.df, a.lddf, local, c0, a.C);
  float gp[NV][8], gq[NV][8], bp[BETA ? NV : 1][8];
  load_param<SL>(a.gp, 1.f, c0, a.C, gp);
  load_param<SL>(a.gq, 1.f, c0, a.C, gq);
  if constexpr (BETA) load_param<SL>(a.bp, 0.f, c0, a.C, bp);
  float acc_gp[NV][8] = {}, acc_gq[NV][8] = {}, acc_bp[BETA ? NV : 1][8] = {}, acc_bq[BETA ? NV : 1][8] = {};

  // the gate: its values, or (not SHARED) a sigmoid's tails
  const bool sig = a.gate && a.gate_act == EL_GATE_SIGMOID;
  float g[NV][8], gsum[NV][8] = {};
  Raw8<T> rg[NV];
  int grow = 0, left = 0;  // SHARED: gate row of the current row, rows of it left in this slot's run
  // those of the workgroup's rows (its first slot has at least one)
  const RowRange wg_gates = SHARED ? gates_of_rows(wg.first, static_cast<long>(PER) * wg.n, a.gate_rows, a.M) : RowRange{};
  const int g0 = wg_gates.first;
  const auto gate_values = [&]() {
    vg.settle(rg);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      to_floats<T>(rg[j], g[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // 16 bits without a branch between the loads, fp32 with one (the registers are short): unshared
        // gates and betas, 65536 x 1024 in bf16 212 us, 216 with the branch; 213031 x 128 in fp32 223, 196
        if constexpr (sizeof(typename T::S) == 2) {
          g[j][e] = a.gate ? (sig ? (SHARED ? sigmoid(g[j][e]) : gate_tail(g[j][e])) : g[j][e]) : 1.f;
        } else {
          if (sig) g[j][e] = SHARED ? sigmoid(g[j][e]) : gate_tail(g[j][e]);
          else if (!a.gate) g[j][e] = 1.f;
        }
      }
    }
  };
  if constexpr (SHARED) {
    grow = mine.first / a.gate_rows;
    left = static_cast<int>(min((grow + 1l) * a.gate_rows, static_cast<long>(mine.first) + mine.n) - mine.first);
    vg.init(a.gate, a.ldg, grow - g0, c0, a.C), vdg.init(a.dgate, a.lddg, grow - g0, c0, a.C);
    vg.load(vg.span(g0, wg_gates.n, a.C), rg, 0, mine.n > 0);
    gate_values();
  } else {
    vg.init(a.gate, a.ldg, sl, c0, a.C), vdg.init(a.dgate, a.lddg, sl, c0, a.C);
  }

  Raw8<T> rdy[NV], rdh[NV], ry[NV], rf[NV];
  u32x2 spre, spost;
  const auto first_of = [&](int t) { return SHARED ? static_cast<long>(wg.first) : static_cast<long>(t) * slots + blockIdx.x * PER; };
  const auto rows_at = [&](int t) {
    if constexpr (SHARED) return min(a.M - wg.first, PER * wg.n);
    else return static_cast<int>(max(0l, min(static_cast<long>(PER), a.M - first_of(t))));
  };
  const auto valid_at = [&](int t) { return !SHARED || t < mine.n; };
  const auto fetch = [&](int t) {
    const long first = first_of(t);
    const int rows = rows_at(t), tt = SHARED ? t : 0;
    const bool ok = valid_at(t);
    vdy.load(vdy.span(first, rows, a.C), rdy, tt, ok);
    vdh.load(vdh.span(first, rows, a.C), rdh, tt, ok);
    vy.load(vy.span(first, a.dh ? rows : 0, a.C), ry, tt, ok);
    vf.load(vf.span(first, rows, a.C), rf, tt, ok);
    if constexpr (!SHARED) vg.load(vg.span(first, rows, a.C), rg);
    const uint32_t at = ok ? static_cast<uint32_t>(local + tt) * 8u : kNowhere;
    spre = __builtin_amdgcn_raw_buffer_load_b64(stats_span(a.pre_stats, first, rows), at, 0, 0);
    spost = __builtin_amdgcn_raw_buffer_load_b64(stats_span(a.post_stats, first, rows), at, 0, 0);
  };
  fetch(0);
  for (int t = 0; t < steps; ++t) {
    const long first = first_of(t);
    const int rows = rows_at(t), tt = SHARED ? t : 0;
    const bool ok = valid_at(t);
    float D[NV][8], v[NV][8], fh[NV][8], dy[NV][8];
    const float mq = __uint_as_float(spre[0]), rq = __uint_as_float(spre[1]);
    const float mp = a.post != EL_NORM_NONE ? __uint_as_float(spost[0]) : 0.f;
    const float rp = a.post != EL_NORM_NONE ? __uint_as_float(spost[1]) : 1.f;
    vdh.settle(rdh), vy.settle(ry), vf.settle(rf), vdy.settle(rdy);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      to_floats<T>(rdh[j], D[j]), to_floats<T>(ry[j], v[j]), to_floats<T>(rf[j], fh[j]), to_floats<T>(rdy[j], dy[j]);
    if constexpr (!SHARED) gate_values();
    fetch(t + 1);
    if (a.dh) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[j][e] = (v[j][e] - mq) * rq;
          acc_gq[j][e] = fmaf(D[j][e], v[j][e], acc_gq[j][e]);
          if constexpr (BETA) acc_bq[j][e] += D[j][e];
          D[j][e] *= gq[j][e];
        }
      norm_grad<SL>(D, v, a.pre, rq, a, lds, turn);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) D[j][e] += dy[j][e];
    vdx.store(vdx.span(first, rows, a.C), D, tt, ok);
    if (a.f) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          fh[j][e] = (fh[j][e] - mp) * rp;
          const float sD = a.scale * D[j][e];
          float tv;
          if constexpr (BETA) tv = fmaf(fh[j][e], gp[j][e], bp[j][e]);
          else tv = fh[j][e] * gp[j][e];
          if constexpr (SHARED) gsum[j][e] = fmaf(sD, tv, gsum[j][e]);
          else gsum[j][e] = sD * tv;
          const float u = (!SHARED && sig ? gate_of_tail(g[j][e]) : g[j][e]) * sD;
          acc_gp[j][e] = fmaf(u, fh[j][e], acc_gp[j][e]);
          if constexpr (BETA) acc_bp[j][e] += u;
          D[j][e] = u * gp[j][e];
        }
      if (!SHARED && sig)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) gsum[j][e] *= slope_of_tail(g[j][e]);
    }
    if constexpr (!SHARED) vdg.store(vdg.span(first, rows, a.C), gsum);  // (in front of the sums: fewer registers)
    if (a.f && a.df && a.post != EL_NORM_NONE) norm_grad<SL>(D, fh, a.post, rp, a, lds, turn);
    vdf.store(vdf.span(first, rows, a.C), D, tt, ok);
    if (SHARED && ok && --left == 0) {
      // the last row of this gate row in the run
      const long gfirst = static_cast<long>(grow) * a.gate_rows, row = static_cast<long>(mine.first) + t;
      const bool begins = gfirst >= mine.first, ends = row + 1 == min(gfirst + a.gate_rows, static_cast<long>(a.M));
      if (a.dgate) {
        if (begins && ends) {
          if (sig) {  // the gate row once more, from the cache: its values alone are kept
            vg.load(vg.span(g0, wg_gates.n, a.C), rg);
            vg.settle(rg);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              float raw[8];
              to_floats<T>(rg[j], raw);
#pragma unroll
              for (int e = 0; e < 8; ++e) gsum[j][e] *= slope_of_tail(gate_tail(raw[e]));
            }
          }
          vdg.store(vdg.span(g0, wg_gates.n, a.C), gsum);
        } else {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SL::L * SL::W * 8;
            if (c < a.C) store8<F32T>(a.gate_part + (2l * slot + begins) * a.C + c, gsum[j], a.C - c);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) gsum[j][e] = 0.f;
      ++grow;
      left = static_cast<int>(min((grow + 1l) * a.gate_rows, static_cast<long>(mine.first) + mine.n) - (row + 1));
      vg.at(grow - g0, c0, a.C), vdg.at(grow - g0, c0, a.C);
      if (left > 0) {
        vg.load(vg.span(g0, wg_gates.n, a.C), rg);
        gate_values();
      } else {  // (an infinite gate times the zeros of a step behind this slot's last row)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) g[j][e] = 0.f;
      }
    }
  }
  // The workgroup's sums of each asked parameter: its slots' added in slot order.
  const auto put = [&](int k, const float (&acc)[NV][8]) {
    if (!(a.want >> k & 1)) return;
    float* out = a.part + (static_cast<long>(blockIdx.x) * 4 + k) * a.C;
    if constexpr (PER == 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * SL::L * SL::W * 8;
        if (c < a.C) store8<F32T>(out + c, acc[j], a.C - c);
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) join[sl * SL::COLS + c0 + j * SL::L * SL::W * 8 + e] = acc[j][e];
      __syncthreads();
      for (int c = threadIdx.x; c < SL::COLS && c < a.C; c += SL::THREADS) {
        float s = join[c];
        for (int p = 1; p < PER; ++p) s += join[p * SL::COLS + c];
        out[c] = s;
      }
    }
  };
  put(0, acc_gp);
  put(2, acc_gq);
  if constexpr (BETA) put(1, acc_bp), put(3, acc_bq);
}

constexpr int kJoin = 256;

// dgate of the gate rows that lie in several slots: their partial sums in slot order, times the
// gate's derivative.  A thread takes eight columns of a gate row (few partial sums a row).
template <class T>
__device__ inline void finish_gate(const NormArgs& a, long r, int c, float (&v)[8]) {
  if (a.gate_act == EL_GATE_SIGMOID) {
    float g[8];
    to_floats<T>(load8_row<T>(static_cast<const typename T::S*>(a.gate) + r * a.ldg, c, a.C), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= slope_of_tail(gate_tail(g[e]));
  }
  store8<T>(static_cast<typename T::S*>(a.dgate) + r * a.lddg + c, v, a.C - c);
}
template <class T>
__device__ inline void join_gate(const NormArgs& a, unsigned block, int gates, int slots) {
  const int vecs = (a.C + 7) / 8;
  const long i = static_cast<long>(block) * kJoin + threadIdx.x;
  const long r = i / vecs;
  if (r >= gates) return;
  const int c = static_cast<int>(i - r * vecs) * 8;
  const int s0 = slot_of_row(static_cast<int>(r * a.gate_rows), slots, a.M);
  const int s1 = slot_of_row(static_cast<int>(min((r + 1) * a.gate_rows, static_cast<long>(a.M)) - 1), slots, a.M);
  if (s0 == s1) return;
  float v[8];
  to_floats<F32T>(load8_row<F32T>(a.gate_part + (2l * s0 + 1) * a.C, c, a.C), v);
  for (int s = s0 + 1; s <= s1; ++s) {
    float p[8];
    to_floats<F32T>(load8_row<F32T>(a.gate_part + 2l * s * a.C, c, a.C), p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += p[e];
  }
  finish_gate<T>(a, r, c, v);
}
// The same where a gate row lies in many slots: a workgroup takes eight columns of a gate row, thread
// p the slots s0 + p, s0 + p + 256, ...; the threads' sums are added by halves.  (One gate row for 65536
// rows of 16: 81 us of 94, what one CU reads.  1024 threads: 102, and 219 against 174 for 64 gate rows of
// 1024 columns.)
template <class T>
__device__ inline void join_gate_long(const NormArgs& a, unsigned block, int slots, float (*red)[9]) {
  const int vecs = (a.C + 7) / 8;
  const long r = block / vecs;
  const int c = static_cast<int>(block - r * vecs) * 8, p = threadIdx.x;
  const int s0 = slot_of_row(static_cast<int>(r * a.gate_rows), slots, a.M);
  const int s1 = slot_of_row(static_cast<int>(min((r + 1) * a.gate_rows, static_cast<long>(a.M)) - 1), slots, a.M);
  if (s0 == s1) return;
  float v[8] = {};
#pragma unroll 4
  for (int s = s0 + p; s <= s1; s += kJoin) {
    float q[8];
    to_floats<F32T>(load8_row<F32T>(a.gate_part + (2l * s + (s == s0)) * a.C, c, a.C), q);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += q[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) red[p][e] = v[e];
  for (int h = kJoin / 2; h > 0; h >>= 1) {
    __syncthreads();
    if (p < h)
#pragma unroll
      for (int e = 0; e < 8; ++e) red[p][e] += red[p + h][e];
  }
  if (p == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = red[0][e];
    finish_gate<T>(a, r, c, v);
  }
}
// Sixteen columns of one parameter: 16 threads share a column's parts (thread s: parts s, s + 16, ...),
// their sums are added in thread order.
__device__ inline void join_params(const JoinArgs& a, unsigned block, float (*red)[9]) {
  const int blocks = (a.C + 15) / 16, k = block / blocks;
  if (!a.out[k]) return;
  const int col = threadIdx.x & 15, s = threadIdx.x >> 4, c = (block - k * blocks) * 16 + col;
  float* sums = &red[0][0];  // [16][17]
  float v = 0.f;
  if (c < a.C)
#pragma unroll 4
    for (int p = s; p < a.parts; p += 16) v += a.part[(static_cast<long>(p) * 4 + k) * a.C + c];
  sums[s * 17 + col] = v;
  __syncthreads();
  if (s == 0 && c < a.C) {
    for (int i = 1; i < 16; ++i) v += sums[i * 17 + col];
    a.out[k][c] = v;
  }
}
// All of a call's joins in one launch (a launch of its own for each: 6 us more from call to call).
template <class T, bool LONG>
__global__ __launch_bounds__(kJoin) void k_join(NormArgs a, JoinArgs j, unsigned param_blocks, int gates, int slots) {
  __shared__ float red[kJoin][9];
  if (blockIdx.x < param_blocks) join_params(j, blockIdx.x, red);
  else if (LONG) join_gate_long<T>(a, blockIdx.x - param_blocks, slots, red);
  else join_gate<T>(a, blockIdx.x - param_blocks, gates, slots);
}

template <class T, class SL, template <class, class> class View, bool BETA>
void launch_one_bwd(const NormArgs& a, bool shared, int grid, hipStream_t st) {
  constexpr bool loose = std::is_same_v<View<T, SL>, Loose<T, SL>>;
  const auto kernel = shared ? k_norm_bwd<T, SL, View, true, BETA, kBwdWaves<SL, loose>> : k_norm_bwd<T, SL, View, false, BETA, kBwdWaves<SL, false>>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(SL::THREADS), 0, st, a);
}

}  // namespace

template <class T>
void launch_norm_bwd(const NormArgs& a, const JoinArgs& j, bool aligned, bool lean, bool shared, int grid, hipStream_t st) {
  constexpr bool two = sizeof(typename T::S) == 2;
  with_bwd_slot<two>(a.C, lean, [&](auto s) {
    using SL = decltype(s);
    if constexpr (SL::COLS <= kMaxAlignedCols) {
      if (lean) return launch_one_bwd<T, SL, Aligned, false>(a, shared, grid, st);
      if constexpr (!kLeanOnly<SL>)
        if (aligned) return launch_one_bwd<T, SL, Aligned, true>(a, shared, grid, st);
    }
    if constexpr (!kLeanOnly<SL>) launch_one_bwd<T, SL, Loose, true>(a, shared, grid, st);
  });
  const unsigned param_blocks = a.want ? 4 * static_cast<unsigned>(ceil_div(a.C, 16)) : 0;
  const bool join = shared && a.dgate;
  if (!param_blocks && !join) return;
  int per = 1;
  with_bwd_slot<two>(a.C, lean, [&](auto s) { per = decltype(s)::PER_WG; });
  const int slots = grid * per, gates = join ? static_cast<int>(ceil_div(a.M, a.gate_rows)) : 0;
  const long vecs = (a.C + 7) / 8;
  // A gate row in more than 32 slots is worth a workgroup: the backward of 426062 x 128 in bf16 with a
  // gate row's slots joined by a thread and by a workgroup: 6 slots each 142 and 184 us, 29 slots 149 and
  // 150, 1170 slots 515 and 145.
  const bool longer = join && slots / gates > 32;
  const long gate_blocks = longer ? gates * vecs : ceil_div(gates * vecs, kJoin);
  const auto kernel = longer ? k_join<T, true> : k_join<T, false>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(param_blocks + gate_blocks)), dim3(kJoin), 0, st, a, j, param_blocks, gates, slots);
}

}  // namespace el
