// group_norm.hip -- channels-last group norm with an activation, forward and backward.
//
// Per sample b and group g, over the n = len Cg values of the group's Cg channels at the
// sample's first len positions:
//   mean = sum x / n,  var = sum (x - mean)^2 / n,  rstd = 1 / sqrt(var + eps)
//   y    = act(u),  u = gamma xh + beta,  xh = (x - mean) rstd
// and backward, with du = dy act'(u), dh = du gamma:
//   dx     = rstd (dh - avg(dh) - xh avg(dh xh))
//   dgamma = sum_{b,s} du xh,  dbeta = sum_{b,s} du
//
// Bound by memory: x in, y out (forward); x, dy in, dx out (backward).  Three forms:
//   wavefront  a sample sits in the registers of some lanes of one wavefront, which exchange its
//              sums: read once, no barrier (16384 samples of 26 x 128 in 8 groups, bf16, SiLU:
//              forward 42 us, 5.2 TB/s, the rate of a copy; backward 76.8 us, 4.3 TB/s, without an
//              activation 72.8: two wavefronts per SIMD, which its 223 registers leave, do not keep
//              more loads in flight; at three it spills and takes 214 us);
//   resident   a sample sits in the registers of one workgroup's threads, which join its sums in
//              LDS: read once, any width and group size (16384 samples of 26 x 96 in 6 groups, bf16:
//              forward 71 us, backward 127, floors 32 and 47; 65536 rows of 1024: 128 and 160, floors
//              52 and 78: one to four vectors a thread in flight, and four barriers for every join
//              of sums, of which the forward has two a sample);
//   streamed   samples too large for that are cut into chunks of positions: one kernel leaves
//              per-channel statistics of each chunk, one joins them per group (the forward of a
//              sample in one chunk does both in one), one applies them
//              (x, and dy, are read twice, the second time from the caches where they fit: 6
//              samples of up to 5001 x 256 in 32 groups, fp16: stats 7.4 us, join 5.0, apply 9.4;
//              backward 11.4, 4.8 with the parameters' sums, 10.9: six dependent launches).
// A thread owns eight consecutive channels of some positions, so every access is a 16-byte
// vector whatever the group width; sums are kept per channel and joined into groups afterwards
// where a vector crosses groups.
#include <algorithm>

#include "tower_common.hpp"

namespace el {
namespace {

constexpr int kResident = 512;  // most threads of a resident workgroup

struct GnArgs {
  const void *x, *dy;
  void* out;  // y or dx
  long ldx, lddy, ldo;
  int B, S, C, G, Cg, CV;  // CV: vectors of eight channels per position
  const int32_t* lengths;
  const float *gamma, *beta;
  float eps;
  uint32_t act;
  float *mean, *rstd;  // written by the forward, read by the backward
  float2* part;        // workspace, see the kernels
  float* gsum;         // [2][B][G]: avg(dh), avg(dh xh)
  float *dgamma, *dbeta;
  // resident
  int TR, team, spw, E, E1, E1_rows, E1_cols;  // E1 = E1_rows (entries of a group's row) + E1_cols
  int blocks;
  // streamed
  int chunks, per_chunk, pieces, per_piece, colblocks, TC;  // chunks: statistics; pieces: their use
};

__device__ inline int sample_len(const GnArgs& a, int b) {
  return a.lengths ? min(max(a.lengths[b], 0), a.S) : a.S;
}

// ---------------------------------------------------------------------------------------
// Resident form.
// ---------------------------------------------------------------------------------------
// Sums over the group, for NVAL values at once.  In: the thread's sums p[v][i] for its
// channels (i < 8), or p[v][0] for all eight where a vector lies inside one group (VECG).
// Out: p[v][i] = the sum over the group of channel i (VECG: p[v][0]).  Every thread of the
// workgroup calls it; the order of additions is fixed.  LDS: `red` holds NVAL arrays of one
// entry per thread (VECG) or eight, then `mid` NVAL x spw x G x E1, then `tot` NVAL x spw x G.
template <bool VECG, int NVAL>
__device__ inline void group_sums(const GnArgs& a, float* lds, int tid, int team_id, int r, int cv, bool on,
                                  float (&p)[NVAL][8]) {
  const int nt = blockDim.x;
  const int per_thread = VECG ? 1 : 8;
  const int cols = VECG ? a.CV : a.CV * 8;        // entries of one thread row of a team
  const int gc = VECG ? a.Cg / 8 : a.Cg;          // of them in one group
  const int red_n = nt * per_thread, items = a.spw * a.G;
  float* red = lds;
  float* mid = lds + NVAL * red_n;
  float* tot = mid + NVAL * items * a.E1;
  __syncthreads();
  if (on) {
#pragma unroll
    for (int v = 0; v < NVAL; ++v)
#pragma unroll
      for (int i = 0; i < (VECG ? 1 : 8); ++i) red[v * red_n + (team_id * a.team + r) * per_thread + i] = p[v][i];
  }
  __syncthreads();
  for (int j = tid; j < items * a.E1; j += nt) {
    const int it = j / a.E1, e0 = j - it * a.E1;
    const int smp = it / a.G, g = it - smp * a.G;
    float s[NVAL] = {};
    int row = e0 / gc, col = e0 - row * gc;
    const float* from = red + smp * a.team * per_thread + g * gc;
    for (int e = e0; e < a.E; e += a.E1) {
#pragma unroll
      for (int v = 0; v < NVAL; ++v) s[v] += from[v * red_n + row * cols + col];
      row += a.E1_rows;
      col += a.E1_cols;
      if (col >= gc) col -= gc, ++row;
    }
#pragma unroll
    for (int v = 0; v < NVAL; ++v) mid[v * items * a.E1 + j] = s[v];
  }
  __syncthreads();
  for (int j = tid; j < items; j += nt) {
#pragma unroll
    for (int v = 0; v < NVAL; ++v) {
      float s = 0.f;
      for (int e = 0; e < a.E1; ++e) s += mid[(v * items + j) * a.E1 + e];
      tot[v * items + j] = s;
    }
  }
  __syncthreads();
  if (on) {
#pragma unroll
    for (int v = 0; v < NVAL; ++v)
    {
      if (VECG)
        p[v][0] = tot[v * items + team_id * a.G + cv * 8 / a.Cg];
      else
        load_groups(a, tot + v * items + team_id * a.G, cv, p[v]);
    }
  }
}

template <bool VECG>
__device__ inline float of_channel(const float (&p)[8], int i) { return p[VECG ? 0 : i]; }

// xh = (x - mean) rstd and du of eight values.  (Centred before it is scaled, as in the forward:
// x rstd - mean rstd loses |mean| rstd steps of fp32, also where x - mean is exact.)
template <class T, bool VECG>
__device__ inline void grad8(const GnArgs& a, const Raw8<T>& rx, const Raw8<T>& rd, const float (&mean)[8],
                             const float (&rstd)[8], const float (&gamma)[8], const float (&beta)[8], float (&xh)[8],
                             float (&du)[8]) {
  float u[8];
  to_floats<T>(rx, xh);
  to_floats<T>(rd, du);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    xh[q] = (xh[q] - of_channel<VECG>(mean, q)) * of_channel<VECG>(rstd, q);
    u[q] = fmaf(xh[q], gamma[q], beta[q]);
  }
  act8_grad(a.act, u, du);
}

// Hides a vector's value from the compiler: what was computed from it before is computed again
// instead of being kept.  (The backward holds x as raw 16-byte vectors; xh beside du in fp32 would
// spill.)
template <class T>
__device__ inline void forget(Raw8<T>& r) {
#pragma unroll
  for (int w = 0; w < Raw8<T>::W; ++w) asm volatile("" : "+v"(r.v[w]));
}

__device__ inline void load_params(const GnArgs& a, int cv, float (&gamma)[8], float (&beta)[8]) {
  const auto load = [&](const float* p, float (&v)[8], float other) {
    if (p && cv * 8 + 8 <= a.C) {
      to_floats<F32T>(load8_raw<F32T>(p + cv * 8), v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p && cv * 8 + i < a.C ? p[cv * 8 + i] : other;
    }
  };
  load(a.gamma, gamma, 1.f);
  load(a.beta, beta, 0.f);
}

// v[i] = p[group of channel 8 cv + i] (of the last channel past it), with one division.
__device__ inline void load_groups(const GnArgs& a, const float* p, int cv, float (&v)[8]) {
  int g = cv * 8 / a.Cg, r = cv * 8 - g * a.Cg;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = p[min(g, a.G - 1)];
    if (++r == a.Cg) r = 0, ++g;
  }
}

template <class T, int NV, bool VECG>
__global__ __launch_bounds__(kResident) void k_gn_fwd_resident(GnArgs a) {
  extern __shared__ float lds[];
  using St = typename T::S;
  const int tid = threadIdx.x, team_id = tid / a.team, r = tid - team_id * a.team;
  const int tr = r / a.CV, cv = r - tr * a.CV;
  const long b = static_cast<long>(blockIdx.x) * a.spw + team_id;
  const bool on = team_id < a.spw && b < a.B;
  const int n = min(8, a.C - cv * 8);
  const int len = on ? sample_len(a, static_cast<int>(b)) : 0;
  const St* x = static_cast<const St*>(a.x) + (on ? b * a.S * a.ldx : 0) + cv * 8;
  Raw8<T> raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int s = tr + i * a.TR;
    if (s < len) raw[i] = load8_raw<T>(x + s * a.ldx, n);
  }
  const float inv_n = len > 0 ? 1.f / (static_cast<float>(len) * a.Cg) : 0.f;
  float p[1][8] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tr + i * a.TR < len) {
      float f[8];
      to_floats<T>(raw[i], f);
#pragma unroll
      for (int q = 0; q < 8; ++q) p[0][VECG ? 0 : q] += f[q];
    }
  group_sums<VECG, 1>(a, lds, tid, team_id, r, cv, on, p);
  float mean[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) mean[q] = of_channel<VECG>(p[0], q) * inv_n;
#pragma unroll
  for (int q = 0; q < 8; ++q) p[0][q] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tr + i * a.TR < len) {
      float f[8];
      to_floats<T>(raw[i], f);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (VECG || q < n) p[0][VECG ? 0 : q] += (f[q] - mean[q]) * (f[q] - mean[q]);
    }
  group_sums<VECG, 1>(a, lds, tid, team_id, r, cv, on, p);
  if (!on) return;
  float rstd[8], gamma[8], beta[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) rstd[q] = 1.f / sqrtf(of_channel<VECG>(p[0], q) * inv_n + a.eps);
  load_params(a, cv, gamma, beta);
  if (tr == 0)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = cv * 8 + q;
      if (c < a.C && c % a.Cg == 0) {
        a.mean[b * a.G + c / a.Cg] = mean[q];
        a.rstd[b * a.G + c / a.Cg] = rstd[q];
      }
    }
  St* y = static_cast<St*>(a.out) + b * a.S * a.ldo + cv * 8;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int s = tr + i * a.TR;
    if (s >= a.S) continue;
    float f[8] = {};
    if (s < len) {
      to_floats<T>(raw[i], f);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = (f[q] - mean[q]) * rstd[q] * gamma[q] + beta[q];
      act8(a.act, f);
    }
    store8<T>(y + s * a.ldo, f, n);
  }
}

// Every workgroup takes samples blockIdx.x * spw + team, then gridDim.x * spw further on, and
// keeps dgamma / dbeta of its samples in registers; part[workgroup][c] = (dbeta, dgamma).  A sample's
// mean and rstd are one value each where a vector lies inside a group (65536 rows of 1024 bf16: 161
// us, eight of each 244).
template <class T, int NV, bool VECG>
__global__ __launch_bounds__(kResident) void k_gn_bwd_resident(GnArgs a) {
  extern __shared__ float lds[];
  using St = typename T::S;
  const int tid = threadIdx.x, team_id = tid / a.team, r = tid - team_id * a.team;
  const int tr = r / a.CV, cv = r - tr * a.CV;
  const int n = min(8, a.C - cv * 8), group = VECG ? cv * 8 / a.Cg : 0;
  float gamma[8], beta[8], sb[8] = {}, sg[8] = {};
  load_params(a, cv, gamma, beta);
  const long first = static_cast<long>(blockIdx.x) * a.spw, step = static_cast<long>(gridDim.x) * a.spw;
  // VECG: pointers walk from sample to sample and a thread's rows lie a uniform stride apart.  With
  // per-channel statistics the scalar registers do not hold that too: a sample's pointers are
  // computed and the rows' offsets kept (65536 rows of 600 in 50 groups 165 us, walking 178).
  const auto place = [&](int i, long ld) { return VECG ? i * (a.TR * ld) : (tr + i * a.TR) * ld; };
  const long row0 = (first + team_id) * a.S + (VECG ? tr : 0), rows = step * a.S;
  const St* x = static_cast<const St*>(a.x) + row0 * a.ldx + cv * 8;
  const St* dy = static_cast<const St*>(a.dy) + row0 * a.lddy + cv * 8;
  St* dx = static_cast<St*>(a.out) + row0 * a.ldo + cv * 8;
  for (long b0 = first; b0 < a.B; b0 += step, x += rows * a.ldx, dy += rows * a.lddy, dx += rows * a.ldo) {
    const long b = b0 + team_id;
    const bool on = team_id < a.spw && b < a.B;
    if constexpr (!VECG) {
      x = static_cast<const St*>(a.x) + (on ? b * a.S * a.ldx : 0) + cv * 8;
      dy = static_cast<const St*>(a.dy) + (on ? b * a.S * a.lddy : 0) + cv * 8;
      dx = static_cast<St*>(a.out) + b * a.S * a.ldo + cv * 8;
    }
    const int len = on ? sample_len(a, static_cast<int>(b)) : 0;
    float mean[8], rstd[8];  // before the sample's vectors, so that those are waited for once
    const long at = on ? b * a.G : 0;
    if constexpr (VECG) {
      rstd[0] = a.rstd[at + group];
      mean[0] = a.mean[at + group];
    } else {
      load_groups(a, a.rstd + at, cv, rstd);
      load_groups(a, a.mean + at, cv, mean);
    }
    Raw8<T> rx[NV], rd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int s = tr + i * a.TR;
      if (s < len) {
        rx[i] = load8_raw<T>(x + place(i, a.ldx), n);
        rd[i] = load8_raw<T>(dy + place(i, a.lddy), n);
      }
    }
    const float inv_n = len > 0 ? 1.f / (static_cast<float>(len) * a.Cg) : 0.f;
    float p[2][8] = {}, cb[8] = {}, cg[8] = {}, du[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (tr + i * a.TR < len) {
        float xh[8];
        grad8<T, VECG>(a, rx[i], rd[i], mean, rstd, gamma, beta, xh, du[i]);  // du is zero past the last channel
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          cb[q] += du[i][q];
          cg[q] = fmaf(du[i][q], xh[q], cg[q]);
        }
      }
#pragma unroll
    for (int q = 0; q < 8; ++q) {  // the sample's channel sums serve both the groups and the parameters
      sb[q] += cb[q];
      sg[q] += cg[q];
      p[0][VECG ? 0 : q] = fmaf(cb[q], gamma[q], p[0][VECG ? 0 : q]);
      p[1][VECG ? 0 : q] = fmaf(cg[q], gamma[q], p[1][VECG ? 0 : q]);
    }
    group_sums<VECG, 2>(a, lds, tid, team_id, r, cv, on, p);
    if (on) {
#pragma unroll
      for (int q = 0; q < (VECG ? 1 : 8); ++q) p[0][q] *= -inv_n, p[1][q] *= -inv_n * rstd[q];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int s = tr + i * a.TR;
        if (s >= a.S) continue;
        float f[8] = {};
        if (s < len) {
          forget(rx[i]);
          to_floats<T>(rx[i], f);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            f[q] -= of_channel<VECG>(mean, q);
            f[q] = of_channel<VECG>(rstd, q) * fmaf(du[i][q], gamma[q], fmaf(f[q], of_channel<VECG>(p[1], q), of_channel<VECG>(p[0], q)));
          }
        }
        store8<T>(dx + place(i, a.ldo), f, n);
      }
    }
  }
  if (!a.part) return;
  // the thread rows of all teams into row 0, by halving the rows
  float2* red = reinterpret_cast<float2*>(lds);
  const int nt = blockDim.x, row = team_id * a.TR + tr;
  __syncthreads();
  for (int left = a.spw * a.TR; left > 1;) {
    const int half = (left + 1) / 2;
    if (row >= half && row < left) {
#pragma unroll
      for (int q = 0; q < 8; ++q) red[q * nt + tid] = make_float2(sb[q], sg[q]);
    }
    __syncthreads();
    if (row < half && row + half < left) {  // (the next rows to be written lie before these)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 v = red[q * nt + tid + half * a.CV];
        sb[q] += v.x;
        sg[q] += v.y;
      }
    }
    left = half;
  }
  if (row == 0) {
    float2* part = a.part + static_cast<long>(blockIdx.x) * a.C + cv * 8;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) part[q] = make_float2(sb[q], sg[q]);
  }
}

// ---------------------------------------------------------------------------------------
// Wavefront form: a sample of at most 512 vectors whose channels and groups are powers of two.
// 2^k lanes (a team) own a sample: lane = row * CV + cv inside the team, `TR` rows, so a group's
// values sit in lanes that differ in some bits of their number and its sums are exchanges
// between lanes, with no LDS and no barrier.  A wavefront holds 64 / team samples.
// ---------------------------------------------------------------------------------------
constexpr int kWave = 256;  // threads of a workgroup: four independent wavefronts

struct WavePos {
  long b;
  int cv, tr, len;
  bool on;
};
__device__ inline WavePos wave_pos(const GnArgs& a, long first) {
  WavePos q;
  const int t = threadIdx.x;
  q.b = first + t / a.team;
  q.cv = t & (a.CV - 1);
  q.tr = (t & (a.team - 1)) / a.CV;
  q.on = q.b < a.B;
  q.len = q.on ? sample_len(a, static_cast<int>(q.b)) : 0;
  return q;
}

// Sums over the group of each channel, over its lanes and rows.  VECG: p[0] stands for all eight
// channels; otherwise Cg is 1, 2 or 4 and p[i] becomes the sum of channel i's group.
template <bool VECG>
__device__ inline void lane_sums(const GnArgs& a, float (&p)[8]) {
#pragma unroll
  for (int i = 0; i < (VECG ? 1 : 8); ++i) {
    if (VECG)
      for (int m = 1; m * 8 < a.Cg; m <<= 1) p[i] += __shfl_xor(p[i], m);
    for (int m = a.CV; m < a.team; m <<= 1) p[i] += __shfl_xor(p[i], m);
  }
  if (!VECG && a.Cg > 1) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) p[i] = p[i + 1] = p[i] + p[i + 1];
    if (a.Cg > 2)
#pragma unroll
      for (int i = 0; i < 8; i += 4) p[i] = p[i + 1] = p[i + 2] = p[i + 3] = p[i] + p[i + 2];
  }
}

template <class T, int NV, bool VECG>
__global__ __launch_bounds__(kWave) void k_gn_fwd_wave(GnArgs a) {
  using St = typename T::S;
  const WavePos w = wave_pos(a, static_cast<long>(blockIdx.x) * (kWave / a.team));
  const St* x = static_cast<const St*>(a.x) + w.b * a.S * a.ldx + w.cv * 8;
  Raw8<T> raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int s = w.tr + i * a.TR;
    if (s < w.len) raw[i] = load8_raw<T>(x + s * a.ldx);
  }
  float gamma[8], beta[8];
  load_params(a, w.cv, gamma, beta);
  const float inv_n = w.len > 0 ? 1.f / (static_cast<float>(w.len) * a.Cg) : 0.f;
  float f[NV][8], p[8] = {}, mean[8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (w.tr + i * a.TR < w.len) {
      to_floats<T>(raw[i], f[i]);
#pragma unroll
      for (int q = 0; q < 8; ++q) p[VECG ? 0 : q] += f[i][q];
    }
  lane_sums<VECG>(a, p);
#pragma unroll
  for (int q = 0; q < 8; ++q) mean[q] = of_channel<VECG>(p, q) * inv_n;
#pragma unroll
  for (int q = 0; q < 8; ++q) p[q] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (w.tr + i * a.TR < w.len) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        f[i][q] -= mean[q];
        p[VECG ? 0 : q] += f[i][q] * f[i][q];
      }
    }
  lane_sums<VECG>(a, p);
  if (!w.on) return;
  float rstd[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) rstd[q] = VECG && q > 0 ? rstd[0] : 1.f / sqrtf(p[q] * inv_n + a.eps);
  if (w.tr == 0)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = w.cv * 8 + q;
      if ((c & (a.Cg - 1)) == 0) {
        a.mean[w.b * a.G + c / a.Cg] = mean[q];
        a.rstd[w.b * a.G + c / a.Cg] = rstd[q];
      }
    }
#pragma unroll
  for (int q = 0; q < 8; ++q) gamma[q] *= rstd[q];
  St* y = static_cast<St*>(a.out) + w.b * a.S * a.ldo + w.cv * 8;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int s = w.tr + i * a.TR;
    if (s >= a.S) continue;
    if (s < w.len) {
#pragma unroll
      for (int q = 0; q < 8; ++q) f[i][q] = f[i][q] * gamma[q] + beta[q];
      act8(a.act, f[i]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) f[i][q] = 0.f;
    }
    store8<T>(y + s * a.ldo, f[i], 8);
  }
}

// part[workgroup][c] = (dbeta, dgamma) of the workgroup's samples, as in the resident form.
// Pointers walk from sample to sample and rows lie a uniform stride apart, so that no lane keeps an
// offset per vector (48 registers; 16384 samples of 26 x 128 bf16, 8 groups: 76.8 us against 91.1).
// Two wavefronts per SIMD; one where eight fp32 vectors and per-channel sums would spill (8192
// samples of 26 x 128, 32 groups: 102.6 us, spilling 134.8).  du stays in registers between the sums
// and dx (KEEP: the activation's derivative, two transcendental instructions a value, is taken once),
// unless that spills, with eight fp32 vectors a lane at two wavefronts per SIMD: 16384 samples of
// bf16, 8 groups 76.8 us against 101.7 taken twice, 32 groups 94.1 against 108.5; 8192 of fp32, 32
// groups 102.6 against 114.6, but 8 groups 113.2 against 79.0.
template <class T, int NV, bool VECG>
__global__ __launch_bounds__(kWave, NV == 8 && !VECG && sizeof(typename T::S) == 4 ? 1 : 2) void k_gn_bwd_wave(GnArgs a) {
  using St = typename T::S;
  constexpr bool KEEP = NV < 8 || !VECG || sizeof(St) == 2;
  float gamma[8], beta[8], sb[8] = {}, sg[8] = {};
  load_params(a, threadIdx.x & (a.CV - 1), gamma, beta);
  const int per = kWave / a.team;
  const long step = static_cast<long>(gridDim.x) * per, rows = step * a.S;
  const WavePos w0 = wave_pos(a, static_cast<long>(blockIdx.x) * per);
  const long row0 = w0.b * a.S + w0.tr;
  const St* x = static_cast<const St*>(a.x) + row0 * a.ldx + w0.cv * 8;
  const St* dy = static_cast<const St*>(a.dy) + row0 * a.lddy + w0.cv * 8;
  St* dx = static_cast<St*>(a.out) + row0 * a.ldo + w0.cv * 8;
  for (long first = static_cast<long>(blockIdx.x) * per; first < a.B;
       first += step, x += rows * a.ldx, dy += rows * a.lddy, dx += rows * a.ldo) {
    const WavePos w = wave_pos(a, first);
    Raw8<T> rx[NV], rd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int s = w.tr + i * a.TR;
      if (s < w.len) {
        rx[i] = load8_raw<T>(x + i * (a.TR * a.ldx));
        rd[i] = load8_raw<T>(dy + i * (a.TR * a.lddy));
      }
    }
    float mean[8], rstd[8], p0[8] = {}, p1[8] = {}, cb[8] = {}, cg[8] = {}, du[KEEP ? NV : 1][8];
#pragma unroll
    for (int q = 0; q < (VECG ? 1 : 8); ++q) {
      const long at = w.on ? w.b * a.G + (w.cv * 8 + q) / a.Cg : 0;
      rstd[q] = a.rstd[at];
      mean[q] = a.mean[at];
    }
    const float inv_n = w.len > 0 ? 1.f / (static_cast<float>(w.len) * a.Cg) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.tr + i * a.TR < w.len) {
        float xh[8];
        float(&d)[8] = du[KEEP ? i : 0];
        grad8<T, VECG>(a, rx[i], rd[i], mean, rstd, gamma, beta, xh, d);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          cb[q] += d[q];
          cg[q] = fmaf(d[q], xh[q], cg[q]);
        }
        __builtin_amdgcn_sched_barrier(0);  // one vector's values in registers at a time
      }
#pragma unroll
    for (int q = 0; q < 8; ++q) {  // the sample's channel sums serve both the groups and the parameters
      sb[q] += cb[q];
      sg[q] += cg[q];
      p0[VECG ? 0 : q] = fmaf(cb[q], gamma[q], p0[VECG ? 0 : q]);
      p1[VECG ? 0 : q] = fmaf(cg[q], gamma[q], p1[VECG ? 0 : q]);
    }
    lane_sums<VECG>(a, p0);
    lane_sums<VECG>(a, p1);
    if (!w.on) continue;
#pragma unroll
    for (int q = 0; q < (VECG ? 1 : 8); ++q) p0[q] *= -inv_n, p1[q] *= KEEP ? -inv_n * rstd[q] : -inv_n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int s = w.tr + i * a.TR;
      if (s >= a.S) continue;
      float f[8] = {};
      if (s < w.len) {
        float(&d)[8] = du[KEEP ? i : 0];
        forget(rx[i]);
        if constexpr (KEEP) {
          to_floats<T>(rx[i], f);
#pragma unroll
          for (int q = 0; q < 8; ++q) f[q] -= of_channel<VECG>(mean, q);
        } else {
          forget(rd[i]);
          grad8<T, VECG>(a, rx[i], rd[i], mean, rstd, gamma, beta, f, d);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          f[q] = of_channel<VECG>(rstd, q) * fmaf(d[q], gamma[q], fmaf(f[q], of_channel<VECG>(p1, q), of_channel<VECG>(p0, q)));
        __builtin_amdgcn_sched_barrier(0);
      }
      store8<T>(dx + i * (a.TR * a.ldo), f, 8);
    }
  }
  if (!a.part) return;
  // all lanes of a channel vector: the wavefront's, then the four wavefronts'
  __shared__ float2 red[4][64][9];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    for (int m = a.CV; m < 64; m <<= 1) {
      sb[q] += __shfl_xor(sb[q], m);
      sg[q] += __shfl_xor(sg[q], m);
    }
    if (lane < a.CV) red[wave][lane][q] = make_float2(sb[q], sg[q]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.C; c += kWave) {
    float2 s = red[0][c >> 3][c & 7];
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      s.x += red[k][c >> 3][c & 7].x;
      s.y += red[k][c >> 3][c & 7].y;
    }
    a.part[static_cast<long>(blockIdx.x) * a.C + c] = s;
  }
}

// ---------------------------------------------------------------------------------------
// Streamed form.  The statistics want few chunks (each leaves a row of channel sums to be joined),
// the passes that use them leave nothing behind and want many small pieces, so the two are cut
// differently.
// ---------------------------------------------------------------------------------------
constexpr int kStream = 256;
constexpr int kAhead = 4;  // positions whose loads a thread has in flight

struct StreamPos {
  int b, chunk, cv, tr, TR, s0, s1, n;
  bool on;
};
// The workgroup's chunk of `per` positions, `chunks` of them to a sample.
__device__ inline StreamPos stream_pos(const GnArgs& a, int chunks, int per) {
  StreamPos q;
  long id = blockIdx.x;
  const int cb = static_cast<int>(id % a.colblocks);
  id /= a.colblocks;
  q.chunk = static_cast<int>(id % chunks);
  q.b = static_cast<int>(id / chunks);
  q.TR = kStream / a.TC;
  q.tr = threadIdx.x / a.TC;
  q.cv = cb * a.TC + threadIdx.x - q.tr * a.TC;
  q.on = q.tr < q.TR && q.cv < a.CV;
  q.s0 = q.chunk * per;
  q.s1 = min(a.S, q.s0 + per);
  q.n = min(8, a.C - q.cv * 8);
  return q;
}

// Joins the eight (x, y) pairs of the workgroup's thread rows, n values behind each, into row 0 by
// halving the rows: join(x, y, other pair, n, other's n) for each channel.
template <class F>
__device__ inline void join_rows(const StreamPos& q, int TC, float (&x)[8], float (&y)[8], float n, F&& join) {
  __shared__ float2 red[8][kStream / 2];
  __shared__ float cnt[kStream / 2];
  const int col = q.cv % TC;
  int h = 1;
  while (h * 2 < q.TR) h *= 2;
  for (int width = q.TR; width > 1; width = h, h /= 2) {  // rows 0 .. width-1 are left
    __syncthreads();
    if (q.on && q.tr >= h && q.tr < width) {
      const int at = (q.tr - h) * TC + col;
#pragma unroll
      for (int i = 0; i < 8; ++i) red[i][at] = make_float2(x[i], y[i]);
      cnt[at] = n;
    }
    __syncthreads();
    if (q.on && q.tr + h < width) {
      const int at = q.tr * TC + col;
      const float nb = cnt[at];
#pragma unroll
      for (int i = 0; i < 8; ++i) join(x[i], y[i], red[i][at], n, nb);
      n += nb;
    }
  }
}

// Row 0's threads write their channels' pairs.
__device__ inline void write_part(const GnArgs& a, const StreamPos& q, const float (&x)[8], const float (&y)[8]) {
  if (!q.on || q.tr != 0) return;
  float2* part = a.part + (static_cast<long>(q.b) * a.chunks + q.chunk) * a.C + q.cv * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < q.n) part[i] = make_float2(x[i], y[i]);
}

// mean and rstd of the sample's groups from row 0's channel statistics, where the workgroup has the
// whole sample: up to 64 lanes share a group's channels.
__device__ inline void group_stats(const GnArgs& a, const StreamPos& q, const float (&mean)[8], const float (&m2)[8]) {
  __shared__ float2 chan[kStream * 8];
  if (q.on && q.tr == 0)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < q.n) chan[q.cv * 8 + i] = make_float2(mean[i], m2[i]);
  __syncthreads();
  const int len = sample_len(a, q.b);
  const float inv_n = len > 0 ? 1.f / (static_cast<float>(len) * a.Cg) : 0.f;
  int lanes = 1;
  while (lanes < a.Cg && lanes < 64) lanes *= 2;
  const int lane = threadIdx.x % lanes;
  for (int g = threadIdx.x / lanes; g < a.G; g += kStream / lanes) {
    const float2* ch = chan + g * a.Cg;
    float s = 0.f, v = 0.f;
    for (int c = lane; c < a.Cg; c += lanes) s += ch[c].x;
    for (int m = lanes / 2; m > 0; m /= 2) s += __shfl_xor(s, m);
    s /= static_cast<float>(a.Cg);
    for (int c = lane; c < a.Cg; c += lanes) v += ch[c].y + static_cast<float>(len) * (ch[c].x - s) * (ch[c].x - s);
    for (int m = lanes / 2; m > 0; m /= 2) v += __shfl_xor(v, m);
    if (lane == 0) {
      a.mean[static_cast<long>(q.b) * a.G + g] = s;
      a.rstd[static_cast<long>(q.b) * a.G + g] = 1.f / sqrtf(v * inv_n + a.eps);
    }
  }
}

// part[b][chunk][c] = (mean, sum of squares about it) of channel c over the chunk's valid
// positions.  A thread sums differences from its mean so far, which is brought up to date each time
// the positions have doubled (differences from its first value all along lose the others behind a
// large one: 4000 positions, the first 1000 standard deviations away, left the mean off by 5e-4 of
// them and rstd by 1 %); threads are joined by the pairwise update of Chan, Golub and LeVeque
// (1979).  WHOLE: the workgroup has the whole sample and writes the groups' mean and rstd instead.
template <class T, bool WHOLE>
__global__ __launch_bounds__(kStream) void k_gn_stats(GnArgs a) {
  using St = typename T::S;
  const StreamPos q = stream_pos(a, a.chunks, a.per_chunk);
  const int end = min(q.s1, sample_len(a, q.b));
  float mean[8] = {}, m2[8] = {}, cnt = 0.f;
  if (q.on) {
    const St* x = static_cast<const St*>(a.x) + static_cast<long>(q.b) * a.S * a.ldx + q.cv * 8;
    float s1[8] = {}, s2[8] = {}, fresh = 0.f;  // of the positions since the last fold
    const auto fold = [&] {
      cnt += fresh;
      const float inv = 1.f / cnt;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = s1[i] * inv;
        mean[i] += d;
        m2[i] += s2[i] - s1[i] * d;
        s1[i] = s2[i] = 0.f;
      }
      fresh = 0.f;
    };
    for (int s = q.s0 + q.tr; s < end; s += kAhead * q.TR) {
      Raw8<T> r[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (s + u * q.TR < end) r[u] = load8_raw<T>(x + (s + u * q.TR) * a.ldx, q.n);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (s + u * q.TR >= end) break;
        float f[8];
        to_floats<T>(r[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (cnt + fresh == 0.f) mean[i] = f[i];
          const float d = f[i] - mean[i];
          s1[i] += d;
          s2[i] = fmaf(d, d, s2[i]);
        }
        fresh += 1.f;
      }
      if (fresh >= cnt) fold();
    }
    if (fresh > 0.f) fold();
#pragma unroll
    for (int i = 0; i < 8; ++i) m2[i] = fmaxf(m2[i], 0.f);
  }
  join_rows(q, a.TC, mean, m2, cnt, [](float& m, float& s, const float2& o, float na, float nb) {
    if (nb > 0.f) {
      const float w = nb / (na + nb), d = o.x - m;
      m += d * w;
      s += o.y + d * d * (na * w);
    }
  });
  if constexpr (WHOLE) group_stats(a, q, mean, m2);
  else write_part(a, q, mean, m2);
}

// Sum of v over the workgroup's threads, in a fixed order, for every thread.
__device__ inline float sum_all(float v) {
  __shared__ float red[16];
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
  for (unsigned w = 1; w < blockDim.x / 64; ++w) s += red[w];
  return s;
}

// Walks the group's chunks * Cg channel entries, thread t from entry t in steps of the workgroup:
// f(chunk, channel in the group).
template <class F>
__device__ inline void each_entry(const GnArgs& a, F&& f) {
  const int nt = blockDim.x, rows = nt / a.Cg, cols = nt % a.Cg;
  int ch = threadIdx.x / a.Cg, c = threadIdx.x % a.Cg;
#pragma unroll 4
  for (int j = threadIdx.x; j < a.chunks * a.Cg; j += nt) {
    f(ch, c);
    ch += rows;
    c += cols;
    if (c >= a.Cg) c -= a.Cg, ++ch;
  }
}

// One workgroup per (sample, group): mean and rstd from the chunks' channel statistics.
__global__ __launch_bounds__(1024) void k_gn_join(GnArgs a) {
  const int b = blockIdx.x / a.G, g = blockIdx.x - b * a.G;
  const int len = sample_len(a, b);
  const float inv_n = len > 0 ? 1.f / (static_cast<float>(len) * a.Cg) : 0.f;
  const float2* part = a.part + static_cast<long>(b) * a.chunks * a.C + g * a.Cg;
  const auto count = [&](int ch) { return static_cast<float>(min(max(len - ch * a.per_chunk, 0), a.per_chunk)); };
  float s = 0.f;
  each_entry(a, [&](int ch, int c) { s += count(ch) * inv_n * part[static_cast<long>(ch) * a.C + c].x; });
  const float mean = sum_all(s);
  float v = 0.f;
  each_entry(a, [&](int ch, int c) {
    const float2 q = part[static_cast<long>(ch) * a.C + c];
    v += q.y + count(ch) * (q.x - mean) * (q.x - mean);
  });
  v = sum_all(v);
  if (threadIdx.x == 0) {
    a.mean[blockIdx.x] = mean;
    a.rstd[blockIdx.x] = 1.f / sqrtf(v * inv_n + a.eps);
  }
}

// (mean, rstd) of the thread's channels.
__device__ inline void load_stats(const GnArgs& a, const StreamPos& q, float (&mean)[8], float (&rstd)[8]) {
  load_groups(a, a.rstd + static_cast<long>(q.b) * a.G, q.cv, rstd);
  load_groups(a, a.mean + static_cast<long>(q.b) * a.G, q.cv, mean);
}

template <class T>
__global__ __launch_bounds__(kStream) void k_gn_apply(GnArgs a) {
  using St = typename T::S;
  const StreamPos q = stream_pos(a, a.pieces, a.per_piece);
  if (!q.on) return;
  const int len = sample_len(a, q.b);
  const St* x = static_cast<const St*>(a.x) + static_cast<long>(q.b) * a.S * a.ldx + q.cv * 8;
  St* y = static_cast<St*>(a.out) + static_cast<long>(q.b) * a.S * a.ldo + q.cv * 8;
  float gamma[8], beta[8], mean[8], rstd[8];
  load_params(a, q.cv, gamma, beta);
  load_stats(a, q, mean, rstd);
  for (int s0 = q.s0 + q.tr; s0 < q.s1; s0 += kAhead * q.TR) {
    Raw8<T> r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (s0 + u * q.TR < min(len, q.s1)) r[u] = load8_raw<T>(x + (s0 + u * q.TR) * a.ldx, q.n);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = s0 + u * q.TR;
      if (s >= q.s1) break;
      float f[8] = {};
      if (s < len) {
        to_floats<T>(r[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (f[i] - mean[i]) * rstd[i] * gamma[i] + beta[i];
        act8(a.act, f);
      }
      store8<T>(y + s * a.ldo, f, q.n);
    }
  }
}

// part[b][chunk][c] = (sum du, sum du xh) of channel c over the chunk's valid positions.
template <class T>
__global__ __launch_bounds__(kStream) void k_gn_bwd_stats(GnArgs a) {
  using St = typename T::S;
  const StreamPos q = stream_pos(a, a.chunks, a.per_chunk);
  const int end = min(q.s1, sample_len(a, q.b));
  float s1[8] = {}, s2[8] = {};
  if (q.on) {
    const St* x = static_cast<const St*>(a.x) + static_cast<long>(q.b) * a.S * a.ldx + q.cv * 8;
    const St* dy = static_cast<const St*>(a.dy) + static_cast<long>(q.b) * a.S * a.lddy + q.cv * 8;
    float gamma[8], beta[8], mean[8], rstd[8];
    load_params(a, q.cv, gamma, beta);
    load_stats(a, q, mean, rstd);
    for (int s = q.s0 + q.tr; s < end; s += kAhead * q.TR) {
      Raw8<T> rx[kAhead], rd[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (s + u * q.TR < end) {
          rx[u] = load8_raw<T>(x + (s + u * q.TR) * a.ldx, q.n);
          rd[u] = load8_raw<T>(dy + (s + u * q.TR) * a.lddy, q.n);
        }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (s + u * q.TR >= end) break;
        float f[8], d[8];
        grad8<T, false>(a, rx[u], rd[u], mean, rstd, gamma, beta, f, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s1[i] += d[i];
          s2[i] += d[i] * f[i];
        }
      }
    }
  }
  join_rows(q, a.TC, s1, s2, 0.f, [](float& x, float& y, const float2& o, float, float) {
    x += o.x;
    y += o.y;
  });
  write_part(a, q, s1, s2);
}

// dbeta[c], dgamma[c] = the sums over `rows` of part[row][c]: 4 channels per workgroup, the rest
// of its threads (T = blockDim.x / 4 per channel, thread t: rows t, t + T, ...) share out the rows,
// and their sums are joined in a fixed tree.
__device__ inline void sum_params(const GnArgs& a, long rows, int block) {
  __shared__ float2 red[256][4];
  const int q = threadIdx.x & 3, c = block * 4 + q, t = threadIdx.x >> 2, C = a.C, T = blockDim.x >> 2;
  float2 s = make_float2(0.f, 0.f);
  if (c < C)
#pragma unroll 4
    for (long r = t; r < rows; r += T) {
      const float2 v = a.part[r * C + c];
      s.x += v.x;
      s.y += v.y;
    }
  red[t][q] = s;
  for (int h = T / 2; h > 0; h >>= 1) {
    __syncthreads();
    if (t < h) {
      s.x += red[t + h][q].x;
      s.y += red[t + h][q].y;
      red[t][q] = s;
    }
  }
  if (t == 0 && c < C) {
    if (a.dbeta) a.dbeta[c] = s.x;
    if (a.dgamma) a.dgamma[c] = s.y;
  }
}

__global__ __launch_bounds__(1024) void k_gn_params(GnArgs a, long rows) { sum_params(a, rows, blockIdx.x); }

// One workgroup per (sample, group): (avg dh, avg dh xh) from the chunks' channel sums.  The
// workgroups past those sum the parameters' gradients, where the launch has them.
__global__ __launch_bounds__(1024) void k_gn_bwd_join(GnArgs a) {
  const int block = blockIdx.x, groups = a.B * a.G;
  if (block >= groups) {
    sum_params(a, static_cast<long>(a.B) * a.chunks, block - groups);
    return;
  }
  const int b = blockIdx.x / a.G, g = blockIdx.x - b * a.G;
  const int len = sample_len(a, b);
  const float2* part = a.part + static_cast<long>(b) * a.chunks * a.C + g * a.Cg;
  float s1 = 0.f, s2 = 0.f;
  each_entry(a, [&](int ch, int c) {
    const float2 v = part[static_cast<long>(ch) * a.C + c];
    const float gm = a.gamma ? a.gamma[g * a.Cg + c] : 1.f;
    s1 += gm * v.x;
    s2 += gm * v.y;
  });
  s1 = sum_all(s1);
  s2 = sum_all(s2);
  const float inv_n = len > 0 ? 1.f / (static_cast<float>(len) * a.Cg) : 0.f;
  if (threadIdx.x == 0) {
    a.gsum[blockIdx.x] = s1 * inv_n;
    a.gsum[static_cast<long>(a.B) * a.G + blockIdx.x] = s2 * inv_n;
  }
}

template <class T>
__global__ __launch_bounds__(kStream) void k_gn_bwd_apply(GnArgs a) {
  using St = typename T::S;
  const StreamPos q = stream_pos(a, a.pieces, a.per_piece);
  if (!q.on) return;
  const int len = sample_len(a, q.b);
  const St* x = static_cast<const St*>(a.x) + static_cast<long>(q.b) * a.S * a.ldx + q.cv * 8;
  const St* dy = static_cast<const St*>(a.dy) + static_cast<long>(q.b) * a.S * a.lddy + q.cv * 8;
  St* dx = static_cast<St*>(a.out) + static_cast<long>(q.b) * a.S * a.ldo + q.cv * 8;
  float gamma[8], beta[8], mean[8], rstd[8], m1[8], m2[8];
  load_params(a, q.cv, gamma, beta);
  load_stats(a, q, mean, rstd);
  load_groups(a, a.gsum + static_cast<long>(q.b) * a.G, q.cv, m1);
  load_groups(a, a.gsum + (static_cast<long>(a.B) + q.b) * a.G, q.cv, m2);
  for (int s0 = q.s0 + q.tr; s0 < q.s1; s0 += kAhead * q.TR) {
    Raw8<T> rx[kAhead], rd[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (s0 + u * q.TR < min(len, q.s1)) {
        rx[u] = load8_raw<T>(x + (s0 + u * q.TR) * a.ldx, q.n);
        rd[u] = load8_raw<T>(dy + (s0 + u * q.TR) * a.lddy, q.n);
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = s0 + u * q.TR;
      if (s >= q.s1) break;
      float f[8] = {};
      if (s < len) {
        float d[8];
        grad8<T, false>(a, rx[u], rd[u], mean, rstd, gamma, beta, f, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = rstd[i] * (d[i] * gamma[i] - m1[i] - f[i] * m2[i]);
      }
      store8<T>(dx + s * a.ldo, f, q.n);
    }
  }
}

// ---------------------------------------------------------------------------------------
// Plans and launches.
// ---------------------------------------------------------------------------------------
enum Form { WAVE, RESIDENT, STREAMED };

struct GnPlan {
  Form form = STREAMED;
  int NV = 1, TR = 0, team = 0, spw = 1, threads = 0, blocks_fwd = 0, blocks_bwd = 0;
  int chunks = 1, per_chunk = 1, pieces = 1, per_piece = 1, colblocks = 1, TC = 1;
  bool whole = false;                // streamed: one workgroup has a sample's statistics
  size_t fwd_bytes = 0, bwd_bytes = 0;
  size_t part_bytes = 0;             // streamed backward: the channel sums, before gsum
};

// LDS of group_sums for nval values: entries, their first sums, the groups' sums.
size_t resident_lds(long Cg, long G, long tr, long spw, long threads, int nval) {
  const long per = Cg % 8 == 0 ? 1 : 8, entries = tr * (Cg % 8 == 0 ? Cg / 8 : Cg);
  return sizeof(float) * nval * (threads * per + spw * G * ((entries + 15) / 16 + 1));
}

GnPlan plan_gn(int B, int S, int C, int G) {
  GnPlan p;
  const long CV = (C + 7l) / 8;
  const auto round256 = [](size_t n) { return (n + 255) / 256 * 256; };
  // wavefront: powers of two all the way, at most eight vectors per lane
  const long Cg = C / G;
  const auto pow2 = [](long n) { return (n & (n - 1)) == 0; };
  if (C % 8 == 0 && CV <= 64 && pow2(CV) && pow2(Cg) && S <= 8 * (64 / CV)) {
    p.form = WAVE;
    p.TR = static_cast<int>(64 / CV);
    while (p.TR > 1 && p.TR / 2 >= S) p.TR /= 2;
    p.team = static_cast<int>(p.TR * CV);
    p.NV = 1;
    while (p.NV * p.TR < S) p.NV *= 2;
    p.threads = kWave;
    p.spw = kWave / p.team;
  }
  // resident: the smallest number of vectors per thread (1, 2, 4) that leaves a sample to one
  // wavefront (no other one to wait for), to 256 threads, or to kResident
  for (int limit : {64, 256, kResident}) {
    for (int nv = 1; nv <= 4 && p.form == STREAMED; nv *= 2) {
      const long tr = (S + (nv - 1l)) / nv;
      const long spw = tr * CV <= limit && limit < kResident ? limit / (tr * CV) : 1;
      if (tr * CV <= limit && resident_lds(Cg, G, tr, spw, limit, 2) <= 65536) {
        p.form = RESIDENT;
        p.NV = nv;
        p.TR = static_cast<int>(tr);
        p.team = static_cast<int>(tr * CV);
        p.spw = static_cast<int>(spw);
        p.threads = limit < kResident ? limit : (p.team + 63) / 64 * 64;
      }
    }
  }
  if (p.form != STREAMED) {
    const long wgs = (B + p.spw - 1l) / p.spw;
    p.blocks_fwd = static_cast<int>(wgs);
    // the backward's workgroups walk samples and leave one row of channel sums each: as many as
    // are resident at once (two to a CU where a thread holds eight vectors in 256 registers, 16
    // of one wavefront, about four otherwise), fewer, down to one, where their rows take over 8 MB
    const long most = p.threads == 64 ? 4096 : p.NV == 8 ? 512 : 1024;
    const long few = std::max<long>(256, std::min<long>(most, (1l << 20) / C));
    p.blocks_bwd = static_cast<int>(std::min(wgs, few));
    p.bwd_bytes = round256(static_cast<size_t>(p.blocks_bwd) * C * sizeof(float2));
    return p;
  }
  p.TC = static_cast<int>(std::min<long>(CV, kStream));
  p.colblocks = static_cast<int>((CV + p.TC - 1) / p.TC);
  const long rows = kStream / p.TC;
  const long want = std::max<long>(1, 512 / (static_cast<long>(B) * p.colblocks));
  const long most = std::max<long>(1, S / (rows * kAhead));  // at least one batch of loads per thread
  // and channel statistics of at most 8 MB where the samples alone do not take more
  const long cap = std::max<long>(1, (1l << 20) / (static_cast<long>(B) * C));
  p.chunks = static_cast<int>(std::min({want, most, cap}));
  p.per_chunk = static_cast<int>((S + static_cast<long>(p.chunks) - 1) / p.chunks);
  p.chunks = static_cast<int>((S + static_cast<long>(p.per_chunk) - 1) / p.per_chunk);
  // the passes that use the statistics leave nothing behind, so their pieces are smaller: one
  // batch of loads per thread, more where the launch would have over 2^22 workgroups
  p.per_piece = static_cast<int>(std::min<long>(S, rows * kAhead));
  while (static_cast<long>(B) * p.colblocks * ((S + static_cast<long>(p.per_piece) - 1) / p.per_piece) > (1l << 22) && p.per_piece < S)
    p.per_piece = static_cast<int>(std::min<long>(S, 2l * p.per_piece));
  p.pieces = static_cast<int>((S + static_cast<long>(p.per_piece) - 1) / p.per_piece);
  // The forward leaves channel statistics only where they have to be joined across workgroups, so
  // the 8 MB above hold for every batch of up to 8 kStream channels (1492 samples of 9 x 1888 bf16:
  // 45.1 us, with channel statistics of 22 MB and a join 65.9; 600 of 200 x 128: 26.2, 30.0).
  p.whole = p.chunks == 1 && p.colblocks == 1;
  p.part_bytes = round256(static_cast<size_t>(B) * p.chunks * C * sizeof(float2));
  p.fwd_bytes = p.whole ? 0 : p.part_bytes;
  p.bwd_bytes = p.part_bytes + round256(static_cast<size_t>(B) * G * 2 * sizeof(float));
  return p;
}

void fill(GnArgs& a, const GnPlan& p) {
  a.CV = (a.C + 7) / 8;
  a.Cg = a.C / a.G;
  a.TR = p.TR, a.team = p.team, a.spw = p.spw;
  a.chunks = p.chunks, a.per_chunk = p.per_chunk, a.pieces = p.pieces, a.per_piece = p.per_piece, a.colblocks = p.colblocks, a.TC = p.TC;
  if (p.form == RESIDENT) {
    a.E = p.TR * (a.Cg % 8 == 0 ? a.Cg / 8 : a.Cg);
    a.E1 = (a.E + 15) / 16;
    const int gc = a.Cg % 8 == 0 ? a.Cg / 8 : a.Cg;
    a.E1_rows = a.E1 / gc;
    a.E1_cols = a.E1 % gc;
  }
}

template <class T, bool BWD, bool VECG>
void launch_resident(const GnArgs& a, const GnPlan& p, hipStream_t st) {
  const size_t lds = std::max(resident_lds(a.Cg, a.G, p.TR, p.spw, p.threads, BWD ? 2 : 1), BWD ? 8 * p.threads * sizeof(float2) : 0);
  const dim3 grid(BWD ? p.blocks_bwd : p.blocks_fwd), block(p.threads);
#define GN_CASE(NV)                                                                                        \
  case NV:                                                                                                 \
    if constexpr (BWD) hipLaunchKernelGGL((k_gn_bwd_resident<T, NV, VECG>), grid, block, lds, st, a); \
    else hipLaunchKernelGGL((k_gn_fwd_resident<T, NV, VECG>), grid, block, lds, st, a);               \
    break;
  switch (p.NV) { GN_CASE(1) GN_CASE(2) GN_CASE(4) }
#undef GN_CASE
}

template <class T, bool BWD, bool VECG>
void launch_wave(const GnArgs& a, const GnPlan& p, hipStream_t st) {
  const dim3 grid(BWD ? p.blocks_bwd : p.blocks_fwd), block(kWave);
#define GN_CASE(NV)                                                                                  \
  case NV:                                                                                           \
    if constexpr (BWD) hipLaunchKernelGGL((k_gn_bwd_wave<T, NV, VECG>), grid, block, 0, st, a);      \
    else hipLaunchKernelGGL((k_gn_fwd_wave<T, NV, VECG>), grid, block, 0, st, a);                    \
    break;
  switch (p.NV) { GN_CASE(1) GN_CASE(2) GN_CASE(4) GN_CASE(8) }
#undef GN_CASE
}

template <class T, bool BWD>
void launch_gn(const GnArgs& a, const GnPlan& p, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(static_cast<long>(a.B) * p.chunks * p.colblocks)), block(kStream);
  const dim3 pieces(static_cast<unsigned>(static_cast<long>(a.B) * p.pieces * p.colblocks));
  // enough threads for a few entries each
  const long entries = static_cast<long>(p.chunks) * a.Cg;
  const int threads = entries <= 256 ? 64 : entries <= 2048 ? 256 : 1024;
  const dim3 join(threads);
  const dim3 groups(static_cast<unsigned>(static_cast<long>(a.B) * a.G));
  const unsigned quads = static_cast<unsigned>((a.C + 3) / 4);
  const long rows = p.form != STREAMED ? p.blocks_bwd : static_cast<long>(a.B) * p.chunks;
  bool params = BWD && (a.dgamma || a.dbeta);
  if (p.form == WAVE) {
    a.Cg % 8 == 0 ? launch_wave<T, BWD, true>(a, p, st) : launch_wave<T, BWD, false>(a, p, st);
  } else if (p.form == RESIDENT) {
    a.Cg % 8 == 0 ? launch_resident<T, BWD, true>(a, p, st) : launch_resident<T, BWD, false>(a, p, st);
  } else if constexpr (BWD) {
    hipLaunchKernelGGL((k_gn_bwd_stats<T>), grid, block, 0, st, a);
    // a parameter's sums beside the groups' where they take at most 16 rows a thread (six samples
    // of 5001 x 256, forward and backward: 45.4 us, in a launch of their own 47.3)
    const bool beside = params && rows <= 4 * threads;
    hipLaunchKernelGGL(k_gn_bwd_join, dim3(groups.x + (beside ? quads : 0)), join, 0, st, a);
    params = params && !beside;
    hipLaunchKernelGGL((k_gn_bwd_apply<T>), pieces, block, 0, st, a);
  } else {
    if (p.whole) {
      hipLaunchKernelGGL((k_gn_stats<T, true>), grid, block, 0, st, a);
    } else {
      hipLaunchKernelGGL((k_gn_stats<T, false>), grid, block, 0, st, a);
      hipLaunchKernelGGL(k_gn_join, groups, join, 0, st, a);
    }
    hipLaunchKernelGGL((k_gn_apply<T>), pieces, block, 0, st, a);
  }
  if (params) hipLaunchKernelGGL(k_gn_params, dim3(quads), dim3(1024), 0, st, a, rows);
}

template <bool BWD>
el_status run_gn(const char* fn, const GnArgs& a, const GnPlan& p, el_dtype dtype, hipStream_t st) {
  if (dtype == EL_F32) launch_gn<F32T, BWD>(a, p, st);
  else if (dtype == EL_F16) launch_gn<F16T, BWD>(a, p, st);
  else launch_gn<BF16T, BWD>(a, p, st);
  return check_launch(fn);
}

// What one launch's grid can hold (2^32 threads): samples that fit a workgroup take up to one
// workgroup each, streamed ones a workgroup per group and per block of columns.
bool gn_sizes_ok(int32_t B, int32_t S, int32_t C, int32_t G) {
  if (B < 1 || S < 1 || C < 1 || G < 1 || C % G != 0 || C > (1 << 20) || S > (1 << 30)) return false;
  if (static_cast<int64_t>(B) * G >= (int64_t{1} << 25)) return false;
  const GnPlan p = plan_gn(B, S, C, G);
  if (p.form != STREAMED) return static_cast<int64_t>(p.blocks_fwd) * p.threads < (int64_t{1} << 32);
  return static_cast<int64_t>(B) * G < (int64_t{1} << 22) && static_cast<int64_t>(B) * p.colblocks <= (int64_t{1} << 22);
}

el_status check_gn(const char* fn, const void* x, int64_t ldx, int32_t B, int32_t S, int32_t C, int32_t G,
                   const int32_t* lengths, const float* gamma, const float* beta, const float* mean, const float* rstd,
                   uint32_t act, el_dtype dtype) {
  if (B < 0) return tower::bad(fn, "B must be >= 0");
  if (S < 0) return tower::bad(fn, "S must be >= 0");
  if (C < 1) return tower::bad(fn, "C must be >= 1");
  if (G < 1 || C % G != 0) return tower::bad(fn, "G must be >= 1 and divide C");
  if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
  if (B > 0 && S > 0 && !gn_sizes_ok(B, S, C, G))
    return tower::unsupported(fn, "more channels (2^20), positions (2^30), groups in all (2^25) or samples than one launch takes");
  const el_status s = tower::check_act(fn, act);
  if (s != EL_OK) return s;
  if (!tower::al(lengths, 4) || !tower::al(gamma, 4) || !tower::al(beta, 4))
    return tower::bad(fn, "lengths, gamma and beta must be aligned to their elements");
  if (B > 0 && (!mean || !rstd)) return tower::bad(fn, "mean or rstd is null");
  if (!tower::al(mean, 4) || !tower::al(rstd, 4)) return tower::bad(fn, "mean and rstd must be aligned to their elements");
  return tower::check_rows(fn, "x", x, ldx, C, B > 0 && S > 0, dtype_size(dtype));
}

// No positions at all: mean 0, rstd 1 / sqrt(eps); zero parameter gradients.
__global__ __launch_bounds__(256) void k_gn_empty(float* mean, float* rstd, long n, float r, float* a, float* b, long c) {
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) mean[i] = 0.f, rstd[i] = r;
  if (i < c) {
    if (a) a[i] = 0.f;
    if (b) b[i] = 0.f;
  }
}

}  // namespace
}  // namespace el

using namespace el;

extern "C" {

size_t el_group_norm_fwd_workspace_bytes(int32_t B, int32_t S, int32_t C, int32_t G) {
  return gn_sizes_ok(B, S, C, G) ? plan_gn(B, S, C, G).fwd_bytes : 0;
}

size_t el_group_norm_bwd_workspace_bytes(int32_t B, int32_t S, int32_t C, int32_t G) {
  return gn_sizes_ok(B, S, C, G) ? plan_gn(B, S, C, G).bwd_bytes : 0;
}

el_status el_group_norm_fwd(const void* x, int64_t ldx, int32_t B, int32_t S, int32_t C, int32_t G,
                            const int32_t* lengths, const float* gamma, const float* beta, float eps, uint32_t act,
                            void* y, int64_t ldy, float* mean, float* rstd, el_dtype dtype, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "el_group_norm_fwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_gn(fn, x, ldx, B, S, C, G, lengths, gamma, beta, mean, rstd, act, dtype));
    if (!(eps >= 0.f) || std::isinf(eps)) return tower::bad(fn, "eps must be >= 0 and finite");
    EL_TRY(tower::check_rows(fn, "y", y, ldy, C, B > 0 && S > 0, dtype_size(dtype)));
    if (B == 0) return EL_OK;
    if (S == 0) {
      const long n = static_cast<long>(B) * G;
      hipLaunchKernelGGL(k_gn_empty, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream, mean, rstd, n,
                         1.f / std::sqrt(eps), nullptr, nullptr, 0l);
      return check_launch(fn);
    }
    const GnPlan p = plan_gn(B, S, C, G);
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, p.fwd_bytes));
    GnArgs a{};
    a.x = x, a.ldx = ldx, a.out = y, a.ldo = ldy, a.B = B, a.S = S, a.C = C, a.G = G;
    a.lengths = lengths, a.gamma = gamma, a.beta = beta, a.eps = eps, a.act = act, a.mean = mean, a.rstd = rstd;
    a.part = static_cast<float2*>(workspace);
    fill(a, p);
    return run_gn<false>(fn, a, p, dtype, stream);
  });
}

el_status el_group_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, int32_t B, int32_t S, int32_t C,
                            int32_t G, const int32_t* lengths, const float* gamma, const float* beta,
                            const float* mean, const float* rstd, uint32_t act, void* dx, int64_t lddx, float* dgamma,
                            float* dbeta, el_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "el_group_norm_bwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_gn(fn, x, ldx, B, S, C, G, lengths, gamma, beta, mean, rstd, act, dtype));
    EL_TRY(tower::check_rows(fn, "dy", dy, lddy, C, B > 0 && S > 0, dtype_size(dtype)));
    EL_TRY(tower::check_rows(fn, "dx", dx, lddx, C, B > 0 && S > 0, dtype_size(dtype)));
    if (!tower::al(dgamma, 4) || !tower::al(dbeta, 4)) return tower::bad(fn, "dgamma and dbeta must be aligned to their elements");
    if (B == 0 || S == 0) {
      hipLaunchKernelGGL(k_gn_empty, dim3(static_cast<unsigned>((C + 255) / 256)), dim3(256), 0, stream, nullptr, nullptr,
                         0l, 0.f, dgamma, dbeta, static_cast<long>(C));
      return check_launch(fn);
    }
    const GnPlan p = plan_gn(B, S, C, G);
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, p.bwd_bytes));
    GnArgs a{};
    a.x = x, a.ldx = ldx, a.dy = dy, a.lddy = lddy, a.out = dx, a.ldo = lddx, a.B = B, a.S = S, a.C = C, a.G = G;
    a.lengths = lengths, a.gamma = gamma, a.beta = beta, a.act = act, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
    a.dgamma = dgamma, a.dbeta = dbeta;
    fill(a, p);
    if (p.form != STREAMED) {
      a.part = dgamma || dbeta ? static_cast<float2*>(workspace) : nullptr;
    } else {
      a.part = static_cast<float2*>(workspace);
      a.gsum = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_bytes);
    }
    return run_gn<true>(fn, a, p, dtype, stream);
  });
}

}  // extern "C"
