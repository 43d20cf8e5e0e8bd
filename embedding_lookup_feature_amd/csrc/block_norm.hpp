// block_norm.hpp -- what the block norm's forward and backward share: arguments, the slots that
// own a row, sums over a slot, the checks of the parameters.
//
// Rows are independent but for the sums of the parameters' and the shared gates' gradients.  A slot
// (L lanes of a wavefront, or W whole wavefronts) owns a row: its columns stay in registers, eight
// to a vector, NV vectors a lane, between the one read of the row and the one write.
//
// The kernels see their operands through views, of two kinds.  The aligned view (rows of whole,
// 16-byte aligned vectors, C <= 8192) is a buffer descriptor of the rows at hand: an operand that is
// left out, a row behind the last and a lane behind the last column all read zeros and write
// nothing, without a branch, so the number of loads and stores in flight is known at every wait (they
// share one in-order counter) and the next rows' loads stay in flight behind this row's arithmetic
// and stores.  The loose view takes any alignment, width and stride with a branch around each access.
// 65536 x 1024 in bf16, forward and backward: 120 and 201 us through aligned views, 143 and 237 at odd
// addresses; 426062 x 128: 101 and 165, 149 and 235.
#pragma once

#include <algorithm>

#include "micro.hpp"

namespace el {

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
  float* gate_part;  // [slots][2][C]: sums of the gate rows that a slot's rows begin and end in
  float* part;       // [grid][4][C]: the parameters' partial sums
  uint32_t want;     // bit k: parameter sum k is asked for
};

// out[k][c] = sum over p < parts of part[(p * 4 + k) * C + c], for the k that are asked for.
struct JoinArgs {
  const float* part;
  float* out[4];
  int parts, C;
};

namespace {

constexpr int kMaxCols = 32768;
constexpr int kMaxAlignedCols = 8192;  // wider rows do not fit the registers of the aligned form (one vector a lane)

// A slot: L lanes of one wavefront (W = 1), or W whole wavefronts (L = 64), NV vectors a lane.  A
// workgroup holds PER_WG of them, which go through the same number of rows.
template <int L_, int W_, int NV_>
struct Slot {
  static constexpr int L = L_, W = W_, NV = NV_;
  static constexpr int COLS = L * W * NV * 8;
  static constexpr int THREADS = W > 4 ? W * 64 : 256;
  static constexpr int PER_WG = THREADS / (L * W);
  static constexpr int WAVES = THREADS / 64;
};

// Adds the value of another lane: within 16 lanes by data-parallel-primitive moves (pairs, pairs of
// pairs, mirrored halves of 8 and 16: the lanes of a half hold equal sums by then), beyond by the
// swaps of rows of 16 and of 32 lanes.  No LDS latency, and the same bits in every lane.
template <int CTRL>
__device__ inline float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ inline float lane_sum(float v) {
  if constexpr (L >= 2) v = dpp_add<0xB1>(v);   // lane ^ 1
  if constexpr (L >= 4) v = dpp_add<0x4E>(v);   // lane ^ 2
  if constexpr (L >= 8) v = dpp_add<0x141>(v);  // 7 - lane of eight
  if constexpr (L >= 16) v = dpp_add<0x140>(v); // 15 - lane of sixteen
  if constexpr (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// Sums of N values over a slot; the same in all its lanes.
template <class SL, int N>
__device__ inline void slot_sums(float (&v)[N], float (*lds)[SL::WAVES][2], int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lane_sum<SL::L>(v[k]);
  if constexpr (SL::W > 1) {
    // two buffers in turn: a wavefront that writes one has passed the barrier behind which nobody
    // reads it any more
    float(*b)[2] = lds[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) b[threadIdx.x >> 6][k] = v[k];
    __syncthreads();
    if constexpr (SL::PER_WG > 1) b += threadIdx.x / (64 * SL::W) * SL::W;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = b[0][k];
#pragma unroll
      for (int w = 1; w < SL::W; ++w) s += b[w][k];
      v[k] = s;
    }
  }
}

// Row statistics are two fp32 numbers a row; absent ones read (0, 0) and are not written.
__device__ inline __amdgpu_buffer_rsrc_t stats_span(const float* p, long first, int rows) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p) + first * 2, 0, p && rows > 0 ? rows * 8 : 0, 0x00027000);
}

// Mean and rstd of a slot's row (values past its end are zero).
template <class SL>
__device__ inline void row_stats(const float (&v)[SL::NV][8], uint32_t kind, const NormArgs& a, int c0,
                                 float (*lds)[SL::WAVES][2], int& turn, float& mean, float& rstd) {
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

// ---------------------------------------------------------------------------------------
// Views of one operand's rows: init() and at() fix this lane's slot's row of the view and its
// columns, span() the rows that the view covers, load() and store() row `t` behind the slot's row;
// settle() comes between load() and the use of what it loaded.
// ---------------------------------------------------------------------------------------
constexpr uint32_t kNowhere = 0x80000000u;  // behind the end of every view (they are shorter than 2^31)
constexpr int kStream = 2;                  // non-temporal: rows are read and written once

template <class T, class SL>
struct Aligned {
  static constexpr int ES = sizeof(typename T::S), STEP = SL::L * SL::W * 8 * ES;
  typedef __amdgpu_buffer_rsrc_t Span;
  const char* base;
  int row_bytes;
  uint32_t voff[SL::NV];
  __device__ inline void init(const void* p, long ld, long slot_row, int c0, int C) {
    base = static_cast<const char*>(p);
    row_bytes = static_cast<int>(ld * ES);
    at(slot_row, c0, C);
  }
  __device__ inline void at(long slot_row, int c0, int C) {
#pragma unroll
    for (int j = 0; j < SL::NV; ++j)
      voff[j] = c0 + j * SL::L * SL::W * 8 < C ? static_cast<uint32_t>(slot_row) * row_bytes + c0 * ES + j * STEP : kNowhere;
  }
  // `rows` rows from row `first` on (0: nothing there), C columns of the last.
  __device__ inline Span span(long first, int rows, int C) const {
    const int bytes = base && rows > 0 ? (rows - 1) * row_bytes + C * ES : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base) + first * row_bytes, 0, bytes, 0x00027000);
  }
  __device__ inline uint32_t place(int j, int t, bool valid) const { return valid ? voff[j] + static_cast<uint32_t>(t) * row_bytes : kNowhere; }
  __device__ inline void load(Span rs, Raw8<T> (&raw)[SL::NV], int t = 0, bool valid = true) const {
#pragma unroll
    for (int j = 0; j < SL::NV; ++j)
#pragma unroll
      for (int w = 0; w < Raw8<T>::W; ++w)
        raw[j].v[w] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, place(j, t, valid) + 16 * w, 0, kStream));
  }
  __device__ inline void settle(Raw8<T> (&)[SL::NV]) const {}
  __device__ inline void store(Span rs, const float (&v)[SL::NV][8], int t = 0, bool valid = true) const {
#pragma unroll
    for (int j = 0; j < SL::NV; ++j) {
      u32x4 q[Raw8<T>::W];
      if constexpr (Raw8<T>::W == 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) q[0][e] = __float_as_uint(v[j][e]), q[1][e] = __float_as_uint(v[j][4 + e]);
      } else {
        q[0] = to_16bit<T>(v[j]);
      }
#pragma unroll
      for (int w = 0; w < Raw8<T>::W; ++w) __builtin_amdgcn_raw_buffer_store_b128(q[w], rs, place(j, t, valid) + 16 * w, 0, kStream);
    }
  }
};

template <class T, class SL>
struct Loose {
  typedef typename T::S S;
  struct Span {
    S* p;
    int rows;
  };
  S* base;
  long ld;
  long row;
  int c, cols;
  __device__ inline void init(const void* p, long ld_, long slot_row, int c0, int C) {
    base = static_cast<S*>(const_cast<void*>(p));
    ld = ld_, row = slot_row, c = c0, cols = C;
  }
  __device__ inline void at(long slot_row, int, int) { row = slot_row; }
  __device__ inline Span span(long first, int rows, int) const { return Span{base ? base + first * ld : nullptr, rows}; }
  __device__ inline void load(Span s, Raw8<T> (&raw)[SL::NV], int t = 0, bool valid = true) const {
    const S* p = s.p + (row + t) * ld;
#pragma unroll
    for (int j = 0; j < SL::NV; ++j) {
      const int cj = c + j * SL::L * SL::W * 8;
      if (s.p && valid && row + t < s.rows && cj < cols) raw[j] = cols >= 8 ? load8_cut<T>(p, cj, cols) : load8_raw<T>(p + cj, cols - cj);
      else
#pragma unroll
        for (int w = 0; w < Raw8<T>::W; ++w) raw[j].v[w] = u32x4{0, 0, 0, 0};
    }
  }
  __device__ inline void settle(Raw8<T> (&raw)[SL::NV]) const {
    if (cols < 8) return;
#pragma unroll
    for (int j = 0; j < SL::NV; ++j) settle8<T>(raw[j], c + j * SL::L * SL::W * 8, cols);
  }
  __device__ inline void store(Span s, const float (&v)[SL::NV][8], int t = 0, bool valid = true) const {
    S* p = s.p + (row + t) * ld;
#pragma unroll
    for (int j = 0; j < SL::NV; ++j) {
      const int cj = c + j * SL::L * SL::W * 8;
      if (s.p && valid && row + t < s.rows && cj < cols) store8<T>(p + cj, v[j], cols - cj);
    }
  }
};

// A parameter's columns of this lane, kept over all its rows (`fill` where there is none, zeros behind
// the last column).
template <class SL>
__device__ inline void load_param(const float* p, float fill, int c0, int C, float (&v)[SL::NV][8]) {
#pragma unroll
  for (int j = 0; j < SL::NV; ++j) {
    const int c = c0 + j * SL::L * SL::W * 8;
    if (p && c < C) {
      to_floats<F32T>(load8_row<F32T>(p, c, C), v[j]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = e < C - c ? fill : 0.f;
    }
  }
}

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
constexpr int kCus = 256;

long ceil_div(long a, long b) { return (a + b - 1) / b; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Calls f with the narrowest slot that holds v vectors: of at most a wavefront with one vector a lane,
// and of sixteen wavefronts.
template <class F>
void with_narrow_slot(int v, F&& f) {
  if (v <= 2) f(Slot<2, 1, 1>{});
  else if (v <= 4) f(Slot<4, 1, 1>{});
  else if (v <= 8) f(Slot<8, 1, 1>{});
  else if (v <= 16) f(Slot<16, 1, 1>{});
  else if (v <= 32) f(Slot<32, 1, 1>{});
  else f(Slot<64, 1, 1>{});
}
template <class F>
void with_wide_slot(int v, F&& f) {
  if (v <= 1024) f(Slot<64, 16, 1>{});
  else if (v <= 2048) f(Slot<64, 16, 2>{});
  else f(Slot<64, 16, 4>{});
}
// The forward's slots.
template <class F>
void with_slot(int C, F&& f) {
  const int v = (C + 7) / 8;
  if (v <= 64) with_narrow_slot(v, f);
  else if (v <= 128) f(Slot<64, 1, 2>{});
  else if (v <= 256) f(Slot<64, 4, 1>{});
  else if (v <= 512) f(Slot<64, 4, 2>{});
  else with_wide_slot(v, f);
}
// The backward's: one vector a lane as far as possible, for the parameters' sums stay in registers
// beside the row (65536 rows of 1024 in bf16 with betas: two vectors a lane spill, 386 us, two
// wavefronts a row take 211; 16384 rows of 4096: 286 and 187).  Only a wavefront with two vectors of an
// aligned row of 16-bit values without betas (`lean`, for types of which TWO holds) fits, and then has no
// barriers: 65536 rows of 1024 202 us against 206, with gate rows shared by 26 169 against 179 (in fp32 it
// spills: 32768 rows of 1024 349 against 219).
template <bool TWO, class F>
void with_bwd_slot(int C, bool lean, F&& f) {
  const int v = (C + 7) / 8;
  if (v <= 64) with_narrow_slot(v, f);
  else if (v <= 128) {
    if constexpr (TWO)
      if (lean) return f(Slot<64, 1, 2>{});
    f(Slot<64, 2, 1>{});
  }
  else if (v <= 256) f(Slot<64, 4, 1>{});
  else if (v <= 512) f(Slot<64, 8, 1>{});
  else with_wide_slot(v, f);
}
template <class SL>
constexpr bool kLeanOnly = SL::W == 1 && SL::NV == 2;
// Wavefronts a SIMD that the backward's registers leave room for.  Eight to a row: one workgroup a CU
// (with two, 128 registers a lane, 16384 rows of 4096 with betas spill: 447 us).  Loose rows with shared
// gates (FULL) spill at three: 30000 rows of 1001 228 us against 122; without shared gates three are
// better, 128 against 147.
template <class SL, bool FULL>
constexpr int kBwdWaves = SL::W == 16 ? 4 : SL::W == 8 || SL::NV == 2 || FULL ? 2 : 3;

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


// An operand as the aligned view takes it: absent, or rows of 16-byte aligned vectors so close that
// `rows` of them span less than 2^30 bytes.
bool aligned_rows(const void* p, int64_t ld, size_t elem, int64_t rows) {
  return !p || (tower::al(p, 16) && ld * static_cast<int64_t>(elem) % 16 == 0 && ld * static_cast<int64_t>(elem) < (int64_t{1} << 30) / rows);
}

}  // namespace

// One direction's launch for a type of data, each in a source file of its own (dozens of kernels).
template <class T>
void launch_norm_fwd(const NormArgs& a, bool aligned, hipStream_t st);
template <class T>
void launch_norm_bwd(const NormArgs& a, const JoinArgs& j, bool aligned, bool lean, bool shared, int grid, hipStream_t st);

}  // namespace el
