// dense_fp4.hip -- microscaled 4-bit numbers (e2m1): packing and unpacking, and the dense layer on
// them, y = residual + act(x4 w4^T + bias).
#include "fp4_plan.hpp"
#include "micro.hpp"

namespace el {
namespace {

using namespace fp4;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// Eight values of a 16-bit type straight to 4 bits: the largest magnitude is found on the bits
// (ordered like unsigned numbers), and the conversion divides by the scale.
template <class T>
__device__ inline uint32_t pack4_raw(const Raw8<T>& raw, uint32_t& byte) {
  if constexpr (T::code == EL_F32) {
    float v[8];
    to_floats<T>(raw, v);
    return pack4(v, byte);
  } else {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, raw.v[0][i] & 0x7fff7fffu));
    const uint32_t top = quad_max(max(static_cast<uint32_t>(m[0]), static_cast<uint32_t>(m[1])));
    const uint32_t amax = __float_as_uint(T::to_f(static_cast<uint16_t>(top)));
    if (amax >= 0x7f800000u) {  // NaN and infinities compare as the largest
      byte = 255u;
      return 0u;
    }
    byte = scale_byte<true>(amax);
    const float scale = scale_of(byte);
    const uint32_t w0 = raw.v[0][0], w1 = raw.v[0][1], w2 = raw.v[0][2], w3 = raw.v[0][3];
    uint32_t q = 0;
    if constexpr (T::code == EL_BF16) {
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w0), scale, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w1), scale, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w2), scale, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w3), scale, 3);
    } else {
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w0), scale, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w1), scale, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w2), scale, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w3), scale, 3);
    }
    return q;
  }
}

// Lane d of the result holds what lane `from` (the same in no two lanes) holds.
__device__ inline u32x4 lanes_from(int from, const u32x4& v) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from * 4, static_cast<int>(v[i])));
  return r;
}

__device__ inline void store8_raw(uint16_t* p, const u32x4& v, int n) {
  if (n >= 8) {
    *reinterpret_cast<u32x4_any*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
  }
}

template <class T>
__device__ inline Raw8<T> zeros8() {
  Raw8<T> r;
#pragma unroll
  for (int w = 0; w < Raw8<T>::W; ++w) r.v[w] = u32x4{0, 0, 0, 0};
  return r;
}

struct PackArgs {
  const void* x;
  long ldx;
  int M, K, steps;
  uint8_t *codes, *scales;
};

// 16 lanes pack the 128 columns of a step of one row; a workgroup takes four steps of 16 rows at a
// time, so that whole words of scales and whole lines of codes are written.  Memory bounds it: 65536 x
// 1024 from bf16 32 us, 5.3 TB/s.
template <class T>
__global__ __launch_bounds__(kThreads) void k_fp4_pack(PackArgs a) {
  __shared__ __attribute__((aligned(4))) uint8_t sc[16][4][4];  // [row][block][step], read as words
  const int groups = (a.steps + 3) / 4;
  const int64_t rows16 = blockIdx.x / groups;
  const int grp = static_cast<int>(blockIdx.x - rows16 * groups);
  const int u = threadIdx.x >> 4, q = threadIdx.x & 15;
  const int64_t row = rows16 * 16 + u;
  Raw8<T> raw[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = grp * 4 + s, c = k * kPad + q * 8, n = a.K - c;
    raw[s] = zeros8<T>();
    if (row < a.M && n > 0) raw[s] = load8_raw<T>(static_cast<const typename T::S*>(a.x) + row * a.ldx + c, n);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = grp * 4 + s;
    uint32_t byte;
    const uint32_t w = pack4_raw<T>(raw[s], byte);
    if (k < a.steps) *reinterpret_cast<uint32_t*>(a.codes + code_at(row, k, q, a.steps)) = w;
    if ((q & 3) == 0) sc[u][q >> 2][s] = static_cast<uint8_t>(byte);
  }
  __syncthreads();
  if (threadIdx.x < 64) {  // (steps behind the last have the scales of zeros)
    const int r = threadIdx.x >> 2, g = threadIdx.x & 3;
    *reinterpret_cast<uint32_t*>(a.scales + scale_at(rows16 * 16 + r, grp * 4, g, groups)) = *reinterpret_cast<const uint32_t*>(sc[r][g]);
  }
}

// Back, row by row: a wavefront writes whole lines and gathers its codes from fragments in pieces of 16
// bytes, scales byte by byte, which bounds it: 65536 x 1024 to bf16 46 us, 3.7 TB/s (32768 rows, whose
// codes the caches hold once they were just packed, 20 us).
struct UnpackArgs {
  const uint8_t *codes, *scales;
  void* y;
  long ldy;
  int K, steps, vecs;
  int64_t items;  // M * vecs
};
template <class T>
__global__ __launch_bounds__(kThreads) void k_fp4_unpack(UnpackArgs a) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;
  if (first + threadIdx.x >= a.items) return;
  const int64_t row0 = first / a.vecs;
  const uint32_t local = static_cast<uint32_t>(first - row0 * a.vecs) + threadIdx.x;
  const uint32_t dr = local / static_cast<uint32_t>(a.vecs), grp = local - dr * a.vecs;
  const int64_t row = row0 + dr;
  const int k = static_cast<int>(grp >> 4), q = static_cast<int>(grp & 15);
  float v[8];
  unpack4(*reinterpret_cast<const uint32_t*>(a.codes + code_at(row, k, q, a.steps)),
          a.scales[scale_at(row, k, q >> 2, (a.steps + 3) / 4)], v);
  put_whole8<T>(static_cast<typename T::S*>(a.y) + row * a.ldy + grp * 8l, v, a.K - static_cast<int>(grp) * 8);
}

// ---------------------------------------------------------------------------------------
// The product.  A workgroup of four wavefronts packs 16 J rows of x into LDS once (their whole
// length), then walks over its columns, 32 to a wavefront; the weights' fragments come straight
// from the L2, which holds them all.
// ---------------------------------------------------------------------------------------
struct DenseArgs {
  const void* x;             // 16-bit rows, packed here
  const uint8_t *xc, *xs;    // or rows packed before (XG)
  const uint8_t *wc, *ws;
  long ldx;
  int M, N, K, steps;        // steps of 128 columns
  int passes, row_blocks;    // column passes of a workgroup; blocks of 16 J rows
  const float* bias;
  const uint16_t* add;
  uint16_t* out;
  long ldadd, ldo;
  uint32_t act;
};

// 16 x 16 outputs from 128 columns; the scale of a lane's block is byte SEL of its scale word.  The
// accumulators of lane l are rows 4 (l / 16) .. +3 of the first operand's fragment and row l % 16
// of the second's.
template <int SEL>
__device__ inline f32x4 mfma_fp4(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb, const f32x4& c) {
  const i32x8 av = {static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]), 0, 0, 0, 0};
  const i32x8 bv = {static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3]), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, SEL, static_cast<int>(sa), SEL, static_cast<int>(sb));
}

// The columns of a bias vector that was loaded from the last eight, moved to the front.
__device__ inline void settle_cut(float (&v)[8], int n) {
  const int s = n > 0 && n < 8 ? 8 - n : 0;
#pragma unroll
  for (int b = 4; b; b >>= 1)
    if (s & b)
#pragma unroll
      for (int e = 0; e + b < 8; ++e) v[e] = v[e + b];
}

// What bounds it, and the shape that follows.  Loads and stores share one in-order counter, so every
// load is issued at a fixed distance in front of its use, without a branch around it (a wait that
// cannot count waits for everything, the stores before it too: 124 us against 118).  The weights of
// the step three ahead, of the next columns where the row ends, are fetched while a step multiplies;
// the residual during a pass's last three steps.  65536 x 1024 x 1024 in bf16 with GELU and a residual
// take 118 us, 3.4 TB/s of x, residual and y (79 us at a copy's rate); no one part bounds it: without the
// products it takes 93, without packing 96, without the stores 98, without the residual 97, and the
// products alone 44.  Three wavefronts a SIMD for J = 4: at four the residual spills (131072 rows 220
// against 206, 24000 rows 49.6 against 46.4).  EIGHT: K and N are at least 8.
template <class T, int J, bool XG, bool EIGHT, bool ADD>
__global__ __launch_bounds__(kThreads, J == 4 ? 3 : 4) void k_dense_fp4(DenseArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // [step][J][64 lanes][16], then [group][J][64 lanes][4]
  constexpr int BR = 16 * J, WC = 32;
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rb = blockIdx.x % a.row_blocks, cb = blockIdx.x / a.row_blocks;
  const int row0 = rb * BR, groups = (a.steps + 3) / 4;
  const int x_frags = frags_of(a.M);
  uint8_t* lsc = lds + a.steps * J * kFrag;
  if constexpr (!XG) {
    // 16 lanes pack the 128 columns of a step of one row
    const int u = threadIdx.x >> 4, q = threadIdx.x & 15;
    const uint16_t* px = static_cast<const uint16_t*>(a.x);
    const uint16_t* p[J];
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = px + static_cast<long>(min(row0 + j * 16 + u, a.M - 1)) * a.ldx;
#pragma unroll 2
    for (int k = 0; k < a.steps; ++k) {
      const int c = k * kPad + q * 8, n = a.K - c;
      Raw8<T> raw[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if constexpr (EIGHT) {
          raw[j] = load8_cut<T>(p[j], c, a.K);
        } else {
          raw[j] = zeros8<T>();
          if (n > 0) raw[j] = load8_raw<T>(p[j] + c, n);
        }
      }
      const bool cut = k * kPad + kPad > a.K;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (EIGHT && cut) settle8<T>(raw[j], c, a.K);
        uint32_t byte;
        const uint32_t w = pack4_raw<T>(raw[j], byte);
        *reinterpret_cast<uint32_t*>(lds + (k * J + j) * kFrag + ((q >> 2) * 16 + u) * 16 + (q & 3) * 4) = w;
        if ((q & 3) == 0) lsc[((k >> 2) * J + j) * 256 + ((q >> 2) * 16 + u) * 4 + (k & 3)] = static_cast<uint8_t>(byte);
      }
    }
    __syncthreads();
  }
  constexpr int SETS = 4;  // steps of w in flight or in use
  u32x4 w[SETS][2];
  uint32_t wsc[2][2], xsc[J];
  const int tiles = (a.N + kTileRows - 1) / kTileRows;
  int tile = cb * a.passes * 4 + wave;
  if (tile >= tiles) return;
  const auto rc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.wc), 0, tiles * a.steps * 2 * kFrag, 0x00027000);
  const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.ws), 0, tiles * groups * 512, 0x00027000);
  const auto rbias = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.bias), 0, a.bias ? a.N * 4 : 0, 0x00027000);  // none: zeros
  // Step k of the tile, or of the tile after it from 4 groups on; what does not exist is replaced by
  // what does, and not used.
  const auto fetch = [&](int set, int k) {
    const bool next = k >= groups * 4;
    const int t = min(next ? tile + 4 : tile, tiles - 1), kk = min(next ? k - groups * 4 : k, a.steps - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[set][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, lane * 16, ((t * a.steps + kk) * 2 + i) * kFrag, 0));
  };
  const auto fetch_scales = [&](int set, int group) {
    const bool next = group >= groups;
    const int t = min(next ? tile + 4 : tile, tiles - 1), gg = next ? 0 : group;
#pragma unroll
    for (int i = 0; i < 2; ++i) wsc[set][i] = __builtin_amdgcn_raw_buffer_load_b32(rs, lane * 4, ((t * groups + gg) * 2 + i) * 256, 0);
  };
  fetch_scales(0, 0);
#pragma unroll
  for (int t = 0; t < SETS - 1; ++t) fetch(t, t);
  // Fragment j's row of this lane in memory is row_of(j, l) = first row of the fragment + l (or l's
  // place in a tile): the lane's part of its address is formed once.
  const int lrow = XG ? row_of_lane(0, lane >> 2) : lane >> 2;
  const auto frag_row = [&](int j) { return XG ? row_of_lane(rb * J + j, 0) : row0 + j * 16; };
  const long add_lane = lrow * a.ldadd, out_lane = lrow * a.ldo;
  for (int pass = 0; pass < a.passes && tile < tiles; ++pass, tile += 4) {
    const int c = tile * WC + 8 * g;              // this lane's columns in the accumulators,
    const int cm = tile * WC + 8 * (lane & 3);    // and in memory, where four neighbours share a row
    f32x4 acc[2][J] = {};
    float bias[8] = {};
    Raw8<T> add[J];
    const auto fetch_ends = [&]() {  // the bias and the residual
      if constexpr (EIGHT) {
        const int at = min(c, a.N - 8) * 4;
        const f32x4 lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rbias, at, 0, 0));
        const f32x4 hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rbias, at + 16, 0, 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = lo[e], bias[4 + e] = hi[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rbias, min(c + e, a.N - 1) * 4, 0, 0));
      }
      if constexpr (ADD)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int fr = frag_row(j);  // (a row that does not exist is replaced by the workgroup's first)
          const uint16_t* p = a.add + (lrow < a.M - fr ? fr * a.ldadd + add_lane : min(row0, a.M - 1) * a.ldadd);
          if constexpr (EIGHT) add[j] = load8_cut<T>(p, cm, a.N);
          else if (cm < a.N) add[j] = load8_raw<T>(p + cm, a.N - cm);
        }
    };
    const auto step = [&](int k, auto sel) {
      constexpr int SEL = decltype(sel)::value;
      fetch((SEL + SETS - 1) % SETS, k + SETS - 1);
      if (k >= a.steps) return;
      u32x4 x[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if constexpr (XG) {
          const int f = frag_read(rb, J, j, x_frags);
          x[j] = *reinterpret_cast<const u32x4*>(a.xc + frag_code_at(f, k, a.steps) + lane * 16);
          if (SEL == 0) xsc[j] = *reinterpret_cast<const uint32_t*>(a.xs + frag_scale_at(f, k, groups) + lane * 4);
        } else {
          x[j] = *reinterpret_cast<const u32x4*>(lds + (k * J + j) * kFrag + lane * 16);
          if (SEL == 0) xsc[j] = *reinterpret_cast<const uint32_t*>(lsc + ((k >> 2) * J + j) * 256 + lane * 4);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[i][j] = mfma_fp4<SEL>(w[SEL][i], wsc[0][i], x[j], xsc[j], acc[i][j]);
    };
    static_assert(SETS == 4, "one set for each scale byte");
    const auto group = [&](int k, auto last) {
      fetch_scales(1, (k >> 2) + 1);
      step(k, std::integral_constant<int, 0>{});
      if constexpr (decltype(last)::value) fetch_ends();
      step(k + 1, std::integral_constant<int, 1>{});
      step(k + 2, std::integral_constant<int, 2>{});
      step(k + 3, std::integral_constant<int, 3>{});
      wsc[0][0] = wsc[1][0], wsc[0][1] = wsc[1][1];
    };
    int k = 0;
    for (; k < groups * 4 - 4; k += 4) group(k, std::false_type{});
    group(k, std::true_type{});
    const bool cut = tile * WC + WC > a.N;
    if (EIGHT && cut) settle_cut(bias, a.N - c);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float v[8], f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = acc[0][j][e] + bias[e], v[4 + e] = acc[1][j][e] + bias[4 + e];
      if (a.act == EL_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_elementwise_maximum(v[e], 0.f);  // (keeps the NaN of NaN blocks)
      } else {
        act8(a.act, v);
      }
      if constexpr (ADD) {
        Raw8<T> mine = add[j];
        if (EIGHT && cut) settle8<T>(mine, cm, a.N);
        mine.v[0] = lanes_from(l16 * 4 + g, mine.v[0]);
        to_floats<T>(mine, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += f[e];
      }
      const u32x4 o = lanes_from((lane & 3) * 16 + (lane >> 2), to_16bit<T>(v));
      const int fr = frag_row(j);
      uint16_t* p = a.out + (fr * a.ldo + out_lane) + cm;
      if (lrow < a.M - fr) {
        if (!cut) *reinterpret_cast<u32x4_any*>(p) = o;
        else if (cm < a.N) store8_raw(p, o, a.N - cm);
      }
      __builtin_amdgcn_sched_barrier(0);  // one vector's values at a time in registers
    }
  }
}

template <class F>
void with_type(el_dtype dtype, F&& f) {
  if (dtype == EL_F32) f(F32T{});
  else if (dtype == EL_F16) f(F16T{});
  else f(BF16T{});
}

void launch_pack(const void* x, long ldx, int M, int K, el_dtype dtype, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const PackArgs a{x, ldx, M, K, static_cast<int>(steps_of(K)), codes, scales};
  const long units = tile_rows(M) / 16 * groups_of(K);
  with_type(dtype, [&](auto t) {
    hipLaunchKernelGGL((k_fp4_pack<decltype(t)>), dim3(static_cast<unsigned>(units)), dim3(kThreads), 0, st, a);
  });
}

template <class T, int J, bool XG, bool EIGHT>
void launch_tiles(const Plan& p, const DenseArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(p.blocks));
  const size_t lds = XG ? 0 : x_lds(16 * J, a.K);
  if (a.add) hipLaunchKernelGGL((k_dense_fp4<T, J, XG, EIGHT, true>), grid, dim3(kThreads), lds, st, a);
  else hipLaunchKernelGGL((k_dense_fp4<T, J, XG, EIGHT, false>), grid, dim3(kThreads), lds, st, a);
}
template <class T, int J>
void launch_rows(const Plan& p, const DenseArgs& a, hipStream_t st) {
  const bool eight = a.K >= 8 && a.N >= 8;
  if (p.packed) eight ? launch_tiles<T, J, true, true>(p, a, st) : launch_tiles<T, J, true, false>(p, a, st);
  else eight ? launch_tiles<T, J, false, true>(p, a, st) : launch_tiles<T, J, false, false>(p, a, st);
}
template <class T>
void launch_dense(const Plan& p, const DenseArgs& a, hipStream_t st) {
  if (p.J == 4) launch_rows<T, 4>(p, a, st);
  else if (p.J == 2) launch_rows<T, 2>(p, a, st);
  else launch_rows<T, 1>(p, a, st);
}

bool dense_fp4_sizes_ok(int64_t M, int64_t K, int64_t N) {
  return M >= 1 && K >= 1 && N >= 1 && K <= tower::kMaxMicroCols && N <= tower::kMaxMicroCols && N * K < (int64_t{1} << 29) &&
         ceil_div(M, 256) * ceil_div(N, 256) < (1l << 21) && tower::pad_to(M, kTileRows) * tower::pad_to(K, kPad) <= (int64_t{1} << 34);
}

}  // namespace
}  // namespace el

using namespace el;

extern "C" {

el_status el_fp4_pack(const void* x, int64_t ldx, int32_t M, int32_t K, el_dtype dtype, uint8_t* codes, uint8_t* scales,
                      hipStream_t stream) {
  const char* fn = "el_fp4_pack";
  return tower::guarded(fn, [&]() -> el_status {
    if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
    EL_TRY(tower::check_packed_sizes(fn, M, K, kPad, kTileRows));
    EL_TRY(tower::check_rows(fn, "x", x, ldx, K, M > 0, dtype_size(dtype)));
    EL_TRY(tower::check_packed(fn, "the output", codes, scales, M > 0));
    if (M == 0) return EL_OK;
    launch_pack(x, ldx, M, K, dtype, codes, scales, stream);
    return check_launch(fn);
  });
}

el_status el_fp4_unpack(const uint8_t* codes, const uint8_t* scales, int32_t M, int32_t K, void* y, int64_t ldy,
                        el_dtype dtype, hipStream_t stream) {
  const char* fn = "el_fp4_unpack";
  return tower::guarded(fn, [&]() -> el_status {
    if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
    EL_TRY(tower::check_packed_sizes(fn, M, K, kPad, kTileRows));
    EL_TRY(tower::check_packed(fn, "x", codes, scales, M > 0));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, K, M > 0, dtype_size(dtype)));
    if (M == 0) return EL_OK;
    UnpackArgs a{codes, scales, y, ldy, K, static_cast<int>(steps_of(K)), (K + 7) / 8, 0};
    a.items = static_cast<int64_t>(M) * a.vecs;
    with_type(dtype, [&](auto t) {
      hipLaunchKernelGGL((k_fp4_unpack<decltype(t)>), dim3(static_cast<unsigned>(ceil_div(a.items, kThreads))), dim3(kThreads), 0, stream, a);
    });
    return check_launch(fn);
  });
}

size_t el_dense_fwd_fp4_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  if (!dense_fp4_sizes_ok(M, K, N) || !plan_dense(M, K, N).packed) return 0;
  return code_bytes(M, K) + scale_bytes(M, K);
}

el_status el_dense_fwd_fp4(const void* x, int64_t ldx, int32_t M, int32_t K, const uint8_t* w_codes,
                           const uint8_t* w_scales, const float* bias, int32_t N, uint32_t act, const void* residual,
                           int64_t ldr, void* y, int64_t ldy, el_dtype dtype, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  const char* fn = "el_dense_fwd_fp4";
  return tower::guarded(fn, [&]() -> el_status {
    if (dtype != EL_BF16 && dtype != EL_F16)
      return dtype_valid(dtype) ? tower::unsupported(fn, "dtype must be EL_BF16 or EL_F16") : tower::bad(fn, "unknown dtype");
    if (M < 0) return tower::bad(fn, "M must be >= 0");
    if (K < 1) return tower::bad(fn, "K must be >= 1");
    if (N < 1) return tower::bad(fn, "N must be >= 1");
    if (!dense_fp4_sizes_ok(std::max(M, 1), K, N))
      return tower::unsupported(fn, "K and N must be <= 2^20, N * K < 2^29, outputs below 2^21 tiles of 256 x 256 and M times padded K <= 2^34");
    EL_TRY(tower::check_act(fn, act));
    EL_TRY(tower::check_packed(fn, "w", w_codes, w_scales, true));
    if (!tower::al(bias, 4)) return tower::bad(fn, "bias must be aligned to its elements");
    EL_TRY(tower::check_rows(fn, "x", x, ldx, K, M > 0, 2));
    EL_TRY(tower::check_rows(fn, "residual", residual, ldr, N, false, 2));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, N, M > 0, 2));
    if (M == 0) return EL_OK;
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, el_dense_fwd_fp4_workspace_bytes(M, K, N)));
    const Plan p = plan_dense(M, K, N);
    DenseArgs a{};
    a.x = x, a.ldx = ldx, a.wc = w_codes, a.ws = w_scales, a.M = M, a.N = N, a.K = K, a.steps = static_cast<int>(steps_of(K));
    a.passes = p.passes, a.row_blocks = p.row_blocks;
    a.bias = bias, a.add = static_cast<const uint16_t*>(residual), a.ldadd = ldr;
    a.out = static_cast<uint16_t*>(y), a.ldo = ldy, a.act = act;
    if (p.packed) {
      uint8_t* xc = static_cast<uint8_t*>(workspace);
      uint8_t* xs = xc + code_bytes(M, K);
      launch_pack(x, ldx, M, K, dtype, xc, xs, stream);
      EL_TRY(check_launch(fn));
      a.xc = xc, a.xs = xs;
    }
    if (dtype == EL_BF16) launch_dense<BF16T>(p, a, stream);
    else launch_dense<F16T>(p, a, stream);
    return check_launch(fn);
  });
}

}  // extern "C"
