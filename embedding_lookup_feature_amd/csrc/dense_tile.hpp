// dense_tile.hpp -- the tile kernels of the dense products (dense_epi.hip describes them) and the
// host code that plans and launches them, shared by the dense layers on 16-bit activations and on
// activations kept in 8 bits.
#pragma once

#include <algorithm>

#include "micro.hpp"

namespace el {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

enum Product { FWD = 0, DGRAD = 1, WGRAD = 2 };

struct GemmArgs {
  const uint16_t *P, *Q;
  long ldp, ldq;
  int R, C;        // output rows, columns
  int red;         // reduction length (of P's rows, zeros included)
  int red_q;       // of Q
  int per_split;   // reduction per split (weight gradient; a multiple of BK)
  int tiles_c;     // column tiles
  int tiles;       // tiles of one split
  // forward: out = y, aux = pre (or null), add = residual (or null)
  // data gradient: out = dx, aux = dzb (or null), add = dres (or null), pre = the layer below's
  // weight gradient: part = fp32 [split][R][C], dbp = fp32 [split * tiles_c * WC][R] (or null)
  const uint16_t *add, *pre;
  uint16_t *out, *aux;
  long ldadd, ldpre, ldo, ldaux;
  const float* bias;
  float *part, *dbp;
  DropArgs drop;
  uint32_t act;
  // activations kept in 8 bits: pre of the data gradient, Q of the weight gradient, rows of kp codes
  const uint8_t *codes, *scales;
  long kp;
};

// Eight columns of the data gradient's pre-activation, in 16 or in 8 bits.
template <class T, bool KEPT>
struct Pre8 {
  Raw8<T> raw;
  __device__ inline void floats(float (&f)[8]) const { to_floats<T>(raw, f); }
};
template <class T>
struct Pre8<T, true> {
  uint2 q;
  uint32_t scale;
  __device__ inline void floats(float (&f)[8]) const { unpack8(q.x, q.y, scale_of(scale), f); }
};

// ---------------------------------------------------------------------------------------
// Epilogue of eight columns c .. c+7 (the first n of them exist) of row r, from the product v;
// `add` and `pre` are the eight values already loaded.  Non-temporal accesses (NT) where the
// arrays are larger than the caches.
// ---------------------------------------------------------------------------------------
template <class T, bool NT>
__device__ inline void put8(uint16_t* p, const float (&f)[8], int n) {
  if (NT && n >= 8) {
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = static_cast<uint32_t>(T::from_f(f[2 * i])) | (static_cast<uint32_t>(T::from_f(f[2 * i + 1])) << 16);
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4_any*>(p));
  } else {
    store8<T>(p, f, n);
  }
}

template <class T, bool NT>
__device__ inline Raw8<T> get8(const uint16_t* p, int n) {
  if (!NT || n < 8) return load8_raw<T>(p, n);
  Raw8<T> r;
  r.v[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
  return r;
}

template <class T, int PROD, bool NT, class PRE>
__device__ inline void epilogue8(const GemmArgs& a, uint64_t offset, long r, int c, int n, float (&v)[8],
                                 const Raw8<T>& add, const PRE& pre) {
  float f[8];
  if (a.add) to_floats<T>(add, f);
  if constexpr (PROD == FWD) {
    if (a.aux) put8<T, NT>(a.aux + r * a.ldaux + c, v, n);
    act8(a.act, v);
  } else {
    if (a.add)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += f[e];
    put8<T, NT>(a.out + r * a.ldo + c, v, n);
    if (!a.aux) return;
    if (a.act != EL_ACT_NONE) {
      pre.floats(f);
      act8_grad(a.act, f, v);
    }
  }
  float scale = 1.f;
  if (a.drop.top) {
    const u32x4 bits = philox8(static_cast<uint32_t>(c) >> 3, static_cast<uint32_t>(r), offset, a.drop.k0, a.drop.k1);
    scale = a.drop.scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = keep_of(bits, e, a.drop.top) ? v[e] : 0.f;
  }
  if (PROD == FWD && a.add) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], scale, f[e]);
  } else if (a.drop.top) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= scale;
  }
  put8<T, NT>((PROD == FWD ? a.out : a.aux) + r * (PROD == FWD ? a.ldo : a.ldaux) + c, v, n);
}

// ---------------------------------------------------------------------------------------
// Operand tiles: global memory -> LDS -> fragments.
// ---------------------------------------------------------------------------------------
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A buffer offset past the end of every buffer used here (their sizes are cut to less than 2^31;
// a stage spans at most 2^30 bytes): the load reads zeros and touches no memory.
constexpr uint32_t kOut = 0x80000000u;

__device__ inline uint32_t uniform(uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))); }

// 64 lanes x 16 bytes from the buffer to LDS at `lds` + 16 lane.  (One wait state between the
// write of M0 and its use.)  The load has no register result; wait_and_meet waits for it.
__device__ inline void load_lds16(uint32_t lds, uint32_t voff, const u32x4& rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               ::"s"(lds), "v"(voff), "s"(rsrc) : "memory");
}

// At most N of this wavefront's loads to LDS are still in flight and its LDS reads are done;
// then the same holds for every wavefront of the workgroup.
template <int N>
__device__ inline void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One operand's W x BK share of the stages, loaded by NW wavefronts in pieces of 1 KiB.
//   RC: [W rows][BK], row r's 16-byte unit c at position c ^ (r / rows per 256 bytes), so that
//       the 32 rows of a fragment read (one unit each) spread over all banks;
//   OC: [BK][W], row k's unit c at c ^ (4 * place of k among the 4 rows of a transposing read),
//       so that the 64-byte pieces which such a read takes from four rows lie in four places.
// Rows past the operand's end fall behind the buffer's size and read as zeros; vectors past the
// reduction's end (RC) or past the last column (OC) are sent to kOut.
template <int W, int BK, bool RC, int NW>
struct Operand {
  static_assert(BK == 64, "the permutations below are for rows of 64 reductions");
  static constexpr int BYTES = W * BK * 2;
  static constexpr int N = BYTES / 1024 / NW;  // pieces per wavefront
  static_assert(N >= 1 && BYTES % (1024 * NW) == 0, "whole pieces");
  uint64_t base;   // where the next stage to load begins
  uint64_t left;   // bytes from there to the operand's end
  uint32_t step;   // bytes per stage
  int rem;         // reductions left
  uint32_t voff[N];
  int kc[N];       // RC: the reduction index of this lane's vector inside the stage

  __device__ static inline int perm(int row_or_k) {
    if constexpr (RC) return (row_or_k >> 1) & 7;
    return W == 64 ? ((row_or_k >> 1) & 1) << 2 : (row_or_k & 3) << 2;
  }
  // rows i0 .. i0+W-1 of n, reductions kbeg .. kend-1
  __device__ inline void init(const uint16_t* p, long ld, int i0, int n, int kbeg, int kend, int wave, int lane) {
    const int rows = min(W, n - i0);
    rem = kend - kbeg;
    if constexpr (RC) {
      left = static_cast<uint64_t>((rows - 1) * ld + rem) * 2;
      base = reinterpret_cast<uint64_t>(p + i0 * ld + kbeg);
      step = BK * 2;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int u = (j * NW + wave) * 64 + lane;
        const int row = u / (BK / 8), c = (u % (BK / 8)) ^ perm(row);
        voff[j] = static_cast<uint32_t>(row * ld * 2) + c * 16;
        kc[j] = c * 8;
      }
    } else {
      left = static_cast<uint64_t>((rem - 1l) * ld + ((n + 7) / 8 * 8 - i0)) * 2;  // rows hold whole vectors
      base = reinterpret_cast<uint64_t>(p + kbeg * ld + i0);
      step = static_cast<uint32_t>(BK * ld * 2);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int u = (j * NW + wave) * 64 + lane;
        const int k = u / (W / 8), c = (u % (W / 8)) ^ perm(k);
        voff[j] = c * 8 < rows ? static_cast<uint32_t>(k * ld * 2) + c * 16 : kOut;
      }
    }
  }
  __device__ inline u32x4 rsrc() const {
    return u32x4{uniform(static_cast<uint32_t>(base)), uniform(static_cast<uint32_t>(base >> 32) & 0xffffu),
                 uniform(rem > 0 ? static_cast<uint32_t>(min(left, uint64_t{0x7fffffff})) : 0u), 0x00027000u};
  }
  __device__ inline void load(uint32_t lds, int j, const u32x4& rs) const {
    uint32_t v = voff[j];
    if constexpr (RC) v = kc[j] < rem ? v : kOut;
    load_lds16(lds + j * NW * 1024, v, rs);
  }
  __device__ inline void advance() {
    base += step;
    left -= step;
    rem -= BK;
  }
  // The fragment of 32 rows from `i`, reductions 16 kk .. 16 kk + 15: lane l holds row l % 32,
  // eight reductions from 8 (l / 32).
  __device__ static inline u32x4 frag(const lds_char* tile, int i, int kk, int lane) {
    if constexpr (RC) {
      const int r = i + (lane & 31), c = (kk * 2 + (lane >> 5)) ^ perm(r);
      return *reinterpret_cast<const lds_u32x4*>(tile + r * (BK * 2) + c * 16);
    } else {
      // each group of 16 lanes reads a 4 x 16 block (lane q: row q / 4, columns 4 (q % 4) .. +3)
      // and gets it transposed (lane q: column q, four rows)
      const int g = lane >> 4, q = lane & 15;
      const int k = kk * 16 + (g >> 1) * 8 + (q >> 2);
      const int col = i + (g & 1) * 16 + (q & 3) * 4;
      const lds_char* p = tile + k * (W * 2) + ((col >> 3) ^ perm(k)) * 16 + (col & 7) * 2;
      struct { s16x4 lo, hi; } v;
      v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
      v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (W * 2)));  // perm(k + 4) = perm(k)
      return __builtin_bit_cast(u32x4, v);
    }
  }
};

// The weight gradient's Q kept in 8 bits: the same tile in LDS (output-contiguous, [BK][W] of 16-bit
// values, the same permutation), but its codes pass through registers, where they get their scales.
// A stage's codes are loaded when its slot is freed and written to it one stage later.
template <class T, int W, int BK, int NW>
struct Operand8 {
  using Tile = Operand<W, BK, false, NW>;
  static constexpr int BYTES = Tile::BYTES, N = Tile::N;
  const uint8_t *codes, *scales;  // where the next stage to load begins
  int64_t left;                   // rows from there to the end
  int kp;
  uint32_t voff[N], soff[N];
  uint2 q[N];
  uint32_t sc[N];
  __device__ inline void init(const uint8_t* c8, const uint8_t* s8, long kp_, int i0, int n, long kbeg, long kend, int wave, int lane) {
    kp = static_cast<int>(kp_);
    codes = c8 + kbeg * kp_ + i0;
    scales = s8 + kbeg * (kp_ / kMicroBlock) + i0 / kMicroBlock;
    left = kend - kbeg;
    const int cols = min(W, n - i0);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int u = (j * NW + wave) * 64 + lane;
      const int k = u / (W / 8), c = (u % (W / 8)) ^ Tile::perm(k);
      voff[j] = c * 8 < cols ? static_cast<uint32_t>(k) * kp + c * 8 : kOut;
      soff[j] = c * 8 < cols ? static_cast<uint32_t>(k) * (kp / kMicroBlock) + c * 8 / kMicroBlock : kOut;
    }
  }
  __device__ inline void load(int j) {
    const int rows = static_cast<int>(max(int64_t{0}, min(left, int64_t{BK})));
    const auto rc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(codes), 0, rows * kp, 0x00027000);
    const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(scales), 0, rows * (kp / kMicroBlock), 0x00027000);
    const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, voff[j], 0, 0));
    q[j] = uint2{v[0], v[1]};
    sc[j] = __builtin_amdgcn_raw_buffer_load_b8(rs, soff[j], 0, 0);
  }
  __device__ inline void advance() {
    codes += static_cast<long>(BK) * kp;
    scales += static_cast<long>(BK) * (kp / kMicroBlock);
    left -= BK;
  }
  // This lane's vectors to their places behind `tile` (this wavefront's first piece).
  __device__ inline void put(lds_char* tile, int lane) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float s = scale_of(sc[j]);
      u32x4 v;
      if constexpr (T::code == EL_BF16) {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[j].x, s, false));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[j].x, s, true));
        v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[j].y, s, false));
        v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[j].y, s, true));
      } else {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[j].x, s, false));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[j].x, s, true));
        v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[j].y, s, false));
        v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[j].y, s, true));
      }
      *reinterpret_cast<lds_u32x4*>(tile + j * NW * 1024 + lane * 16) = v;
    }
  }
  __device__ static inline u32x4 frag(const lds_char* tile, int i, int kk, int lane) { return Tile::frag(tile, i, kk, lane); }
};

// Orders this wavefront's LDS writes before its later reads by other lanes (the hardware keeps a
// wavefront's LDS accesses in order; this keeps the compiler from moving them).
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The hardware hands workgroups to the 8 XCDs in turn; this gives each XCD one contiguous run of
// the n logical ones, so that tiles which share operand panels share an L2.
__device__ inline int xcd_order(int bid, int n) {
  const int x = bid & 7, per = n >> 3, rem = n & 7;
  return x * per + min(x, rem) + (bid >> 3);
}

// Tile shapes: WR x WC wavefronts own BR x BC outputs of a workgroup; ST stages of 64 reductions.
// 16 wavefronts on the large tile and 8 on the middle one: more wavefronts share the epilogue's
// latency (L forward 232 us at 16, 244 at 8; backward 376, 387).
template <int BR_, int BC_, int WR_, int WC_, int ST_, int WPE_, bool NT_, int AHEAD_>
struct Cfg {
  static constexpr int BR = BR_, BC = BC_, BK = 64, WR = WR_, WC = WC_, ST = ST_, NW = WR * WC;
  static constexpr int FR = BR / WR / 32, FC = BC / WC / 32;  // 32 x 32 blocks per wavefront
  static constexpr int WPE = WPE_;                            // wavefronts per SIMD the registers allow
  static constexpr bool NT = NT_;                             // non-temporal epilogue
  static constexpr int AHEAD = AHEAD_;                        // row blocks whose residual / pre are on their way
  static constexpr int PITCH = FC * 32 + 4;                   // floats per row of the epilogue's LDS blocks
  static constexpr int LDS = std::max(ST * (BR + BC) * BK * 2, NW * 32 * PITCH * 4);
};
using CfgL = Cfg<256, 256, 4, 4, 2, 4, true, 1>;   // 136 KB of LDS, one workgroup of 16 wavefronts per CU
using CfgM = Cfg<128, 128, 2, 4, 2, 4, false, 2>;  // 64 KB, two of 8 wavefronts per CU
using CfgS = Cfg<64, 64, 2, 2, 4, 2, false, 1>;    // 64 KB, two per CU
using CfgS2 = Cfg<64, 64, 2, 2, 2, 4, false, 1>;   // 32 KB, four per CU: for codes, of which the registers hold one stage
                                                   // (4099 x 479 x 256, fp16: 25 us; unpacked first for CfgS 27.7)

// One tile (of one split): `lid` in tiles of all splits, in the order that shares panels.
// KEPT: the data gradient's pre or the weight gradient's Q is read from 8 bits.
template <class T, class C, int PROD, bool KEPT = false>
__device__ __forceinline__ void dense_tile(const GemmArgs& a, int lid, char* lds) {
  constexpr int NW = C::NW, FR = C::FR, FC = C::FC, BK = C::BK, ST = C::ST, WC = C::WC;
  using OP = Operand<C::BR, BK, PROD != WGRAD, NW>;
  constexpr bool Q8 = KEPT && PROD == WGRAD;
  static_assert(!Q8 || ST == 2, "the registers hold one stage of codes");
  using OQ = std::conditional_t<Q8, Operand8<T, C::BC, BK, NW>, Operand<C::BC, BK, PROD == FWD, NW>>;
  constexpr int SB = OP::BYTES + OQ::BYTES, LOADS = OP::N + OQ::N;
  const int lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = static_cast<int>(uniform(threadIdx.x >> 6));
  const int split = lid / a.tiles, t = lid - split * a.tiles;
  const int tr = t / a.tiles_c, tc = t - tr * a.tiles_c;
  const int row0 = tr * C::BR, col0 = tc * C::BC;
  const int kbeg = split * a.per_split;
  const int kend = a.red - kbeg < a.per_split ? a.red : kbeg + a.per_split;  // (the sum may pass 2^31)
  const int nk = (kend - kbeg + BK - 1) / BK;
  const int wr = wave / WC, wc = wave % WC;
  OP op;
  OQ oq;
  op.init(a.P, a.ldp, row0, a.R, kbeg, kend, wave, lane);
  if constexpr (Q8) oq.init(a.codes, a.scales, a.kp, col0, a.C, kbeg, min(kend, a.red_q), wave, lane);
  else oq.init(a.Q, a.ldq, col0, a.C, kbeg, min(kend, a.red_q), wave, lane);
  const lds_char* base = (const lds_char*)lds;
  const uint32_t mine = uniform(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(base)) + wave * 1024);
  const auto rsrc_q = [&]() {
    if constexpr (Q8) return u32x4{};
    else return oq.rsrc();
  };
  const auto load_one = [&](int m, uint32_t slot, const u32x4& rp, const u32x4& rq) {
    if (m < OP::N) op.load(mine + slot, m, rp);
    else if constexpr (Q8) oq.load(m - OP::N);
    else oq.load(mine + slot + OP::BYTES, m - OP::N, rq);
  };
  const auto put_q = [&](uint32_t slot) {
    if constexpr (Q8) oq.put((lds_char*)lds + slot + OP::BYTES + wave * 1024, lane);
  };
  f32x16 acc[FC][FR];
  // register 4 g + e of acc[i][j]: column 32 i + 8 g + 4 half + e of row 32 j + l32; the forward's
  // accumulators start from the bias
#pragma unroll
  for (int i = 0; i < FC; ++i) {
    f32x16 z = f32x16{};
    if (PROD == FWD && a.bias)
#pragma unroll
      for (int k = 0; k < 16; ++k) z[k] = a.bias[min(col0 + (wc * FC + i) * 32 + acc_row(k, lane), a.C - 1)];
#pragma unroll
    for (int j = 0; j < FR; ++j) acc[i][j] = z;
  }
  float dbs[FR] = {};

  // Fill the ring.  Stages past the reduction's end load zeros without touching memory, so the
  // number of loads in flight at every wait is known at compile time.
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    const u32x4 rp = op.rsrc(), rq = rsrc_q();
#pragma unroll
    for (int m = 0; m < LOADS; ++m) load_one(m, s * SB, rp, rq);
    op.advance();
    oq.advance();
    if (s < ST - 1) put_q(s * SB);  // (the last stage's codes wait for the loop)
  }

  // Two register sets of fragments: while one K16 step multiplies, the next one's are read.  The
  // matrix A operand is Q's fragment, so a lane's accumulators are consecutive output columns.
  constexpr int KK = BK / 16;
  u32x4 q[2][FC], p[2][FR];
  const auto read = [&](int set, uint32_t slot, int kk) {
#pragma unroll
    for (int i = 0; i < FC; ++i) q[set][i] = OQ::frag(base + slot + OP::BYTES, (wc * FC + i) * 32, kk, lane);
#pragma unroll
    for (int j = 0; j < FR; ++j) p[set][j] = OP::frag(base + slot, (wr * FR + j) * 32, kk, lane);
  };
  // Bias gradient: the column tiles and their wavefront columns share the stages out, so every
  // row's sum is taken once and no tile does more than its part.
  const auto add_rows = [&](int set, int kt) {
    if (PROD == WGRAD && a.dbp && kt % (a.tiles_c * WC) == tc * WC + wc)
#pragma unroll
      for (int j = 0; j < FR; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dbs[j] += T::to_f(static_cast<uint16_t>(p[set][j][e] & 0xffffu)) + T::to_f(static_cast<uint16_t>(p[set][j][e] >> 16));
  };
  wait_and_meet<LOADS*(ST - 1)>();
  __builtin_amdgcn_sched_barrier(0);
  read(0, 0, 0);
  uint32_t slot = 0;
  for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
    for (int kk = 0; kk < KK - 1; ++kk) {
      // the next stage's codes, loaded a stage ago, to the slot that was freed then
      if (Q8 && kk == KK - 2) put_q(slot + SB == ST * SB ? 0 : slot + SB);
      read((kk + 1) & 1, slot, kk + 1);
#pragma unroll
      for (int j = 0; j < FR; ++j)
#pragma unroll
        for (int i = 0; i < FC; ++i) acc[i][j] = mfma32<T>(q[kk & 1][i], p[kk & 1][j], acc[i][j]);
      add_rows(kk & 1, kt);
      // one LDS read (two where a fragment takes two) behind each product
#pragma unroll
      for (int m = 0; m < FC * FR; ++m) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, PROD == FWD ? 1 : 2, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // The stage's last fragments are in registers: its slot is free, and the next stage has
    // arrived.  The refill's loads are issued one behind each product of the last K16 step.
    wait_and_meet<LOADS*(ST - 2)>();
    __builtin_amdgcn_sched_barrier(0);
    const uint32_t freed = slot;
    slot = slot + SB == ST * SB ? 0 : slot + SB;
    const u32x4 rp = op.rsrc(), rq = rsrc_q();
    add_rows((KK - 1) & 1, kt);
    read(0, slot, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < (FC * FR > LOADS ? FC * FR : LOADS); ++m) {
      if (m < FC * FR) acc[m % FC][m / FC] = mfma32<T>(q[1][m % FC], p[1][m / FC], acc[m % FC][m / FC]);
      __builtin_amdgcn_sched_barrier(0);
      if (m < LOADS) load_one(m, freed, rp, rq);
      __builtin_amdgcn_sched_barrier(0);
    }
    op.advance();
    oq.advance();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  if constexpr (PROD == WGRAD) {
    if (a.dbp) {
#pragma unroll
      for (int j = 0; j < FR; ++j) {
        const float s = dbs[j] + __shfl_xor(dbs[j], 32);
        const int r = row0 + (wr * FR + j) * 32 + l32;
        if (half == 0 && r < a.R) a.dbp[((static_cast<long>(split) * a.tiles_c + tc) * WC + wc) * a.R + r] = s;
      }
    }
#pragma unroll
    for (int j = 0; j < FR; ++j) {
      const int r = row0 + (wr * FR + j) * 32 + l32;
      float* o = a.part + (static_cast<long>(split) * a.R + r) * a.C;
#pragma unroll
      for (int i = 0; i < FC; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = col0 + (wc * FC + i) * 32 + g * 8 + half * 4;
          if (r >= a.R || c >= a.C) continue;
          if (a.C % 4 == 0) {
            *reinterpret_cast<u32x4_f32*>(o + c) =
                u32x4{__float_as_uint(acc[i][j][4 * g]), __float_as_uint(acc[i][j][4 * g + 1]),
                      __float_as_uint(acc[i][j][4 * g + 2]), __float_as_uint(acc[i][j][4 * g + 3])};
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (c + e < a.C) o[c + e] = acc[i][j][4 * g + e];
          }
        }
    }
  } else {
    // Accumulators go through LDS (each wavefront's own 32 x (32 FC) floats at a time), so that a
    // lane gets eight consecutive columns: they share one call of the mask's generator, and a
    // row's accesses to residual, pre, y, ... are whole cache lines (222 us against 298 with the
    // epilogue straight from the accumulators' four columns a lane).
    constexpr int WCOLS = FC * 32, GR = WCOLS / 8, RPP = 64 / GR, PASS = 32 / RPP, PITCH = C::PITCH, AHEAD = C::AHEAD;
    static_assert(AHEAD <= FR, "no block is fetched twice");
    const uint64_t offset = a.drop.top ? drop_offset(a.drop) : 0;
    float* blk = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
    const int gr = lane % GR, rr = lane / GR;
    const int c = col0 + wc * WCOLS + gr * 8, n = min(8, a.C - c);
    constexpr bool P8 = KEPT && PROD == DGRAD;
    Raw8<T> add[AHEAD][PASS];
    Pre8<T, P8> pre[AHEAD][PASS];
    const auto fetch = [&](int j) {
#pragma unroll
      for (int s = 0; s < PASS; ++s) {
        const long r = row0 + (wr * FR + j) * 32 + rr + s * RPP;
        if (r < a.R && n > 0) {
          constexpr bool NTL = C::NT && PROD == DGRAD;
          if (a.add) add[j % AHEAD][s] = get8<T, NTL>(a.add + r * a.ldadd + c, n);
          if constexpr (P8) {
            if (a.codes) {
              pre[j % AHEAD][s].q = *reinterpret_cast<const uint2*>(a.codes + r * a.kp + c);
              pre[j % AHEAD][s].scale = a.scales[r * (a.kp / kMicroBlock) + c / kMicroBlock];
            }
          } else {
            if (PROD == DGRAD && a.pre) pre[j % AHEAD][s].raw = get8<T, NTL>(a.pre + r * a.ldpre + c, n);
          }
        }
      }
    };
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) fetch(j);
    __syncthreads();  // the ring is no longer read
#pragma unroll
    for (int j = 0; j < FR; ++j) {
#pragma unroll
      for (int i = 0; i < FC; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<float4*>(blk + l32 * PITCH + i * 32 + g * 8 + half * 4) =
              make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
      wave_sync();
#pragma unroll
      for (int s = 0; s < PASS; ++s) {
        const int r = row0 + (wr * FR + j) * 32 + rr + s * RPP;
        float v[8];
        const float4 lo = *reinterpret_cast<const float4*>(blk + (rr + s * RPP) * PITCH + gr * 8);
        const float4 hi = *reinterpret_cast<const float4*>(blk + (rr + s * RPP) * PITCH + gr * 8 + 4);
        v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
        if (r < a.R && n > 0) epilogue8<T, PROD, C::NT>(a, offset, r, c, n, v, add[j % AHEAD][s], pre[j % AHEAD][s]);
      }
      wave_sync();
      if (j + AHEAD < FR) fetch(j + AHEAD);
    }
  }
}

template <class T, class C, int PROD, bool KEPT>
__global__ __launch_bounds__(C::NW * 64, C::WPE) void k_dense(GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  dense_tile<T, C, PROD, KEPT>(a, xcd_order(blockIdx.x, gridDim.x), lds);
}

// The two products of the backward in one launch: nd tiles of the data gradient `d`, and the
// weight gradient `w`'s, which do not depend on them.  Each XCD gets its run of both, the weight
// gradient's long tiles first, so that the data gradient's short ones fill the gaps behind them
// and one tail replaces two (65536 x 1024 x 1024: 374 us; two launches 383; every third
// workgroup a weight gradient's 394).
template <class T, class CD, class CW, bool KD, bool KW>
__global__ __launch_bounds__(CD::NW * 64, CD::WPE) void k_dense_bwd(GemmArgs d, GemmArgs w, int nd) {
  static_assert(CD::NW == CW::NW, "one workgroup shape");
  __shared__ __attribute__((aligned(1024))) char lds[std::max(CD::LDS, CW::LDS)];
  const int n = gridDim.x, x = blockIdx.x & 7, i = blockIdx.x >> 3;
  const int count = (n >> 3) + (x < (n & 7)), first = x * (n >> 3) + min(x, n & 7);  // this XCD's workgroups
  const int dcount = (nd >> 3) + (x < (nd & 7)), dfirst = x * (nd >> 3) + min(x, nd & 7);
  const int wcount = count - dcount;
  if (i < wcount)
    dense_tile<T, CW, WGRAD, KW>(w, first - dfirst + i, lds);
  else
    dense_tile<T, CD, DGRAD, KD>(d, dfirst + i - wcount, lds);
}

// ---------------------------------------------------------------------------------------
// Operands whose rows are not whole aligned vectors are copied once, rows padded with zeros: the
// direct loads to LDS take whole 16-byte units only (4099 x 479 and 1001 x 479: 5.1 us, beside
// 24.7 for the product; its floor in memory 5.8 us).
// ---------------------------------------------------------------------------------------
struct PackJob {
  const uint16_t* src;
  uint16_t* dst;
  long ld, rows;
  int cols, vecs;
  unsigned blocks;  // 0: nothing to copy
};
__device__ inline void pack_rows(const PackJob& j, unsigned blk) {
  const long i = static_cast<long>(blk) * 256 + threadIdx.x;
  const long r = i / j.vecs;
  const int v = static_cast<int>(i - r * j.vecs);
  if (r >= j.rows) return;
  // (bits: one loader serves both 16-bit types)
  reinterpret_cast<u32x4*>(j.dst)[i] = load8_raw<BF16T>(j.src + r * j.ld + v * 8, j.cols - v * 8).v[0];
}
__global__ __launch_bounds__(256) void k_pack(PackJob a, PackJob b, PackJob c) {
  unsigned blk = blockIdx.x;
  PackJob j = a;
  if (blk >= a.blocks) {
    blk -= a.blocks;
    j = b;
    if (blk >= b.blocks) {
      blk -= b.blocks;
      j = c;
    }
  }
  pack_rows(j, blk);
}

// out[i] = the sum over p < parts of part[p][i], i < n: 16 threads share one vector's parts
// (thread s: parts s, s + 16, ...), their sums are added in thread order.
struct Sums {
  const float* part;
  float* out;
  long n;
  int parts;
};
template <int VEC>
__device__ inline void sum_parts(const Sums& a, long blk, float (&red)[16][65]) {
  const int cv = threadIdx.x & 15, s = threadIdx.x >> 4;
  const long c = (blk * 16 + cv) * VEC;
  float v[VEC] = {};
  if (c < a.n)
#pragma unroll 4
    for (int p = s; p < a.parts; p += 16) {
      float x[VEC];
      __builtin_memcpy(x, __builtin_assume_aligned(a.part + p * a.n + c, 4 * VEC), sizeof x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] += x[e];
    }
#pragma unroll
  for (int e = 0; e < VEC; ++e) red[s][cv * VEC + e] = v[e];
  __syncthreads();
  if (threadIdx.x < 16 * VEC) {
    const long i = blk * 16 * VEC + threadIdx.x;
    if (i < a.n) {
      float t = red[0][threadIdx.x];
      for (int k = 1; k < 16 && k < a.parts; ++k) t += red[k][threadIdx.x];
      a.out[i] = t;
    }
  }
}
// The weight gradient's partials (the first `blocks` workgroups) and the bias gradient's.
template <int VEC>
__global__ __launch_bounds__(256) void k_sum_parts(Sums w, Sums b, int blocks) {
  __shared__ float red[16][65];
  const int blk = blockIdx.x;
  if (blk < blocks) sum_parts<VEC>(w, blk, red);
  else sum_parts<1>(b, blk - blocks, red);
}

__global__ __launch_bounds__(256) void k_zero(float* p, long n) {
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

void launch_zero(float* p, long n, hipStream_t st) {
  hipLaunchKernelGGL(k_zero, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st, p, n);
}

// ---------------------------------------------------------------------------------------
// Plans and launches.
// ---------------------------------------------------------------------------------------
long ceil_div(long a, long b) { return (a + b - 1) / b; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
long pad8(long n) { return (n + 7) / 8 * 8; }

constexpr int kMaxCols = 1 << 20;  // widest layer; a stage of 256 rows then spans at most 2^30 bytes

enum Shape { SHAPE_L, SHAPE_M, SHAPE_S };
constexpr int kEdge[3] = {256, 128, 64};

// Forward and data gradient: the largest tile that still gives every CU one.
Shape plan_tiles(long R, long C) {
  for (Shape s : {SHAPE_L, SHAPE_M})
    if (ceil_div(R, kEdge[s]) * ceil_div(C, kEdge[s]) >= 256) return s;
  return SHAPE_S;
}

// Weight gradient: tiles x batch slices that fill the CUs once (L) or twice.  A slice has to be
// long enough to pay for its fp32 partial tile, which is written and read again: at 1024 x 1024
// the shapes meet near 2048 rows a slice for L (16384 rows: L 63 us, M 55; 65536: 156, 167) and
// near 512 for M (4096 rows: M 32, S 33; 2048: 31, 27).  Beside the data gradient's L tiles
// (`shared`) half the CUs are enough: the others begin with those tiles, and the partials halve
// (65536 x 1024 x 1024, both products: 382 us against 390; 65536 x 512 x 1024: 192, 206).
struct WgradPlan {
  Shape shape;
  int splits, per, db_rows;
  size_t dw_bytes, bytes;
};
WgradPlan plan_wgrad(int M, int K, int N, bool shared) {
  WgradPlan p{};
  long splits = 1;
  for (Shape s : {SHAPE_L, SHAPE_M, SHAPE_S}) {
    const long tiles = ceil_div(N, kEdge[s]) * ceil_div(K, kEdge[s]);
    splits = std::max<long>(1, (s != SHAPE_L ? 512 : shared ? 128 : 256) / tiles);
    p.shape = s;
    if (s == SHAPE_S) splits = std::min(splits, ceil_div(M, 256));
    else if (M / splits >= (s == SHAPE_L ? 2048 : 512)) break;
  }
  p.per = static_cast<int>(std::min(ceil_div(ceil_div(M, splits), 64) * 64, (1l << 31) - 64));
  p.splits = static_cast<int>(ceil_div(M, p.per));
  const int wc = p.shape == SHAPE_L ? CfgL::WC : p.shape == SHAPE_M ? CfgM::WC : CfgS::WC;
  p.db_rows = p.splits * static_cast<int>(ceil_div(K, kEdge[p.shape])) * wc;
  p.dw_bytes = round256(static_cast<size_t>(p.splits) * N * K * 4);
  p.bytes = p.dw_bytes + round256(static_cast<size_t>(p.db_rows) * N * 4);
  return p;
}

// What one launch takes of the forward's and the data gradient's R x C outputs (shape L, where there
// are many); the weight gradient's, N K < 2^29 of them, are always fewer.
bool tiles_fit(long R, long C) { return ceil_div(R, kEdge[SHAPE_L]) * ceil_div(C, kEdge[SHAPE_L]) < (1l << 21); }
el_status too_many_tiles(const char* fn) { return tower::unsupported(fn, "an output must have fewer than 2^21 tiles of 256 x 256"); }

// Tiles of `a` (all splits) in shape C.
template <class C>
int set_tiles(GemmArgs& a, int splits) {
  a.tiles_c = static_cast<int>(ceil_div(a.C, C::BC));
  a.tiles = static_cast<int>(ceil_div(a.R, C::BR) * a.tiles_c);
  return a.tiles * splits;
}

template <class T, class C, int PROD, bool KEPT>
el_status launch_tiles(const char* fn, GemmArgs a, int splits, hipStream_t st) {
  const int n = set_tiles<C>(a, splits);
  hipLaunchKernelGGL((k_dense<T, C, PROD, KEPT>), dim3(n), dim3(C::NW * 64), 0, st, a);
  return check_launch(fn);
}
template <class T, int PROD, bool KEPT = false>
el_status launch_product(const char* fn, const GemmArgs& a, Shape s, int splits, hipStream_t st) {
  using S = std::conditional_t<KEPT, CfgS2, CfgS>;
  return s == SHAPE_L   ? launch_tiles<T, CfgL, PROD, KEPT>(fn, a, splits, st)
         : s == SHAPE_M ? launch_tiles<T, CfgM, PROD, KEPT>(fn, a, splits, st)
                        : launch_tiles<T, S, PROD, KEPT>(fn, a, splits, st);
}

template <class T, class CD, class CW, bool KD, bool KW>
el_status launch_both(const char* fn, GemmArgs d, GemmArgs w, int splits, hipStream_t st) {
  const int nd = set_tiles<CD>(d, 1), nw = set_tiles<CW>(w, splits);
  hipLaunchKernelGGL((k_dense_bwd<T, CD, CW, KD, KW>), dim3(nd + nw), dim3(CD::NW * 64), 0, st, d, w, nd);
  return check_launch(fn);
}
// The backward's two products: in one launch where their workgroups have one shape.
template <class T, bool KEPT = false>
el_status launch_backward(const char* fn, const GemmArgs& d, Shape sd, const GemmArgs& w, Shape sw, int splits, hipStream_t st) {
  if (sd == SHAPE_L && sw == SHAPE_L) return launch_both<T, CfgL, CfgL, KEPT, KEPT>(fn, d, w, splits, st);
  using S = std::conditional_t<KEPT, CfgS2, CfgS>;
  if (sd == SHAPE_M && sw == SHAPE_M) return launch_both<T, CfgM, CfgM, KEPT, KEPT>(fn, d, w, splits, st);
  if (sd == SHAPE_S && sw == SHAPE_S) return launch_both<T, S, S, KEPT, KEPT>(fn, d, w, splits, st);
  const el_status s = launch_product<T, DGRAD, KEPT>(fn, d, sd, 1, st);
  return s == EL_OK ? launch_product<T, WGRAD, KEPT>(fn, w, sw, splits, st) : s;
}

bool wgrad_shares(long M, long K, const void* dx) { return dx && plan_tiles(M, K) == SHAPE_L; }

// The operand as the tile kernels take it: 16-byte aligned rows of whole vectors.
bool whole_vectors(const void* p, int64_t ld, int64_t cols) {
  return tower::al(p, 16) && ld % 8 == 0 && cols % 8 == 0 && ld <= 2 * kMaxCols;
}
size_t packed_bytes(long rows, long cols) { return round256(static_cast<size_t>(rows) * pad8(cols) * 2); }

// The copies that a call's operands need, in one launch: `add` an operand, its pointer and stride
// become the copy's behind `ws` (which moves on) unless it is whole already, then `run`.
struct Packs {
  PackJob job[3] = {};
  int n = 0;
  void add(const uint16_t** p, long* ld, long rows, int cols, char** ws) {
    if (whole_vectors(*p, *ld, cols)) return;
    const int vecs = static_cast<int>(pad8(cols) / 8);
    uint16_t* dst = reinterpret_cast<uint16_t*>(*ws);
    job[n++] = PackJob{*p, dst, *ld, rows, cols, vecs, static_cast<unsigned>(std::min<long>(ceil_div(rows * vecs, 256), 1l << 24))};
    *p = dst;
    *ld = vecs * 8l;
    *ws += packed_bytes(rows, cols);
  }
  el_status run(const char* fn, hipStream_t st) const {
    const long blocks = static_cast<long>(job[0].blocks) + job[1].blocks + job[2].blocks;
    if (blocks == 0) return EL_OK;
    if (blocks >= (1l << 24)) return tower::unsupported(fn, "unaligned operands of more than 2^35 elements");
    hipLaunchKernelGGL(k_pack, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, job[0], job[1], job[2]);
    return check_launch(fn);
  }
};

void launch_sums(const Sums& w, const Sums& b, hipStream_t st) {
  const bool vec = w.n % 4 == 0;
  const long nw = ceil_div(w.n, vec ? 64 : 16), nb = ceil_div(b.n, 16);
  if (nw + nb == 0) return;
  const dim3 grid(static_cast<unsigned>(nw + nb));
  if (vec) hipLaunchKernelGGL((k_sum_parts<4>), grid, dim3(256), 0, st, w, b, static_cast<int>(nw));
  else hipLaunchKernelGGL((k_sum_parts<1>), grid, dim3(256), 0, st, w, b, static_cast<int>(nw));
}

bool dense_sizes_ok(int32_t M, int32_t K, int32_t N) {
  return M >= 1 && K >= 1 && N >= 1 && K <= kMaxCols && N <= kMaxCols && static_cast<int64_t>(N) * K < (int64_t{1} << 29);
}

// The sizes and the type of a dense layer.
el_status check_dense_sizes(const char* fn, int32_t M, int32_t K, int32_t N, el_dtype dtype) {
  if (dtype != EL_BF16 && dtype != EL_F16) {
    if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
    return tower::unsupported(fn, "dtype must be EL_BF16 or EL_F16");
  }
  if (M < 0) return tower::bad(fn, "M must be >= 0");
  if (K < 1) return tower::bad(fn, "K must be >= 1");
  if (N < 1) return tower::bad(fn, "N must be >= 1");
  if (!dense_sizes_ok(std::max(M, 1), K, N)) return tower::unsupported(fn, "K and N must be <= 2^20 and N * K < 2^29");
  return EL_OK;
}

el_status check_dense_layer(const char* fn, const void* x, int64_t ldx, int32_t M, int32_t K, const void* w, int32_t N,
                            uint32_t act, el_dtype dtype) {
  EL_TRY(check_dense_sizes(fn, M, K, N, dtype));
  if (!w) return tower::bad(fn, "w is null");
  if (!tower::al(w, 2)) return tower::bad(fn, "w must be aligned to its elements");
  EL_TRY(tower::check_act(fn, act));
  return tower::check_rows(fn, "x", x, ldx, K, M > 0, 2);
}

const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

// Device bytes of the copies that these operands need (none when they are whole vectors).
size_t copy_bytes(const void* p, int64_t ld, long rows, long cols) {
  return whole_vectors(p, ld, cols) ? 0 : packed_bytes(rows, cols);
}

}  // namespace
}  // namespace el
