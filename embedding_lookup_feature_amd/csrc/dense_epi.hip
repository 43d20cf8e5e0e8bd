// dense_epi.hip -- a dense layer with bias, activation, dropout and residual in its epilogue,
// and its backward.
//
//   forward      y  = residual + drop(act(x w^T + bias)),  pre = x w^T + bias
//   data grad    dx = dz w + dres,  dzb = drop(dx * act'(pre))
//   weight grad  dw = dz^T x,  db = column sums of dz
//
// The three products are one kernel over operands P (output rows) and Q (output columns),
// out[r][c] = sum_k P(r, k) Q(c, k), each operand either reduction-contiguous (element (i, k)
// at i * ld + k: x, dz and w in the first two) or output-contiguous (at k * ld + i).
//
// Operands travel from global memory straight into LDS (no staging registers, no LDS store
// instructions), `ST` stages of BK reductions in a ring; a stage's slot is refilled as soon as
// every wavefront holds its last fragments in registers.  Reduction-contiguous fragments are
// plain 16-byte LDS reads, output-contiguous ones gfx950's transposing LDS reads, both from
// layouts whose 16-byte units are permuted so that the reads touch every bank once.
//
// What bounds it: the large products run at the matrix units' rate under the power limit (65536 x
// 1024 x 1024 bf16, y alone stored: 148 us, a library's product 115; with operands of zeros, the
// same work, 107 and 87), and behind each tile's products its epilogue moves residual, pre and y at
// the memory's rate with the matrix units idle, the generator and the activation beside it: 215 us
// forward with GELU, dropout, residual and pre, 363 us for both products of the backward, their
// partials' sums included (floors 121 and 242 of products, 105 and 158 of memory).
#include <algorithm>

#include "tower_common.hpp"

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

template <class T, int PROD, bool NT>
__device__ inline void epilogue8(const GemmArgs& a, uint64_t offset, long r, int c, int n, float (&v)[8],
                                 const Raw8<T>& add, const Raw8<T>& pre) {
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
      to_floats<T>(pre, f);
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

// One tile (of one split): `lid` in tiles of all splits, in the order that shares panels.
template <class T, class C, int PROD>
__device__ __forceinline__ void dense_tile(const GemmArgs& a, int lid, char* lds) {
  constexpr int NW = C::NW, FR = C::FR, FC = C::FC, BK = C::BK, ST = C::ST, WC = C::WC;
  using OP = Operand<C::BR, BK, PROD != WGRAD, NW>;
  using OQ = Operand<C::BC, BK, PROD == FWD, NW>;
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
  oq.init(a.Q, a.ldq, col0, a.C, kbeg, min(kend, a.red_q), wave, lane);
  const lds_char* base = (const lds_char*)lds;
  const uint32_t mine = uniform(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(base)) + wave * 1024);
  const auto load_one = [&](int m, uint32_t slot, const u32x4& rp, const u32x4& rq) {
    if (m < OP::N) op.load(mine + slot, m, rp);
    else oq.load(mine + slot + OP::BYTES, m - OP::N, rq);
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
    const u32x4 rp = op.rsrc(), rq = oq.rsrc();
#pragma unroll
    for (int m = 0; m < LOADS; ++m) load_one(m, s * SB, rp, rq);
    op.advance();
    oq.advance();
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
    const u32x4 rp = op.rsrc(), rq = oq.rsrc();
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
    Raw8<T> add[AHEAD][PASS], pre[AHEAD][PASS];
    const auto fetch = [&](int j) {
#pragma unroll
      for (int s = 0; s < PASS; ++s) {
        const long r = row0 + (wr * FR + j) * 32 + rr + s * RPP;
        if (r < a.R && n > 0) {
          constexpr bool NTL = C::NT && PROD == DGRAD;
          if (a.add) add[j % AHEAD][s] = get8<T, NTL>(a.add + r * a.ldadd + c, n);
          if (PROD == DGRAD && a.pre) pre[j % AHEAD][s] = get8<T, NTL>(a.pre + r * a.ldpre + c, n);
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

template <class T, class C, int PROD>
__global__ __launch_bounds__(C::NW * 64, C::WPE) void k_dense(GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  dense_tile<T, C, PROD>(a, xcd_order(blockIdx.x, gridDim.x), lds);
}

// The two products of the backward in one launch: nd tiles of the data gradient `d`, and the
// weight gradient `w`'s, which do not depend on them.  Each XCD gets its run of both, the weight
// gradient's long tiles first, so that the data gradient's short ones fill the gaps behind them
// and one tail replaces two (65536 x 1024 x 1024: 374 us; two launches 383; every third
// workgroup a weight gradient's 394).
template <class T, class CD, class CW>
__global__ __launch_bounds__(CD::NW * 64, CD::WPE) void k_dense_bwd(GemmArgs d, GemmArgs w, int nd) {
  static_assert(CD::NW == CW::NW, "one workgroup shape");
  __shared__ __attribute__((aligned(1024))) char lds[std::max(CD::LDS, CW::LDS)];
  const int n = gridDim.x, x = blockIdx.x & 7, i = blockIdx.x >> 3;
  const int count = (n >> 3) + (x < (n & 7)), first = x * (n >> 3) + min(x, n & 7);  // this XCD's workgroups
  const int dcount = (nd >> 3) + (x < (nd & 7)), dfirst = x * (nd >> 3) + min(x, nd & 7);
  const int wcount = count - dcount;
  if (i < wcount)
    dense_tile<T, CW, WGRAD>(w, first - dfirst + i, lds);
  else
    dense_tile<T, CD, DGRAD>(d, dfirst + i - wcount, lds);
}

// ---------------------------------------------------------------------------------------
// Few outputs (a forward of one to a few hundred rows): the weights' bytes and latency count.  A
// workgroup's wavefronts share out the reduction of one 16 x 16 tile, fragments straight from
// global memory (64 contiguous bytes of a row per read), and the partial tiles are added in
// wavefront order in LDS.  Any alignment.  1 x 1024 x 1024 takes 4.2 us and 77 x 512 x 1024 4.7
// (an empty kernel 2.1): a round of loads or two and a barrier, no longer the bytes.
// ---------------------------------------------------------------------------------------
constexpr int kFewWaves = 8;

template <class T>
__device__ inline f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  if constexpr (T::code == EL_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <class T>
__global__ __launch_bounds__(kFewWaves * 64) void k_dense_few(GemmArgs a) {
  constexpr int PITCH = 20, AHEAD = 4;
  __shared__ float lds[kFewWaves][16 * PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int tr = blockIdx.x / a.tiles_c, tc = blockIdx.x - tr * a.tiles_c;
  const int row0 = tr * 16, col0 = tc * 16;
  const int k0 = wave * a.per_split, kend = min(a.red, k0 + a.per_split);
  const uint16_t* q = a.Q + static_cast<long>(min(col0 + l16, a.C - 1)) * a.ldq;  // rows past the end: never stored
  const uint16_t* p = a.P + static_cast<long>(min(row0 + l16, a.R - 1)) * a.ldp;
  // the epilogue's operands are on their way while the products run
  const int r = row0 + threadIdx.x / 2, c = col0 + threadIdx.x % 2 * 8, n = min(8, a.C - c);
  const bool mine = threadIdx.x < 32 && r < a.R && n > 0;
  float v[8] = {};
  Raw8<T> add;
  if (mine) {
    if (a.add) add = load8_raw<T>(a.add + r * a.ldadd + c, n);
    if (a.bias)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = a.bias[min(c + e, a.C - 1)];
  }
  f32x4 acc = {};
  for (int k = k0; k < kend; k += 32 * AHEAD) {
    Raw8<T> fq[AHEAD], fp[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int at = k + u * 32 + g * 8;
      if (at < kend) {
        fq[u] = load8_raw<T>(q + at, kend - at);
        fp[u] = load8_raw<T>(p + at, kend - at);
      } else {
        fq[u].v[0] = fp[u].v[0] = u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) acc = mfma16<T>(fq[u].v[0], fp[u].v[0], acc);
  }
  // register e: column 4 g + e of row l16
  *reinterpret_cast<f32x4*>(&lds[wave][l16 * PITCH + g * 4]) = acc;
  __syncthreads();
  if (!mine) return;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += lds[w][threadIdx.x / 2 * PITCH + threadIdx.x % 2 * 8 + e];
  epilogue8<T, FWD, false>(a, a.drop.top ? drop_offset(a.drop) : 0, r, c, n, v, add, add);
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
  const long i = static_cast<long>(blk) * 256 + threadIdx.x;
  const long r = i / j.vecs;
  const int v = static_cast<int>(i - r * j.vecs);
  if (r >= j.rows) return;
  // (bits: one loader serves both 16-bit types)
  reinterpret_cast<u32x4*>(j.dst)[i] = load8_raw<BF16T>(j.src + r * j.ld + v * 8, j.cols - v * 8).v[0];
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

template <class T, class C, int PROD>
el_status launch_tiles(const char* fn, GemmArgs a, int splits, hipStream_t st) {
  const int n = set_tiles<C>(a, splits);
  hipLaunchKernelGGL((k_dense<T, C, PROD>), dim3(n), dim3(C::NW * 64), 0, st, a);
  return check_launch(fn);
}
template <class T, int PROD>
el_status launch_product(const char* fn, const GemmArgs& a, Shape s, int splits, hipStream_t st) {
  return s == SHAPE_L   ? launch_tiles<T, CfgL, PROD>(fn, a, splits, st)
         : s == SHAPE_M ? launch_tiles<T, CfgM, PROD>(fn, a, splits, st)
                        : launch_tiles<T, CfgS, PROD>(fn, a, splits, st);
}

template <class T, class CD, class CW>
el_status launch_both(const char* fn, GemmArgs d, GemmArgs w, int splits, hipStream_t st) {
  const int nd = set_tiles<CD>(d, 1), nw = set_tiles<CW>(w, splits);
  hipLaunchKernelGGL((k_dense_bwd<T, CD, CW>), dim3(nd + nw), dim3(CD::NW * 64), 0, st, d, w, nd);
  return check_launch(fn);
}
// The backward's two products: in one launch where their workgroups have one shape.
template <class T>
el_status launch_backward(const char* fn, const GemmArgs& d, Shape sd, const GemmArgs& w, Shape sw, int splits, hipStream_t st) {
  if (sd == SHAPE_L && sw == SHAPE_L) return launch_both<T, CfgL, CfgL>(fn, d, w, splits, st);
  if (sd == SHAPE_M && sw == SHAPE_M) return launch_both<T, CfgM, CfgM>(fn, d, w, splits, st);
  if (sd == SHAPE_S && sw == SHAPE_S) return launch_both<T, CfgS, CfgS>(fn, d, w, splits, st);
  const el_status s = launch_product<T, DGRAD>(fn, d, sd, 1, st);
  return s == EL_OK ? launch_product<T, WGRAD>(fn, w, sw, splits, st) : s;
}

bool wgrad_shares(long M, long K, const void* dx) { return dx && plan_tiles(M, K) == SHAPE_L; }

// A forward of few outputs: at most 64 tiles of 64 x 64 (512 x 512 x 512: 7.6 us against 9.1 in
// tiles; 300 x 1024 x 1024, 80 tiles: 14.7 against 13.8).
bool plan_few(long M, long N) { return ceil_div(M, 64) * ceil_div(N, 64) <= 64; }

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

el_status check_dense_layer(const char* fn, const void* x, int64_t ldx, int32_t M, int32_t K, const void* w, int32_t N,
                            uint32_t act, el_dtype dtype) {
  if (dtype != EL_BF16 && dtype != EL_F16) {
    if (!dtype_valid(dtype)) return tower::bad(fn, "unknown dtype");
    return tower::unsupported(fn, "dtype must be EL_BF16 or EL_F16");
  }
  if (M < 0) return tower::bad(fn, "M must be >= 0");
  if (K < 1) return tower::bad(fn, "K must be >= 1");
  if (N < 1) return tower::bad(fn, "N must be >= 1");
  if (!dense_sizes_ok(std::max(M, 1), K, N)) return tower::unsupported(fn, "K and N must be <= 2^20 and N * K < 2^29");
  if (!w) return tower::bad(fn, "w is null");
  if (!tower::al(w, 2)) return tower::bad(fn, "w must be aligned to its elements");
  const el_status s = tower::check_act(fn, act);
  if (s != EL_OK) return s;
  return tower::check_rows(fn, "x", x, ldx, K, M > 0, 2);
}

const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

template <class T>
el_status run_fwd(const char* fn, GemmArgs a, char* ws, hipStream_t st) {
  if (plan_few(a.R, a.C)) {
    a.tiles_c = static_cast<int>(ceil_div(a.C, 16));
    a.per_split = static_cast<int>(ceil_div(ceil_div(a.red, kFewWaves), 32) * 32);
    hipLaunchKernelGGL((k_dense_few<T>), dim3(static_cast<unsigned>(ceil_div(a.R, 16) * a.tiles_c)), dim3(kFewWaves * 64), 0,
                       st, a);
    return check_launch(fn);
  }
  Packs packs;
  packs.add(&a.P, &a.ldp, a.R, a.red, &ws);
  packs.add(&a.Q, &a.ldq, a.C, a.red, &ws);
  const el_status s = packs.run(fn, st);
  if (s != EL_OK) return s;
  a.red = static_cast<int>(pad8(a.red));  // the copies' padding is zero; whole rows need none
  a.red_q = a.per_split = a.red;
  return launch_product<T, FWD>(fn, a, plan_tiles(a.R, a.C), 1, st);
}

}  // namespace
}  // namespace el

using namespace el;

namespace {

// Device bytes of the copies that these operands need (none when they are whole vectors).
size_t copy_bytes(const void* p, int64_t ld, long rows, long cols) {
  return whole_vectors(p, ld, cols) ? 0 : packed_bytes(rows, cols);
}

template <class T>
el_status run_bwd(const char* fn, const uint16_t* x, long ldx, int M, int K, const uint16_t* w, int N, const uint16_t* dz,
                  long lddz, GemmArgs a, float* dw, float* db, char* ws, hipStream_t st) {
  Packs packs;
  packs.add(&dz, &lddz, M, N, &ws);
  packs.add(&x, &ldx, M, K, &ws);
  long ldw = K;
  if (a.out) packs.add(&w, &ldw, N, K, &ws);
  EL_TRY(packs.run(fn, st));
  const WgradPlan pl = plan_wgrad(M, K, N, wgrad_shares(M, K, a.out));
  GemmArgs b{};
  b.P = dz, b.ldp = lddz, b.Q = x, b.ldq = ldx, b.R = N, b.C = K, b.red = b.red_q = M, b.per_split = pl.per;
  b.part = pl.splits > 1 ? reinterpret_cast<float*>(ws) : dw;
  float* dbp = reinterpret_cast<float*>(ws + pl.dw_bytes);
  b.dbp = db ? dbp : nullptr;
  if (a.out) {
    // a copied dz has rows that end in zeros; the rows of w behind N read as zeros
    a.P = dz, a.ldp = lddz, a.Q = w, a.ldq = ldw, a.R = M, a.C = K;
    a.red = a.per_split = static_cast<int>(pad8(N));
    a.red_q = N;
    EL_TRY(launch_backward<T>(fn, a, plan_tiles(M, K), b, pl.shape, pl.splits, st));
  } else {
    EL_TRY((launch_product<T, WGRAD>(fn, b, pl.shape, pl.splits, st)));
  }
  launch_sums(Sums{b.part, dw, pl.splits > 1 ? static_cast<long>(N) * K : 0, pl.splits},
              Sums{dbp, db, db ? static_cast<long>(N) : 0, pl.db_rows}, st);
  return check_launch(fn);
}

}  // namespace

extern "C" {

size_t el_dense_fwd_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  if (!dense_sizes_ok(M, K, N) || plan_few(M, N) || !tiles_fit(M, N)) return 0;
  return packed_bytes(M, K) + packed_bytes(N, K);
}

size_t el_dense_bwd_workspace_bytes(int32_t M, int32_t K, int32_t N) {
  if (!dense_sizes_ok(M, K, N)) return 0;
  return packed_bytes(M, N) + packed_bytes(M, K) + packed_bytes(N, K) +
         std::max(plan_wgrad(M, K, N, false).bytes, plan_wgrad(M, K, N, true).bytes);
}

el_status el_dense_fwd(const void* x, int64_t ldx, int32_t M, int32_t K, const void* w, const float* bias, int32_t N,
                       uint32_t act, const el_dropout* drop, const void* residual, int64_t ldr, void* pre,
                       int64_t ldpre, void* y, int64_t ldy, el_dtype dtype, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  const char* fn = "el_dense_fwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_dense_layer(fn, x, ldx, M, K, w, N, act, dtype));
    GemmArgs a{};
    EL_TRY(tower::drop_args(fn, drop, &a.drop));
    if (!tower::al(bias, 4)) return tower::bad(fn, "bias must be aligned to its elements");
    EL_TRY(tower::check_rows(fn, "residual", residual, ldr, N, false, 2));
    EL_TRY(tower::check_rows(fn, "pre", pre, ldpre, N, false, 2));
    EL_TRY(tower::check_rows(fn, "y", y, ldy, N, M > 0, 2));
    if (M == 0) return EL_OK;
    if (!tiles_fit(M, N)) return too_many_tiles(fn);
    const size_t need = plan_few(M, N) ? 0 : copy_bytes(x, ldx, M, K) + copy_bytes(w, K, N, K);
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, need));
    a.P = u16(x), a.ldp = ldx, a.Q = u16(w), a.ldq = K, a.R = M, a.C = N, a.red = K, a.act = act;
    a.add = u16(residual), a.ldadd = ldr, a.aux = static_cast<uint16_t*>(pre), a.ldaux = ldpre;
    a.out = static_cast<uint16_t*>(y), a.ldo = ldy, a.bias = bias;
    char* ws = static_cast<char*>(workspace);
    return dtype == EL_BF16 ? run_fwd<BF16T>(fn, a, ws, stream) : run_fwd<F16T>(fn, a, ws, stream);
  });
}

el_status el_dense_bwd(const void* x, int64_t ldx, int32_t M, int32_t K, const void* w, int32_t N, const void* dz,
                       int64_t lddz, const void* dres, int64_t lddres, void* dx, int64_t lddx, uint32_t act,
                       const el_dropout* drop, const void* pre, int64_t ldpre, void* dzb, int64_t lddzb, float* dw,
                       float* db, el_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "el_dense_bwd";
  return tower::guarded(fn, [&]() -> el_status {
    EL_TRY(check_dense_layer(fn, x, ldx, M, K, w, N, act, dtype));
    GemmArgs a{};
    EL_TRY(tower::drop_args(fn, drop, &a.drop));
    EL_TRY(tower::check_rows(fn, "dz", dz, lddz, N, M > 0, 2));
    EL_TRY(tower::check_rows(fn, "dres", dres, lddres, K, false, 2));
    EL_TRY(tower::check_rows(fn, "dx", dx, lddx, K, false, 2));
    EL_TRY(tower::check_rows(fn, "pre", pre, ldpre, K, dzb && act != EL_ACT_NONE && M > 0, 2));
    EL_TRY(tower::check_rows(fn, "dzb", dzb, lddzb, K, false, 2));
    if ((dzb || dres) && !dx) return tower::bad(fn, "dzb and dres need dx");
    if (!dw || !tower::al(dw, 4) || !tower::al(db, 4)) return tower::bad(fn, "dw must be non-null, dw and db aligned to their elements");
    const long nk = static_cast<long>(N) * K;
    if (M == 0) {  // an empty batch: zero gradients, by a kernel (a captured fill stays a kernel node)
      hipLaunchKernelGGL(k_zero, dim3(static_cast<unsigned>(ceil_div(nk, 256))), dim3(256), 0, stream, dw, nk);
      if (db) hipLaunchKernelGGL(k_zero, dim3(static_cast<unsigned>(ceil_div(N, 256))), dim3(256), 0, stream, db, static_cast<long>(N));
      return check_launch(fn);
    }
    if (dx && !tiles_fit(M, K)) return too_many_tiles(fn);
    const size_t need = copy_bytes(dz, lddz, M, N) + copy_bytes(x, ldx, M, K) + (dx ? copy_bytes(w, K, N, K) : 0) +
                        plan_wgrad(M, K, N, wgrad_shares(M, K, dx)).bytes;
    EL_TRY(tower::check_workspace(fn, workspace, workspace_bytes, need));
    a.add = u16(dres), a.ldadd = lddres, a.out = static_cast<uint16_t*>(dx), a.ldo = lddx, a.act = act;
    a.aux = static_cast<uint16_t*>(dzb), a.ldaux = lddzb, a.pre = dzb && act != EL_ACT_NONE ? u16(pre) : nullptr, a.ldpre = ldpre;
    char* ws = static_cast<char*>(workspace);
    return dtype == EL_BF16
               ? run_bwd<BF16T>(fn, u16(x), ldx, M, K, u16(w), N, u16(dz), lddz, a, dw, db, ws, stream)
               : run_bwd<F16T>(fn, u16(x), ldx, M, K, u16(w), N, u16(dz), lddz, a, dw, db, ws, stream);
  });
}

}  // extern "C"
