// Calls every entry point of embblock.h with arguments its checks must refuse, and the pure size
// queries over ordinary and extreme sizes, in a build with host sanitizers.  No GPU is touched.
#include <cstdio>
#include <limits>

#include "embblock.h"

static int failures = 0;
static void refuse(el_status s, const char* what) {
  if (s == EL_OK || s == EL_ERR_HIP) {
    std::printf("not refused: %s (%d)\n", what, static_cast<int>(s));
    ++failures;
  }
}

int main() {
  char* const A = reinterpret_cast<char*>(0x7f0000000000ull);
  float* const F = reinterpret_cast<float*>(A);
  uint8_t* const U = reinterpret_cast<uint8_t*>(A);
  const int big = std::numeric_limits<int>::max(), low = std::numeric_limits<int>::min();
  const long lbig = std::numeric_limits<long>::max(), llow = std::numeric_limits<long>::min();
  const float inf = std::numeric_limits<float>::infinity(), nan = std::numeric_limits<float>::quiet_NaN();
  const el_block_norm ok{EL_NORM_RMS, EL_NORM_LAYER, EL_GATE_SIGMOID, 2, 1.f, 1e-5f, F, F, F, F};
  const auto fwd = [&](const el_block_norm* p, int M, int C, long ld, el_dtype dt) {
    return el_block_norm_fwd(p, A, ld, A, ld, A, ld, M, C, A, ld, A, ld, F, F, dt, nullptr);
  };
  const auto bwd = [&](const el_block_norm* p, int M, int C, long ld, el_dtype dt, size_t ws) {
    return el_block_norm_bwd(p, A, ld, A, ld, A, ld, A, ld, A, ld, M, C, F, F, A, ld, A, ld, A, ld, F, F, F, F, dt, A, ws, nullptr);
  };
  for (int dt : {-7, 3, 99, big, low}) {
    const el_dtype d = static_cast<el_dtype>(dt);
    refuse(fwd(&ok, 4, 8, 8, d), "norm dtype");
    refuse(bwd(&ok, 4, 8, 8, d, 1 << 30), "norm bwd dtype");
    refuse(el_ckpt_pack(A, 8, 4, 8, d, U, U, nullptr), "pack dtype");
    refuse(el_ckpt_act_dropout_fwd(U, U, 4, 8, 1, nullptr, A, 8, d, nullptr), "act dtype");
    refuse(el_ckpt_act_dropout_bwd(A, 8, U, U, 4, 8, 1, nullptr, A, 8, d, nullptr), "act bwd dtype");
    refuse(el_dense_bwd_ckpt(U, U, 4, 8, A, 8, A, 8, nullptr, 0, A, 8, 0, nullptr, nullptr, nullptr, nullptr, 0, F, F, d, A, 1, nullptr), "dense dtype");
    refuse(el_fp4_pack(A, 8, 4, 8, d, U, U, nullptr), "fp4 dtype");
    refuse(el_fp4_unpack(U, U, 4, 8, A, 8, d, nullptr), "fp4 unpack dtype");
    refuse(el_dense_fwd_fp4(A, 8, 4, 8, U, U, F, 8, 0, nullptr, 0, A, 8, d, A, 1, nullptr), "fp4 dense dtype");
  }
  for (long ld : {-1l, 7l, lbig, llow}) {
    refuse(fwd(&ok, 4, 8, ld, EL_BF16), "norm ld");
    refuse(bwd(&ok, 4, 8, ld, EL_BF16, 1 << 30), "norm bwd ld");
    refuse(el_ckpt_pack(A, ld, 4, 8, EL_F32, U, U, nullptr), "pack ld");
    refuse(el_ckpt_act_dropout_bwd(A, ld, U, U, 4, 8, 1, nullptr, A, 8, EL_F32, nullptr), "act bwd ld");
    refuse(el_fp4_unpack(U, U, 4, 8, A, ld, EL_F32, nullptr), "unpack ld");
    refuse(el_dense_fwd_fp4(A, ld, 4, 8, U, U, F, 8, 0, nullptr, 0, A, 8, EL_BF16, A, 1, nullptr), "fp4 dense ld");
    refuse(el_dense_bwd_ckpt(U, U, 4, 8, A, 8, A, ld, nullptr, 0, A, 8, 0, nullptr, nullptr, nullptr, nullptr, 0, F, F, EL_BF16, A, 1, nullptr), "dense ld");
  }
  for (float v : {inf, -inf, nan}) {
    el_block_norm p = ok;
    p.scale = v;
    refuse(fwd(&p, 4, 8, 8, EL_BF16), "scale");
    p = ok;
    p.eps = v;
    refuse(bwd(&p, 4, 8, 8, EL_BF16, 1 << 30), "eps");
  }
  for (int n : {low, -1, 0}) {
    el_block_norm p = ok;
    p.gate_rows = n;
    refuse(fwd(&p, 4, 8, 8, EL_BF16), "gate_rows");
    refuse(fwd(&ok, 4, n, 8, EL_BF16), "C");
    refuse(el_ckpt_pack(A, 8, 4, n, EL_F32, U, U, nullptr), "K");
  }
  refuse(bwd(&ok, big, 32768, 32768, EL_F32, 1), "norm workspace");
  refuse(el_ckpt_pack(A, lbig >> 30, big, 1 << 20, EL_F32, U, U, nullptr), "huge pack");
  refuse(el_fp4_pack(A, lbig >> 30, big, 1 << 20, EL_F32, U, U, nullptr), "huge fp4 pack");
  refuse(el_fp4_pack(A, big, big, big, EL_F32, U, U, nullptr), "huge K");
  refuse(el_dense_fwd_fp4(A, big, big, big, U, U, F, big, 0, nullptr, 0, A, big, EL_BF16, A, 1, nullptr), "huge fp4 dense");
  refuse(el_dense_fwd_fp4(A, 1 << 17, 4000, 1 << 17, U, U, F, 4000, 0, nullptr, 0, A, 4000, EL_BF16, A, 1, nullptr), "fp4 dense workspace");
  refuse(el_dense_bwd_ckpt(U, U, big, 1024, A, 1024, A, 1024, nullptr, 0, A, 1024, 0, nullptr, nullptr, nullptr, nullptr, 0, F, F, EL_BF16, A, 1, nullptr), "huge dense bwd");

  size_t sum = 0;
  const int sizes[] = {low, -1, 0, 1, 2, 7, 8, 31, 64, 65, 127, 1000, 1024, 4099, 32768, 32769, 65536, 1 << 20, 1 << 24, big - 1, big};
  for (int a : sizes)
    for (int b : sizes)
      for (int c : sizes) {
        sum += el_block_norm_bwd_workspace_bytes(a, b, c) & 255;
        sum += el_dense_bwd_ckpt_workspace_bytes(a, b, c) & 255;
        sum += el_dense_fwd_fp4_workspace_bytes(a, b, c) & 255;
      }
  if (sum) std::printf("workspace sizes are not multiples of 256\n"), ++failures;
  std::printf(failures ? "failed\n" : "ok\n");
  return failures != 0;
}
