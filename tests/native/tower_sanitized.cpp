// Calls every entry point of embtower.h with arguments its checks must refuse, and the pure size
// queries over ordinary and extreme sizes, in a build with host sanitizers.  No GPU is touched.
#include <cstdio>
#include <cstdlib>
#include <limits>

#include "embtower.h"

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
  const int big = std::numeric_limits<int>::max(), low = std::numeric_limits<int>::min();
  const long lbig = std::numeric_limits<long>::max(), llow = std::numeric_limits<long>::min();
  const el_dropout bad_p{1.5, 1, 2, nullptr}, nan_p{std::numeric_limits<double>::quiet_NaN(), 1, 2, nullptr};
  const el_dropout bad_step{0.5, 1, 2, reinterpret_cast<const uint64_t*>(A + 1)};

  for (int dt : {-7, 3, 99, big, low}) {
    refuse(el_act_dropout_fwd(A, 8, nullptr, 0, 4, 8, 0, nullptr, A, 8, static_cast<el_dtype>(dt), nullptr), "fwd dtype");
    refuse(el_act_dropout_bwd(A, 8, A, 8, 4, 8, 1, nullptr, A, 8, static_cast<el_dtype>(dt), nullptr), "bwd dtype");
    refuse(el_dense_fwd(A, 8, 4, 8, A, F, 8, 0, nullptr, nullptr, 0, nullptr, 0, A, 8, static_cast<el_dtype>(dt), A, 1, nullptr), "dense dtype");
    refuse(el_dense_bwd(A, 8, 4, 8, A, 8, A, 8, nullptr, 0, A, 8, 0, nullptr, nullptr, 0, nullptr, 0, F, F, static_cast<el_dtype>(dt), A, 1, nullptr), "dense bwd dtype");
    refuse(el_group_norm_fwd(A, 8, 2, 2, 8, 2, nullptr, F, F, 1e-5f, 0, A, 8, F, F, static_cast<el_dtype>(dt), A, 1, nullptr), "gn dtype");
    refuse(el_group_norm_bwd(A, 8, A, 8, 2, 2, 8, 2, nullptr, F, F, F, F, 0, A, 8, F, F, static_cast<el_dtype>(dt), A, 1, nullptr), "gn bwd dtype");
  }
  for (const el_dropout* d : {&bad_p, &nan_p, &bad_step}) {
    refuse(el_act_dropout_fwd(A, 8, nullptr, 0, 4, 8, 0, d, A, 8, EL_F32, nullptr), "dropout");
    refuse(el_dense_fwd(A, 8, 4, 8, A, F, 8, 0, d, nullptr, 0, nullptr, 0, A, 8, EL_BF16, A, 1, nullptr), "dense dropout");
    refuse(el_dense_bwd(A, 8, 4, 8, A, 8, A, 8, nullptr, 0, A, 8, 0, d, nullptr, 0, A, 8, F, F, EL_BF16, A, 1, nullptr), "dense bwd dropout");
  }
  for (long ld : {-1l, 7l, lbig, llow}) {
    refuse(el_act_dropout_fwd(A, ld, nullptr, 0, 4, 8, 0, nullptr, A, 8, EL_F32, nullptr), "ldx");
    refuse(el_dense_fwd(A, ld, 4, 8, A, F, 8, 0, nullptr, nullptr, 0, nullptr, 0, A, 8, EL_BF16, A, 1, nullptr), "dense ldx");
    refuse(el_dense_bwd(A, 8, 4, 8, A, 8, A, ld, nullptr, 0, A, 8, 0, nullptr, nullptr, 0, nullptr, 0, F, F, EL_BF16, A, 1, nullptr), "lddz");
    refuse(el_group_norm_fwd(A, ld, 2, 2, 8, 2, nullptr, F, F, 1e-5f, 0, A, 8, F, F, EL_F32, A, 1, nullptr), "gn ldx");
    refuse(el_group_norm_bwd(A, ld, A, 8, 2, 2, 8, 2, nullptr, F, F, F, F, 0, A, 8, F, F, EL_F32, A, 1, nullptr), "gn lddy");
  }
  refuse(el_act_dropout_fwd(A, 1l << 39, nullptr, 0, big, big, 0, nullptr, A, 1l << 39, EL_F32, nullptr), "huge");
  refuse(el_dense_fwd(A, big, big, big, A, F, big, 0, nullptr, nullptr, 0, nullptr, 0, A, big, EL_BF16, A, 1, nullptr), "huge dense");
  refuse(el_dense_bwd(A, big, big, big, A, big, A, big, nullptr, 0, A, big, 0, nullptr, nullptr, 0, nullptr, 0, F, F, EL_BF16, A, 1, nullptr), "huge bwd");
  refuse(el_dense_bwd(A, 1024, big, 1024, A, 1024, A, 1024, nullptr, 0, A, 1024, 0, nullptr, nullptr, 0, nullptr, 0, F, F, EL_BF16, A, 1, nullptr), "no workspace");
  refuse(el_group_norm_fwd(A, big, big, big, big, 1, nullptr, F, F, 1e-5f, 0, A, big, F, F, EL_F32, A, 1, nullptr), "huge gn");
  refuse(el_group_norm_bwd(A, 64, A, 64, 1 << 20, 4096, 64, 1, nullptr, F, F, F, F, 0, A, 64, F, F, EL_F32, A, 1, nullptr), "gn workspace");

  size_t sum = 0;
  const int sizes[] = {low, -1, 0, 1, 2, 7, 8, 63, 64, 65, 1000, 1024, 4099, 65536, 1 << 20, 1 << 24, big - 1, big};
  for (int a : sizes)
    for (int b : sizes)
      for (int c : sizes) {
        sum += el_dense_fwd_workspace_bytes(a, b, c) & 255;
        sum += el_dense_bwd_workspace_bytes(a, b, c) & 255;
        for (int g : {1, 8, 1024, big}) {
          sum += el_group_norm_fwd_workspace_bytes(a, b, c, g) & 255;
          sum += el_group_norm_bwd_workspace_bytes(a, b, c, g) & 255;
        }
      }
  if (sum) std::printf("workspace sizes are not multiples of 256\n"), ++failures;
  std::printf(failures ? "failed\n" : "ok\n");
  return failures != 0;
}
