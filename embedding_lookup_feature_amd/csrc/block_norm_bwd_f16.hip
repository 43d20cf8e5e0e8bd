// block_norm_bwd_f16.hip -- the block norm's backward kernels for one type of data.
#include "block_norm_bwd.hpp"

namespace el {
template void launch_norm_bwd<F16T>(const NormArgs&, const JoinArgs&, bool, bool, bool, int, hipStream_t);
}
