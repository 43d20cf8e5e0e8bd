// block_norm_bwd_f32.hip -- the block norm's backward kernels for one type of data.
#include "block_norm_bwd.hpp"

namespace el {
template void launch_norm_bwd<F32T>(const NormArgs&, const JoinArgs&, bool, bool, bool, int, hipStream_t);
}
