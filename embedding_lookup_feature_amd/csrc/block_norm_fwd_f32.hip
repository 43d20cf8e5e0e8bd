// block_norm_fwd_f32.hip -- the block norm's forward kernels for one type of data.
#include "block_norm_fwd.hpp"

namespace el {
template void launch_norm_fwd<F32T>(const NormArgs&, bool, hipStream_t);
}
