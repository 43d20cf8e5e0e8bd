// block_norm_fwd_f16.hip -- the block norm's forward kernels for one type of data.
#include "block_norm_fwd.hpp"

namespace el {
template void launch_norm_fwd<F16T>(const NormArgs&, bool, hipStream_t);
}
