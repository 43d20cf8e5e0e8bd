// block_norm_fwd_bf16.hip -- the block norm's forward kernels for one type of data.
#include "block_norm_fwd.hpp"

namespace el {
template void launch_norm_fwd<BF16T>(const NormArgs&, bool, hipStream_t);
}
