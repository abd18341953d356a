// attention_f16.hip -- the attention kernels for fp16 tensors.
#include "attention_launch.hpp"

namespace finetune {
template int launch_fwd<F16>(const FwdCall&);
template int launch_bwd<F16>(const BwdCall&);
}  // namespace finetune
