// attention_bf16.hip -- the attention kernels for bf16 tensors.
#include "attention_launch.hpp"

namespace finetune {
template int launch_fwd<Bf16>(const FwdCall&);
template int launch_bwd<Bf16>(const BwdCall&);
}  // namespace finetune
