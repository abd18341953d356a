// attention_f32.hip -- the attention kernels for fp32 tensors.
#include "attention_launch.hpp"

namespace finetune {
template int launch_fwd<F32>(const FwdCall&);
template int launch_bwd<F32>(const BwdCall&);
}  // namespace finetune
