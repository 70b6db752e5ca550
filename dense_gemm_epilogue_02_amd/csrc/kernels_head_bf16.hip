// kernels_head_bf16.hip -- the products of the output head's losses in bf16
#include "head_kernels.hpp"

namespace mg {

const HeadLaunch &head_launch_bf16() { return HeadKernels<FAM_BF16>::table; }

}  // namespace mg
