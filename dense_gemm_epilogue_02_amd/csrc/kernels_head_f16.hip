// kernels_head_f16.hip -- the products of the output head's losses in f16
#include "head_kernels.hpp"

namespace mg {

const HeadLaunch &head_launch_f16() { return HeadKernels<FAM_F16>::table; }

}  // namespace mg
