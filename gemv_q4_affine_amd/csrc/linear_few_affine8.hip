// linear_few_affine8.hip -- the few-row product (linear_few.hpp) on its format.
#include "linear_few.hpp"

namespace q4 {

hipError_t launch_few_affine8(const LinearArgs& a, hipStream_t s) { return few_format<WF_AFFINE8>(a, s); }

}  // namespace q4
