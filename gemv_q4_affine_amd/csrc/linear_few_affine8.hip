// linear_few_affine8.hip -- the few-row product (linear_few.hpp) on its format.
#include "linear_few.hpp"

namespace q4 {

hipError_t launch_few_affine8(const LinearArgs& a, const FewPlan& p, const FewSplit& split, hipStream_t s) {
    return few_format<WF_AFFINE8>(a, p, split, s);
}

}  // namespace q4
