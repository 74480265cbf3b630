// linear_pair_forward.cu -- instances of linear_pair.cuh for C = A B with the
// full epilogue, one per activation.
#include "linear_pair.cuh"

namespace gbr {

void* linear_pair_forward_kernel(int act) {
    using namespace linear;
    switch (act) {
        case kActRelu: return reinterpret_cast<void*>(&linear_pair_kernel<false, true, kActRelu, false>);
        case kActGelu: return reinterpret_cast<void*>(&linear_pair_kernel<false, true, kActGelu, false>);
        case kActGeluTanh: return reinterpret_cast<void*>(&linear_pair_kernel<false, true, kActGeluTanh, false>);
        case kActSilu: return reinterpret_cast<void*>(&linear_pair_kernel<false, true, kActSilu, false>);
        default: return reinterpret_cast<void*>(&linear_pair_kernel<false, true, kActNone, false>);
    }
}

}  // namespace gbr
