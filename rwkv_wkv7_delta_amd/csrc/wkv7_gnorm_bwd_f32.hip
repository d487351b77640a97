// wkv7_gnorm_bwd_f32.hip -- gradients of the group norm, fp32 tokens.

#include "wkv7_gnorm_bwd.h"

namespace wkv7 {

hipError_t launch_gnorm_backward_f32(const GnArgs& p, hipStream_t stream) {
    WKV7_GN_F32
    return hipErrorInvalidValue;
}

}  // namespace wkv7
