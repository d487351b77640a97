// wkv7_gnorm_bwd_bf16.hip -- gradients of the group norm, bf16 tokens.

#include "wkv7_gnorm_bwd.h"

namespace wkv7 {

hipError_t launch_gnorm_backward_bf16(const GnArgs& p, hipStream_t stream) {
    WKV7_GN_BF16
    return hipErrorInvalidValue;
}

}  // namespace wkv7
