// The layer of a mixture of experts in float16 (moe_few_impl.h).
#include "moe_few_impl.h"

namespace qaff {

hipError_t launch_moe_ffn_f16(const MoeArgs& a, hipStream_t stream) { return launch_moe<true>(a, stream); }

}  // namespace qaff
