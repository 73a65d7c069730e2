// The layer of a mixture of experts for few rows an expert, in bf16 (moe_few_impl.h).
#include "moe_few_impl.h"

namespace qaff {

hipError_t launch_moe_few_bf16(const MoeArgs& a, hipStream_t stream) { return launch_few_any<false>(a, stream); }

}  // namespace qaff
