// The layer of a mixture of experts in float16 (moe_few_impl.h: few rows an expert, moe_gemm_impl.h: many).
#include "moe_gemm_impl.h"

namespace qaff {

hipError_t launch_moe_ffn_f16(const MoeArgs& a, hipStream_t stream) { return launch_moe<true>(a, stream); }

}  // namespace qaff
