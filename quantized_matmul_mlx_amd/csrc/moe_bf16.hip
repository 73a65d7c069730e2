// The layer of a mixture of experts in bf16 (moe_few_impl.h: few rows an expert, moe_gemm_impl.h: many).
#include "moe_gemm_impl.h"

namespace qaff {

hipError_t launch_moe_ffn_bf16(const MoeArgs& a, hipStream_t stream) { return launch_moe<false>(a, stream); }

size_t moe_ffn_workspace(int64_t tokens, int64_t width, int64_t hidden, int64_t top_k, int64_t experts) {
    return (size_t)moe_gemm_space(tokens, width, hidden, top_k, experts).bytes;  // the few rows' is smaller
}

hipError_t launch_moe_ffn(const MoeArgs& a, bool f16, hipStream_t stream) {
    return f16 ? launch_moe_ffn_f16(a, stream) : launch_moe_ffn_bf16(a, stream);
}

}  // namespace qaff
