// The layer of a mixture of experts: which kernels serve a call (moe_few_impl.h: few rows an expert, moe_gemm_impl.h:
// many), and its workspace.
#include "moe_gemm_impl.h"

namespace qaff {

size_t moe_ffn_workspace(int64_t tokens, int64_t width, int64_t hidden, int64_t top_k, int64_t experts) {
    return (size_t)moe_gemm_space(tokens, width, hidden, top_k, experts).bytes;  // the few rows' is smaller
}

hipError_t launch_moe_ffn(const MoeArgs& a, bool f16, hipStream_t stream) {
    if (a.top_k == 0 || a.experts == 0 || a.hidden == 0)
        return f16 ? launch_combine<true>(a, nullptr, stream) : launch_combine<false>(a, nullptr, stream);
    if (gemm_path(a)) return launch_moe_many(a, f16, stream);
    return f16 ? launch_moe_few_f16(a, stream) : launch_moe_few_bf16(a, stream);
}

}  // namespace qaff
