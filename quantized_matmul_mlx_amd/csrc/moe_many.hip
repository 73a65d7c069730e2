// The layer of a mixture of experts for many rows an expert (moe_gemm_impl.h).
#include "moe_gemm_impl.h"

namespace qaff {

hipError_t launch_moe_many(const MoeArgs& a, bool f16, hipStream_t stream) {
    switch (a.bits) {
        case 1: return launch_gemm_path<1>(a, f16, stream);
        case 2: return launch_gemm_path<2>(a, f16, stream);
        case 3: return launch_gemm_path<3>(a, f16, stream);
        case 4: return launch_gemm_path<4>(a, f16, stream);
        case 5: return launch_gemm_path<5>(a, f16, stream);
        case 6: return launch_gemm_path<6>(a, f16, stream);
        case 8: return launch_gemm_path<8>(a, f16, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace qaff
