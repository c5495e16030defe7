// linear_fwd.cu -- the tensor-core kernels of y = act(x w^T + b) + residual.
#include "linear_tc.cuh"

namespace moe {

cudaError_t lin_launch_fwd(const LinArgs& a, const LtPlan& p, const LtMaps& m, bool tma, cudaStream_t s) {
    return a.a[1] ? lt_launch<LIN_FWD, true>(a, p, m, tma, s) : lt_launch<LIN_FWD, false>(a, p, m, tma, s);
}

cudaError_t lin_allow_fwd(int bytes) {
    const cudaError_t e = lt_allow<LIN_FWD, false>(bytes);
    return e == cudaSuccess ? lt_allow<LIN_FWD, true>(bytes) : e;
}

}  // namespace moe
