// The forward and backward kernels whose rows see first keys beside their
// window, in a translation unit of their own (they compile beside the others).
#include "launch.cuh"

namespace tab_host {

attn_status_t dispatch_fwd_sinks(const tab::FwdParams &p, int grid, int D, int exp_mode, int mod,
                                 cudaStream_t stream) {
    if (D == 128) return dispatch_exp<128, kStagesD128, true>(p, grid, exp_mode, mod, stream);
    return dispatch_exp<64, kStagesD64, true>(p, grid, exp_mode, mod, stream);
}

attn_status_t dispatch_bwd_sinks(const tab::BwdParams &p, int D, int mod, cudaStream_t stream) {
    return D == 128 ? dispatch_bwd<128, true>(p, mod, stream) : dispatch_bwd<64, true>(p, mod, stream);
}

}  // namespace tab_host
