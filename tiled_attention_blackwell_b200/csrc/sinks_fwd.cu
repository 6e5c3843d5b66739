// The forward kernels whose rows see first keys beside their window.
#include "launch.cuh"

attn_status_t tab_host::dispatch_fwd_sinks(const tab::FwdParams &p, int grid, int D, int exp_mode,
                                           int mod, cudaStream_t stream) {
    return D == 128 ? dispatch_exp<128, kStagesD128, 1>(p, grid, exp_mode, mod, stream)
                    : dispatch_exp<64, kStagesD64, 1>(p, grid, exp_mode, mod, stream);
}
