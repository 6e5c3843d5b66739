// The backward kernels whose rows see first keys beside their window.
#include "launch.cuh"

attn_status_t tab_host::dispatch_bwd_sinks(const tab::BwdParams &p, int D, int mod, cudaStream_t stream) {
    return D == 128 ? dispatch_bwd<128, true>(p, mod, stream) : dispatch_bwd<64, true>(p, mod, stream);
}
