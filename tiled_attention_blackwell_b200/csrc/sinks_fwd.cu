// The forward under a window with first keys that stay visible.
#include "launch.cuh"

attn_status_t tab_host::dispatch_fwd_sinks(const tab::WindowParams &p, int D, int exp_mode, int mod,
                                           cudaStream_t stream) {
    return D == 128 ? dispatch_window<128, kStagesD128, false>(p, exp_mode, mod, stream)
                    : dispatch_window<64, kStagesD64, false>(p, exp_mode, mod, stream);
}
