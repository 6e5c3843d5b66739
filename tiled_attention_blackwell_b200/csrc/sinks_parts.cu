// The same for few items: each item's steps in p.parts parts, and their join.
#include "launch.cuh"

attn_status_t tab_host::dispatch_fwd_parts(const tab::WindowParams &p, int D, int exp_mode, int mod,
                                           cudaStream_t stream) {
    const attn_status_t s = D == 128 ? dispatch_window<128, kStagesD128, true>(p, exp_mode, mod, stream)
                                     : dispatch_window<64, kStagesD64, true>(p, exp_mode, mod, stream);
    if (s != ATTN_OK) return s;
    const long long rows = (long long)p.B * p.Sq * p.Hq, per = tab::kFwdJoinThreads / (D / 4);
    return launch_dependent(D == 128 ? tab::attn_fwd_join_kernel<128> : tab::attn_fwd_join_kernel<64>,
                            dim3((unsigned)((rows + per - 1) / per)), dim3(tab::kFwdJoinThreads), stream, 0, p);
}
