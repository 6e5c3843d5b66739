// Launching of the forward and backward kernels, shared by the translation
// units that hold their variants.
#pragma once

#include <algorithm>

#include "bwd_kernel.cuh"
#include "fwd_kernel.cuh"
#include "fwd_persistent.cuh"
#include "fwd_window.cuh"
#include "host_common.h"

namespace tab_host {

// Windows with first keys that stay visible: the forward (one CTA per item, or
// p.parts of them) and the backward, in translation units of their own: they
// compile side by side.  sinks_fwd.cu, sinks_parts.cu, sinks_bwd.cu
attn_status_t dispatch_fwd_sinks(const tab::WindowParams &p, int D, int exp_mode, int mod, cudaStream_t stream);
attn_status_t dispatch_fwd_parts(const tab::WindowParams &p, int D, int exp_mode, int mod, cudaStream_t stream);
attn_status_t dispatch_bwd_sinks(const tab::BwdParams &p, int D, int mod, cudaStream_t stream);

}  // namespace tab_host

namespace {

using tab_host::fail;
using tab_host::kMaxDevices;
using tab_host::ok;

// A forward kernel of kFwdThreads threads that moves registers between its
// warpgroups (setmaxnreg), and what is asked of it once per device.
struct PreparedFwd {
    std::once_flag once[kMaxDevices];
    cudaError_t err[kMaxDevices];
    cudaFuncAttributes attrs[kMaxDevices];
};
template <class Params>
attn_status_t launch_fwd_kernel(PreparedFwd &st, void (*kernel)(Params), const Params &p, dim3 grid, size_t smem,
                                cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    std::call_once(st.once[dev], [&]() {
        st.err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (st.err[dev] == cudaSuccess) st.err[dev] = cudaFuncGetAttributes(&st.attrs[dev], kernel);
    });
    if (st.err[dev] != cudaSuccess)
        return fail(ATTN_ERR_LAUNCH, "kernel attributes: %s", cudaGetErrorString(st.err[dev]));
    // If the compiled per-thread count does not cover the register split, the
    // increase would wait forever, so never launch such a build.
    if (st.attrs[dev].numRegs < tab::kLaunchRegs)
        return fail(ATTN_ERR_LAUNCH, "kernel compiled with %d registers per thread, %d needed",
                    st.attrs[dev].numRegs, tab::kLaunchRegs);
    kernel<<<grid, tab::kFwdThreads, smem, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
    return ok();
}

// PERSIST selects the persistent kernel (fwd_persistent.cuh: one CTA per SM
// running many items), otherwise one CTA per item.
template <int D, int NS, int EXP, int MOD = 0, int PREC = 0, bool PERSIST = false>
attn_status_t launch_fwd(const tab::FwdParams &p, int grid, cudaStream_t stream) {
    using Smem = std::conditional_t<PERSIST, tab::FwdSmemPersistent<D, NS, PREC == 1 ? 1 : 2>,
                                    tab::FwdSmem<D, NS, PREC == 1 ? 1 : 2>>;
    constexpr size_t smem = sizeof(Smem) + 1024;
    static_assert(smem <= 232448, "shared memory budget");
    static PreparedFwd st;
    if constexpr (PERSIST)
        return launch_fwd_kernel(st, tab::attn_fwd_persistent_kernel<D, NS, EXP, MOD, PREC>, p, grid, smem, stream);
    else
        return launch_fwd_kernel(st, tab::attn_fwd_kernel<D, NS, EXP, MOD, PREC>, p, grid, smem, stream);
}

template <int D, int NS, int EXP, int MOD, bool PARTS>
attn_status_t launch_window(const tab::WindowParams &p, cudaStream_t stream) {
    constexpr size_t smem = sizeof(tab::WindowSmem<D, NS>) + 1024;
    static_assert(smem <= 232448, "shared memory budget");
    static PreparedFwd st;
    return launch_fwd_kernel(st, tab::attn_fwd_window_kernel<D, NS, EXP, MOD, PARTS>, p,
                             dim3(p.head_group, p.num_qblocks, p.groups * p.parts), smem, stream);
}

constexpr int kStagesD128 = 4;
constexpr int kStagesD64 = 8;

// With a score modifier the exponentials all run on MUFU.
template <int D, int NS>
attn_status_t dispatch_exp(const tab::FwdParams &p, int grid, int exp_mode, int mod,
                           cudaStream_t s) {
    switch (mod) {
        case 1: return launch_fwd<D, NS, 0, 1>(p, grid, s);
        case 2: return launch_fwd<D, NS, 0, 2>(p, grid, s);
        case 3: return launch_fwd<D, NS, 0, 3>(p, grid, s);
        default: break;
    }
    switch (exp_mode) {
        case 0: return launch_fwd<D, NS, 0>(p, grid, s);
        case 1: return launch_fwd<D, NS, 1>(p, grid, s);
        default: return launch_fwd<D, NS, 2>(p, grid, s);
    }
}

template <int D, int NS, bool PARTS>
attn_status_t dispatch_window(const tab::WindowParams &p, int exp_mode, int mod, cudaStream_t s) {
    switch (mod) {
        case 1: return launch_window<D, NS, 0, 1, PARTS>(p, s);
        case 2: return launch_window<D, NS, 0, 2, PARTS>(p, s);
        case 3: return launch_window<D, NS, 0, 3, PARTS>(p, s);
        default: break;
    }
    switch (exp_mode) {
        case 0: return launch_window<D, NS, 0, 0, PARTS>(p, s);
        case 1: return launch_window<D, NS, 1, 0, PARTS>(p, s);
        default: return launch_window<D, NS, 2, 0, PARTS>(p, s);
    }
}

template <class Kernel>
attn_status_t prepare_kernel(Kernel kernel, size_t smem, int threads, int min_regs) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess)
        return fail(ATTN_ERR_LAUNCH, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    cudaFuncAttributes attrs;
    e = cudaFuncGetAttributes(&attrs, kernel);
    if (e != cudaSuccess)
        return fail(ATTN_ERR_LAUNCH, "cudaFuncGetAttributes: %s", cudaGetErrorString(e));
    if (attrs.numRegs < min_regs || attrs.maxThreadsPerBlock < threads)
        return fail(ATTN_ERR_LAUNCH, "kernel build cannot be launched (%d regs, %d threads)",
                    attrs.numRegs, attrs.maxThreadsPerBlock);
    return ATTN_OK;
}

constexpr int kBwdStagesQ = 2;
// dQ kernel: K and V ring depths (224 KB of SMEM with Q and dO at D = 128).
constexpr int bwd_k_stages(int D) { return D == 128 ? 3 : 6; }
constexpr int bwd_v_stages(int D) { return D == 128 ? 2 : 4; }

template <int D, int MOD, bool SINKS>
attn_status_t launch_bwd(const tab::BwdParams &p, cudaStream_t stream) {
    using DkdvS = tab::DkdvSmem<D, kBwdStagesQ>;
    using DqS = tab::DqSmem<D, bwd_k_stages(D), bwd_v_stages(D)>;
    constexpr size_t smem_dkdv = sizeof(DkdvS) + 1024;
    constexpr size_t smem_dq = sizeof(DqS) + 1024;
    static_assert(smem_dkdv <= 232448 && smem_dq <= 232448, "shared memory budget");
    auto k_dkdv = tab::attn_bwd_dkdv_kernel<D, kBwdStagesQ, MOD, SINKS>;
    auto k_dq = tab::attn_bwd_dq_kernel<D, bwd_k_stages(D), bwd_v_stages(D), MOD, SINKS>;
    static std::once_flag once[kMaxDevices];
    static attn_status_t prep[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    std::call_once(once[dev], [&]() {
        prep[dev] = prepare_kernel(k_dkdv, smem_dkdv, tab::kBwdThreads, 0);
        if (prep[dev] == ATTN_OK) prep[dev] = prepare_kernel(k_dq, smem_dq, tab::kBwdThreads, 0);
    });
    if (prep[dev] != ATTN_OK) return fail(prep[dev], "backward kernels could not be prepared");
    // dQ first: it also computes D_i into the workspace, which the dK/dV
    // kernel reads.
    k_dq<<<p.num_qb * p.Hq * p.B, tab::kBwdThreads, smem_dq, stream>>>(p);
    if constexpr (SINKS) {
        // A CTA per part of a key block, and the sum of the parts.
        const int rows = p.sink_blocks * p.sink_parts + (p.num_kb - p.sink_blocks) * p.other_parts;
        k_dkdv<<<rows * p.Hkv * p.B, tab::kBwdThreads, smem_dkdv, stream>>>(p);
        const int blocks = p.other_parts > 1 ? p.num_kb : p.sink_parts > 1 ? p.sink_blocks : 0;
        const long long n = (long long)blocks * p.Hkv * p.B * 2 * 128 * (D / 4);
        const int grid = (int)std::min<long long>((n + 255) / 256, 148 * 8);
        if (blocks > 0) tab::attn_bwd_part_sum_kernel<D><<<grid, 256, 0, stream>>>(p, blocks);
    } else {
        k_dkdv<<<p.num_kb * p.Hkv * p.B, tab::kBwdThreads, smem_dkdv, stream>>>(p);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
    return ok();
}

template <int D, bool SINKS = false>
attn_status_t dispatch_bwd(const tab::BwdParams &p, int mod, cudaStream_t stream) {
    switch (mod) {
        case 1: return launch_bwd<D, 1, SINKS>(p, stream);
        case 2: return launch_bwd<D, 2, SINKS>(p, stream);
        case 3: return launch_bwd<D, 3, SINKS>(p, stream);
        default: return launch_bwd<D, 0, SINKS>(p, stream);
    }
}

}  // namespace
