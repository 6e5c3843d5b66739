// C ABI of the operators around the attention kernels: head norms with
// rotation (forward, backward, and into a paged cache) and the decode over
// that cache.  See include/attn.h for the contract of every entry point.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/attn.h"
#include "decode_paged.cuh"
#include "host_common.h"
#include "norm_rope.cuh"

using tab_host::aligned16;
using tab_host::aligned4;
using tab_host::device_state;
using tab_host::DeviceState;
using tab_host::encode_fn;
using tab_host::fail;
using tab_host::kMaxDevices;
using tab_host::launch_dependent;
using tab_host::ok;

namespace {

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// ------------------------------------------------------------- norm + rope

// Blocks of the backward, per SM: each leaves one share of dw.  A fixed
// bound, so that the workspace's size needs no device.
constexpr int kNormBwdMaxBlocks = 592;
constexpr int kNormBwdBlocksPerSm = 4;  // as many as are resident

// A bf16 (or wider) [tokens][H][D] argument: a pointer and the distance of
// its tokens.
attn_status_t check_rows(const char *name, const void *ptr, long long stride, int H, int D) {
    if (!ptr) return fail(ATTN_ERR_INVALID_ARG, "%s is null", name);
    if (!aligned16(ptr)) return fail(ATTN_ERR_MISALIGNED, "%s must be 16-byte aligned", name);
    if (stride < (long long)H * D || stride % 8 != 0)
        return fail(ATTN_ERR_INVALID_ARG, "%s: token stride %lld must be a multiple of 8 and >= H * D",
                    name, stride);
    return ATTN_OK;
}

// Checks of what every form shares; no CUDA call.
attn_status_t check_norm(const void *qw, const void *kw, int w_fp32, const float *cos,
                         const float *sin, const int *positions, long long tokens, int Hq, int Hkv,
                         int D, int rot, int max_positions, float eps, int interleaved,
                         long long chunks) {
    if (!qw || !kw || !cos || !sin || !positions) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (tokens < 1 || Hq < 1 || Hkv < 1) return fail(ATTN_ERR_INVALID_ARG, "tokens, Hq, Hkv must be >= 1");
    if (D != 64 && D != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d (built: 64, 128)", D);
    if (rot < 16 || rot > D || rot % 16 != 0)
        return fail(ATTN_ERR_INVALID_ARG, "rotated values (%d) must be a multiple of 16 in [16, D]", rot);
    if (max_positions < 1) return fail(ATTN_ERR_INVALID_ARG, "max_positions must be >= 1");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(ATTN_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    if ((w_fp32 != 0 && w_fp32 != 1) || (interleaved != 0 && interleaved != 1))
        return fail(ATTN_ERR_INVALID_ARG, "w_fp32 and interleaved must be 0 or 1");
    if (!aligned16(qw) || !aligned16(kw) || !aligned16(cos) || !aligned16(sin))
        return fail(ATTN_ERR_MISALIGNED, "weights, cos and sin must be 16-byte aligned");
    if (!aligned4(positions)) return fail(ATTN_ERR_MISALIGNED, "positions must be 4-byte aligned");
    if ((double)tokens * (double)chunks >= 2147483648.0 - 65536.0)
        return fail(ATTN_ERR_UNSUPPORTED, "too many tokens for one call");
    return ATTN_OK;
}

int chunks_of(int heads, int per) { return (heads + per - 1) / per; }

// Parameters that every form has, in one place: a field that a form forgot would
// be a zero.  `rows`: heads of a token that the form's kernel takes together.
tab::NormRopeParams norm_params(const void *q, const void *k, void *q_out, void *k_out,
                                long long q_stride, long long k_stride, long long q_out_stride,
                                long long k_out_stride, const void *qw, const void *kw, int w_fp32,
                                const float *cos, const float *sin, const int *positions,
                                long long tokens, int Hq, int Hkv, int rot, int max_positions,
                                float eps, int rows, int *status) {
    tab::NormRopeParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.qw = qw;
    p.kw = kw;
    p.w_fp32 = w_fp32;
    p.cos = cos;
    p.sin = sin;
    p.positions = positions;
    p.status = status;
    p.tokens = tokens;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.rot = rot;
    p.max_positions = max_positions;
    p.chunks_q = chunks_of(Hq, rows);
    p.chunks_k = chunks_of(Hkv, rows);
    p.eps = eps;
    return p;
}

template <int KV, bool INTERLEAVED>
attn_status_t launch_norm(const tab::NormRopeParams &p, int D, cudaStream_t stream) {
    const long long items = p.tokens * (p.chunks_q + (KV ? 2 : 1) * p.chunks_k);
    const int groups = tab::kNormThreads / (D / 8);
    const unsigned grid = (unsigned)((items + groups - 1) / groups);
    return launch_dependent(D == 128 ? tab::norm_rope_kernel<128, KV, INTERLEAVED>
                                     : tab::norm_rope_kernel<64, KV, INTERLEAVED>,
                            dim3(grid), dim3(tab::kNormThreads), stream, 0, p);
}

template <int KV>
attn_status_t dispatch_norm(const tab::NormRopeParams &p, int D, int interleaved, cudaStream_t stream) {
    return interleaved ? launch_norm<KV, true>(p, D, stream) : launch_norm<KV, false>(p, D, stream);
}

template <int D, bool INTERLEAVED>
attn_status_t launch_norm_bwd(const tab::NormRopeParams &p, int num_sms, float *dqw, float *dkw,
                              cudaStream_t stream) {
    const int groups = tab::kNormThreads / (D / 8);
    const long long items = p.tokens * std::max(p.chunks_q, p.chunks_k);
    const int blocks = (int)std::min<long long>(
        (items + groups - 1) / groups, std::min(kNormBwdMaxBlocks, kNormBwdBlocksPerSm * num_sms));
    const attn_status_t s = launch_dependent(tab::norm_rope_bwd_kernel<D, INTERLEAVED>, dim3(blocks),
                                             dim3(tab::kNormThreads), stream, 0, p);
    if (s != ATTN_OK) return s;
    return launch_dependent(tab::norm_rope_dw_kernel, dim3(2 * D / tab::kDwCols),
                            dim3(tab::kDwCols, tab::kDwRows), stream, 0,
                            static_cast<const float *>(p.partial), blocks, D, dqw, dkw);
}

// ------------------------------------------------------------------ decode

// Bound of the decode's blocks (two per SM of a 148-SM device): the
// workspace's size needs no device.
constexpr int kDecodeMaxBlocks = 296;

struct DecodeLayout {
    size_t part_ml, record, total;
};
DecodeLayout decode_layout(int D) {
    // Key heads of a pair: at most what makes 256 bytes of 8-bit values.
    const size_t rows = (size_t)kDecodeMaxBlocks * 2 * std::max(1, 256 / D) * tab::kDecRows;
    DecodeLayout L;
    L.part_ml = align256(rows * D * sizeof(float));
    L.record = L.part_ml + align256(rows * sizeof(float2));
    L.total = L.record + align256((size_t)kDecodeMaxBlocks * sizeof(int4));
    return L;
}

// Boxes of 16 keys of `heads` heads; the rows of a box are 128-byte pieces with
// the 128-byte swizzle (64 bytes for D = 64 in 8 bits).
attn_status_t make_cache_map(CUtensorMap *map, const void *base, int pages, int page_size, int Hkv,
                             int D, int eb, int heads) {
    tab_host::EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    const int row = D * eb, piece = std::min(row, 128);
    const cuuint64_t dims[5] = {(cuuint64_t)(piece / eb), (cuuint64_t)page_size,
                                (cuuint64_t)(row / piece), (cuuint64_t)Hkv, (cuuint64_t)pages};
    const cuuint64_t strides[4] = {(cuuint64_t)Hkv * row, (cuuint64_t)piece, (cuuint64_t)row,
                                   (cuuint64_t)page_size * Hkv * row};
    const cuuint32_t box[5] = {(cuuint32_t)(piece / eb), (cuuint32_t)tab::kDecBlock,
                               (cuuint32_t)(row / piece), (cuuint32_t)heads, 1};
    const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(
        map, eb == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
        const_cast<void *>(base), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
        piece == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled (cache) failed (%d)", (int)r);
    return ATTN_OK;
}

template <int D, bool F8, int kHeads, int NB, int kBlocks, int kStages>
attn_status_t launch_decode_nb(tab::DecodeParams &p, const void *k_cache, const void *v_cache,
                            int blocks, cudaStream_t stream) {
    using Smem = tab::DecodeSmem<D, F8, kHeads, NB, kBlocks, kStages>;
    constexpr size_t smem = sizeof(Smem) + 1024;
    static_assert(tab::kDecCtasPerSm * (smem + 1024) <= 233472, "shared memory budget");
    auto kernel = tab::decode_paged_kernel<D, F8, kHeads, NB, kBlocks, kStages>;
    static std::once_flag once[kMaxDevices];
    static cudaError_t attr_err[kMaxDevices];
    static cudaFuncAttributes attrs[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    std::call_once(once[dev], [&]() {
        attr_err[dev] =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (attr_err[dev] == cudaSuccess) attr_err[dev] = cudaFuncGetAttributes(&attrs[dev], kernel);
    });
    if (attr_err[dev] != cudaSuccess)
        return fail(ATTN_ERR_LAUNCH, "kernel attributes: %s", cudaGetErrorString(attr_err[dev]));
    // The register split (setmaxnreg) counts on this allocation: with less,
    // the increase would wait forever, so never launch such a build.
    if (attrs[dev].numRegs < tab::kDecLaunchRegs)
        return fail(ATTN_ERR_LAUNCH, "kernel compiled with %d registers per thread, %d needed",
                    attrs[dev].numRegs, tab::kDecLaunchRegs);
    attn_status_t s;
    const int eb = F8 ? 1 : 2;
    if ((s = make_cache_map(&p.tm_k, k_cache, p.num_pages, p.page_size, p.Hkv, D, eb, kHeads)) != ATTN_OK ||
        (s = make_cache_map(&p.tm_v, v_cache, p.num_pages, p.page_size, p.Hkv, D, eb, kHeads)) != ATTN_OK)
        return s;
    // No more blocks than runs: pairs of one tile, or a team's tiles each.
    const double pairs = (double)p.B * (p.Hkv / kHeads) * p.hchunks;
    const double tiles = ((double)p.max_pages * p.page_size + Smem::kTile - 1) / Smem::kTile;
    blocks = (int)std::min<double>(blocks, pairs * std::max(1.0, std::ceil(tiles / Smem::kTeams)));
    if ((s = launch_dependent(kernel, dim3(blocks), dim3(tab::kDecThreads), stream, smem, p)) != ATTN_OK)
        return s;
    const tab::JoinParams jp = {p.part_o, p.part_ml, p.record, p.o, p.lse, p.Hq, p.group, p.v_descale};
    return launch_dependent(tab::decode_join_kernel<D, kHeads>,
                            dim3(blocks, std::min(p.group, Smem::kRows), kHeads),
                            dim3(tab::kJoinThreads), stream, 0, jp);
}

// One block of 8 query heads where that holds a key head's, else two.
template <int D, bool F8, int kHeads, int kBlocks, int kStages>
attn_status_t launch_decode(tab::DecodeParams &p, const void *k_cache, const void *v_cache,
                            int blocks, cudaStream_t stream) {
    return p.group <= 8 ? launch_decode_nb<D, F8, kHeads, 1, kBlocks, kStages>(p, k_cache, v_cache, blocks, stream)
                        : launch_decode_nb<D, F8, kHeads, 2, kBlocks, kStages>(p, k_cache, v_cache, blocks, stream);
}

// The variant by the bytes of a key's head: pairs of as many key heads as make
// 256 bytes and divide Hkv; rings of 64 KB per block (128 KB per SM; with 96
// KB the bf16 cases read 5 % slower), in tiles of 32 keys, or of 16 for heads
// of 256 bytes.
attn_status_t dispatch_decode(tab::DecodeParams &p, const void *k, const void *v, int D, bool f8,
                              int blocks, cudaStream_t s) {
    const bool two = p.Hkv % 2 == 0, four = p.Hkv % 4 == 0;
    if (!f8 && D == 128) return launch_decode<128, false, 1, 1, 8>(p, k, v, blocks, s);
    if (!f8) return two ? launch_decode<64, false, 2, 2, 4>(p, k, v, blocks, s)
                        : launch_decode<64, false, 1, 2, 8>(p, k, v, blocks, s);
    if (D == 128) return two ? launch_decode<128, true, 2, 2, 4>(p, k, v, blocks, s)
                             : launch_decode<128, true, 1, 2, 8>(p, k, v, blocks, s);
    if (four) return launch_decode<64, true, 4, 2, 4>(p, k, v, blocks, s);
    return two ? launch_decode<64, true, 2, 2, 8>(p, k, v, blocks, s)
               : launch_decode<64, true, 1, 2, 16>(p, k, v, blocks, s);
}

}  // namespace

extern "C" {

attn_status_t attn_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out,
                                long long q_stride, long long k_stride, long long q_out_stride,
                                long long k_out_stride, const void *q_weight, const void *k_weight,
                                int w_fp32, const float *cos, const float *sin,
                                const int *positions, long long tokens, int Hq, int Hkv, int D,
                                int rot, int max_positions, float eps, int interleaved,
                                void *stream) {
    const int cq = chunks_of(Hq, tab::kNormRows), ck = chunks_of(Hkv, tab::kNormRows);
    attn_status_t s = check_norm(q_weight, k_weight, w_fp32, cos, sin, positions, tokens, Hq, Hkv, D,
                                 rot, max_positions, eps, interleaved, (long long)cq + ck);
    if (s != ATTN_OK) return s;
    if ((s = check_rows("q", q, q_stride, Hq, D)) != ATTN_OK ||
        (s = check_rows("k", k, k_stride, Hkv, D)) != ATTN_OK ||
        (s = check_rows("q_out", q_out, q_out_stride, Hq, D)) != ATTN_OK ||
        (s = check_rows("k_out", k_out, k_out_stride, Hkv, D)) != ATTN_OK)
        return s;
    DeviceState *st = nullptr;
    if ((s = device_state(&st)) != ATTN_OK) return s;
    const tab::NormRopeParams p = norm_params(
        q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, q_weight, k_weight, w_fp32,
        cos, sin, positions, tokens, Hq, Hkv, rot, max_positions, eps, tab::kNormRows, st->status);
    return dispatch_norm<0>(p, D, interleaved, static_cast<cudaStream_t>(stream));
}

attn_status_t attn_qk_norm_rope_cache(const void *q, const void *k, const void *v, void *q_out,
                                      long long q_stride, long long k_stride, long long v_stride,
                                      long long q_out_stride, const void *q_weight,
                                      const void *k_weight, int w_fp32, const float *cos,
                                      const float *sin, const int *positions, const int *slots,
                                      void *k_cache, void *v_cache, int kv_dtype, float k_descale,
                                      float v_descale, long long num_slots, long long tokens, int Hq,
                                      int Hkv, int D, int rot, int max_positions, float eps,
                                      int interleaved, void *stream) {
    const int cq = chunks_of(Hq, tab::kNormRows), ck = chunks_of(Hkv, tab::kNormRows);
    attn_status_t s = check_norm(q_weight, k_weight, w_fp32, cos, sin, positions, tokens, Hq, Hkv, D,
                                 rot, max_positions, eps, interleaved, (long long)cq + 2LL * ck);
    if (s != ATTN_OK) return s;
    if ((s = check_rows("q", q, q_stride, Hq, D)) != ATTN_OK ||
        (s = check_rows("k", k, k_stride, Hkv, D)) != ATTN_OK ||
        (s = check_rows("v", v, v_stride, Hkv, D)) != ATTN_OK ||
        (s = check_rows("q_out", q_out, q_out_stride, Hq, D)) != ATTN_OK)
        return s;
    if (!slots || !k_cache || !v_cache) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(ATTN_ERR_MISALIGNED, "k_cache and v_cache must be 16-byte aligned");
    if (!aligned4(slots)) return fail(ATTN_ERR_MISALIGNED, "slots must be 4-byte aligned");
    if (num_slots < 1) return fail(ATTN_ERR_INVALID_ARG, "num_slots must be >= 1");
    if (kv_dtype != ATTN_KV_BF16 && kv_dtype != ATTN_KV_E4M3)
        return fail(ATTN_ERR_INVALID_ARG, "kv_dtype must be ATTN_KV_BF16 or ATTN_KV_E4M3");
    for (float d : {k_descale, v_descale})
        if (!(d > 0.0f) || !std::isfinite(d) || !std::isfinite(1.0f / d) ||
            (kv_dtype == ATTN_KV_BF16 && d != 1.0f))
            return fail(ATTN_ERR_INVALID_ARG,
                        "descale factors and their reciprocals must be > 0 and finite, and 1 for a bf16 cache");
    DeviceState *st = nullptr;
    if ((s = device_state(&st)) != ATTN_OK) return s;
    tab::NormRopeParams p = norm_params(
        q, k, q_out, nullptr, q_stride, k_stride, q_out_stride, 0, q_weight, k_weight, w_fp32, cos, sin,
        positions, tokens, Hq, Hkv, rot, max_positions, eps, tab::kNormRows, st->status);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.v_stride = v_stride;
    p.slots = slots;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.num_slots = num_slots;
    p.k_scale = 1.0f / k_descale;
    p.v_scale = 1.0f / v_descale;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return kv_dtype == ATTN_KV_E4M3 ? dispatch_norm<2>(p, D, interleaved, cs)
                                    : dispatch_norm<1>(p, D, interleaved, cs);
}

size_t attn_qk_norm_rope_bwd_workspace_size(int D) {
    return D < 1 ? 0 : align256((size_t)kNormBwdMaxBlocks * 2 * D * sizeof(float));
}

attn_status_t attn_qk_norm_rope_bwd(const void *dq, const void *dk, int dq_fp32, int dk_fp32,
                                    const void *q, const void *k, void *dq_in, void *dk_in,
                                    float *dq_weight, float *dk_weight, long long dq_stride,
                                    long long dk_stride, long long q_stride, long long k_stride,
                                    long long dq_in_stride, long long dk_in_stride,
                                    const void *q_weight, const void *k_weight, int w_fp32,
                                    const float *cos, const float *sin, const int *positions,
                                    long long tokens, int Hq, int Hkv, int D, int rot,
                                    int max_positions, float eps, int interleaved, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    const int cq = chunks_of(Hq, tab::kNormBwdRows), ck = chunks_of(Hkv, tab::kNormBwdRows);
    attn_status_t s = check_norm(q_weight, k_weight, w_fp32, cos, sin, positions, tokens, Hq, Hkv, D,
                                 rot, max_positions, eps, interleaved, (long long)cq + ck);
    if (s != ATTN_OK) return s;
    if ((s = check_rows("dq", dq, dq_stride, Hq, D)) != ATTN_OK ||
        (s = check_rows("dk", dk, dk_stride, Hkv, D)) != ATTN_OK ||
        (s = check_rows("q", q, q_stride, Hq, D)) != ATTN_OK ||
        (s = check_rows("k", k, k_stride, Hkv, D)) != ATTN_OK ||
        (s = check_rows("dq_in", dq_in, dq_in_stride, Hq, D)) != ATTN_OK ||
        (s = check_rows("dk_in", dk_in, dk_in_stride, Hkv, D)) != ATTN_OK)
        return s;
    if (!dq_weight || !dk_weight || !workspace) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned4(dq_weight) || !aligned4(dk_weight))
        return fail(ATTN_ERR_MISALIGNED, "dq_weight and dk_weight must be 4-byte aligned");
    if (!aligned16(workspace)) return fail(ATTN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    for (int f : {dq_fp32, dk_fp32})
        if (f != 0 && f != 1) return fail(ATTN_ERR_INVALID_ARG, "dq_fp32 and dk_fp32 must be 0 or 1");
    const size_t need = attn_qk_norm_rope_bwd_workspace_size(D);
    if (workspace_bytes < need)
        return fail(ATTN_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    DeviceState *st = nullptr;
    if ((s = device_state(&st)) != ATTN_OK) return s;
    tab::NormRopeParams p = norm_params(
        q, k, dq_in, dk_in, q_stride, k_stride, dq_in_stride, dk_in_stride, q_weight, k_weight, w_fp32,
        cos, sin, positions, tokens, Hq, Hkv, rot, max_positions, eps, tab::kNormBwdRows, st->status);
    p.dq = dq;
    p.dk = dk;
    p.dq_stride = dq_stride;
    p.dk_stride = dk_stride;
    p.dq_fp32 = dq_fp32;
    p.dk_fp32 = dk_fp32;
    p.partial = static_cast<float *>(workspace);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (D == 128)
        return interleaved ? launch_norm_bwd<128, true>(p, st->num_sms, dq_weight, dk_weight, cs)
                           : launch_norm_bwd<128, false>(p, st->num_sms, dq_weight, dk_weight, cs);
    return interleaved ? launch_norm_bwd<64, true>(p, st->num_sms, dq_weight, dk_weight, cs)
                       : launch_norm_bwd<64, false>(p, st->num_sms, dq_weight, dk_weight, cs);
}

size_t attn_decode_paged_workspace_size(int D) { return D < 1 ? 0 : decode_layout(D).total; }

attn_status_t attn_decode_paged(const void *q, const void *k_cache, const void *v_cache,
                                int kv_dtype, float k_descale, float v_descale,
                                const int *page_table, const int *seq_lens, void *o, float *lse,
                                int B, int Hq, int Hkv, int D, int num_pages, int page_size,
                                int max_pages, float scale, int window_left, int sinks,
                                float softcap, const float *alibi_slopes, void *workspace,
                                size_t workspace_bytes, void *stream) {
    // ----- validation (no CUDA call before this block completes)
    for (const void *ptr : {q, k_cache, v_cache, (const void *)o, (const void *)workspace}) {
        if (!ptr) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
        if (!aligned16(ptr))
            return fail(ATTN_ERR_MISALIGNED, "q, caches, o and workspace must be 16-byte aligned");
    }
    if (!page_table || !seq_lens || !lse) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (q == o) return fail(ATTN_ERR_INVALID_ARG, "o must not be q: blocks that share a sequence read q late");
    if (!aligned4(page_table) || !aligned4(seq_lens) || !aligned4(lse) || !aligned4(alibi_slopes))
        return fail(ATTN_ERR_MISALIGNED, "page_table, seq_lens, lse, alibi_slopes must be 4-byte aligned");
    if (B < 1 || Hq < 1 || Hkv < 1 || num_pages < 1 || max_pages < 1)
        return fail(ATTN_ERR_INVALID_ARG, "B, Hq, Hkv, num_pages, max_pages must be >= 1");
    if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (D != 64 && D != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d (built: 64, 128)", D);
    if (page_size < 16 || page_size % 16 != 0)
        return fail(ATTN_ERR_UNSUPPORTED, "page size %d (built: multiples of 16)", page_size);
    if (kv_dtype != ATTN_KV_BF16 && kv_dtype != ATTN_KV_E4M3)
        return fail(ATTN_ERR_INVALID_ARG, "kv_dtype must be ATTN_KV_BF16 or ATTN_KV_E4M3");
    for (float d : {k_descale, v_descale})
        if (!(d > 0.0f) || !std::isfinite(d) || (kv_dtype == ATTN_KV_BF16 && d != 1.0f))
            return fail(ATTN_ERR_INVALID_ARG,
                        "descale factors must be > 0 and finite, and 1 for a bf16 cache");
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return fail(ATTN_ERR_INVALID_ARG, "scale must be positive and finite");
    if (window_left < -1 || sinks < 0)
        return fail(ATTN_ERR_INVALID_ARG, "window_left must be -1 or >= 0, sinks >= 0");
    if (!(softcap >= 0.0f) || !std::isfinite(softcap))
        return fail(ATTN_ERR_INVALID_ARG, "softcap must be >= 0 and finite");
    const size_t need = attn_decode_paged_workspace_size(D);
    if (workspace_bytes < need)
        return fail(ATTN_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    const int group = Hq / Hkv, hchunks = (group + tab::kDecRows - 1) / tab::kDecRows;
    const double keys = (double)max_pages * page_size;
    const double tiles = (keys / tab::kDecBlock + 1.0) * Hkv * hchunks;  // of one sequence, at most
    if (keys > 2147483647.0 - 4096.0 || tiles > 2147483647.0 || tiles * B > 2.0 * 2147483647.0)
        return fail(ATTN_ERR_UNSUPPORTED, "sequences too long for one call");
    if ((double)page_size * Hkv * D * 2.0 >= 1099511627776.0)
        return fail(ATTN_ERR_UNSUPPORTED, "pages too large for a TMA descriptor");

    // ----- set-up
    DeviceState *st = nullptr;
    attn_status_t s = device_state(&st);
    if (s != ATTN_OK) return s;
    const bool f8 = kv_dtype == ATTN_KV_E4M3;
    tab::DecodeParams p;
    memset(&p, 0, sizeof p);
    const DecodeLayout L = decode_layout(D);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.status = st->status;
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + L.part_ml);
    p.record = reinterpret_cast<int4 *>(ws + L.record);
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = group;
    p.hchunks = hchunks;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.window_left = window_left;
    p.sinks = window_left < 0 ? 0 : sinks;
    p.scale_log2 = (float)((double)scale * k_descale * 1.4426950408889634);
    p.v_descale = v_descale;
    if (softcap > 0.0f) {
        p.softcap_in = (float)((double)scale * k_descale / softcap);
        p.softcap_out = (float)((double)softcap * 1.4426950408889634);
    }
    p.alibi_slopes = alibi_slopes;
    const int blocks = std::min(kDecodeMaxBlocks, tab::kDecCtasPerSm * st->num_sms);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return dispatch_decode(p, k_cache, v_cache, D, f8, blocks, cs);
}

}  // extern "C"
