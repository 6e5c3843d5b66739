// The forward under a sliding window with first keys that stay visible.
//
// Beside its interval (window, causal) a row sees keys j < sinks up to the
// interval's upper end.  The key blocks of a tile of 128 rows are those of the
// first keys before its window, [0, min(sink_blocks, lo)), and [lo, hi].
//
// The roles, barriers and tensor memory are those of attn_fwd_kernel (two
// query tiles per CTA, in turn on the tensor cores and in the softmax warps).
// What differs, since a window leaves a CTA about ten key blocks:
//  - The tiles walk together (TileWalk): first the blocks that both see, then
//    side by side those that only one of them sees.
//  - The load warp finds its blocks and starts the first copies before the CTA
//    meets; results leave through shared memory by TMA.
//  - Blocks that the mask cuts are handled by groups of 32 keys: one that no
//    row of a warp sees is left out, one that all see is not masked.
//  - PARTS, for few items: the walk's steps are cut into parts, a CTA each,
//    which attn_fwd_join_kernel joins by their LSEs.
//
// Measured on 2 x 8192 tokens, 16 heads of 128, four first tokens, in turn with
// the plain kernel under this mask: window 1024 209 -> 193 us, window 512 148 ->
// 132, window 128 100 -> 84.  Of a CTA's 43000 cycles at window 1024 the first
// scores take 4000 and the ends 5000; a step takes 3600 for both tiles, as in
// the plain forward (softmax warps).  One tile per CTA and two CTAs per SM ran
// as long (a ring of two slots: 3600 cycles a step too); multiplying only the
// 32 first keys of a block that has no more cost the issuing warp more than it
// saved (198 us).
//
// P is rounded to bf16, as in the plain forward: the tensor cores take no wider
// operand beside a bf16 V, and a second product for the rest would add half to
// their work.  The output is normalised by the sum of the rounded P and is off
// by 0.0021 of its norm, 0.0017 of which is its own rounding; maxima, sums and
// LSE are in fp32.
#pragma once

#include "fwd_kernel.cuh"

namespace tab {

// The grid is (head_group, query blocks, groups x parts), which has the order of
// attn_fwd_kernel's items without its divisions.
struct WindowParams : FwdParams {
    CUtensorMap tm_o;  // as tm_q
    int groups;        // of (batch, query head) pairs
    // First keys that stay visible; parts of each item's steps (1: none), and
    // the parts' results: fp32 O [part][B][Sq][Hq][D], each normalised, and LSE
    // [part][B][Hq][Sq].
    int sinks, parts;
    float *part_o, *part_lse;
};

// row_key_range without a document mask.
__device__ __forceinline__ KeyRange window_range(const WindowParams &p, int row) {
    long long lo = 0, hi = (long long)p.Sk - 1;
    const long long diag = (long long)row + p.Sk - p.Sq;
    if (p.causal) hi = min(hi, diag);
    if (p.window_right >= 0) hi = min(hi, diag + p.window_right);
    lo = max(lo, diag - p.window_left);
    if (lo > hi) return {1, 0};
    return {(int)lo, (int)hi};
}

// The steps of a CTA's two tiles: the blocks that both see, one a step; then,
// side by side, those that only the upper tile sees (its window begins a block
// earlier) and those that only the lower one sees (its window ends a block
// later), so that the tiles begin and end together.
struct TileWalk {
    int first, shared, next;  // the shared blocks: [0, first), then next, next + 1, ...
    int own0, own1;           // first block of each tile's own
    int n0, n1;               // steps of each tile, from step 0 on

    // Tiles of blocks [lo, hi] (none if lo > hi), the second one 128 rows below
    // the first: lo0 <= lo1 <= lo0 + 1 and hi0 <= hi1.
    __device__ __forceinline__ TileWalk(int lo0, int hi0, int lo1, int hi1, int sink_blocks) {
        const bool has0 = lo0 <= hi0, has1 = lo1 <= hi1;
        if (has0 && has1) {
            const int s1 = min(sink_blocks, lo1);
            first = s1 > lo0 ? min(s1, hi0 + 1) : min(sink_blocks, lo0);
            next = max(lo1, first);
            shared = first + max(0, hi0 - next + 1);
            own0 = max(lo0, first);
            own1 = max(lo1, hi0 + 1);
            n0 = shared + max(0, min(lo1 - 1, hi0) - own0 + 1);
            n1 = shared + max(0, hi1 - own1 + 1);
        } else {
            const int lo = has0 ? lo0 : lo1, hi = has0 ? hi0 : hi1;
            first = min(sink_blocks, lo);
            next = own0 = own1 = lo;
            shared = has0 || has1 ? first + hi - lo + 1 : 0;
            n0 = has0 ? shared : 0;
            n1 = has1 ? shared : 0;
        }
    }
    __device__ __forceinline__ int steps() const { return max(n0, n1); }
    __device__ __forceinline__ bool active(int i, int t) const { return t < (i == 0 ? n0 : n1); }
    // Both tiles in step t, each with a block of its own.
    __device__ __forceinline__ bool apart(int t) const { return t >= shared && t < min(n0, n1); }
    __device__ __forceinline__ int block(int i, int t) const {
        return t >= shared ? (i == 0 ? own0 : own1) + t - shared : t < first ? t : next + t - first;
    }
};

// exp_pack_half for 32 scores of a masked block, all on MUFU: ex2(-inf) = 0 exactly.
__device__ __forceinline__ void exp_pack_group(const float *s, float c, float neg_m, uint32_t *pk,
                                               float &sum, float &sum_pv) {
    float sum0 = 0.0f, sum1 = 0.0f, r0s = 0.0f, r1s = 0.0f;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float x0, x1;
        fma2(x0, x1, s[e], s[e + 1], c, c, neg_m, neg_m);
        const float p0 = ex2_mufu(x0), p1 = ex2_mufu(x1);
        add2(sum0, sum1, sum0, sum1, p0, p1);
        const uint32_t h = pack_bf16x2(p0, p1);
        pk[e >> 1] = h;
        add_bf16x2_f32(r0s, r1s, h);
    }
    sum += sum0 + sum1;
    sum_pv += r0s + r1s;
}

template <int D, int NS>
struct WindowSmem {
    static constexpr int kChunkBytes = kBlockM * 128;  // 16 KB: 128 rows x 128 bytes
    static constexpr int kChunks = D / 64;
    uint8_t q[2][kChunks][kChunkBytes];  // and O, on its way out
    uint8_t kv[NS][kChunks][kChunkBytes];
    uint64_t q_full[2];
    uint64_t kv_full[NS];
    uint64_t kv_empty[NS];
    uint64_t s_full[2];
    uint64_t p_half[2];  // P of keys [0, 64) of the block is in TMEM
    uint64_t p_full[2];  // all of P (and any O correction) is in TMEM
    uint64_t o_final[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int range[2][2];  // per query tile: first and last key block (inclusive)
    int walk[2][4];   // per tile: what gives a step's block (TileWalk::block)
    int item[3];      // batch, query head, part: for the epilogue
};

template <int D, int NS, int EXP_MODE, int MOD, bool PARTS>
__global__ void __launch_bounds__(kFwdThreads, 1)
attn_fwd_window_kernel(const __grid_constant__ WindowParams p) {
    using Smem = WindowSmem<D, NS>;
    constexpr uint32_t kTileBytes = kBlockM * D * 2;
    static_assert((NS & (NS - 1)) == 0 && NS >= 4, "a step may need four slots");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_off = smem_u32(smem_raw);
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (raw_off & 1023u)) & 1023u));
    const int warp = warp_id(), lane = lane_id();

    const int part = PARTS ? (int)blockIdx.z / p.groups : 0;
    const int grp = PARTS ? (int)blockIdx.z - part * p.groups : (int)blockIdx.z;
    const int bh = grp * p.head_group + (int)blockIdx.x;
    if (bh >= p.Hq * p.B) return;  // the last group may be smaller
    if constexpr (PARTS) launch_dependents();
    const int q0 = (p.num_qblocks - 1 - (int)blockIdx.y) * 2 * kBlockM;  // the longest first
    const int b = bh / p.Hq;
    const int hq = bh - b * p.Hq;
    const int hkv = hq / p.group;

    // The walk, from sm.range, and this CTA's steps [t0, t1) of it.
    auto make_walk = [&]() -> TileWalk {
        return TileWalk(sm.range[0][0], sm.range[0][1], sm.range[1][0], sm.range[1][1],
                        (p.sinks + kBlockN - 1) / kBlockN);
    };
    auto first_step = [&](int steps) -> int { return PARTS ? (int)((long long)steps * part / p.parts) : 0; };
    auto end_step = [&](int steps) -> int {
        return PARTS ? (int)((long long)steps * (part + 1) / p.parts) : steps;
    };
    // Copy `it` of this CTA: K or V of the key block kb.
    auto copy_kv = [&](uint32_t it, bool v, int kb) {
        // Testing only: the first CTA withholds its first K copy.
        if (p.debug_withhold_kv && it == 0 && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) return;
        mbar_arrive_expect_tx(&sm.kv_full[it % NS], kTileBytes);
        for (int c = 0; c < Smem::kChunks; ++c)
            tma_load_4d(sm.kv[it % NS][c], v ? &p.tm_v : &p.tm_k, &sm.kv_full[it % NS], c * 64, kb * kBlockN, hkv, b);
    };

    // ------------------------------------------------------------ prologue
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_half[i], kBlockM);
            mbar_init(&sm.p_full[i], kBlockM);
            mbar_init(&sm.o_final[i], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        sm.item[0] = b;
        sm.item[1] = hq;
        sm.item[2] = part;
        fence_mbar_init();
    }
    if (warp == 9) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) mbar_init(&sm.q_full[i], 1);
            for (int s = 0; s < NS; ++s) {
                mbar_init(&sm.kv_full[s], 1);
                mbar_init(&sm.kv_empty[s], 1);
            }
            fence_mbar_init();
            auto copy_q = [&](int i) {
                mbar_arrive_expect_tx(&sm.q_full[i], kTileBytes);
                for (int c = 0; c < Smem::kChunks; ++c)
                    tma_load_4d(sm.q[i][c], &p.tm_q, &sm.q_full[i], c * 64, q0 + i * kBlockM, hq, b);
            };
            copy_q(0);
            // Key blocks of each query tile: from the first row's to the last's; in a tile
            // whose first rows have no key, the first row with one sees key 0.
            for (int i = 0; i < 2; ++i) {
                const int r0 = q0 + i * kBlockM;
                const KeyRange a = window_range(p, min(r0, p.Sq - 1));
                const KeyRange z = window_range(p, min(r0 + kBlockM, p.Sq) - 1);
                const bool none = r0 >= p.Sq || z.lo > z.hi;
                sm.range[i][0] = none ? 1 : a.lo > a.hi ? 0 : a.lo / kBlockN;
                sm.range[i][1] = none ? 0 : z.hi / kBlockN;
            }
            const TileWalk walk = make_walk();
            const int t0 = first_step(walk.steps());
            if (t0 < end_step(walk.steps())) {
                copy_kv(0, false, walk.block(walk.active(0, t0) ? 0 : 1, t0));
                if (walk.apart(t0)) copy_kv(1, false, walk.block(1, t0));
            }
            copy_q(1);
            for (int i = 0; i < 2; ++i) {
                sm.walk[i][0] = walk.shared;
                sm.walk[i][1] = (i == 0 ? walk.own0 : walk.own1) - walk.shared;
                sm.walk[i][2] = walk.first;
                sm.walk[i][3] = walk.next - walk.first;
            }
        }
        __syncwarp();
    }
    if (warp == 8) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem = sm.tmem_base;
    volatile int *abort_flag = &sm.abort_flag;

    if (warp >= 8) {
        setmaxnreg_dec<kOtherRegs>();
        if (warp == 9) {
            // ------------------------------------------------------ TMA producer
            if (lane == 0) {
                const TileWalk walk = make_walk();
                const int t0 = first_step(walk.steps()), t1 = end_step(walk.steps());
                uint32_t n = 0;
                bool ok = true;
                for (int t = t0; t < t1 && ok; ++t) {
                    // K, then V, of the step's block or of both tiles' blocks; the first K
                    // (of each tile) is under way.
                    const uint32_t apart = walk.apart(t) ? 1u : 0u;
                    uint32_t x = t == t0 ? 1 + apart : 0;
                    for (n += x; x < 2 + 2 * apart && ok; ++x, ++n) {
                        if (n >= NS)
                            ok = wait_bounded(&sm.kv_empty[n % NS], ((n / NS) & 1u) ^ 1u, abort_flag, p.status, true,
                                              p.timeout_ns);
                        if (!ok) break;
                        copy_kv(n, (x >> apart) != 0, walk.block(apart ? x & 1 : walk.active(0, t) ? 0 : 1, t));
                    }
                }
                // Every copy still in flight lands before the CTA can exit.
                for (int i = 0; i < 2; ++i)
                    wait_bounded(&sm.q_full[i], 0, abort_flag, p.status, false, p.timeout_ns);
                for (uint32_t L = n > NS ? n - NS : 0; L < n; ++L)
                    wait_bounded(&sm.kv_full[L % NS], (L / NS) & 1u, abort_flag, p.status, false, p.timeout_ns);
            }
            __syncwarp();
        } else if (warp == 8) {
            // --------------------------------------------------- MMA issuer
            // The whole warp runs the schedule; one elected lane issues.
            const TileWalk walk = make_walk();
            const int t0 = first_step(walk.steps()), t1 = end_step(walk.steps());
            if (t0 < t1) {
                const bool leader = elect_one();
                constexpr uint32_t kIdescQK = idesc_bf16_f32(kBlockM, kBlockN, 0, 0);
                constexpr uint32_t kIdescPV = idesc_bf16_f32(kBlockM, D, 0, 1);
                constexpr uint32_t kChunkBytes = Smem::kChunkBytes;
                const uint64_t q_desc = smem_desc_sw128(smem_u32(&sm.q[0][0][0]), 16, 1024);
                const uint64_t k_desc = smem_desc_sw128(smem_u32(&sm.kv[0][0][0]), 16, 1024);
                const uint64_t v_desc = smem_desc_sw128(smem_u32(&sm.kv[0][0][0]), kChunkBytes, 1024);
                bool ok = true;
                auto wait = [&](uint64_t *bar, uint32_t parity) {
                    if (ok)
                        ok = __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, p.status, true,
                                                                  p.timeout_ns));
                    tc_fence_after();
                };
                auto wait_kv = [&](uint32_t L) { wait(&sm.kv_full[L % NS], (L / NS) & 1u); };
                auto issue_s = [&](int i, uint32_t L) {
                    const uint64_t a0 = q_desc + ((i * kTileBytes) >> 4);
                    const uint64_t b0 = k_desc + (((L % NS) * kTileBytes) >> 4);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t off = ((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4;
                            mma_ss_k<false>(tmem + i * kBlockN, a0 + off, b0 + off, kIdescQK, ks > 0 ? 1u : 0u);
                        }
                        tc_commit(&sm.s_full[i]);
                    }
                    __syncwarp();
                };
                // Steps [t0, n_i) are tile i's.  Of step t, whose copies begin at `at`:
                // K of tile i at at + i, V at at + 2 + i where the tiles are apart, else
                // at and at + 1.
                const int n0 = min(walk.n0, t1), n1 = min(walk.n1, t1);
                const int apart0 = walk.shared, apart1 = min(n0, n1);  // steps that are apart
                uint32_t at = 0;
                uint32_t apart = t0 >= apart0 && t0 < apart1 ? 1u : 0u;
                for (int i = 0; i < 2 && ok; ++i) {
                    if (t0 >= (i == 0 ? n0 : n1)) continue;
                    wait(&sm.q_full[i], 0);
                    wait_kv(i * apart);
                    if (ok) issue_s(i, i * apart);
                }
                if (ok && leader) {
                    tc_commit(&sm.kv_empty[0]);
                    if (apart) tc_commit(&sm.kv_empty[1]);
                }
                __syncwarp();

                for (int t = t0; t < t1 && ok; ++t) {
                    const uint32_t par = (uint32_t)(t - t0) & 1u, first = t > t0 ? 1u : 0u;
                    const uint32_t at_next = at + 2 + 2 * apart;
                    const uint32_t apart_next = t + 1 >= apart0 && t + 1 < apart1 ? 1u : 0u;
                    const uint32_t v0 = at + 1 + apart, v1 = v0 + apart;                // V of this step
                    const uint32_t k0 = at_next, k1 = at_next + apart_next;             // K of the next
                    const bool more0 = t + 1 < n0, more1 = t + 1 < n1;
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        const bool here = t < (i == 0 ? n0 : n1), more = i == 0 ? more0 : more1;
                        const uint32_t L = i == 0 ? v0 : v1;
                        if (here) {
                            const uint64_t vb = v_desc + (((L % NS) * kTileBytes) >> 4);
                            const uint32_t o_tmem = tmem + 2 * kBlockN + i * D;
                            const uint32_t p_tmem = tmem + i * kBlockN;
                            if (i == 0 || apart || t >= n0) wait_kv(L);
                            // PV in two halves of 64 keys, each as soon as its P is in TMEM.
                            wait(&sm.p_half[i], par);
                            if (!ok) break;
                            if (leader) {
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    mma_ts_k<false>(o_tmem, p_tmem + ks * 8, vb + ((ks * 16 * 128) >> 4), kIdescPV,
                                                    ks > 0 ? 1u : first);
                            }
                            __syncwarp();
                            wait(&sm.p_full[i], par);
                            if (!ok) break;
                            if (leader) {
#pragma unroll
                                for (int ks = 4; ks < 8; ++ks)
                                    mma_ts_k<false>(o_tmem, p_tmem + ks * 8, vb + ((ks * 16 * 128) >> 4), kIdescPV, 1u);
                                if (!more) tc_commit(&sm.o_final[i]);
                            }
                            __syncwarp();
                        }
                        if (more) {
                            if (i == 0 || apart_next || !more0) wait_kv(i == 0 ? k0 : k1);
                            if (!ok) break;
                            issue_s(i, i == 0 ? k0 : k1);
                        }
                    }
                    if (ok && leader) {
                        tc_commit(&sm.kv_empty[v0 % NS]);
                        if (apart) tc_commit(&sm.kv_empty[v1 % NS]);
                        if (more0 || more1) tc_commit(&sm.kv_empty[k0 % NS]);
                        if (apart_next) tc_commit(&sm.kv_empty[k1 % NS]);
                    }
                    __syncwarp();
                    at = at_next;
                    apart = apart_next;
                }
                if (!ok) {
                    // Let every MMA already issued finish before TMEM is freed.
                    if (leader) tc_commit(&sm.drain);
                    __syncwarp();
                    wait_bounded(&sm.drain, 0, abort_flag, p.status, false, p.timeout_ns);
                }
            }
            __syncwarp();
        }
        // warps 10-11: idle
    } else {
        // ------------------------------------- softmax / correction / epilogue
        setmaxnreg_inc<kSoftmaxRegs>();
        const int i = warp >> 2;
        const int row_in_tile = threadIdx.x & (kBlockM - 1);
        const int row = q0 + i * kBlockM + row_in_tile;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_base + i * kBlockN;
        const uint32_t o_tmem = tmem + lane_base + 2 * kBlockN + i * D;
        // Rows behind the last see what it sees (their results go nowhere).
        KeyRange kr = window_range(p, min(row, p.Sq - 1));
        if (kr.lo > kr.hi) kr.hi = -1;  // no key, so no first key either
        const float c = p.scale_log2;
        const float tau = p.rescale_threshold;
        // With a modifier the scores are transformed into log2 units before
        // the max, so the exponent step multiplies by 1 instead of c.
        const float c_exp = MOD ? 1.0f : c;
        const float slope2 = (MOD & 2) ? __ldg(p.alibi_slopes + hq) * kLog2eF : 0.0f;
        const float k1 = p.softcap_in * (2.0f * kLog2eF);  // soft-cap: 2 log2(e) scale / cap
        const float diag_f = (float)(row + p.Sk - p.Sq);
        float m_run = -INFINITY;
        float l_run = 0.0f;   // row sum of the unrounded p (the LSE's normaliser)
        float l_pv = 0.0f;    // row sum of the p that PV consumes (the output's normaliser)
        bool ok = true;
        int t0, blocks;  // this tile's steps: [t0, t0 + blocks)
        {
            const TileWalk walk = make_walk();
            t0 = first_step(walk.steps());
            blocks = max(0, min(i == 0 ? walk.n0 : walk.n1, end_step(walk.steps())) - t0);
        }
        for (int t = 0; t < blocks; ++t) {
            // The step's block; from shared memory, so that no register holds the walk.
            const volatile int *w = sm.walk[i];
            int j = t0 + t;
            j += j >= w[0] ? w[1] : j < w[2] ? 0 : w[3];
            ok = wait_bounded(&sm.s_full[i], (uint32_t)t & 1u, abort_flag, p.status, true, p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();

            uint32_t sr[kBlockN];
            tmem_ld32(s_tmem + 0, sr + 0);
            tmem_ld32(s_tmem + 32, sr + 32);
            tmem_ld32(s_tmem + 64, sr + 64);
            tmem_ld32(s_tmem + 96, sr + 96);
            tmem_wait_ld();
            reg_fence32(sr + 0);
            reg_fence32(sr + 32);
            reg_fence32(sr + 64);
            reg_fence32(sr + 96);
            float *s = reinterpret_cast<float *>(sr);

            const int key0 = j * kBlockN;
            const float dist0 = diag_f - (float)key0;  // distance to key0 of this block
            const bool need_mask = (key0 < kr.lo && key0 + kBlockN > p.sinks) || key0 + kBlockN - 1 > kr.hi;
            const bool masked = __any_sync(0xffffffffu, need_mask);
            float row_max = -INFINITY;
            uint32_t unseen = 0u;  // groups of 32 keys that no row of the warp sees
            if (masked) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint32_t bits = visible_bits(key0 + 32 * g, kr.lo, kr.hi, p.sinks);
                    if (!__any_sync(0xffffffffu, bits != 0u)) {
                        unseen |= 1u << g;
                        continue;
                    }
                    if (MOD)
                        modify_scores<MOD, 32>(s + 32 * g, c, k1, p.softcap_out, slope2,
                                               dist0 - (float)(32 * g));
                    if (!__all_sync(0xffffffffu, bits == ~0u)) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((bits >> e) & 1u)) s[32 * g + e] = -INFINITY;
                    }
                    row_max = fmaxf(row_max, block_max32(s + 32 * g));
                }
            } else {
                if (MOD) modify_scores<MOD, kBlockN>(s, c, k1, p.softcap_out, slope2, dist0);
                float mx[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) mx[u] = fmax3(s[u], s[u + 4], s[u + 8]);
#pragma unroll
                for (int e = 12; e < kBlockN - 4; e += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = fmax3(mx[u], s[e + u], s[e + 4 + u]);
#pragma unroll
                for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], s[kBlockN - 4 + u]);
                row_max = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
            }
            const float m_cand = MOD ? row_max : row_max * c;
            float alpha = 1.0f;
            if (m_cand > m_run + tau) {
                alpha = ex2_mufu(m_run - m_cand);
                m_run = m_cand;
            }
            const float neg_m = m_run == -INFINITY ? 0.0f : -m_run;
            l_run *= alpha;
            l_pv *= alpha;

            // Correction first: rescale this row of O in TMEM (rare once the
            // max settles) before any P of this block is handed over.  PV of
            // the previous block is complete: the commit that signalled S of
            // this block covers every earlier MMA.
            if (t > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t r[32];
                    tmem_ld32(o_tmem + ch * 32, r);
                    tmem_wait_ld();
                    reg_fence32(r);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a0, a1;
                        mul2(a0, a1, __uint_as_float(r[e]), __uint_as_float(r[e + 1]), alpha, alpha);
                        r[e] = __float_as_uint(a0);
                        r[e + 1] = __float_as_uint(a1);
                    }
                    tmem_st32(o_tmem + ch * 32, r);
                }
            }

            // Probabilities p = 2^(s*c - m) in pairs, row sums, bf16 pairs to
            // TMEM, in two halves: the MMA warp starts PV on keys [0, 64) while
            // this warp computes keys [64, 128).
            uint32_t pk[kBlockN / 2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (masked) {
#pragma unroll
                    for (int g = 2 * h; g < 2 * h + 2; ++g) {
                        if ((unseen >> g) & 1u) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[16 * g + e] = 0u;
                        } else {
                            exp_pack_group(s + 32 * g, c_exp, neg_m, pk + 16 * g, l_run, l_pv);
                        }
                    }
                } else {
                    exp_pack_half<EXP_MODE>(s + 64 * h, c_exp, neg_m, pk + 32 * h, l_run, l_pv);
                }
                __syncwarp();
                tmem_st32(s_tmem + 32 * h, pk + 32 * h);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(h == 0 ? &sm.p_half[i] : &sm.p_full[i]);
            }
        }

        // ----------------------------------------------------------- epilogue
        // A tile without a key block writes zeros, through Q's buffer: Q must have
        // landed there first.
        if (ok) {
            ok = wait_bounded(blocks > 0 ? &sm.o_final[i] : &sm.q_full[i], 0, abort_flag, p.status, true,
                              p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        }
        if (ok) {
            const bool row_ok = row < p.Sq;
            // Normalise by the sum of the rounded weights that PV applied.
            const float inv_l = l_pv > 0.0f ? 1.0f / l_pv : 0.0f;
            // (From shared memory, so that no register holds them till here.)
            const int eb = *(volatile int *)&sm.item[0];
            const int eh = *(volatile int *)&sm.item[1];
            const int ep = *(volatile int *)&sm.item[2];
#pragma unroll
            for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t r[32];
                if (blocks > 0) {
                    tmem_ld32(o_tmem + ch * 32, r);
                    tmem_wait_ld();
                    reg_fence32(r);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = 0u;
                }
                if constexpr (PARTS) {
                    if (row_ok) {
                        float4 *dst = reinterpret_cast<float4 *>(
                            p.part_o + ((((size_t)ep * p.B + eb) * p.Sq + row) * p.Hq + eh) * (size_t)D + ch * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_float4(__uint_as_float(r[4 * e]) * inv_l, __uint_as_float(r[4 * e + 1]) * inv_l,
                                                 __uint_as_float(r[4 * e + 2]) * inv_l,
                                                 __uint_as_float(r[4 * e + 3]) * inv_l);
                    }
                } else {
                    // Into Q's buffer (its last product is done), laid out as TMA has it:
                    // 16-byte piece c of a row's 128 bytes at c ^ (row & 7).
                    uint8_t *dst = sm.q[i][ch / 2] + row_in_tile * 128;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint4 w4;
                        uint32_t *w = reinterpret_cast<uint32_t *>(&w4);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            w[x] = pack_bf16x2(__uint_as_float(r[8 * e + 2 * x]) * inv_l,
                                               __uint_as_float(r[8 * e + 2 * x + 1]) * inv_l);
                        *reinterpret_cast<uint4 *>(dst + (((ch & 1) * 4 + e) ^ (row_in_tile & 7)) * 16) = w4;
                    }
                }
            }
            if (row_ok) {
                float lse = l_run > 0.0f ? (m_run + log2f(l_run)) * 0.69314718055994531f : -INFINITY;
                if (PARTS && l_run != l_run) lse = l_run;  // the join must not take NaN for a part without a key
                float *dst = PARTS ? p.part_lse + (size_t)ep * p.B * p.Hq * p.Sq : p.lse;
                dst[((size_t)eb * p.Hq + eh) * p.Sq + row] = lse;
            }
        }
        if constexpr (!PARTS) {
            fence_proxy_async_smem();
            named_bar_sync(1 + i, kBlockM);  // every warp of the tile, after a wait that ran out too
            if (ok && (warp & 3) == 0 && lane == 0 && row < p.Sq) {  // the tile's first row: not behind the last
                for (int ch = 0; ch < Smem::kChunks; ++ch)
                    tma_store_4d(&p.tm_o, sm.q[i][ch], ch * 64, row, sm.item[1], sm.item[0]);
                bulk_store_wait();
            }
        }
    }

    // ------------------------------------------------------------ teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of attn_fwd_window_kernel<..., PARTS = true>: O = sum_s w_s O_s, w_s =
// exp(LSE_s - LSE).  D / 4 lanes per row of O; the parts in order.
constexpr int kFwdJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kFwdJoinThreads)
attn_fwd_join_kernel(const __grid_constant__ WindowParams p) {
    constexpr int kLanes = D / 4;
    wait_for_primary();
    const long long rows = (long long)p.B * p.Sq * p.Hq;
    const long long r = (long long)blockIdx.x * (kFwdJoinThreads / kLanes) + threadIdx.x / kLanes;
    const int d = (threadIdx.x % kLanes) * 4;
    if (r >= rows) return;
    const int hq = (int)(r % p.Hq), row = (int)(r / p.Hq % p.Sq), b = (int)(r / p.Hq / p.Sq);
    const size_t at = ((size_t)b * p.Hq + hq) * p.Sq + row;
    const size_t lses = (size_t)p.B * p.Hq * p.Sq;
    float m = -INFINITY;
    for (int s = 0; s < p.parts; ++s) m = fmaxf(m, p.part_lse[s * lses + at]);
    float sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < p.parts; ++s) {
        const float l = p.part_lse[s * lses + at];
        const float4 v = *reinterpret_cast<const float4 *>(p.part_o + ((size_t)s * rows + r) * D + d);
        if (l == -INFINITY) continue;  // no key of this part
        const float w = ex2_mufu((l - m) * kLog2eF);
        sum += w;
        o.x = fmaf(v.x, w, o.x);
        o.y = fmaf(v.y, w, o.y);
        o.z = fmaf(v.z, w, o.z);
        o.w = fmaf(v.w, w, o.w);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    *reinterpret_cast<uint2 *>(p.o + (size_t)r * D + d) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (d == 0) p.lse[at] = sum > 0.0f ? m + log2f(sum) * 0.69314718055994531f : -INFINITY;
}

}  // namespace tab
