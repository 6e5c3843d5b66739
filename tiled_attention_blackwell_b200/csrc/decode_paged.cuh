// Attention of one new token per sequence over a paged key/value cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - max s),  s_j = scale <q, k_j>
// over the keys j < len that a window and its first tokens leave visible.
//
// Bound by memory: every visible key's K and V are read once (4 D bytes per
// key and key head in bf16) for 4 D operations per query head, far below the
// tensor cores' rate for any group of heads.  So the work is cut by bytes,
// not by heads: the tiles of kTile keys of all (sequence, key head) pairs
// form one list, and each block takes an equal run of it, whatever the
// lengths are.  A block that holds all of a pair's tiles writes its output;
// a pair that crosses a block's end leaves partial results (maximum, sums,
// unnormalised output), which decode_join_kernel joins in the order of the
// blocks, so the result does not depend on the timing.
//
// A pair here is a sequence and kHeads neighbouring key heads, whose rows in
// the cache are adjacent: kHeads * D * bytes is 256 where the heads allow it.
// (Read head by head, a key's 128 or 64 bytes lie 1 KB and more apart, and
// the copies run at 67 % and 41 % of the copy rate instead of 95 %.)
//
// Warp roles: warps 0-3 compute, warps 4-7 copy.  Warp
// w works on head w % kHeads, as part of team w / kHeads; team t takes the
// tiles g = t, t + kTeams, ... of the block's run and keeps the running
// maximum, sums and output of its head in registers.  The teams' results are
// joined through shared memory at the end of a pair.  The copying warps walk
// the block's whole run ahead of the computing ones, across the ends of
// pairs, so the copies never pause: 16 keys of K and of V are one TMA box
// each (a page holds a multiple of 16 keys), in a ring of kStages tiles.
//
// Products: mma.sync m16n8k16 with 16 keys (S^T = K Q^T), then 16 values (O^T =
// V^T P^T) as rows and the query heads of one key head as columns, in blocks of
// 8: eight heads or fewer waste nothing.  P goes from the layout of a result to
// that of an operand by a transposition within the warp.  (tcgen05 needs 64
// rows or more of the other operand's heads; here the tensor pipe is idle most
// of the time either way, and the registers hold S, P and O without a trip
// through tensor memory.)  An e4m3 cache is widened to f16 in registers,
// exactly; Q is scaled by a power of two per head so that f16 holds it.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace tab {

constexpr int kDecWarps = 4;                         // computing warps
constexpr int kDecCopyWarps = 4;
constexpr int kDecThreads = (kDecWarps + kDecCopyWarps) * 32;
constexpr int kDecRows = 16;                         // query heads of a key head per pair, at most
constexpr int kDecBlock = 16;                        // keys per TMA box
constexpr int kDecCtasPerSm = 2;
// Registers: 512 threads per SM launch with 128 each; setmaxnreg moves them
// from the copying to the computing warpgroup of a block.  The split must not
// exceed the launch allocation (a larger request would wait forever), and the
// host checks the compiled count.
constexpr int kDecLaunchRegs = 128;
constexpr int kDecComputeRegs = 200;
constexpr int kDecCopyRegs = 56;
static_assert(kDecComputeRegs + kDecCopyRegs <= 2 * kDecLaunchRegs, "register split exceeds the launch allocation");
// A row's maximum moves only when a tile raises it by more than this (log2
// units), as in the forward; P stays below 2^8.
constexpr float kDecTau = 8.0f;
// f16 weights (e4m3 caches) are 2^kDecBias times P, so at most 2^15, within f16:
// its smallest step, 2^-24, is then 2^-31 of a weight of 1.  Without it many small
// weights beside a first token 17 nats above them became zero in the products,
// though not in the sum below.  Partial results scale alike; maxima are
// handed on less the bias, so that only the weights know of it.
constexpr float kDecBias = 7.0f;

struct DecodeParams {
    CUtensorMap tm_k, tm_v;  // [pages][page_size][Hkv][D], box 16 keys of kHeads heads
    const __nv_bfloat16 *q;  // [B][Hq][D]
    __nv_bfloat16 *o;        // [B][Hq][D]
    float *lse;              // [B][Hq]
    const int *page_table;   // [B][max_pages]
    const int *seq_lens;     // [B], the new token counted
    int *status;
    // Workspace: per block two partial results (a pair that begins before
    // the block, one that ends behind it) and one record.
    float *part_o;           // [blocks][2][kHeads][16][D], relative to the partial's maximum
    float2 *part_ml;         // [blocks][2][kHeads][16]: maximum (log2), sum
    int4 *record;            // [blocks]: the pair that is first cut at this block's end
    int B, Hq, Hkv, group, hchunks;  // hchunks: parts of a key head's query heads
    int max_pages, page_size, num_pages;
    int window_left, sinks;
    float scale_log2;        // scale * k_descale * log2(e)
    float v_descale;
    float softcap_in, softcap_out;  // scale * k_descale / cap, cap * log2(e); 0: none
    const float *alibi_slopes;
};

// The visible tiles of a sequence: ns tiles from key 0 on (first tokens),
// then those from tile w0 on.  `lo` is the window's first key.
struct SeqTiles {
    int len, lo, ns, w0, n;
};

template <int kTile>
__device__ __forceinline__ SeqTiles seq_tiles(const DecodeParams &p, int b) {
    SeqTiles s;
    s.len = min(max(__ldg(p.seq_lens + b), 0), p.max_pages * p.page_size);
    s.lo = p.window_left >= 0 ? max(0, s.len - 1 - p.window_left) : 0;
    s.w0 = s.lo / kTile;
    s.ns = min((min(p.sinks, s.lo) + kTile - 1) / kTile, s.w0);
    s.n = s.ns + (s.len + kTile - 1) / kTile - s.w0;
    return s;
}

// 16-bit operand type of the products: bf16, or f16 for an e4m3 cache.
template <bool F8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (F8)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// The f16 pairs of the low and the high two e4m3 codes of a word (exact).
__device__ __forceinline__ void widen_e4m3x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Transposes an 8 x 8 matrix of 16-bit values held as lane (row, column pair).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Weights of two heads in the operand type.  bf16: in two words, what the first
// rounding leaves in `rest`, so that a weight is off by 2^-17, and their sum in
// fp32 normalises them.  (One word, normalised by the sum of what it held, put
// the output off by sqrt(2) of its own rounding.  The time is the keys' bytes
// either way: 64 ragged sequences of 32 / 8 heads of 128 172.9 us, as with one
// word; 48 of 16 / 16 heads of 64 128.0 against 127.4.)  f16 weights are off by
// 2^-11 of themselves or by 2^-32 of the largest (kDecBias): less than the
// output's own rounding, 2^-8 of the largest V, for the 2^23 keys that n 2^-32
// allows.
template <bool F8>
__device__ __forceinline__ uint32_t pack_weights(float p0, float p1, uint32_t &rest) {
    if constexpr (F8) {
        return pack_f16x2(p0, p1);
    } else {
        const uint32_t h = pack_bf16x2(p0, p1);
        rest = pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
        return h;
    }
}

// kBlocks boxes of 16 keys of kHeads heads per tile; NB blocks of 8 query heads.
template <int D, bool F8, int kHeads, int NB, int kBlocks, int kStages>
struct DecodeSmem {
    static constexpr int kRowBytes = D * (F8 ? 1 : 2);
    static constexpr int kHeadBytes = kDecBlock * kRowBytes;  // one head's part of a box
    static constexpr int kBoxBytes = kHeads * kHeadBytes;
    static constexpr int kPitch = kRowBytes < 128 ? kRowBytes : 128;  // bytes per key in a chunk
    static constexpr int kChunkBytes = kDecBlock * kPitch;            // 128 bytes of every key
    static constexpr int kTile = kDecBlock * kBlocks;
    static constexpr int kTeams = kDecWarps / kHeads;
    uint8_t k[kStages][kBlocks][kBoxBytes];
    uint8_t v[kStages][kBlocks][kBoxBytes];
    static constexpr int kRows = 8 * NB;
    float o[kDecWarps][kRows][D + 4];  // + 4: rows start in different banks
    float2 ml[kDecWarps][kRows];
    uint64_t full[kStages], empty[kStages];
    long long start, end, share, base;    // this block's run; tiles before sequence b0
    int b0;
    int abort_flag;
};

// Byte of 16-byte piece `c` of key `r` in a box's first chunk: 128 bytes per
// key with the 128-byte swizzle, or 64 with the 64-byte swizzle.  The next 128
// bytes of the keys are the next chunk, laid out the same.
template <int kRowBytes>
__device__ __forceinline__ uint32_t box_offset(int r, int c) {
    if constexpr (kRowBytes >= 128)
        return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
    else
        return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int D, bool F8, int kHeads, int NB, int kBlocks, int kStages>
__global__ void __launch_bounds__(kDecThreads, kDecCtasPerSm)
decode_paged_kernel(const __grid_constant__ DecodeParams p) {
    using Smem = DecodeSmem<D, F8, kHeads, NB, kBlocks, kStages>;
    constexpr int kTile = Smem::kTile, kTeams = Smem::kTeams;
    constexpr int kPieces = Smem::kRowBytes / 16;  // 16-byte pieces of a row
    // Tile g goes to slot g % kStages, which is one team's and one copying
    // warp's alone: no wait can be two phases behind its slot.
    static_assert(kStages % kTeams == 0 && kStages % kDecCopyWarps == 0, "slots belong to fixed warps");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_off = smem_u32(smem_raw);
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (raw_off & 1023u)) & 1023u));
    const int warp = warp_id(), lane = lane_id();
    const int H = p.Hkv / kHeads * p.hchunks;  // pairs per sequence
    volatile int *abort_flag = &sm.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[s], 2 * kBlocks);  // one arrival per box, copied or not
            mbar_init(&sm.empty[s], kHeads);
        }
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kDecWarps && lane == 0) {
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_v);
    }
    // What stands before this launch in the stream may still be ending; from
    // here on its results are read.  The join may begin to start: its blocks
    // wait in turn for this grid's end.
    wait_for_primary();
    launch_dependents();
    if (warp == kDecWarps) {
        // Tiles of all sequences, then this block's run and where it begins.
        // A run has a tile for each team, or the longest pair's if that has fewer:
        // blocks that are there anyway take short pairs one each.
        long long total = 0;
        int longest = 0;
        for (int b = lane; b < p.B; b += 32) {
            const int n = seq_tiles<kTile>(p, b).n;
            total += (long long)n * H;
            longest = max(longest, n);
        }
        for (int o = 16; o > 0; o >>= 1) {
            total += __shfl_xor_sync(0xffffffffu, total, o);
            longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
        }
        const long long share =
            max((long long)min(kTeams, longest), (total + gridDim.x - 1) / (long long)gridDim.x);
        const long long start = min(total, share * blockIdx.x);
        const long long end = min(total, start + share);
        long long base = 0;
        int b0 = 0;
        for (int c = 0; c < p.B && start < end; c += 32) {
            const long long n = c + lane < p.B ? (long long)seq_tiles<kTile>(p, c + lane).n * H : 0;
            long long upto = n;
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += t;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, base + upto > start);
            if (past) {
                const int at = __ffs(past) - 1;
                b0 = c + at;
                base += __shfl_sync(0xffffffffu, upto - n, at);
                break;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0) {
            sm.start = start;
            sm.end = end;
            sm.share = share;
            sm.base = base;
            sm.b0 = b0;
        }
    }
    __syncthreads();
    const long long start = sm.start, end = sm.end;

    if (warp >= kDecWarps) {
        // ------------------------------------------------------------ copies
        setmaxnreg_dec<kDecCopyRegs>();
        const uint32_t n_tiles = (uint32_t)(end - start);
        // This warp's tiles are w, w + kDecCopyWarps, ...; each lane looks up one of
        // the next 32 of them: its pair and its pages.
        const uint32_t w = warp - kDecWarps;
        const uint32_t n_mine = n_tiles > w ? (n_tiles - w - 1) / kDecCopyWarps + 1 : 0;
        long long base = sm.base;
        int b = sm.b0;
        struct Item {
            int page[kBlocks], row[kBlocks], head;  // page -1: no copy
        };
        auto look_up = [&](uint32_t i) {
            Item it{};
            for (int u = 0; u < kBlocks; ++u) it.page[u] = -1;
            if (i >= n_mine) return it;
            const long long pos = start + w + (long long)i * kDecCopyWarps;
            SeqTiles st = seq_tiles<kTile>(p, b);
            while (b + 1 < p.B && pos >= base + (long long)st.n * H) {
                base += (long long)st.n * H;
                st = seq_tiles<kTile>(p, ++b);
            }
            const uint32_t in_seq = (uint32_t)(pos - base);
            const uint32_t pair = in_seq / (uint32_t)st.n;
            const int t = (int)(in_seq - pair * (uint32_t)st.n);
            const int key0 = (t < st.ns ? t : st.w0 + t - st.ns) * kTile;
            it.head = (int)(pair / (uint32_t)p.hchunks) * kHeads;
#pragma unroll
            for (int u = 0; u < kBlocks; ++u) {
                const int key = key0 + u * kDecBlock;
                // Boxes without a visible key are not copied, nor their pages looked up (a
                // cache may have given them to others).
                if (key < st.len && (key + kDecBlock > st.lo || key < p.sinks)) {
                    const int page = key / p.page_size;
                    it.row[u] = key - page * p.page_size;
                    int at = __ldg(p.page_table + (size_t)b * p.max_pages + page);
                    if (at < 0 || at >= p.num_pages) {  // reported; page 0 stands in
                        atomicCAS(p.status, 0, kStatusRange);
                        at = 0;
                    }
                    it.page[u] = at;
                }
            }
            return it;
        };
        // Lane 2 u + v copies box u of K (v = 0) or V (v = 1).
        const int my_u = lane >> 1;
        const bool my_v = lane & 1;
        bool ok = true;
        uint32_t issued = 0;
        Item next = look_up(lane);
        for (uint32_t i0 = 0; i0 < n_mine && ok; i0 += 32) {
            const Item it = next;
            next = look_up(i0 + 32 + lane);
            const uint32_t n = min(32u, n_mine - i0);
            for (uint32_t i = 0; i < n; ++i) {
                const int head = __shfl_sync(0xffffffffu, it.head, i);
                int page = -1, row = 0;
#pragma unroll
                for (int u = 0; u < kBlocks; ++u) {
                    const int pg = __shfl_sync(0xffffffffu, it.page[u], i);
                    const int rw = __shfl_sync(0xffffffffu, it.row[u], i);
                    if (my_u == u) page = pg, row = rw;
                }
                const uint32_t g = w + issued * kDecCopyWarps;
                const uint32_t s = g % kStages;
                ok = __all_sync(0xffffffffu, wait_bounded(&sm.empty[s], ((g / kStages) & 1u) ^ 1u,
                                                          abort_flag, p.status));
                if (!ok) break;
                if (my_u < kBlocks) {
                    if (page >= 0) {
                        mbar_arrive_expect_tx(&sm.full[s], Smem::kBoxBytes);
                        tma_load_5d(my_v ? sm.v[s][my_u] : sm.k[s][my_u], my_v ? &p.tm_v : &p.tm_k,
                                    &sm.full[s], 0, row, 0, head, page);
                    } else {
                        mbar_arrive(&sm.full[s]);
                    }
                }
                __syncwarp();
                ++issued;
            }
        }
        // Copies still in flight land before the block can exit.
        constexpr uint32_t kMine = kStages / kDecCopyWarps;
        for (uint32_t i = issued > kMine ? issued - kMine : 0; i < issued; ++i) {
            const uint32_t g = w + i * kDecCopyWarps;
            wait_bounded(&sm.full[g % kStages], (g / kStages) & 1u, abort_flag, p.status, false);
        }
        return;
    }

    // --------------------------------------------------------------- compute
    setmaxnreg_inc<kDecComputeRegs>();
    const int head = warp % kHeads, team = warp / kHeads;
    const int fr = lane >> 2, fc = lane & 3;  // row (and row + 8) and column pair of a fragment
    // Sequences without a key: zeros and -inf (each block takes every
    // gridDim.x-th sequence).
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (seq_tiles<kTile>(p, b).n > 0) continue;
        for (int i = threadIdx.x; i < p.Hq * (D / 8); i += kDecWarps * 32)
            *reinterpret_cast<uint4 *>(p.o + (size_t)b * p.Hq * D + (size_t)i * 8) = make_uint4(0u, 0u, 0u, 0u);
        for (int i = threadIdx.x; i < p.Hq; i += kDecWarps * 32) p.lse[(size_t)b * p.Hq + i] = -INFINITY;
    }
    if (blockIdx.x == 0) {  // out-of-range lengths are clamped and reported
        for (int b = threadIdx.x; b < p.B; b += kDecWarps * 32) {
            const int len = __ldg(p.seq_lens + b);
            if (len < 0 || len > p.max_pages * p.page_size) atomicCAS(p.status, 0, kStatusRange);
        }
    }
    if (threadIdx.x == 0) p.record[blockIdx.x] = make_int4(0, 0, 0, 0);

    // Where this lane reads K and V (16 keys, two pieces of a chunk at a time).
    constexpr int kAt = kPieces >= 8 ? 4 : 2;
    uint32_t at[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) at[i] = box_offset<Smem::kRowBytes>(lane & 15, 2 * i + (lane >> 4));
    const bool modified = p.softcap_out > 0.0f || p.alibi_slopes != nullptr;

    // The block's run, pair by pair.
    struct Segment {
        SeqTiles st;
        int b, t0, t1;  // tiles [t0, t1) of the pair
        int rows, hq0;  // query heads of a key head, the first of the pair's first key head
        uint32_t g0;    // the block's tiles before it
    };
    long long pos = start, base = sm.base;
    int next_b = sm.b0;
    auto next_segment = [&](Segment &s) -> bool {
        while (pos < end && next_b < p.B) {
            s.st = seq_tiles<kTile>(p, next_b);
            if (pos >= base + (long long)s.st.n * H) {
                base += (long long)s.st.n * H;
                ++next_b;
                continue;
            }
            const uint32_t in_seq = (uint32_t)(pos - base);
            const int pair = (int)(in_seq / (uint32_t)s.st.n);
            s.b = next_b;
            s.t0 = (int)(in_seq - (uint32_t)pair * (uint32_t)s.st.n);
            s.t1 = (int)min((long long)s.st.n, s.t0 + (end - pos));
            const int heads = pair / p.hchunks, r0 = (pair - heads * p.hchunks) * Smem::kRows;
            s.rows = min(Smem::kRows, p.group - r0);
            s.hq0 = heads * kHeads * p.group + r0;
            s.g0 = (uint32_t)(pos - start);
            pos += s.t1 - s.t0;
            return true;
        }
        return false;
    };
    // Q of a pair as the B operand (this lane: head 8 nb + fr), loaded while the
    // pair before it is joined.  bf16: K index k of step ks is value 16 ks + k.
    // e4m3: the A operand's word holds four neighbouring values, so index (2c,
    // 2c+1, 2c+8, 2c+9) is value 16 ks + 4c + (0..3) on both sides.
    uint32_t qb[NB][D / 16][2];
    auto load_q = [&](const Segment &s) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int r = 8 * nb + fr;
            const bool there = r < s.rows;
            const __nv_bfloat16 *q =
                p.q + ((size_t)s.b * p.Hq + s.hq0 + head * p.group + (there ? r : 0)) * D;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                if constexpr (F8) {
                    const uint2 w = there ? *reinterpret_cast<const uint2 *>(q + 16 * ks + 4 * fc) : make_uint2(0u, 0u);
                    qb[nb][ks][0] = w.x;
                    qb[nb][ks][1] = w.y;
                } else {
                    qb[nb][ks][0] = there ? *reinterpret_cast<const uint32_t *>(q + 16 * ks + 2 * fc) : 0u;
                    qb[nb][ks][1] = there ? *reinterpret_cast<const uint32_t *>(q + 16 * ks + 8 + 2 * fc) : 0u;
                }
            }
        }
    };

    bool ok = true;
    Segment seg, next;
    bool more = next_segment(next);
    if (more) load_q(next);
    while (more) {
        seg = next;
        const SeqTiles &st = seg.st;
        const int rows = seg.rows, t0 = seg.t0, t1 = seg.t1;
        const int hq = seg.hq0 + head * p.group;  // of this warp's head
        // Per head 8 nb + 2 fc + i, which is column i of this lane's results: factor
        // of the scores, soft-cap's, slope.
        float c_head[NB][2], cap_head[NB][2], slope[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float up = 1.0f;
            if constexpr (F8) {
                // To f16, by a power of two per head.
                float amax = 0.0f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qb[nb][ks][i] << 16)),
                                                 fabsf(__uint_as_float(qb[nb][ks][i] & 0xffff0000u))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^-e with amax in [2^e, 2^(e+1)); e within [-100, 120], and 0 for
                // heads of zeros or with infinities (f16 keeps those).
                int e = (int)(__float_as_uint(amax) >> 23) - 127;
                e = amax == 0.0f || e > 127 ? 0 : min(max(e, -100), 120);
                const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qb[nb][ks][i] = pack_f16x2(__uint_as_float(qb[nb][ks][i] << 16) * down,
                                                   __uint_as_float(qb[nb][ks][i] & 0xffff0000u) * down);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float f = F8 ? __shfl_sync(0xffffffffu, up, (2 * fc + i) * 4) : 1.0f;
                c_head[nb][i] = p.scale_log2 * f;
                cap_head[nb][i] = p.softcap_in * (2.0f * kLog2eF) * f;
                const int r = 8 * nb + 2 * fc + i;
                slope[nb][i] =
                    p.alibi_slopes && r < rows ? __ldg(p.alibi_slopes + hq + r) * kLog2eF : 0.0f;
            }
        }

        float acc[D / 16][NB][4];
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][nb][e] = 0.0f;
        float m[NB][2], l[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) m[nb][i] = -INFINITY, l[nb][i] = 0.0f;

        // This team's tiles of the pair.
        const uint32_t g0 = seg.g0;
        int t = t0 + (int)((team + kTeams - g0 % kTeams) % kTeams);
        for (; t < t1; t += kTeams) {
            const uint32_t g = g0 + (uint32_t)(t - t0);
            const uint32_t s = g % kStages;
            if (ok)
                ok = __all_sync(0xffffffffu, wait_bounded(&sm.full[s], (g / kStages) & 1u, abort_flag, p.status));
            if (!ok) break;
            const int key0 = (t < st.ns ? t : st.w0 + t - st.ns) * kTile;
            // S^T of the tile: x[u][nb][2 h + i] is key key0 + 16 u + 8 h + fr, head
            // 8 nb + 2 fc + i.  With one block of heads two chains per block of keys.
            constexpr int kChains = NB == 1 ? 2 : 1;
            float x[kBlocks][NB * kChains][4];
#pragma unroll
            for (int u = 0; u < kBlocks; ++u)
#pragma unroll
                for (int nb = 0; nb < NB * kChains; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[u][nb][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < kPieces; c += 2) {
                uint32_t w[kBlocks][4];
#pragma unroll
                for (int u = 0; u < kBlocks; ++u)
                    ldsm4(w[u], smem_u32(sm.k[s][u]) + head * Smem::kHeadBytes + at[c / 2 % kAt] +
                                    (c / 8) * Smem::kChunkBytes);
#pragma unroll
                for (int u = 0; u < kBlocks; ++u) {
                    if constexpr (F8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t a[4];
                            widen_e4m3x4(w[u][2 * i], a[0], a[2]);
                            widen_e4m3x4(w[u][2 * i + 1], a[1], a[3]);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma16816<true>(x[u][NB == 1 ? i : nb], a, qb[nb][c + i][0], qb[nb][c + i][1]);
                        }
                    } else {
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma16816<false>(x[u][NB == 1 ? (c / 2) & 1 : nb], w[u], qb[nb][c / 2][0],
                                            qb[nb][c / 2][1]);
                    }
                }
            }
            if constexpr (NB == 1) {
#pragma unroll
                for (int u = 0; u < kBlocks; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[u][0][e] += x[u][1][e];
            }
            // With a score modifier the scores become log2 units here, else in the
            // exponent.
            if (modified) {
#pragma unroll
                for (int u = 0; u < kBlocks; ++u)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float &x0 = x[u][nb][i], &x1 = x[u][nb][2 + i];
                            if (p.softcap_out > 0.0f) {
                                float r0, r1;
                                softcap_pair(x0, x1, r0, r1, x0, x1, cap_head[nb][i], p.softcap_out);
                            } else {
                                x0 *= c_head[nb][i];
                                x1 *= c_head[nb][i];
                            }
                            const float dist = (float)(st.len - 1 - (key0 + 16 * u + fr));
                            x0 = fmaf(-slope[nb][i], dist, x0);
                            x1 = fmaf(-slope[nb][i], dist - 8.0f, x1);
                        }
            }
            // Keys that the mask hides: their scores become -inf and their values
            // zero, so what lies in them (NaN too) has no part.  see: the keys 16 u +
            // 8 h + 2 fc + (0, 1), whose values this lane holds, as halves of a word.
            uint32_t see[kBlocks][2];
            const bool masked =
                key0 + kTile > st.len || (key0 < st.lo && key0 + kTile > p.sinks);
            if (masked) {
                auto visible = [&](int key) {
                    return key < st.len && (key >= st.lo || key < p.sinks);
                };
#pragma unroll
                for (int u = 0; u < kBlocks; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int first = key0 + 16 * u + 8 * h;
                        see[u][h] = (visible(first + 2 * fc) ? 0xffffu : 0u) |
                                    (visible(first + 2 * fc + 1) ? 0xffff0000u : 0u);
                        if (!visible(first + fr)) {
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) x[u][nb][2 * h] = x[u][nb][2 * h + 1] = -INFINITY;
                        }
                    }
            }
            // P^T as the B operand; bf16: and what its rounding leaves.
            uint32_t pt[kBlocks][NB][2], rest[kBlocks][NB][2];
            float alpha[NB][2];
            bool moved = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float neg_m[2], c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    c[i] = modified ? 1.0f : c_head[nb][i];
                    float mx = fmaxf(x[0][nb][i], x[0][nb][2 + i]);
#pragma unroll
                    for (int u = 1; u < kBlocks; ++u) mx = fmax3(mx, x[u][nb][i], x[u][nb][2 + i]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    mx *= c[i];
                    alpha[nb][i] = 1.0f;
                    if (mx > m[nb][i] + kDecTau) {
                        alpha[nb][i] = ex2_mufu(m[nb][i] - mx);
                        m[nb][i] = mx;
                        moved = true;
                    }
                    neg_m[i] = m[nb][i] == -INFINITY ? 0.0f : (F8 ? kDecBias : 0.0f) - m[nb][i];
                }
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int u = 0; u < kBlocks; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float e0 = ex2_mufu(fmaf(x[u][nb][2 * h], c[0], neg_m[0]));
                        const float e1 = ex2_mufu(fmaf(x[u][nb][2 * h + 1], c[1], neg_m[1]));
                        sum[0] += e0;
                        sum[1] += e1;
                        uint32_t left = 0u;
                        pt[u][nb][h] = transpose8x8(pack_weights<F8>(e0, e1, left));
                        if (!F8) rest[u][nb][h] = transpose8x8(left);
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i) l[nb][i] = fmaf(l[nb][i], alpha[nb][i], sum[i]);
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][nb][e] *= alpha[nb][e & 1];
            }
            // O^T += V^T P^T.  acc[j][nb][i] and [2 + i]: head 8 nb + 2 fc + i, values
            // (bf16) 16 j + fr and 16 j + 8 + fr, or (e4m3, whose words hold value
            // pairs) 16 j + 2 fr and 16 j + 2 fr + 1.  Boxes without a visible key were
            // not copied: `see` hides what is left in them.
#pragma unroll
            for (int u = 0; u < kBlocks; ++u) {
                const uint32_t vb = smem_u32(sm.v[s][u]) + head * Smem::kHeadBytes;
#pragma unroll
                for (int j = 0; j < kPieces; j += 2) {
                    uint32_t w[4];
                    ldsm4_trans(w, vb + at[j / 2 % kAt] + (j / 8) * Smem::kChunkBytes);
                    if (masked) {
                        w[0] &= see[u][0];
                        w[1] &= see[u][1];
                        w[2] &= see[u][0];
                        w[3] &= see[u][1];
                    }
                    if constexpr (F8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t a[4];
                            widen_e4m3x4(__byte_perm(w[2 * i], 0u, 0x3120), a[0], a[1]);
                            widen_e4m3x4(__byte_perm(w[2 * i + 1], 0u, 0x3120), a[2], a[3]);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma16816<true>(acc[j + i][nb], a, pt[u][nb][0], pt[u][nb][1]);
                        }
                    } else {
                        const uint32_t a[4] = {w[0], w[2], w[1], w[3]};
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma16816<false>(acc[j / 2][nb], a, pt[u][nb][0], pt[u][nb][1]);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma16816<false>(acc[j / 2][nb], a, rest[u][nb][0], rest[u][nb][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the tile
            if (lane == 0) mbar_arrive(&sm.empty[s]);
        }

        more = next_segment(next);
        if (more) load_q(next);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (F8) m[nb][i] -= kDecBias;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], o);
            }
        const bool whole = t0 == 0 && t1 == st.n;
        if (whole && t1 == 1) {
            // A pair of one tile is its team's alone: the team writes the output, and
            // the others are already at their next pair.
            if (team == (int)(g0 % kTeams)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = 8 * nb + 2 * fc + i;
                        if (r >= rows) continue;
                        const size_t row = (size_t)seg.b * p.Hq + hq + r;
                        const float inv = l[nb][i] == 0.0f ? 0.0f : p.v_descale / l[nb][i];
                        __nv_bfloat16 *o = p.o + row * D;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            const float v0 = acc[j][nb][i] * inv, v1 = acc[j][nb][2 + i] * inv;
                            if constexpr (F8) {
                                *reinterpret_cast<uint32_t *>(o + 16 * j + 2 * fr) = pack_bf16x2(v0, v1);
                            } else {
                                o[16 * j + fr] = __float2bfloat16_rn(v0);
                                o[16 * j + 8 + fr] = __float2bfloat16_rn(v1);
                            }
                        }
                        if (fr == 0)
                            p.lse[row] = l[nb][i] == 0.0f
                                             ? -INFINITY
                                             : (m[nb][i] + log2f(l[nb][i])) * 0.69314718055994531f;
                    }
            }
            continue;
        }

        // ------------------------------------------- join the teams' results
        // Every warp comes here for every other pair, with or without a tile of it
        // (and after a wait that ran out), so the barriers below always meet.
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * nb + 2 * fc + i;
                if (r >= rows) continue;
                if (fr == 0)
                    sm.ml[warp][r] = make_float2(m[nb][i], l[nb][i]);
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    if constexpr (F8) {
                        *reinterpret_cast<float2 *>(&sm.o[warp][r][16 * j + 2 * fr]) =
                            make_float2(acc[j][nb][i], acc[j][nb][2 + i]);
                    } else {
                        sm.o[warp][r][16 * j + fr] = acc[j][nb][i];
                        sm.o[warp][r][16 * j + 8 + fr] = acc[j][nb][2 + i];
                    }
                }
            }
        const size_t part = (size_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0);
        named_bar_sync(1, kDecWarps * 32);
        for (int i = threadIdx.x; i < kHeads * rows * (D / 4); i += kDecWarps * 32) {
            const int d = (i % (D / 4)) * 4;
            const int k = i / (D / 4) / rows, r = i / (D / 4) % rows;  // head, row
            float mx = sm.ml[k][r].x;
#pragma unroll
            for (int w = 1; w < kTeams; ++w) mx = fmaxf(mx, sm.ml[k + w * kHeads][r].x);
            float ls = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kTeams; ++w) {
                const float2 ml = sm.ml[k + w * kHeads][r];
                const float f = ml.x == -INFINITY ? 0.0f : ex2_mufu(ml.x - mx);
                const float4 ow = *reinterpret_cast<const float4 *>(&sm.o[k + w * kHeads][r][d]);
                ls = fmaf(ml.y, f, ls);
                o.x = fmaf(ow.x, f, o.x);
                o.y = fmaf(ow.y, f, o.y);
                o.z = fmaf(ow.z, f, o.z);
                o.w = fmaf(ow.w, f, o.w);
            }
            if (whole) {
                const size_t row = (size_t)seg.b * p.Hq + seg.hq0 + k * p.group + r;
                const float inv = ls == 0.0f ? 0.0f : p.v_descale / ls;
                *reinterpret_cast<uint2 *>(p.o + row * D + d) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (d == 0) p.lse[row] = ls == 0.0f ? -INFINITY : (mx + log2f(ls)) * 0.69314718055994531f;
            } else {
                const size_t row = (part * kHeads + k) * kDecRows + r;
                *reinterpret_cast<float4 *>(p.part_o + row * D + d) = o;
                if (d == 0) p.part_ml[row] = make_float2(mx, ls);
            }
        }
        named_bar_sync(1, kDecWarps * 32);  // the buffers are free again
        // A pair that begins here and goes on: the join starts at this block.
        if (t0 == 0 && t1 < st.n && threadIdx.x == 0) {
            const long long last = start + g0 + st.n - 1;
            p.record[blockIdx.x] = make_int4(seg.b, seg.hq0, rows, (int)(last / sm.share));
        }
    }
}

// Joins the partial results of the pair that is first cut at the end of block
// blockIdx.x: row blockIdx.y of head blockIdx.z of it.  The partials are those of that block
// (its second) and of the blocks up to the recorded one (their first).
constexpr int kJoinThreads = 256;

struct JoinParams {
    const float *part_o;
    const float2 *part_ml;
    const int4 *record;
    __nv_bfloat16 *o;
    float *lse;
    int Hq, group;
    float v_descale;
};

template <int D, int kHeads>
__global__ void __launch_bounds__(kJoinThreads)
decode_join_kernel(const JoinParams p) {
    constexpr int kCols = D / 4, kParts = kJoinThreads / kCols;  // float4 columns, rows of threads
    __shared__ float4 sum_o[kParts][kCols];
    __shared__ float2 sum_ml[kParts];
    wait_for_primary();
    const int4 rec = p.record[blockIdx.x];
    const int row = blockIdx.y, head = blockIdx.z;
    if (row >= rec.z) return;
    const int first = blockIdx.x, n = rec.w - first + 1;
    const int part = threadIdx.x / kCols, c = threadIdx.x % kCols;
    // Each row of threads joins every kParts-th partial, in order, under a running
    // maximum; then the rows' results, in order.
    float mx = -INFINITY;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    auto add = [&](const float2 &ml, const float4 &v) {
        const float to = fmaxf(mx, ml.x);
        const float f = mx == to ? 1.0f : mx == -INFINITY ? 0.0f : ex2_mufu(mx - to);
        const float g = ml.x == to ? 1.0f : ml.x == -INFINITY ? 0.0f : ex2_mufu(ml.x - to);
        mx = to;
        l = fmaf(l, f, ml.y * g);
        o.x = fmaf(o.x, f, v.x * g);
        o.y = fmaf(o.y, f, v.y * g);
        o.z = fmaf(o.z, f, v.z * g);
        o.w = fmaf(o.w, f, v.w * g);
    };
    // Four partials' loads at a time, each before the first is used: a sequence of
    // 8000 keys, whose pairs have 36, takes 11.1 us in a graph, and 12.6 with one
    // at a time.
    constexpr int kAhead = 4;
    for (int i0 = part; i0 < n; i0 += kAhead * kParts) {
        float2 ml[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kParts;
            if (i >= n) break;
            const size_t at = (((size_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * kHeads + head) * kDecRows + row;
            ml[u] = p.part_ml[at];
            v[u] = *reinterpret_cast<const float4 *>(p.part_o + at * D + 4 * c);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i0 + u * kParts >= n) break;
            add(ml[u], v[u]);
        }
    }
    sum_o[part][c] = o;
    if (c == 0) sum_ml[part] = make_float2(mx, l);
    __syncthreads();
    if (part == 0) {
#pragma unroll
        for (int w = 1; w < kParts; ++w) add(sum_ml[w], sum_o[w][c]);
        const size_t out = (size_t)rec.x * p.Hq + rec.y + head * p.group + row;
        const float inv = l == 0.0f ? 0.0f : p.v_descale / l;
        *reinterpret_cast<uint2 *>(p.o + out * D + 4 * c) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (c == 0) p.lse[out] = l == 0.0f ? -INFINITY : (mx + log2f(l)) * 0.69314718055994531f;
    }
}

}  // namespace tab
