// RMS norm of every query and key head and the rotation by position, in one
// pass over the data; its backward; and the serving form that writes K and V
// of the new tokens to a paged cache.
//
// Per token and head, with x the D values of the head and w the weights:
//   r = (mean_d x_d^2 + eps)^(-1/2),  u_d = w_d x_d r
//   y = R u: the first `rot` values turn in pairs (a, b) by the angle of the
//   token's position, y_a = u_a c - u_b s, y_b = u_b c + u_a s, where the
//   pair is (i, i + rot/2), or (2i, 2i + 1) when interleaved.
// Backward, with g = R^T dy and h = w g:
//   dx_d = r (h_d - x_d r (r sum_e h_e x_e) / D)
//   dw_d = sum over tokens and heads of g_d x_d r
//
// Bound by memory: two bytes in and two out per value (eight in all for a
// query's value in the backward, whose dy is fp32) against about ten
// operations.  D / 8 lanes hold a head, eight values per lane: the four first
// and the four second members of four pairs, so that the rotation stays
// within a lane and only the sums over the head are shuffles.  In the half
// style those are two runs of four values, rot/2 apart; interleaved, one run
// of eight.  A group of lanes takes kNormRows heads of one token at a time:
// their loads are in flight together, and the angles, with the weights
// multiplied in, serve all of them.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace tab {

// Small blocks: one that ends makes room for the next's loads at once.
// Measured on 16384 tokens of 32 heads of 128 (273 MB in and out): 49 us with
// blocks of 128 threads, eight per SM (64 registers: none spilled in this form,
// 124 to 156 bytes a thread in the one with a bf16 cache, 52 to 56 with an e4m3
// one), as long as a plain copy of the same bytes takes; 51 us with 256 threads, four
// per SM, or with blocks that walk over the items and load one ahead; 59 us
// with 71 registers and three blocks of 256.
constexpr int kNormThreads = 128;

struct NormRopeParams {
    // Inputs: bf16 [tokens][H][D], heads contiguous, tokens `*_stride` values apart.
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_out;
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    const void *qw, *kw;      // [D], bf16 or fp32
    const float *cos, *sin;   // [max_positions][rot / 2]
    const int *positions;     // [tokens]
    int *status;
    long long tokens;
    int Hq, Hkv, rot, max_positions;
    int chunks_q, chunks_k;   // kRows-head chunks of a token's query and key heads
    int w_fp32;
    float eps;
    // Serving form: slots [tokens] (negative: padding, left alone), caches
    // [num_slots][Hkv][D].
    const int *slots;
    void *k_cache, *v_cache;
    long long num_slots;
    float k_scale, v_scale;   // e4m3: codes of value * scale
    // Backward.
    const void *dq, *dk;      // [tokens][H][D], contiguous heads, fp32 or bf16
    long long dq_stride, dk_stride;
    int dq_fp32, dk_fp32;
    float *partial;           // [blocks][2][D]
};

// Where a lane's values of a head lie: `a` and `b` are the first values of its
// two runs of four; `turn` says whether they are rotated (then by the angles
// [angle, angle + 4) of the position).
struct LanePlace {
    int a, b, angle;
    bool turn;
};

template <bool INTERLEAVED>
__device__ __forceinline__ LanePlace lane_place(int l, int rot) {
    LanePlace at;
    at.angle = 4 * l;
    at.turn = 8 * l < rot;
    if (INTERLEAVED || !at.turn) {
        at.a = 8 * l;
        at.b = 8 * l + 4;
    } else {
        at.a = 4 * l;
        at.b = 4 * l + rot / 2;
    }
    return at;
}

// A lane's eight values as the first members p and the second members q of
// its four pairs (interleaved: neighbours; half style: run a and run b).
struct Pairs {
    float p[4], q[4];
};

template <bool INTERLEAVED>
__device__ __forceinline__ Pairs make_pairs(const float (&a)[4], const float (&b)[4]) {
    if (INTERLEAVED) return {{a[0], a[2], b[0], b[2]}, {a[1], a[3], b[1], b[3]}};
    return {{a[0], a[1], a[2], a[3]}, {b[0], b[1], b[2], b[3]}};
}

__device__ __forceinline__ void unpack4(float (&v)[4], uint2 w) {
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
}

// Both runs of a row of bf16 values that an output may overwrite in place
// (each thread reads its values before it writes them): not the read-only path.
struct Raw8 {
    uint2 a, b;
};
__device__ __forceinline__ Raw8 load_raw(const __nv_bfloat16 *row, const LanePlace &at) {
    return {*reinterpret_cast<const uint2 *>(row + at.a), *reinterpret_cast<const uint2 *>(row + at.b)};
}

template <bool INTERLEAVED>
__device__ __forceinline__ Pairs unpack8(const Raw8 &r) {
    float a[4], b[4];
    unpack4(a, r.a);
    unpack4(b, r.b);
    return make_pairs<INTERLEAVED>(a, b);
}

template <bool INTERLEAVED>
__device__ __forceinline__ void store_bf16(__nv_bfloat16 *row, const LanePlace &at, const Pairs &y) {
    uint2 a, b;
    if (INTERLEAVED) {
        a = make_uint2(pack_bf16x2(y.p[0], y.q[0]), pack_bf16x2(y.p[1], y.q[1]));
        b = make_uint2(pack_bf16x2(y.p[2], y.q[2]), pack_bf16x2(y.p[3], y.q[3]));
    } else {
        a = make_uint2(pack_bf16x2(y.p[0], y.p[1]), pack_bf16x2(y.p[2], y.p[3]));
        b = make_uint2(pack_bf16x2(y.q[0], y.q[1]), pack_bf16x2(y.q[2], y.q[3]));
    }
    *reinterpret_cast<uint2 *>(row + at.a) = a;
    *reinterpret_cast<uint2 *>(row + at.b) = b;
}

// e4m3 codes of x * scale (nearest even, saturating).
template <bool INTERLEAVED>
__device__ __forceinline__ void store_e4m3(uint8_t *row, const LanePlace &at, const Pairs &x, float scale) {
    Pairs y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y.p[e] = x.p[e] * scale, y.q[e] = x.q[e] * scale;
    uint32_t a, b;
    if (INTERLEAVED) {
        a = pack_e4m3x4(y.p[0], y.q[0], y.p[1], y.q[1]);
        b = pack_e4m3x4(y.p[2], y.q[2], y.p[3], y.q[3]);
    } else {
        a = pack_e4m3x4(y.p[0], y.p[1], y.p[2], y.p[3]);
        b = pack_e4m3x4(y.q[0], y.q[1], y.q[2], y.q[3]);
    }
    *reinterpret_cast<uint32_t *>(row + at.a) = a;
    *reinterpret_cast<uint32_t *>(row + at.b) = b;
}

__device__ __forceinline__ void load4_f32(float (&v)[4], const float *p) {
    const float4 f = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}

template <bool INTERLEAVED>
__device__ __forceinline__ Pairs load_weights(const void *w, int fp32, const LanePlace &at) {
    float a[4], b[4];
    if (fp32) {
        load4_f32(a, static_cast<const float *>(w) + at.a);
        load4_f32(b, static_cast<const float *>(w) + at.b);
    } else {
        const __nv_bfloat16 *h = static_cast<const __nv_bfloat16 *>(w);
        unpack4(a, __ldg(reinterpret_cast<const uint2 *>(h + at.a)));
        unpack4(b, __ldg(reinterpret_cast<const uint2 *>(h + at.b)));
    }
    return make_pairs<INTERLEAVED>(a, b);
}

// Cosines and sines of a lane's four pairs (1 and 0 past `rot`) at the
// position `pos`; one outside the table is clamped and reported.
__device__ __forceinline__ void load_angles(float (&c)[4], float (&s)[4], const NormRopeParams &p,
                                            int pos, const LanePlace &at) {
    if (pos < 0 || pos >= p.max_positions) {
        atomicCAS(p.status, 0, kStatusRange);
        pos = pos < 0 ? 0 : p.max_positions - 1;
    }
    const size_t i = (size_t)pos * (p.rot / 2) + at.angle;
    if (at.turn) {
        load4_f32(c, p.cos + i);
        load4_f32(s, p.sin + i);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = 1.0f, s[e] = 0.0f;
    }
}

// Sum over the D / 8 lanes of a head.
template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// sum_e x_e y_e of a lane's values.
__device__ __forceinline__ float lane_dot(const Pairs &x, const Pairs &y) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        fma2(s0, s1, x.p[e], x.p[e + 1], y.p[e], y.p[e + 1], s0, s1);
        fma2(s0, s1, x.q[e], x.q[e + 1], y.q[e], y.q[e + 1], s0, s1);
    }
    return s0 + s1;
}

// KV: where K goes.  0: k_out, like Q; 1: a bf16 cache; 2: an e4m3 cache
// (with V beside it in both).
constexpr int kNormRows = 4;  // heads of a token that a group of lanes takes together

template <int D, int KV, bool INTERLEAVED>
__global__ void __launch_bounds__(kNormThreads, 8)
norm_rope_kernel(const NormRopeParams p) {
    wait_for_primary();
    launch_dependents();
    constexpr int kLanes = D / 8, kGroups = kNormThreads / kLanes, U = kNormRows;
    const LanePlace at = lane_place<INTERLEAVED>(threadIdx.x % kLanes, p.rot);
    const uint32_t chunks = p.chunks_q + (KV ? 2 : 1) * p.chunks_k;
    // The host bounds the items by 2^31.
    const uint32_t item = blockIdx.x * kGroups + threadIdx.x / kLanes;
    // Groups past the end do the first token's work once more, for the
    // shuffles, and write nothing.
    bool live = item < (uint32_t)p.tokens * chunks;
    const long long token = live ? item / chunks : 0;
    const int chunk = live ? (int)(item % chunks) : 0;
    const int what = chunk < p.chunks_q ? 0 : chunk < p.chunks_q + p.chunks_k ? 1 : 2;  // Q, K, V
    const int h0 = U * (chunk - (what == 0 ? 0 : what == 1 ? p.chunks_q : p.chunks_q + p.chunks_k));
    const int heads = min(U, (what == 0 ? p.Hq : p.Hkv) - h0);
    const __nv_bfloat16 *src = (what == 0   ? p.q + token * p.q_stride
                                : what == 1 ? p.k + token * p.k_stride
                                            : p.v + token * p.v_stride) +
                               (size_t)h0 * D;
    const int pos = __ldg(p.positions + token);
    const int slot = KV ? __ldg(p.slots + token) : 0;
    Raw8 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = load_raw(src + (u < heads ? u : 0) * D, at);
    if (KV) {
        // Padding tokens write nothing; a slot behind the cache is reported.
        if (live && slot >= p.num_slots) atomicCAS(p.status, 0, kStatusRange);
        live = live && slot >= 0 && slot < p.num_slots;
    }
    // y_p = r (x_p wc_p - x_q ws_q),  y_q = r (x_q wc_q + x_p ws_p)
    Pairs wc, ws;
    {
        float c[4], s[4];
        const bool angles = live && what != 2;
        Pairs w{};
        if (angles) {
            w = load_weights<INTERLEAVED>(what == 0 ? p.qw : p.kw, p.w_fp32, at);
            load_angles(c, s, p, pos, at);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = s[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wc.p[e] = w.p[e] * c[e];
            wc.q[e] = w.q[e] * c[e];
            ws.p[e] = w.p[e] * s[e];
            ws.q[e] = -w.q[e] * s[e];
        }
    }
    float r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Pairs x = unpack8<INTERLEAVED>(raw[u]);
        r[u] = rsqrtf(head_sum<D>(lane_dot(x, x)) * (1.0f / D) + p.eps);
    }
    if (!live) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u >= heads) break;
        const Pairs x = unpack8<INTERLEAVED>(raw[u]);
        Pairs y;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            mul2(y.p[e], y.p[e + 1], x.q[e], x.q[e + 1], ws.q[e], ws.q[e + 1]);
            fma2(y.p[e], y.p[e + 1], x.p[e], x.p[e + 1], wc.p[e], wc.p[e + 1], y.p[e], y.p[e + 1]);
            mul2(y.p[e], y.p[e + 1], y.p[e], y.p[e + 1], r[u], r[u]);
            mul2(y.q[e], y.q[e + 1], x.p[e], x.p[e + 1], ws.p[e], ws.p[e + 1]);
            fma2(y.q[e], y.q[e + 1], x.q[e], x.q[e + 1], wc.q[e], wc.q[e + 1], y.q[e], y.q[e + 1]);
            mul2(y.q[e], y.q[e + 1], y.q[e], y.q[e + 1], r[u], r[u]);
        }
        const size_t head = (size_t)(h0 + u) * D;
        if (KV == 0 || what == 0) {
            store_bf16<INTERLEAVED>((what == 0 ? p.q_out + token * p.q_out_stride
                                               : p.k_out + token * p.k_out_stride) + head, at, y);
        } else {
            const size_t off = (size_t)slot * p.Hkv * D + head;
            if (KV == 1) {
                __nv_bfloat16 *row = static_cast<__nv_bfloat16 *>(what == 1 ? p.k_cache : p.v_cache) + off;
                if (what == 1) {
                    store_bf16<INTERLEAVED>(row, at, y);
                } else {
                    *reinterpret_cast<uint2 *>(row + at.a) = raw[u].a;
                    *reinterpret_cast<uint2 *>(row + at.b) = raw[u].b;
                }
            } else {
                uint8_t *row = static_cast<uint8_t *>(what == 1 ? p.k_cache : p.v_cache) + off;
                store_e4m3<INTERLEAVED>(row, at, what == 1 ? y : x, what == 1 ? p.k_scale : p.v_scale);
            }
        }
    }
}

// ----------------------------------------------------------------- backward

// A fixed number of blocks walks over the items, first Q's, then K's, so that
// each block's share of dw stays in registers until its end, and the sum of
// the blocks' shares (norm_rope_dw_kernel, in the blocks' order) does not
// depend on the timing.  Measured on 16384 tokens of 40 heads of 128 (646
// MB): 112 us, 87 % of the copy rate; two heads at a time, or more blocks
// than four of 128 threads per SM, 122 us and more.
constexpr int kNormBwdRows = 4;

template <int D, bool INTERLEAVED>
__device__ __forceinline__ Pairs norm_rope_bwd_side(const NormRopeParams &p, const LanePlace &at,
                                                    bool is_q, uint32_t first_block) {
    constexpr int kGroups = kNormThreads / (D / 8), U = kNormBwdRows;
    const uint32_t chunks = is_q ? p.chunks_q : p.chunks_k;
    const int H = is_q ? p.Hq : p.Hkv;
    const uint32_t items = (uint32_t)p.tokens * chunks;  // below 2^31
    const __nv_bfloat16 *x_base = is_q ? p.q : p.k;
    __nv_bfloat16 *dx_base = is_q ? p.q_out : p.k_out;
    const long long x_stride = is_q ? p.q_stride : p.k_stride;
    const long long dx_stride = is_q ? p.q_out_stride : p.k_out_stride;
    const long long dy_stride = is_q ? p.dq_stride : p.dk_stride;
    const void *dy_base = is_q ? p.dq : p.dk;
    const int fp32 = is_q ? p.dq_fp32 : p.dk_fp32;
    const Pairs w = load_weights<INTERLEAVED>(is_q ? p.qw : p.kw, p.w_fp32, at);
    Pairs dw{};
    // Whole warps loop together, as the shuffles need.
    for (uint32_t base = first_block * kGroups; base < items; base += gridDim.x * kGroups) {
        const uint32_t mine = base + threadIdx.x / (D / 8);
        const bool live = mine < items;
        const uint32_t item = live ? mine : 0;
        const long long token = item / chunks;
        const int h0 = U * (int)(item % chunks);
        const int heads = live ? min(U, H - h0) : 0;
        const int pos = __ldg(p.positions + token);
        const __nv_bfloat16 *src = x_base + token * x_stride + (size_t)h0 * D;
        const long long dy_at = token * dy_stride + (long long)h0 * D;
        Raw8 raw[U];
        float ga[U][4], gb[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // A row that is not there is read as the chunk's first, and adds nothing.
            const int row = u < heads ? u * D : 0;
            raw[u] = load_raw(src + row, at);
            if (fp32) {
                const float *dy = static_cast<const float *>(dy_base) + dy_at + row;
                load4_f32(ga[u], dy + at.a);
                load4_f32(gb[u], dy + at.b);
            } else {
                const __nv_bfloat16 *dy = static_cast<const __nv_bfloat16 *>(dy_base) + dy_at + row;
                unpack4(ga[u], __ldg(reinterpret_cast<const uint2 *>(dy + at.a)));
                unpack4(gb[u], __ldg(reinterpret_cast<const uint2 *>(dy + at.b)));
            }
        }
        float c[4], s[4];
        load_angles(c, s, p, pos, at);
        __nv_bfloat16 *dst = dx_base + token * dx_stride + (size_t)h0 * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Pairs x = unpack8<INTERLEAVED>(raw[u]);
            const Pairs dy = make_pairs<INTERLEAVED>(ga[u], gb[u]);
            Pairs g, gx;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                mul2(g.p[e], g.p[e + 1], dy.q[e], dy.q[e + 1], s[e], s[e + 1]);
                fma2(g.p[e], g.p[e + 1], dy.p[e], dy.p[e + 1], c[e], c[e + 1], g.p[e], g.p[e + 1]);
                mul2(g.q[e], g.q[e + 1], dy.p[e], dy.p[e + 1], -s[e], -s[e + 1]);
                fma2(g.q[e], g.q[e + 1], dy.q[e], dy.q[e + 1], c[e], c[e + 1], g.q[e], g.q[e + 1]);
                mul2(gx.p[e], gx.p[e + 1], g.p[e], g.p[e + 1], x.p[e], x.p[e + 1]);
                mul2(gx.q[e], gx.q[e + 1], g.q[e], g.q[e + 1], x.q[e], x.q[e + 1]);
            }
            const float r = rsqrtf(head_sum<D>(lane_dot(x, x)) * (1.0f / D) + p.eps);
            // dx = r (h - (x r) (r mean(h x))): x r and r mean(h x) are of the sizes of 1
            // and h, where r^3 leaves fp32 long before the result does (|x| of 1e15).
            const float t = -r * (head_sum<D>(lane_dot(w, gx)) * (1.0f / D));
            if (u >= heads) continue;
            Pairs dx;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                fma2(dw.p[e], dw.p[e + 1], gx.p[e], gx.p[e + 1], r, r, dw.p[e], dw.p[e + 1]);
                fma2(dw.q[e], dw.q[e + 1], gx.q[e], gx.q[e + 1], r, r, dw.q[e], dw.q[e + 1]);
                mul2(g.p[e], g.p[e + 1], g.p[e], g.p[e + 1], w.p[e], w.p[e + 1]);
                mul2(g.q[e], g.q[e + 1], g.q[e], g.q[e + 1], w.q[e], w.q[e + 1]);
                mul2(dx.p[e], dx.p[e + 1], x.p[e], x.p[e + 1], r, r);
                mul2(dx.q[e], dx.q[e + 1], x.q[e], x.q[e + 1], r, r);
                fma2(dx.p[e], dx.p[e + 1], dx.p[e], dx.p[e + 1], t, t, g.p[e], g.p[e + 1]);
                fma2(dx.q[e], dx.q[e + 1], dx.q[e], dx.q[e + 1], t, t, g.q[e], g.q[e + 1]);
                mul2(dx.p[e], dx.p[e + 1], dx.p[e], dx.p[e + 1], r, r);
                mul2(dx.q[e], dx.q[e + 1], dx.q[e], dx.q[e + 1], r, r);
            }
            store_bf16<INTERLEAVED>(dst + u * D, at, dx);
        }
    }
    return dw;
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kNormThreads, 4)
norm_rope_bwd_kernel(const NormRopeParams p) {
    constexpr int kLanes = D / 8, kGroups = kNormThreads / kLanes;
    __shared__ float share[kGroups][D];
    wait_for_primary();
    launch_dependents();  // the sum of the shares: its blocks wait for this grid's end
    const int group = threadIdx.x / kLanes;
    const LanePlace at = lane_place<INTERLEAVED>(threadIdx.x % kLanes, p.rot);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        // K's items start at the other end of the grid: the blocks that had one
        // more of Q's have one fewer.
        const Pairs dw = norm_rope_bwd_side<D, INTERLEAVED>(
            p, at, which == 0, which == 0 ? blockIdx.x : gridDim.x - 1 - blockIdx.x);
        // This block's share: the groups' sums in their order.
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            share[group][INTERLEAVED ? at.a + 2 * e : at.a + e] = dw.p[e];
            share[group][INTERLEAVED ? at.a + 2 * e + 1 : at.b + e] = dw.q[e];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < D; i += kNormThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) sum += share[g][i];
            p.partial[((size_t)blockIdx.x * 2 + which) * D + i] = sum;
        }
    }
}

// dw[i] = sum over blocks of partial[block][i], i < 2 D: 16 columns per block,
// 64 rows of threads that take every 64th partial, then their sums in order.
constexpr int kDwRows = 64, kDwCols = 16;
__global__ void __launch_bounds__(kDwRows * kDwCols)
norm_rope_dw_kernel(const float *partial, int blocks, int D, float *dqw, float *dkw) {
    __shared__ float share[kDwRows][kDwCols + 1];
    wait_for_primary();
    const int i = blockIdx.x * kDwCols + threadIdx.x;
    float sum = 0.0f;
#pragma unroll 8
    for (int b = threadIdx.y; b < blocks; b += kDwRows) sum += partial[(size_t)b * 2 * D + i];
    share[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y == 0) {
        sum = 0.0f;
#pragma unroll
        for (int r = 0; r < kDwRows; ++r) sum += share[r][threadIdx.x];
        (i < D ? dqw[i] : dkw[i - D]) = sum;
    }
}

}  // namespace tab
