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
//   dx_d = r h_d - r^3 x_d (sum_e h_e x_e) / D
//   dw_d = sum over tokens and heads of g_d x_d r
//
// Bound by memory: two bytes in and two out per value (ten in all for a
// query's value in the backward, whose dy is fp32) against about ten
// operations.  D / 8 lanes hold a head, eight values (16 bytes) per lane, so
// the sums over a head are shuffles and every access is 16 bytes wide.  A
// group of lanes takes kRows heads of one token at a time: their loads are
// in flight together and the angles are read once for all of them.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace tab {

constexpr int kNormThreads = 256;

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
    int w_fp32, interleaved;
    float eps;
    // Serving form: slots [tokens] (negative: padding, left alone), caches
    // [num_slots][Hkv][D].
    const int *slots;
    void *k_cache, *v_cache;
    long long num_slots;
    float k_descale, v_descale;
    // Backward.
    const void *dq, *dk;      // [tokens][H][D], contiguous heads, fp32 or bf16
    long long dq_stride, dk_stride;
    int dq_fp32, dk_fp32;
    float *partial;           // [blocks][2][D]
};

struct Lane8 {
    float v[8];
};

// Sixteen bytes of an input that an output may overwrite in place (each
// thread reads its values before it writes them): not the read-only path.
__device__ __forceinline__ uint4 load16(const __nv_bfloat16 *p) {
    return *reinterpret_cast<const uint4 *>(p);
}

__device__ __forceinline__ Lane8 unpack8(uint4 p) {
    Lane8 r;
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r.v[2 * e] = __uint_as_float(w[e] << 16);
        r.v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ uint4 pack8(const Lane8 &x) {
    return make_uint4(pack_bf16x2(x.v[0], x.v[1]), pack_bf16x2(x.v[2], x.v[3]),
                      pack_bf16x2(x.v[4], x.v[5]), pack_bf16x2(x.v[6], x.v[7]));
}

__device__ __forceinline__ Lane8 load8_f32(const float *p) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Eight weights from d on.  The caller guarantees 16-byte alignment.
__device__ __forceinline__ Lane8 load_weights(const void *w, int fp32, int d) {
    if (fp32) return load8_f32(static_cast<const float *>(w) + d);
    return unpack8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(w) + d)));
}

// Cosines and sines of a lane's eight values; `turn` is false past `rot`.
// Half style: one pair of factors per value; interleaved: per pair (the
// first four entries).
struct Angles {
    float c[8], s[8];
    bool turn;
};

__device__ __forceinline__ Angles load_angles(const NormRopeParams &p, int pos, int d) {
    Angles a;
    a.turn = d < p.rot;
    if (!a.turn) return a;
    const size_t row = (size_t)pos * (p.rot / 2);
    if (p.interleaved) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(p.cos + row + d / 2));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(p.sin + row + d / 2));
        a.c[0] = c.x, a.c[1] = c.y, a.c[2] = c.z, a.c[3] = c.w;
        a.s[0] = s.x, a.s[1] = s.y, a.s[2] = s.z, a.s[3] = s.w;
    } else {
        const int i = d < p.rot / 2 ? d : d - p.rot / 2;
        const Lane8 c = load8_f32(p.cos + row + i), s = load8_f32(p.sin + row + i);
#pragma unroll
        for (int e = 0; e < 8; ++e) a.c[e] = c.v[e], a.s[e] = s.v[e];
    }
    return a;
}

// R u (sign = 1) or R^T u (sign = -1) of a lane's eight values.  Whole warps
// call it: in the half style the partner's values come from the lane rot/16
// away.  rot is a multiple of 16, so a lane's eight values lie in one half.
__device__ __forceinline__ Lane8 rotate8(const NormRopeParams &p, const Lane8 &u, const Angles &a,
                                         int d, float sign) {
    Lane8 y = u;
    if (p.interleaved) {
        if (a.turn) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float s = sign * a.s[e];
                y.v[2 * e] = u.v[2 * e] * a.c[e] - u.v[2 * e + 1] * s;
                y.v[2 * e + 1] = u.v[2 * e + 1] * a.c[e] + u.v[2 * e] * s;
            }
        }
    } else {
        const int off = p.rot / 16;
        const bool low = d < p.rot / 2;
        const int partner = !a.turn ? lane_id() : low ? lane_id() + off : lane_id() - off;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float o = __shfl_sync(0xffffffffu, u.v[e], partner);
            if (a.turn) y.v[e] = u.v[e] * a.c[e] + (low ? -sign : sign) * a.s[e] * o;
        }
    }
    return y;
}

// Sum over the D / 8 lanes of a head.
template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Position of a token, clamped into the table (out of range: reported).
__device__ __forceinline__ int token_position(const NormRopeParams &p, long long token) {
    const int pos = __ldg(p.positions + token);
    if (pos >= 0 && pos < p.max_positions) return pos;
    atomicCAS(p.status, 0, kStatusRange);
    return pos < 0 ? 0 : p.max_positions - 1;
}

// Eight values as e4m3 codes of x / descale (nearest even, saturating).
__device__ __forceinline__ uint2 codes8(const Lane8 &x, float descale) {
    return make_uint2(pack_e4m3x4(__fdiv_rn(x.v[0], descale), __fdiv_rn(x.v[1], descale),
                                  __fdiv_rn(x.v[2], descale), __fdiv_rn(x.v[3], descale)),
                      pack_e4m3x4(__fdiv_rn(x.v[4], descale), __fdiv_rn(x.v[5], descale),
                                  __fdiv_rn(x.v[6], descale), __fdiv_rn(x.v[7], descale)));
}

// KV: where K goes.  0: k_out, like Q; 1: a bf16 cache; 2: an e4m3 cache
// (with V beside it in both).
constexpr int kNormRows = 4;  // heads of a token that a group of lanes takes together

template <int D, int KV>
__global__ void __launch_bounds__(kNormThreads)
norm_rope_kernel(const NormRopeParams p) {
    constexpr int kLanes = D / 8, kGroups = kNormThreads / kLanes, U = kNormRows;
    const int group = threadIdx.x / kLanes;
    const int d = (threadIdx.x % kLanes) * 8;
    const int chunks = p.chunks_q + (KV ? 2 : 1) * p.chunks_k;
    const uint32_t item = blockIdx.x * kGroups + group;  // the host bounds the items by 2^31
    long long token = item / (uint32_t)chunks;
    // Groups past the end, and padding tokens, read nothing and write nothing
    // but stay for the shuffles.
    bool live = token < p.tokens;
    if (!live) token = 0;
    const int chunk = (int)(item % (uint32_t)chunks);
    const int what = chunk < p.chunks_q ? 0 : chunk < p.chunks_q + p.chunks_k ? 1 : 2;  // Q, K, V
    const int h0 = U * (chunk - (what == 0 ? 0 : what == 1 ? p.chunks_q : p.chunks_q + p.chunks_k));
    const int heads = min(U, (what == 0 ? p.Hq : p.Hkv) - h0);
    long long slot = 0;
    if (KV && live) {
        slot = __ldg(p.slots + token);
        if (slot >= p.num_slots) atomicCAS(p.status, 0, kStatusRange);
        live = slot >= 0 && slot < p.num_slots;
    }
    const __nv_bfloat16 *src = what == 0   ? p.q + token * p.q_stride
                               : what == 1 ? p.k + token * p.k_stride
                                           : p.v + token * p.v_stride;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (live && u < heads) raw[u] = load16(src + (h0 + u) * D + d);
    }
    Angles ang;
    ang.turn = false;
    Lane8 w{};
    if (live && what != 2) {
        ang = load_angles(p, token_position(p, token), d);
        w = load_weights(what == 0 ? p.qw : p.kw, p.w_fp32, d);
    }
    float r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Lane8 x = unpack8(raw[u]);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) s0 += x.v[e] * x.v[e], s1 += x.v[e + 1] * x.v[e + 1];
        r[u] = rsqrtf(head_sum<D>(s0 + s1) * (1.0f / D) + p.eps);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Lane8 x = unpack8(raw[u]);
        Lane8 y;
#pragma unroll
        for (int e = 0; e < 8; ++e) y.v[e] = x.v[e] * r[u] * w.v[e];
        y = rotate8(p, y, ang, d, 1.0f);
        if (!live || u >= heads) continue;
        const int at = (h0 + u) * D + d;
        if (KV == 0 || what == 0) {
            __nv_bfloat16 *dst = what == 0 ? p.q_out + token * p.q_out_stride : p.k_out + token * p.k_out_stride;
            *reinterpret_cast<uint4 *>(dst + at) = pack8(y);
        } else {
            const size_t off = (size_t)slot * p.Hkv * D + at;
            void *cache = what == 1 ? p.k_cache : p.v_cache;
            if (KV == 1)
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(cache) + off) =
                    what == 1 ? pack8(y) : raw[u];
            else
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + off) =
                    what == 1 ? codes8(y, p.k_descale) : codes8(x, p.v_descale);
        }
    }
}

// ----------------------------------------------------------------- backward

// A fixed number of blocks walks over the items, so that each block's share
// of dw stays in registers until its end and the sum of the blocks' shares
// (norm_rope_dw_kernel, in the blocks' order) does not depend on the timing.
constexpr int kNormBwdRows = 2;

template <int D>
__global__ void __launch_bounds__(kNormThreads)
norm_rope_bwd_kernel(const NormRopeParams p) {
    constexpr int kLanes = D / 8, kGroups = kNormThreads / kLanes, U = kNormBwdRows;
    __shared__ float share[kGroups][D];
    const int group = threadIdx.x / kLanes;
    const int d = (threadIdx.x % kLanes) * 8;
    const int chunks = p.chunks_q + p.chunks_k;
    const uint32_t items = (uint32_t)(p.tokens * chunks);  // below 2^31
    const Lane8 wq = load_weights(p.qw, p.w_fp32, d), wk = load_weights(p.kw, p.w_fp32, d);
    Lane8 dwq{}, dwk{};
    // Whole warps loop together, as the shuffles need.
    for (uint32_t base = blockIdx.x * kGroups; base < items; base += gridDim.x * kGroups) {
        const bool live = base + group < items;
        const uint32_t item = live ? base + group : 0;
        const long long token = item / (uint32_t)chunks;
        const int chunk = (int)(item % (uint32_t)chunks);
        const bool is_q = chunk < p.chunks_q;
        const int h0 = U * (is_q ? chunk : chunk - p.chunks_q);
        const int heads = live ? min(U, (is_q ? p.Hq : p.Hkv) - h0) : 0;
        const __nv_bfloat16 *src = is_q ? p.q + token * p.q_stride : p.k + token * p.k_stride;
        const int fp32 = is_q ? p.dq_fp32 : p.dk_fp32;
        const void *dy = is_q ? p.dq : p.dk;
        const long long dy_at = token * (is_q ? p.dq_stride : p.dk_stride);
        uint4 raw[U];
        Lane8 g[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            g[u] = Lane8{};
            if (u < heads) {
                const long long at = dy_at + (h0 + u) * D + d;
                raw[u] = load16(src + (h0 + u) * D + d);
                if (fp32) g[u] = load8_f32(static_cast<const float *>(dy) + at);
                else g[u] = unpack8(ld_nc_v4(static_cast<const __nv_bfloat16 *>(dy) + at));
            }
        }
        Angles ang;
        ang.turn = false;
        if (live) ang = load_angles(p, token_position(p, token), d);
        __nv_bfloat16 *dst = is_q ? p.q_out + token * p.q_out_stride : p.k_out + token * p.k_out_stride;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Lane8 x = unpack8(raw[u]);
            g[u] = rotate8(p, g[u], ang, d, -1.0f);
            float ss = 0.0f, hx = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss += x.v[e] * x.v[e];
                hx += (is_q ? wq.v[e] : wk.v[e]) * g[u].v[e] * x.v[e];
            }
            const float r = rsqrtf(head_sum<D>(ss) * (1.0f / D) + p.eps);
            const float t = head_sum<D>(hx) * (1.0f / D) * r * r;
            if (u >= heads) continue;
            Lane8 dx;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gx = g[u].v[e] * (x.v[e] * r);
                if (is_q) dwq.v[e] += gx;
                else dwk.v[e] += gx;
                dx.v[e] = r * ((is_q ? wq.v[e] : wk.v[e]) * g[u].v[e] - x.v[e] * t);
            }
            *reinterpret_cast<uint4 *>(dst + (h0 + u) * D + d) = pack8(dx);
        }
    }
    // This block's share: the groups' sums in their order.
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) share[group][d + e] = which ? dwk.v[e] : dwq.v[e];
        __syncthreads();
        for (int i = threadIdx.x; i < D; i += kNormThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) sum += share[g][i];
            p.partial[((size_t)blockIdx.x * 2 + which) * D + i] = sum;
        }
    }
}

// dw[i] = sum over blocks of partial[block][i], i < 2 D: 32 columns per
// block, 32 rows of threads that take every 32nd partial, then their sums in
// order.
__global__ void __launch_bounds__(1024)
norm_rope_dw_kernel(const float *partial, int blocks, int D, float *dqw, float *dkw) {
    __shared__ float share[32][33];
    const int i = blockIdx.x * 32 + threadIdx.x;
    float sum = 0.0f;
#pragma unroll 4
    for (int b = threadIdx.y; b < blocks; b += 32) sum += partial[(size_t)b * 2 * D + i];
    share[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y == 0) {
        sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 32; ++r) sum += share[r][threadIdx.x];
        (i < D ? dqw[i] : dkw[i - D]) = sum;
    }
}

}  // namespace tab
