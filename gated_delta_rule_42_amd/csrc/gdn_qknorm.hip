// Per-head norm of queries and keys with the rotary rotation in the same pass, and its gradients, for gfx950.
//
// One row is one head of one token, x [d]. With n = 1 (L2) or n = d (RMS):
//     r = (sum x^2 / n + eps)^(-1/2),   xh = r x,   z = w * xh,   y = scale * R(p) z,
// R(p) turning pairs of the first `rot` channels by the angle p * inv_freq[j] (and scaling them by rope_scale):
// pairs (j, j + rot/2) in the half layout, (2j, 2j + 1) in the interleaved one.
// Backward: g = scale * R(p)^T dy (the opposite angle, the same rope_scale), dw = sum over rows of xh * g,
//     c = sum(w g xh) / n,   dx = r (w g - xh c).
// Both directions read and write each row once; r is computed again in the backward pass, whose x it has to read
// anyway. Sums are fp32.
//
// A row takes G lanes of 8 channels (G = 8, 16 or 32 by d), so every load and store is 16 bytes wide and the row's
// sums are G-lane butterflies. A work-group takes a run of NP * 256 / G consecutive rows, whatever heads they
// are, with all of its loads issued before the first row is used. The angles of the few tokens these rows belong to are computed
// once per work-group, in fp64 revolutions (a position of a million times a frequency near 1 has lost 5 of its
// digits in fp32), reduced to half a revolution, and their cosines and sines kept in LDS for all heads.
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

constexpr int kNormThreads = 256;
// NP rows per lane group: four where there are enough of them to fill the device many times over, else one, which spreads
// a small call over more work-groups. 64 tokens x 32 heads of 128: 3.6 us with one, 5.3 with four; 32768 x 36 heads of 64,
// rotated: 69 us with one, 57 with four.

enum { ROPE_NONE = 0, ROPE_HALF = 1, ROPE_PAIRS = 2 };

// Eight consecutive channels as they lie in memory, and as fp32: rows wait for their turn as loaded, which halves the
// registers of bf16 rows in flight.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <> struct Raw8<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16_lo_half(w[e]);
            x[2 * e + 1] = bf16_hi_half(w[e]);
        }
    }
};
// NT: past the caches, in the calls of many rows (NP = 4), whose outputs mostly exceed the L2 (the 32768-token call above: 57 us
// against 61). The rule counts rows, not bytes: very short rows go past the caches too.
template <bool NT, typename T>
__device__ __forceinline__ void store_piece(void* p, const T& x) {
    if constexpr (NT) __builtin_nontemporal_store(x, static_cast<T*>(p));
    else *static_cast<T*>(p) = x;
}
template <bool NT>
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    store_piece<NT>(p, f32x4_t{x[0], x[1], x[2], x[3]});
    store_piece<NT>(p + 4, f32x4_t{x[4], x[5], x[6], x[7]});
}
template <bool NT>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    store_piece<NT>(p, u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                               pack_bf16x2(x[6], x[7])});
}

// Sum over the G lanes of a row, in every lane.
template <int G>
__device__ __forceinline__ float row_sum(float x) {
    x += dpp_f32<0xB1>(x);    // quad_perm [1,0,3,2]
    x += dpp_f32<0x4E>(x);    // quad_perm [2,3,0,1]
    x += dpp_f32<0x141>(x);   // row_half_mirror
    if constexpr (G >= 16) x += dpp_f32<0x140>(x);   // row_mirror
    if constexpr (G >= 32) x += __shfl_xor(x, 16, 64);
    return x;
}

// The rows of a work-group and their angles. A block of RB consecutive rows (row = token * (Hq + Hk) + head, queries
// first) touches at most RB / 2 + 2 tokens, since a token has two rows at least.
template <int G, int NP>
struct NormBlock {
    static constexpr int RPP = kNormThreads / G;         // rows per pass
    static constexpr int RB = RPP * NP;
    static constexpr int MAXTOK = RB / 2 + 2;
    static constexpr int PAIRS = 4 * G;                  // rotated pairs of a row at most
};

template <int PAIRS>
__device__ __forceinline__ void fill_angles(const NormProblem& p, float2* cs, long tok0, int ntok, int tid) {
    const int half = p.rot / 2;
    for (int i = tid; i < ntok * half; i += kNormThreads) {
        const int t = i / half, j = i - t * half;
        double u = (double)p.positions[tok0 + t] * (double)p.inv_freq[j] * 0.15915494309189535;   // 1 / (2 pi)
        u -= rint(u);
        float s, c;
        sincospif(2.f * (float)u, &s, &c);
        cs[t * PAIRS + j] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
}

// y = R x for a lane's 8 channels (8 l .. 8 l + 7) of a row; cs are the row's cosines and sines. Called by all lanes of the
// wave (the half layout exchanges channels between the lanes of a row; rot / 2 is a multiple of 8 there, so a
// lane's partners all sit in one other lane).
template <int ROPE, bool BACK>
__device__ __forceinline__ void rotate8(float (&x)[8], const float2* cs, int l, int rot) {
    if constexpr (ROPE == ROPE_PAIRS) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            if (8 * l + e < rot) {
                const float2 w = cs[4 * l + e / 2];
                const float s = BACK ? -w.y : w.y, a = x[e], b = x[e + 1];
                x[e] = a * w.x - b * s;
                x[e + 1] = b * w.x + a * s;
            }
        }
    } else if constexpr (ROPE == ROPE_HALF) {
        const int hl = rot / 16;   // lanes of half the rotated channels
        const bool first = l < hl, in = l < 2 * hl;
        const int shift = in ? (first ? hl : -hl) : 0;
        const int from = (int)(threadIdx.x & 63) + shift;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __shfl(x[e], from, 64);
        if (in) {
            const float2* w = cs + 8 * (first ? l : l - hl);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = (first != BACK) ? -w[e].y : w[e].y;
                x[e] = x[e] * w[e].x + o[e] * s;
            }
        }
    }
}

// Row `row` of the call (at most 2^28 rows): its token, its head, whether that is one of the keys'.
struct NormRow {
    bool ok, key;
    int head, token;
};
__device__ __forceinline__ NormRow norm_row(const NormProblem& p, unsigned row, unsigned nrows) {
    NormRow r;
    r.ok = row < nrows;
    const unsigned ht = p.hq + p.hk, t = r.ok ? row / ht : 0;
    const int h = r.ok ? (int)(row - t * ht) : 0;
    r.key = h >= p.hq;
    r.head = r.key ? h - p.hq : h;
    r.token = (int)t;
    return r;
}
// Element offsets of a row: in q and k, and in dense tensors.
__device__ __forceinline__ long row_in(const NormProblem& p, const NormRow& r) {
    return r.key ? r.token * p.k_token + r.head * p.k_head : r.token * p.q_token + r.head * p.q_head;
}
__device__ __forceinline__ long row_dense(const NormProblem& p, const NormRow& r) {
    return ((long)r.token * (r.key ? p.hk : p.hq) + r.head) * p.d;
}

template <typename TX, typename TY, int G, int ROPE, int NP>
__global__ __launch_bounds__(kNormThreads) void qk_norm_fwd_kernel(NormProblem p) {
    using B = NormBlock<G, NP>;
    __shared__ float2 cs[ROPE ? B::MAXTOK * B::PAIRS : 1];
    const int tid = threadIdx.x, l = tid % G, grp = tid / G;
    const unsigned nrows = (unsigned)(p.tokens * (p.hq + p.hk)), row0 = blockIdx.x * B::RB;
    const bool lane_in = 8 * l < p.d;

    Raw8<TX> raw[NP];
    NormRow rw[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        rw[i] = norm_row(p, row0 + i * B::RPP + grp, nrows);
        raw[i].zero();
        if (rw[i].ok && lane_in) raw[i].load(static_cast<const TX*>(rw[i].key ? p.k : p.q) + row_in(p, rw[i]) + 8 * l);
    }
    int tok0 = 0;
    if constexpr (ROPE != ROPE_NONE) {
        const unsigned ht = p.hq + p.hk, last = min(row0 + B::RB, nrows) - 1;
        tok0 = (int)(row0 / ht);
        fill_angles<B::PAIRS>(p, cs, tok0, (int)(last / ht) - tok0 + 1, tid);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float x[8], ss = 0.f;
        raw[i].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
        ss = row_sum<G>(ss);
        const float r = 1.f / sqrtf(ss * p.inv_n + p.eps);
        const float* w = rw[i].key ? p.k_weight : p.q_weight;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= r;
        if (w && lane_in) {
            Raw8<float> wr;
            float wv[8];
            wr.load(w + 8 * l);
            wr.get(wv);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= wv[e];
        }
        if constexpr (ROPE != ROPE_NONE)
            rotate8<ROPE, false>(x, cs + (rw[i].ok ? (rw[i].token - tok0) : 0) * B::PAIRS, l, p.rot);
        const float scale = rw[i].key ? 1.f : p.q_scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= scale;
        if (rw[i].ok && lane_in) store8<(NP > 1)>(static_cast<TY*>(rw[i].key ? p.k_out : p.q_out) + row_dense(p, rw[i]) + 8 * l, x);
    }
}

// DW: the weights' gradients too. The grid is then at most kNormGradBlocks work-groups, each of which walks its blocks
// of rows in a fixed order, sums its rows' contributions in registers, then over its lane groups in LDS, and writes
// one partial row [2, d] (q, k); norm_weight_grad_kernel adds those. No atomics: the same inputs give the same bits.
template <typename TX, typename TY, int G, int ROPE, int NP, bool DW>
__global__ __launch_bounds__(kNormThreads) void qk_norm_bwd_kernel(NormProblem p) {
    using B = NormBlock<G, NP>;
    __shared__ float2 cs[ROPE ? B::MAXTOK * B::PAIRS : 1];
    __shared__ float part[DW ? 4 * 2 * 8 * G : 1];
    const int tid = threadIdx.x, l = tid % G, grp = tid / G;
    const unsigned nrows = (unsigned)(p.tokens * (p.hq + p.hk)), nblocks = (nrows + B::RB - 1) / B::RB;
    const bool lane_in = 8 * l < p.d;
    float aq[8], ak[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) aq[e] = ak[e] = 0.f;

    for (unsigned blk = blockIdx.x; blk < nblocks; blk += gridDim.x) {
        const unsigned row0 = blk * B::RB;
        Raw8<TX> xr[NP];
        Raw8<TY> gr[NP];
        NormRow rw[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            rw[i] = norm_row(p, row0 + i * B::RPP + grp, nrows);
            xr[i].zero();
            gr[i].zero();
            if (rw[i].ok && lane_in) {
                xr[i].load(static_cast<const TX*>(rw[i].key ? p.k : p.q) + row_in(p, rw[i]) + 8 * l);
                gr[i].load(static_cast<const TY*>(rw[i].key ? p.dk_in : p.dq_in) + row_dense(p, rw[i]) + 8 * l);
            }
        }
        int tok0 = 0;
        if constexpr (ROPE != ROPE_NONE) {
            const unsigned ht = p.hq + p.hk, last = min(row0 + B::RB, nrows) - 1;
            tok0 = (int)(row0 / ht);
            if (DW) __syncthreads();   // the previous block is done with the angles
            fill_angles<B::PAIRS>(p, cs, tok0, (int)(last / ht) - tok0 + 1, tid);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float x[8], g[8];
            xr[i].get(x);
            gr[i].get(g);
            const float scale = rw[i].key ? 1.f : p.q_scale;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] *= scale;
            if constexpr (ROPE != ROPE_NONE)
                rotate8<ROPE, true>(g, cs + (rw[i].ok ? (rw[i].token - tok0) : 0) * B::PAIRS, l, p.rot);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
            ss = row_sum<G>(ss);
            const float r = 1.f / sqrtf(ss * p.inv_n + p.eps);
            const float* w = rw[i].key ? p.k_weight : p.q_weight;
            float c = 0.f, wv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) wv[e] = 1.f;
            if (w && lane_in) {
                Raw8<float> wr;
                wr.load(w + 8 * l);
                wr.get(wv);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] *= r;
                if constexpr (DW) {   // rows past the end hold zeros
                    const float t = x[e] * g[e];
                    aq[e] += rw[i].key ? 0.f : t;
                    ak[e] += rw[i].key ? t : 0.f;
                }
                g[e] *= wv[e];
                c += g[e] * x[e];
            }
            c = row_sum<G>(c) * p.inv_n;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = r * (g[e] - x[e] * c);
            if (rw[i].ok && lane_in) {
                const long o = rw[i].key ? rw[i].token * p.dk_token + rw[i].head * p.dk_head
                                         : rw[i].token * p.dq_token + rw[i].head * p.dq_head;
                store8<(NP > 1)>(static_cast<TX*>(rw[i].key ? p.dk_out : p.dq_out) + o + 8 * l, g);
            }
        }
    }
    if constexpr (DW) {
        // lanes l of a wave's row groups, then the four waves
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int m = G; m < 64; m *= 2) {
                aq[e] += __shfl_xor(aq[e], m, 64);
                ak[e] += __shfl_xor(ak[e], m, 64);
            }
        }
        const int wave = tid >> 6;
        if ((tid & 63) < G) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                part[(wave * 2 + 0) * 8 * G + 8 * l + e] = aq[e];
                part[(wave * 2 + 1) * 8 * G + 8 * l + e] = ak[e];
            }
        }
        __syncthreads();
        for (int i = tid; i < 2 * p.d; i += kNormThreads) {
            const int s = i >= p.d, c = i - s * p.d;
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) a += part[(w * 2 + s) * 8 * G + c];
            p.partial[(long)blockIdx.x * 2 * p.d + i] = a;
        }
    }
}

// The sum of the partial rows: a work-group per 16 columns, 16 lanes across them and 64 down the rows, joined in LDS.
__global__ __launch_bounds__(1024) void norm_weight_grad_kernel(const float* partial, int nparts, int d, float* dqw, float* dkw) {
    __shared__ float sum[64][17];
    const int lc = threadIdx.x & 15, lr = threadIdx.x >> 4, c = blockIdx.x * 16 + lc;
    float a = 0.f;
    // kNormGradBlocks / 64 = 16 rows a lane at most, loaded together
    float x[kNormGradBlocks / 64];
#pragma unroll
    for (int j = 0; j < kNormGradBlocks / 64; ++j) {
        const int i = lr + 64 * j;
        x[j] = i < nparts ? partial[(long)i * 2 * d + c] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kNormGradBlocks / 64; ++j) a += x[j];
    sum[lr][lc] = a;
    __syncthreads();
#pragma unroll
    for (int m = 32; m > 0; m /= 2) {
        if (lr < m) sum[lr][lc] += sum[lr + m][lc];
        __syncthreads();
    }
    if (lr == 0) {
        float* out = c < d ? dqw : dkw;
        if (out) out[c < d ? c : c - d] = sum[0][lc];
    }
}

template <typename TX, typename TY, int G, int ROPE, int NP>
static hipError_t norm_launch(const NormProblem& p, hipStream_t s) {
    const long nrows = p.tokens * (p.hq + p.hk);
    const long nblocks = (nrows + NormBlock<G, NP>::RB - 1) / NormBlock<G, NP>::RB;
    if (!p.backward) {
        if (nblocks == 0) return hipSuccess;
        return launch(qk_norm_fwd_kernel<TX, TY, G, ROPE, NP>, dim3((unsigned)nblocks), dim3(kNormThreads), s, p);
    }
    if (!p.dqw && !p.dkw) {
        if (nblocks == 0) return hipSuccess;
        return launch(qk_norm_bwd_kernel<TX, TY, G, ROPE, NP, false>, dim3((unsigned)nblocks), dim3(kNormThreads), s, p);
    }
    const int parts = norm_grad_blocks(nrows);
    if (nblocks > 0) {
        const hipError_t e = launch(qk_norm_bwd_kernel<TX, TY, G, ROPE, NP, true>, dim3((unsigned)parts), dim3(kNormThreads), s, p);
        if (e != hipSuccess) return e;
    }
    return launch(norm_weight_grad_kernel, dim3((unsigned)(p.d / 8)), dim3(1024), s, (const float*)p.partial, parts, p.d, p.dqw, p.dkw);
}

template <typename TX, typename TY, int G>
static hipError_t norm_rope(const NormProblem& p, hipStream_t s) {
    const bool large = p.tokens * (p.hq + p.hk) >= 2048 * NormBlock<G, 1>::RB;
    if (p.rot == 0) return large ? norm_launch<TX, TY, G, ROPE_NONE, 4>(p, s) : norm_launch<TX, TY, G, ROPE_NONE, 1>(p, s);
    if (p.interleaved)
        return large ? norm_launch<TX, TY, G, ROPE_PAIRS, 4>(p, s) : norm_launch<TX, TY, G, ROPE_PAIRS, 1>(p, s);
    return large ? norm_launch<TX, TY, G, ROPE_HALF, 4>(p, s) : norm_launch<TX, TY, G, ROPE_HALF, 1>(p, s);
}

template <typename TX, typename TY>
static hipError_t norm_dispatch(const NormProblem& p, hipStream_t s) {
    if (p.d <= 64) return norm_rope<TX, TY, 8>(p, s);
    if (p.d <= 128) return norm_rope<TX, TY, 16>(p, s);
    return norm_rope<TX, TY, 32>(p, s);
}

// Work-groups (and partial rows) of the backward pass with weight gradients: enough to fill the device several times
// over, but no more than there are blocks of rows (counted at 32 rows each).
int norm_grad_blocks(long nrows) {
    const long blocks = (nrows + 31) / 32;
    return (int)(blocks < kNormGradBlocks ? blocks : kNormGradBlocks);
}

hipError_t launch_qk_norm(const NormProblem& p, hipStream_t s) {
    if (p.x_bf16) return p.y_bf16 ? norm_dispatch<uint16_t, uint16_t>(p, s) : norm_dispatch<uint16_t, float>(p, s);
    return norm_dispatch<float, float>(p, s);
}

}  // namespace gdn
