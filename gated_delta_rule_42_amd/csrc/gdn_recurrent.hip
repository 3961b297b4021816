// Recurrent form of the gated delta rule for short runs of tokens on a pool of states, for gfx950: the serving side
// of the library, where a batch holds single new tokens, draft tokens and short prompts of different
// sequences, and each sequence's state lives in a slot of one pool.
//
// Per token, value head and state row s_i [dk] (alpha a scalar, or one decay per key channel):
//     s~ = s_i * alpha,   c = beta (v_i - s~ . k),   s_i <- s~ + c k,   o_i = s~ . q + c (k . q).
// The rows of a state are independent given the token's q, k, alpha and beta, so a row never leaves its 16 lanes'
// registers between the tokens of a run: the state is read once and written once per call (or once per token,
// where every token's state goes to a slot of its own).
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

// Four consecutive input elements as fp32.
__device__ __forceinline__ f32x4_t in4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }
__device__ __forceinline__ f32x4_t in4(const uint16_t* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return f32x4_t{bf16_lo_half(w.x), bf16_hi_half(w.x), bf16_lo_half(w.y), bf16_hi_half(w.y)};
}

// One work-group per (sequence, value head, tile of 16 RPG state rows): 16 groups of 16 lanes, RPG rows each. Lane l16
// owns the columns 4 l16 + 0..3 of each 64-column half of a row, so that the state's loads and stores cover whole
// 256-byte runs. The next token's operands are loaded while the current one is computed.
template <typename TS, typename TO, int DK, int DV, int RPG, bool CW>
__global__ __launch_bounds__(256) void recurrent_kernel(RecurrentProblem p) {
    constexpr int EPL = DK / 16, NH = EPL / 4;   // state columns per lane, in runs of four
    constexpr int TILES = DV / (16 * RPG);
    const int tid = threadIdx.x, l16 = tid & 15, grp = tid >> 4;
    const long unit = blockIdx.x / TILES;
    const int tile = (int)(blockIdx.x % TILES);
    const int n = (int)(unit / p.HV), hv = (int)(unit % p.HV), h = hv / (p.HV / p.H);
    int t0 = n, t1 = n + 1;
    if (p.cu_seqlens) {   // offsets outside [0, T] or falling ones are clamped
        t0 = min(max(p.cu_seqlens[n], 0), p.T);
        t1 = min(max(p.cu_seqlens[n + 1], t0), p.T);
    }
    if (t0 >= t1) return;
    const int slot = p.slots[n];
    const int row0 = tile * 16 * RPG + grp;
    TO* op = static_cast<TO*>(p.o) + (long)hv * DV + row0;
    if (slot < 0 || slot >= p.n_slots) {   // a padded entry: zeros for its tokens, no state touched
        if (l16 == 0)
            for (int t = t0; t < t1; ++t)
#pragma unroll
                for (int r = 0; r < RPG; ++r) op[(long)t * p.HV * DV + 16 * r] = from_f32<TO>(0.f);
        return;
    }
    const long srow = (long)hv * DV + row0;   // row within a slot
    const long slot_size = (long)p.HV * DV;
    float* st = p.states + (slot * slot_size + srow) * DK + 4 * l16;
    f32x4_t s[RPG][NH];
#pragma unroll
    for (int r = 0; r < RPG; ++r)
#pragma unroll
        for (int e = 0; e < NH; ++e)
            s[r][e] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(st + (long)16 * r * DK + 64 * e));

    struct Token {
        f32x4_t q[NH], k[NH], g[CW ? NH : 1];
        float v[RPG], g1, beta;
    };
    auto load = [&](Token& x, int t) {
        const TS* qp = static_cast<const TS*>(p.q) + t * p.q_token + h * DK + 4 * l16;
        const TS* kp = static_cast<const TS*>(p.k) + t * p.k_token + h * DK + 4 * l16;
        const TS* vp = static_cast<const TS*>(p.v) + t * p.v_token + hv * DV + row0;
        const long gi = (long)t * p.HV + hv;
#pragma unroll
        for (int e = 0; e < NH; ++e) {
            x.q[e] = in4(qp + 64 * e);
            x.k[e] = in4(kp + 64 * e);
            if constexpr (CW) x.g[e] = *reinterpret_cast<const f32x4_t*>(p.g + gi * DK + 64 * e + 4 * l16);
        }
        if constexpr (!CW) x.g1 = p.g[gi];
        x.beta = p.beta[gi];
#pragma unroll
        for (int r = 0; r < RPG; ++r) x.v[r] = to_f32(vp[16 * r]);
    };
    Token cur, nxt;
    load(cur, t0);
    for (int t = t0; t < t1; ++t) {
        if (t + 1 < t1) load(nxt, t + 1);
        f32x4_t a[NH];
        float kq = 0.f;
#pragma unroll
        for (int e = 0; e < NH; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[e][i] = CW ? __expf(cur.g[CW ? e : 0][i]) : 0.f;
                kq += cur.k[e][i] * cur.q[e][i];
            }
        kq = row16_sum(kq);
        const float a1 = CW ? 1.f : __expf(cur.g1);
#pragma unroll
        for (int r = 0; r < RPG; ++r) {
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int e = 0; e < NH; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[r][e][i] *= CW ? a[e][i] : a1;
                    sk += s[r][e][i] * cur.k[e][i];
                    sq += s[r][e][i] * cur.q[e][i];
                }
            sk = row16_sum(sk);
            sq = row16_sum(sq);
            const float c = cur.beta * (cur.v[r] - sk);
#pragma unroll
            for (int e = 0; e < NH; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[r][e][i] += c * cur.k[e][i];
            if (l16 == 0) op[(long)t * p.HV * DV + 16 * r] = from_f32<TO>(sq + c * kq);
        }
        const int to = p.out_slots ? p.out_slots[t] : -1;
        if (to >= 0 && to < p.n_slots) {
            float* dst = p.states + (to * slot_size + srow) * DK + 4 * l16;
#pragma unroll
            for (int r = 0; r < RPG; ++r)
#pragma unroll
                for (int e = 0; e < NH; ++e)
                    __builtin_nontemporal_store(s[r][e], reinterpret_cast<f32x4_t*>(dst + (long)16 * r * DK + 64 * e));
        }
        cur = nxt;
    }
    if (!p.out_slots) {
#pragma unroll
        for (int r = 0; r < RPG; ++r)
#pragma unroll
            for (int e = 0; e < NH; ++e)
                __builtin_nontemporal_store(s[r][e], reinterpret_cast<f32x4_t*>(st + (long)16 * r * DK + 64 * e));
    }
}

template <typename TS, typename TO, int DK, int DV, int RPG>
static hipError_t recurrent_gate(const RecurrentProblem& p, hipStream_t s) {
    const dim3 grid((unsigned)((long)p.N * p.HV * (DV / (16 * RPG))));
    return p.channel_gate ? launch(recurrent_kernel<TS, TO, DK, DV, RPG, true>, grid, dim3(256), s, p)
                          : launch(recurrent_kernel<TS, TO, DK, DV, RPG, false>, grid, dim3(256), s, p);
}

template <typename TS, typename TO, int DK, int DV>
static hipError_t recurrent_rows(const RecurrentProblem& p, hipStream_t s) {
    const long units = (long)p.N * p.HV;
    if (units * (DV / 64) >= 2048) return recurrent_gate<TS, TO, DK, DV, 4>(p, s);
    return recurrent_gate<TS, TO, DK, DV, 1>(p, s);
}

template <typename TS, typename TO>
static hipError_t recurrent_dispatch(const RecurrentProblem& p, hipStream_t s) {
    if (p.dk == 64)
        return p.dv == 64 ? recurrent_rows<TS, TO, 64, 64>(p, s) : recurrent_rows<TS, TO, 64, 128>(p, s);
    return p.dv == 64 ? recurrent_rows<TS, TO, 128, 64>(p, s) : recurrent_rows<TS, TO, 128, 128>(p, s);
}

hipError_t launch_recurrent(const RecurrentProblem& p, hipStream_t s) {
    if (p.N == 0 || p.T == 0) return hipSuccess;
    if (p.bf16)
        return p.o_bf16 ? recurrent_dispatch<uint16_t, uint16_t>(p, s) : recurrent_dispatch<uint16_t, float>(p, s);
    return p.o_bf16 ? recurrent_dispatch<float, uint16_t>(p, s) : recurrent_dispatch<float, float>(p, s);
}

}  // namespace gdn
