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
// 256-byte runs. Where sequences have about one token each (RUNS false) its operands go straight to registers, which leaves
// room for more waves. Longer runs take their tokens in blocks of TB through
// LDS: the next block's loads are in flight while the current one is computed, and what all 16 groups need (the decay,
// k . q) is computed once per work-group.
template <typename TS, typename TO, int DK, int DV, int RPG, bool CW, bool RUNS>
__global__ __launch_bounds__(256) void recurrent_kernel(RecurrentProblem p) {
    constexpr int NH = DK / 64;                  // a lane's runs of four columns
    constexpr int TILES = DV / (16 * RPG);
    constexpr int TB = 1024 / DK;                // tokens per block: four channels per thread
    constexpr int NVB = TB * 16 * RPG / 256 > 0 ? TB * 16 * RPG / 256 : 1;   // value rows per thread and block
    constexpr int LB = RUNS ? TB : 1;
    __shared__ alignas(16) float sk[LB][DK], sq[LB][DK], sa[CW ? LB : 1][DK], sv[LB][16 * RPG];
    __shared__ float4 sc[LB];                    // alpha (scalar gate), beta, k . q
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
    const long otok = (long)p.HV * DV;
    TO* op = static_cast<TO*>(p.o) + (long)hv * DV + row0;
    if (slot < 0 || slot >= p.n_slots) {   // a padded entry: zeros for its tokens, no state touched
        if (l16 == 0)
            for (int t = t0; t < t1; ++t)
#pragma unroll
                for (int r = 0; r < RPG; ++r) op[t * otok + 16 * r] = from_f32<TO>(0.f);
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
    auto put = [&](float* dst) {
#pragma unroll
        for (int r = 0; r < RPG; ++r)
#pragma unroll
            for (int e = 0; e < NH; ++e)
                __builtin_nontemporal_store(s[r][e], reinterpret_cast<f32x4_t*>(dst + (long)16 * r * DK + 64 * e));
    };
    const TS* qp = static_cast<const TS*>(p.q) + h * DK;
    const TS* kp = static_cast<const TS*>(p.k) + h * DK;
    const TS* vp = static_cast<const TS*>(p.v) + (long)hv * DV + tile * 16 * RPG;

    struct Token {
        f32x4_t q[NH], k[NH], a[NH];   // a: the decay of the lane's columns
        float v[RPG], beta, kq;
    };
    auto step = [&](const Token& x, int t) {
#pragma unroll
        for (int r = 0; r < RPG; ++r) {
            float dk = 0.f, dq = 0.f;
#pragma unroll
            for (int e = 0; e < NH; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[r][e][i] *= x.a[e][i];
                    dk += s[r][e][i] * x.k[e][i];
                    dq += s[r][e][i] * x.q[e][i];
                }
            dk = row16_sum(dk);
            dq = row16_sum(dq);
            const float c = x.beta * (x.v[r] - dk);
#pragma unroll
            for (int e = 0; e < NH; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[r][e][i] += c * x.k[e][i];
            if (l16 == 0) op[t * otok + 16 * r] = from_f32<TO>(dq + c * x.kq);
        }
        if (p.out_slots) {
            const int to = p.out_slots[t];
            if (to >= 0 && to < p.n_slots) put(p.states + (to * slot_size + srow) * DK + 4 * l16);
        }
    };

    if constexpr (!RUNS) {
        for (int t = t0; t < t1; ++t) {
            Token x;
            const long gi = (long)t * p.HV + hv;
            x.kq = 0.f;
#pragma unroll
            for (int e = 0; e < NH; ++e) {
                x.q[e] = in4(qp + t * p.q_token + 64 * e + 4 * l16);
                x.k[e] = in4(kp + t * p.k_token + 64 * e + 4 * l16);
                if constexpr (CW) x.a[e] = *reinterpret_cast<const f32x4_t*>(p.g + gi * DK + 64 * e + 4 * l16);
            }
            const float g1 = CW ? 0.f : p.g[gi];
            x.beta = p.beta[gi];
#pragma unroll
            for (int r = 0; r < RPG; ++r) x.v[r] = to_f32(vp[t * p.v_token + grp + 16 * r]);
            const float a1 = __expf(g1);
#pragma unroll
            for (int e = 0; e < NH; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x.a[e][i] = CW ? __expf(x.a[e][i]) : a1;
                    x.kq += x.k[e][i] * x.q[e][i];
                }
            x.kq = row16_sum(x.kq);
            step(x, t);
        }
    } else {
        // thread's share of a block: four channels of token tid / (DK / 4), one or more values, a token's scalars;
        // tokens past the run's end are the last one again (not used)
        const int bt = tid / (DK / 4), bc = 4 * (tid % (DK / 4));
        f32x4_t fq, fk, fa;
        float fv[NVB], fg = 0.f, fb = 0.f;
        auto fetch = [&](int t) {
            const int tt = min(t + bt, t1 - 1);
            const long gi = (long)tt * p.HV + hv;
            fq = in4(qp + tt * p.q_token + bc);
            fk = in4(kp + tt * p.k_token + bc);
            if constexpr (CW) fa = *reinterpret_cast<const f32x4_t*>(p.g + gi * DK + bc);
            else fg = p.g[gi];
            fb = p.beta[gi];
#pragma unroll
            for (int i = 0; i < NVB; ++i) {
                const int x = (tid + 256 * i) % (TB * 16 * RPG);
                fv[i] = to_f32(vp[min(t + x / (16 * RPG), t1 - 1) * p.v_token + x % (16 * RPG)]);
            }
        };
        fetch(t0);
        for (int tb = t0; tb < t1; tb += TB) {
            __syncthreads();   // the previous block is done with LDS
            *reinterpret_cast<f32x4_t*>(&sk[bt][bc]) = fk;
            *reinterpret_cast<f32x4_t*>(&sq[bt][bc]) = fq;
            if constexpr (CW)
                *reinterpret_cast<f32x4_t*>(&sa[bt][bc]) = f32x4_t{__expf(fa[0]), __expf(fa[1]), __expf(fa[2]), __expf(fa[3])};
            float kq = row16_sum(fk[0] * fq[0] + fk[1] * fq[1] + fk[2] * fq[2] + fk[3] * fq[3]);
            if constexpr (DK == 128) kq += __shfl_xor(kq, 16, 64);
            if (bc == 0) sc[bt] = make_float4(__expf(fg), fb, kq, 0.f);
#pragma unroll
            for (int i = 0; i < NVB; ++i) {
                const int x = (tid + 256 * i) % (TB * 16 * RPG);   // threads past the block write a value again
                sv[x / (16 * RPG)][x % (16 * RPG)] = fv[i];
            }
            __syncthreads();
            if (tb + TB < t1) fetch(tb + TB);
            auto get = [&](Token& x, int i) {
                const float4 c = sc[i];
#pragma unroll
                for (int e = 0; e < NH; ++e) {
                    x.k[e] = *reinterpret_cast<const f32x4_t*>(&sk[i][64 * e + 4 * l16]);
                    x.q[e] = *reinterpret_cast<const f32x4_t*>(&sq[i][64 * e + 4 * l16]);
                    if constexpr (CW) x.a[e] = *reinterpret_cast<const f32x4_t*>(&sa[i][64 * e + 4 * l16]);
                    else x.a[e] = f32x4_t{c.x, c.x, c.x, c.x};
                }
                x.beta = c.y;
                x.kq = c.z;
#pragma unroll
                for (int r = 0; r < RPG; ++r) x.v[r] = sv[i][grp + 16 * r];
            };
            const int nt = min(TB, t1 - tb);
            Token x, y;
            get(x, 0);
            for (int i = 0; i < nt; i += 2) {
                get(y, min(i + 1, TB - 1));
                step(x, tb + i);
                if (i + 1 < nt) {
                    get(x, min(i + 2, TB - 1));
                    step(y, tb + i + 1);
                }
            }
        }
    }
    if (!p.out_slots) put(st);
}

template <typename TS, typename TO, int DK, int DV, int RPG, bool RUNS>
static hipError_t recurrent_gate(const RecurrentProblem& p, hipStream_t s) {
    const dim3 grid((unsigned)((long)p.N * p.HV * (DV / (16 * RPG))));
    return p.channel_gate ? launch(recurrent_kernel<TS, TO, DK, DV, RPG, true, RUNS>, grid, dim3(256), s, p)
                          : launch(recurrent_kernel<TS, TO, DK, DV, RPG, false, RUNS>, grid, dim3(256), s, p);
}

// One row per group streams single tokens fastest at every size (256 sequences x 32 heads of 128 x 128: 179 us, 5.9 TB/s,
// against 185 with two and 196 with four rows; 32 sequences: 24.7, 25.1, 25.4). Runs are bound by vector instructions once
// there are enough of them; more rows then share a token's operands. Work-groups of one row per group: 1,024 (4 runs of 16
// tokens, 32 heads) 10.0 us with one row, 10.8 with two; 16,384 (64 runs of 8) 69 with one, 65 with two, 68 with four;
// 65,536 (256 runs of 4, channel-wise) 237, 210, 190.
// Whether there are runs is judged by the call's average, more than 1.25 tokens a sequence, since the host does not see
// the lengths. In mixed calls that costs something on either side of the border. 255 single tokens beside one run of
// 64, 32 heads of 128 x 128: 197 us on the single-token kernel (the single tokens alone 166, the run alone 18), and with
// 66, on the other one, 228; 4 heads: 42 and 44 (23 and 18). Rows behind the last sequence count as tokens: 256 single tokens
// with 256 such rows 191.
template <typename TS, typename TO, int DK, int DV>
static hipError_t recurrent_rows(const RecurrentProblem& p, hipStream_t s) {
    const bool runs = p.T > p.N + p.N / 4;
    const long groups = (long)p.N * p.HV * (DV / 16);
    if (!runs) return recurrent_gate<TS, TO, DK, DV, 1, false>(p, s);
    if (groups >= 32768) return recurrent_gate<TS, TO, DK, DV, 4, true>(p, s);
    if (groups >= 8192) return recurrent_gate<TS, TO, DK, DV, 2, true>(p, s);
    return recurrent_gate<TS, TO, DK, DV, 1, true>(p, s);
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
