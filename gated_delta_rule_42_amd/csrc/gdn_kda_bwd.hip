// Backward pass of the chunkwise gated delta rule with a channel-wise decay, for gfx950.
//
// The forward pass of one chunk (gdn_kda.hip), with gamma the in-chunk inclusive cumulative sum of g per channel:
//     Kh = K e^gamma,  Qh = Q e^gamma,  Kd = K e^{gamma_last - gamma},  lam = e^{gamma_last}
//     A = strict_lower(diag(beta) G),  G[r,i] = sum_c k_r k_i e^{gamma_r - gamma_i},   T = (I + A)^{-1},  M = T diag(beta)
//     P = lower(sum_c q_r k_i e^{gamma_r - gamma_i})
//     R = V - Kh S^T,   D = M R,   O = Qh S^T + P D,   S' = S Diag(lam) + D^T Kd.
// Its adjoint, from dO and the gradient dS' that reaches the state behind the chunk:
//     dD = P^T dO + Kd dS'^T,   Y = T^T dD,   dR = beta Y = dV
//     dS = dS' Diag(lam) + dO^T Qh - dR^T Kh                           (to the chunk before)
//     dP = lower(dO D^T),   dA = -strict_lower(Y D^T)
//     with the decayed in-chunk sums  aq_r = sum_i dP[r,i] k_i e^{gamma_r - gamma_i},
//         al_r = sum_i dA[r,i] k_i e^{gamma_r - gamma_i},
//         ar_i = sum_r (dP[r,i] q_r + dA[r,i] beta_r k_r) e^{gamma_r - gamma_i}:
//     dq = e^gamma (dO S) + aq,   l = al - e^gamma (Y S),   x = e^{gamma_last - gamma} (D dS')
//     dk = beta l + x + ar,   dbeta_r = Y_r . V_r + k_r . l_r
//     dgamma = q dq + k (beta l - x - ar),   and into every row of dg: sum_r k x + lam colsum(S dS')
//     (the pairs i = r of dq and ar cancel in dgamma and are left out there),
//     dg = the reverse cumulative sum of dgamma in the chunk + that.
// (dbeta needs no second look at A: sum_i dA[r,i] G[r,i] = k_r . al_r, and Y_r . R_r = Y_r . V_r - (Y S)_r . Kh_r.)
//
// Three kernels: the forward pass's stage 1 with fp32 operators (and T in place of M); the two walks over the chunks of each
// sequence, forwards for the state entering each chunk and D, backwards for dS' and Y; and one that takes
// every chunk by itself. All arithmetic is fp32 for both input types (fp32 matrix core, 16x16x4): dg is a reverse cumulative
// sum of differences, so rounding any product operand to 16 bits would show in it many times over.
// No e^{-gamma} is formed: a product over rows of different 16-row blocks is factored through the block
// boundary between them (both factors at most 1), and a pair inside a block takes its own decay. No e^{gamma_r - gamma_i} is
// formed from the two gammas either: see the decays in the chunk kernel.
#include "gdn_device.h"
#include "gdn_internal.h"

#include <type_traits>

namespace gdn {

// Four consecutive gradients, rounded to the output type.
__device__ __forceinline__ void kb_out4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void kb_out4(uint16_t* p, float4 x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// One element through a buffer resource (per-lane byte offset), as fp32.
template <typename TIn>
__device__ __forceinline__ float buf_in(__amdgpu_buffer_rsrc_t r, int off) {
    if constexpr (sizeof(TIn) == 2) return to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
    else return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}
// Keeps the compiler from moving memory accesses across: without it, it reads the operands of whole unrolled sections
// ahead and spills what it read.
__device__ __forceinline__ void pin() { asm volatile("" ::: "memory"); }

// Makes the compiler have x in a register at this point of the program.
__device__ __forceinline__ void hold(float& x) { asm volatile("" : "+v"(x)); }

// ------------------------------------------------------------------- the two walks
// The state walk (S entering each chunk, D) and the reverse walk (dS' leaving each chunk, Y) do not need each other and
// run side by side in one launch (one after the other, on tiles of 32 columns: 357 us for the training shape, against 320).
// One work-group per walk, (sequence, head) and tile of 16 NCG columns of d_v, NHF NCG waves (NCG x NHF is 1 x 4, 2 x 2 or
// 4 x 2, see kNarrowWalks). Wave w has the 16 columns cg = w % NCG and the part hf = w / NCG of the d_k channels:
// S^T [dk/NHF, 16] in accumulator registers. Per chunk each wave forms its part of the products over d_k for all 64 rows,
// the parts are added through LDS, the triangular product (with T or T^T) is shared by row tiles (see TriFrags), and each
// wave updates its own channels. Operators go global -> registers -> LDS a chunk ahead, all of these memory instructions
// placed between the products, whose steps hide them.
constexpr int kWalkPitch = 4;   // pad of an operator row in LDS (floats)

// A [64, W] fp32 operator on its way into LDS (row pitch W + kWalkPitch): NV 16-byte pieces per thread, held in registers
// between load and store.
template <int W, int NT>
struct WalkTile {
    static constexpr int NV = 64 * W / 4 / NT;
    f32x4_t x[NV];
    __device__ __forceinline__ void load(const float* src, int i, int tid) {
        x[i] = *reinterpret_cast<const f32x4_t*>(src + 4 * (tid + NT * i));
    }
    __device__ __forceinline__ void store(float* dst, int i, int tid) const {
        const int e = 4 * (tid + NT * i);
        *reinterpret_cast<f32x4_t*>(&dst[(e / W) * (W + kWalkPitch) + e % W]) = x[i];
    }
};

// Lower triangular [64, 64] matrices keep only their ten lower 16x16 tiles in LDS, tile (I, J) at I (I + 1) / 2 + J, its
// rows permuted so that the four rows 4 lq + s of a column read are in different banks.
constexpr int kTriFloats = 10 * 256;
__device__ __forceinline__ int tri_tile(int I, int J) { return (I * (I + 1) / 2 + J) * 256; }
__device__ __forceinline__ int tri_row(int r) { return ((r & ~3) | ((r ^ (r >> 2)) & 3)) * 16; }
// NM such matrices on their way into LDS, one after the other: 640 pieces each.
template <int NM, int NT>
struct WalkTri {
    static constexpr int NP = 640 * NM, NV = (NP + NT - 1) / NT;
    f32x4_t x[NV];
    static __device__ __forceinline__ void place(int i, int tid, int& m, int& I, int& J, int& r, int& c) {
        const int n = min(tid + NT * i, NP - 1), tile = n % 640 / 64;
        m = n / 640;
        I = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3;
        J = tile - I * (I + 1) / 2;
        r = n % 64 / 4;
        c = 4 * (n % 4);
    }
    __device__ __forceinline__ void load(const float* a, const float* b, int i, int tid) {
        int m, I, J, r, c;
        place(i, tid, m, I, J, r, c);
        x[i] = *reinterpret_cast<const f32x4_t*>((m ? b : a) + (16 * I + r) * 64 + 16 * J + c);
    }
    __device__ __forceinline__ void store(float* dst, int i, int tid) const {   // threads past the end write the last piece again
        int m, I, J, r, c;
        place(i, tid, m, I, J, r, c);
        *reinterpret_cast<f32x4_t*>(&dst[m * kTriFloats + tri_tile(I, J) + tri_row(r) + c]) = x[i];
    }
};

// The pieces j of NV that the i-th of eight shares has.
template <int NV, typename F>
__device__ __forceinline__ void share(int i, F f) {
#pragma unroll
    for (int j = i * NV / 8; j < (i + 1) * NV / 8; ++j) f(j);
}

// A wave's 16 columns of a chunk's [len, H, DV] tokens: 16-byte pieces in registers as loaded (zeros past the end), then
// through 4 KB of LDS of the wave's own into the layout of a right operand (lane (lq, l16): rows 16 t + 4 lq + m of
// column l16, stored in that order, so that the reads are free of bank conflicts).
template <typename TIn, int DV>
struct TokenCols {
    static constexpr int EB = (int)sizeof(TIn), PR = 16 * EB / 16, NV = 64 * PR / 64;   // pieces a row, pieces a lane
    u32x4_t x[NV];
    __device__ __forceinline__ void load(const void* src, long bos, int len, int H, int h, int col0, int i, int lane) {
        const auto rs = make_rsrc(static_cast<const TIn*>(src) + (bos * H + h) * DV, (unsigned)((len - 1) * H * DV + DV) * EB);
        const int n = lane + 64 * i, r = n / PR, c = n % PR;
        x[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, (r * H * DV + col0) * EB + 16 * c, 0, 0);
    }
    __device__ __forceinline__ void store(float* own, int i, int lane) const {
        const int n = lane + 64 * i, r = n / PR, c = n % PR;
        float* dst = own + ((r >> 4) * 4 + (r & 3)) * 64 + ((r >> 2) & 3) * 16 + c * (16 / EB);
        if constexpr (EB == 2) {
            *reinterpret_cast<f32x4_t*>(dst) = f32x4_t{bf16_lo_half(x[i][0]), bf16_hi_half(x[i][0]), bf16_lo_half(x[i][1]), bf16_hi_half(x[i][1])};
            *reinterpret_cast<f32x4_t*>(dst + 4) = f32x4_t{bf16_lo_half(x[i][2]), bf16_hi_half(x[i][2]), bf16_lo_half(x[i][3]), bf16_hi_half(x[i][3])};
        } else {
            *reinterpret_cast<u32x4_t*>(dst) = x[i];
        }
    }
    static __device__ __forceinline__ void get(const float* own, f32x4_t (&v)[4], int lane) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int m = 0; m < 4; ++m) v[t][m] = own[(4 * t + m) * 64 + lane];
    }
};

// acc[t] += the wave's channels (from c0) of the rows of tile t of m [64, P] times b, operands read one block of 16
// channels ahead; step(0) .. step(15) run between the products.
template <int NJ, typename F>
__device__ __forceinline__ void mul_rows(f32x4_t (&acc)[4], const float* m, int pitch, int c0, const f32x4_t (&b)[NJ], int l16, int lq, F step) {
    f32x4_t a[2][4];
    auto read = [&](int j) {
#pragma unroll
        for (int t = 0; t < 4; ++t) a[j & 1][t] = *reinterpret_cast<const f32x4_t*>(&m[(16 * t + l16) * pitch + c0 + 16 * j + 4 * lq]);
    };
    read(0);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s == 0 && j + 1 < NJ) read(j + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t] = mfma4(a[j & 1][t][s], b[j][s], acc[t]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4 / NJ; ++i) step((4 * j + s) * (4 / NJ) + i);
        }
    __builtin_amdgcn_sched_barrier(0);
}
// acc[j] += m^T (its columns c0 + 16 j + l16) times b over the 64 rows, operands read two steps ahead.
template <int NJ, typename F>
__device__ __forceinline__ void mul_cols(f32x4_t (&acc)[NJ], const float* m, int pitch, int c0, const f32x4_t (&b)[4], int l16, int lq, F step) {
    float a[4][NJ];
    auto read = [&](int i) {   // row 16 (i / 4) + 4 lq + i % 4
#pragma unroll
        for (int j = 0; j < NJ; ++j) a[i & 3][j] = m[(16 * (i / 4) + 4 * lq + i % 4) * pitch + c0 + 16 * j + l16];
    };
    read(0);
    read(1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i + 2 < 16) read(i + 2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j] = mfma4(a[i & 3][j], b[i / 4][i % 4], acc[j]);
        __builtin_amdgcn_sched_barrier(0);
        step(i);
    }
    __builtin_amdgcn_sched_barrier(0);
}
// The wave's share of a product with a lower triangular matrix m (TRANS: with m^T). NHF = 2: row tiles 0 and 3 for
// hf = 0, 1 and 2 for hf = 1, five block products either way. NHF = 4: row tile hf.
template <bool TRANS, int NHF>
struct TriFrags {
    static constexpr int NB = NHF == 2 ? 5 : 4;
    f32x4_t a[NB];
    // NHF = 2, block of (row tile, contraction tile) number i: (0,0) (3,0) (3,1) (3,2) (3,3) or (1,0) (1,1) (2,0) (2,1) (2,2);
    // transposed: (3,3) (0,0) (0,1) (0,2) (0,3) or (2,2) (2,3) (1,1) (1,2) (1,3)
    template <int HF>
    static constexpr int row(int i) {
        return TRANS ? (HF == 0 ? (i == 0 ? 3 : 0) : (i < 2 ? 2 : 1)) : (HF == 0 ? (i == 0 ? 0 : 3) : (i < 2 ? 1 : 2));
    }
    template <int HF>
    static constexpr int con(int i) {
        return TRANS ? (HF == 0 ? (i == 0 ? 3 : i - 1) : (i < 2 ? 2 + i : i - 1)) : (HF == 0 ? (i == 0 ? 0 : i - 1) : (i < 2 ? i : i - 2));
    }
    __device__ __forceinline__ void read(const float* m, int hf, int i, int l16, int lq) {   // i = 0 .. NB - 1
        int t = hf, t2 = i;
        if constexpr (NHF == 2) {
            t = hf == 0 ? row<0>(i) : row<1>(i);
            t2 = hf == 0 ? con<0>(i) : con<1>(i);
        } else if (TRANS ? t2 < t : t2 > t) {   // a block of zeros
            a[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            return;
        }
        if constexpr (TRANS) {
#pragma unroll
            for (int s = 0; s < 4; ++s) a[i][s] = m[tri_tile(t2, t) + tri_row(4 * lq + s) + l16];
        } else {
            a[i] = *reinterpret_cast<const f32x4_t*>(&m[tri_tile(t, t2) + tri_row(l16) + 4 * lq]);
        }
    }
    // The wave's row tiles of the product with x (NHF = 4: the first only), each block's product on its own accumulator
    template <int HF>
    __device__ __forceinline__ void mul_of(const f32x4_t (&x)[4], f32x4_t (&y)[2]) const {
        f32x4_t d[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) d[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < NB; ++i) d[i] = mfma4(a[i][s], x[NHF == 2 ? con<HF>(i) : i][s], d[i]);
        if constexpr (NHF == 4) y[0] = (d[0] + d[1]) + (d[2] + d[3]);
        else if constexpr (HF == 0) y[0] = d[0], y[1] = (d[1] + d[2]) + (d[3] + d[4]);
        else y[0] = d[0] + d[1], y[1] = (d[2] + d[3]) + d[4];
    }
    __device__ __forceinline__ void mul(const f32x4_t (&x)[4], int hf, f32x4_t (&y)[2]) const {
        if (NHF == 4 || hf == 0) mul_of<0>(x, y);
        else mul_of<1>(x, y);
    }
    static constexpr int TILES = NHF == 2 ? 2 : 1;
    static __device__ __forceinline__ int tile(int hf, int k) {   // row tile of y[k]
        if (NHF == 4) return hf;
        if (TRANS) return hf == 0 ? (k ? 0 : 3) : (k ? 1 : 2);
        return hf == 0 ? (k ? 3 : 0) : (k ? 2 : 1);
    }
};

template <int DK, int NCG, int NHF>
struct alignas(16) KdaStateSmem {
    float Kh[64 * (DK + kWalkPitch)];
    float Kd[64 * (DK + kWalkPitch)];
    float T[kTriFloats];
    float lam[DK];
    float beta[64];
    f32x4_t ex[NHF * NCG][4][64];    // each wave's partial products, row tile by row tile
    f32x4_t ex2[NCG][4][64];   // the triangular product, per column group
};
template <int DK, int NCG, int NHF>
struct alignas(16) KdaRevSmem {
    float Kd[64 * (DK + kWalkPitch)];
    union {
        float Qh[64 * (DK + kWalkPitch)];
        f32x4_t ex2[NCG][4][64];
    };
    float Kh[64 * (DK + kWalkPitch)];
    float PT[2 * kTriFloats];   // P, then T
    float lam[DK];
    float beta[64];
    f32x4_t ex[NHF * NCG][4][64];
};

// The sum of the NHF partial products of row tile t, the same in every wave.
template <int NCG, int NHF, typename SM>
__device__ __forceinline__ f32x4_t join(const SM& sm, int cg, int t, int lane) {
    const f32x4_t x = sm.ex[cg][t][lane] + sm.ex[cg + NCG][t][lane];
    if constexpr (NHF == 2) return x;
    else return x + (sm.ex[cg + 2 * NCG][t][lane] + sm.ex[cg + 3 * NCG][t][lane]);
}

struct Chain {   // the chunks of the work-group's (sequence, head)
    long pair, sbos, seos, cbase, nchunks;
    int h, tile;
};
template <int NTILE>
__device__ __forceinline__ Chain chain_of(const ChunkProblem& p, long b, long nb) {
    Chain c;
    // Work-groups go to the eight XCDs in turn; the tiles of one pair read the same operators, so in every full group
    // of eight pairs they are eight apart and share an XCD's L2.
    const long full = nb / (8 * NTILE) * (8 * NTILE);
    const long slot = b < full ? b / (8 * NTILE) * 8 + b % 8 : b / NTILE;
    c.tile = (int)(b < full ? b / 8 % NTILE : b % NTILE);
    // packed sequences are taken longest first (the chunk table's order)
    const int n = p.cu_seqlens ? p.chunk_base[p.N + 1 + (int)(slot / p.H)] : (int)(slot / p.H);
    c.h = (int)(slot % p.H);
    c.pair = (long)n * p.H + c.h;
    seq_range(p, n, c.sbos, c.seos);
    c.cbase = (p.cu_seqlens == nullptr) ? (long)n * p.nc_per_seq : (long)p.chunk_base[n];
    c.nchunks = (c.seos - c.sbos + 63) / 64;
    if (c.cbase + c.nchunks > p.nc_bound) c.nchunks = max(0L, p.nc_bound - c.cbase);
    return c;
}

// Barriers of a chunk: (1) its first operators are in LDS; (2) all partial products are exchanged, and the rest of the
// operators are in; (3) the triangular product is exchanged.
template <typename TIn, int DK, int DV, int NCG, int NHF>
__device__ __forceinline__ void walk_states(const KdaBwdProblem& b, KdaStateSmem<DK, NCG, NHF>& sm, const Chain& c, int tid) {
    constexpr int PK = DK + kWalkPitch, HK = DK / NHF, NJ = HK / 16, NT = 64 * NHF * NCG, NV = WalkTile<DK, NT>::NV;
    const ChunkProblem& p = b.f;
    const int lane = tid & 63, l16 = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), cg = wave % NCG, hf = wave / NCG;
    const int H = p.H, col0 = 16 * NCG * c.tile + 16 * cg, col = col0 + l16;

    f32x4_t ST[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        ST[j] = p.h0 ? *reinterpret_cast<const f32x4_t*>(p.h0 + (c.pair * DV + col) * DK + hf * HK + 16 * j + 4 * lq)
                     : f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (c.nchunks == 0) return;

    WalkTile<DK, NT> kh, kd;
    WalkTri<1, NT> tt;
    TokenCols<TIn, DV> v;
    float lam = 0.f, beta = 0.f;
    float* own = reinterpret_cast<float*>(&sm.ex[wave][0][0]);
    // the chunk's first operators (Kh, V) and the rest (Kd, T, lam, beta), each in up to eight shares
    auto load1 = [&](long jc, int i) {
        const long widx = (c.cbase + jc) * H + c.h, bos = c.sbos + jc * 64;
        share<NV>(i, [&](int j) { kh.load(p.khat + widx * 64 * DK, j, tid); });
        share<v.NV>(i, [&](int j) { v.load(p.v, bos, (int)min(64L, c.seos - bos), H, c.h, col0, j, lane); });
    };
    auto store1 = [&](int i) {
        share<NV>(i, [&](int j) { kh.store(sm.Kh, j, tid); });
        share<v.NV>(i, [&](int j) { v.store(own, j, lane); });
    };
    auto load2 = [&](long jc, int i) {
        const long widx = (c.cbase + jc) * H + c.h;
        share<NV>(i, [&](int j) { kd.load(p.kdec + widx * 64 * DK, j, tid); });
        share<tt.NV>(i, [&](int j) { tt.load(p.tmat + widx * 4096, nullptr, j, tid); });
        if (i == 7) {
            const long bos = c.sbos + jc * 64;
            const auto br = make_rsrc(p.beta + bos * H + c.h, (unsigned)((((int)min(64L, c.seos - bos) - 1) * H + 1) * 4));
            lam = p.lam[widx * DK + tid % DK];
            beta = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(br, (tid & 63) * H * 4, 0, 0));
        }
    };
    auto store2 = [&](int i) {
        share<NV>(i, [&](int j) { kd.store(sm.Kd, j, tid); });
        share<tt.NV>(i, [&](int j) { tt.store(sm.T, j, tid); });
        if (i == 7) {
            sm.lam[tid % DK] = lam;
            sm.beta[tid & 63] = beta;
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) load1(0, i);
#pragma unroll
    for (int i = 0; i < 8; ++i) load2(0, i);
#pragma unroll
    for (int i = 0; i < 8; ++i) store1(i);
#pragma unroll
    for (int i = 0; i < 8; ++i) load1(min(1L, c.nchunks - 1), i);

    for (long jc = 0; jc < c.nchunks; ++jc) {
        const long widx = (c.cbase + jc) * H + c.h;
        const long nxt = min(jc + 1, c.nchunks - 1), nxt2 = min(jc + 2, c.nchunks - 1);   // the last chunk again at the end
        f32x4_t X[4], D[4];
        __syncthreads();   // (1)
        TokenCols<TIn, DV>::get(own, D, lane);   // V, until R is formed
        // this part of X = Kh S^T
#pragma unroll
        for (int t = 0; t < 4; ++t) X[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        mul_rows<NJ>(X, sm.Kh, PK, hf * HK, ST, l16, lq, [&](int i) {
            if (i % 2 == 0) store2(i / 2);
            const int j = i / 4;
            if (i % 4 == 1 && j < NJ)
                *reinterpret_cast<f32x4_t*>(p.states + (widx * DV + col) * DK + hf * HK + 16 * j + 4 * lq) = ST[j];
        });
#pragma unroll
        for (int t = 0; t < 4; ++t) sm.ex[wave][t][lane] = X[t];
        __syncthreads();   // (2)
        TriFrags<false, NHF> m;
#pragma unroll
        for (int i = 0; i < m.NB; ++i) m.read(sm.T, hf, i, l16, lq);
#pragma unroll
        for (int t = 0; t < 4; ++t)   // beta R
            X[t] = *reinterpret_cast<const f32x4_t*>(&sm.beta[16 * t + 4 * lq]) * (D[t] - join<NCG, NHF>(sm, cg, t, lane));
        // D = T beta R on the wave's row tiles
        {
            f32x4_t d[2];
            m.mul(X, hf, d);
            float* dst = b.delta + (widx * 64 + 4 * lq) * DV + col;
#pragma unroll
            for (int k = 0; k < m.TILES; ++k) {
                const int t = m.tile(hf, k);
                sm.ex2[cg][t][lane] = d[k];
#pragma unroll
                for (int i = 0; i < 4; ++i) dst[(16 * t + i) * DV] = d[k][i];
            }
        }
        f32x4_t lm[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) lm[j] = *reinterpret_cast<const f32x4_t*>(&sm.lam[hf * HK + 16 * j + 4 * lq]);
        __syncthreads();   // (3)
#pragma unroll
        for (int t = 0; t < 4; ++t) D[t] = sm.ex2[cg][t][lane];
        // S^T <- Diag(lam) S^T + Kd^T D on the wave's channels
#pragma unroll
        for (int j = 0; j < NJ; ++j) ST[j] *= lm[j];
        mul_cols<NJ>(ST, sm.Kd, PK, hf * HK, D, l16, lq, [&](int i) {
            if (i % 2 == 0) store1(i / 2), load2(nxt, i / 2);
            else load1(nxt2, i / 2);
        });
    }
}

// Barriers of a chunk: (1) Kd, P, T and dO are in LDS; (2) all partial products are exchanged, and Qh, Kh, lam and beta
// are in; (3) Qh is dead; (4) the triangular product is exchanged (over Qh).
template <typename TIn, int DK, int DV, int NCG, int NHF>
__device__ __forceinline__ void walk_back(const KdaBwdProblem& b, KdaRevSmem<DK, NCG, NHF>& sm, const Chain& c, int tid) {
    constexpr int PK = DK + kWalkPitch, HK = DK / NHF, NJ = HK / 16, NT = 64 * NHF * NCG, NV = WalkTile<DK, NT>::NV;
    const ChunkProblem& p = b.f;
    const int lane = tid & 63, l16 = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), cg = wave % NCG, hf = wave / NCG;
    const int H = p.H, col0 = 16 * NCG * c.tile + 16 * cg, col = col0 + l16;

    f32x4_t dST[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        dST[j] = b.dhT ? *reinterpret_cast<const f32x4_t*>(b.dhT + (c.pair * DV + col) * DK + hf * HK + 16 * j + 4 * lq)
                       : f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto finish = [&]() {
        if (b.dh0) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                *reinterpret_cast<f32x4_t*>(b.dh0 + (c.pair * DV + col) * DK + hf * HK + 16 * j + 4 * lq) = dST[j];
        }
    };
    if (c.nchunks == 0) return finish();

    WalkTile<DK, NT> kh, qh, kd;
    WalkTri<2, NT> pt;
    TokenCols<TIn, DV> dof;
    float lam = 0.f, beta = 0.f;
    float* own = reinterpret_cast<float*>(&sm.ex[wave][0][0]);
    auto load1 = [&](long jc, int i) {   // Kd, P, T, dO
        const long widx = (c.cbase + jc) * H + c.h, bos = c.sbos + jc * 64;
        share<NV>(i, [&](int j) { kd.load(p.kdec + widx * 64 * DK, j, tid); });
        share<pt.NV>(i, [&](int j) { pt.load(static_cast<const float*>(p.pmat) + widx * 4096, p.tmat + widx * 4096, j, tid); });
        share<dof.NV>(i, [&](int j) { dof.load(b.d_o, bos, (int)min(64L, c.seos - bos), H, c.h, col0, j, lane); });
    };
    auto store1 = [&](int i) {
        share<NV>(i, [&](int j) { kd.store(sm.Kd, j, tid); });
        share<pt.NV>(i, [&](int j) { pt.store(sm.PT, j, tid); });
        share<dof.NV>(i, [&](int j) { dof.store(own, j, lane); });
    };
    auto load2 = [&](long jc, int i) {   // Qh, Kh, lam, beta
        const long widx = (c.cbase + jc) * H + c.h, bos = c.sbos + jc * 64;
        share<NV>(i, [&](int j) {
            qh.load(p.qhat + widx * 64 * DK, j, tid);
            kh.load(p.khat + widx * 64 * DK, j, tid);
        });
        if (i == 7) {
            const int len = (int)min(64L, c.seos - bos);
            lam = p.lam[widx * DK + tid % DK];
            const auto br = make_rsrc(p.beta + bos * H + c.h, (unsigned)(((len - 1) * H + 1) * 4));
            beta = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(br, (tid & 63) * H * 4, 0, 0));
        }
    };
    auto store2 = [&](int i) {
        share<NV>(i, [&](int j) {
            qh.store(sm.Qh, j, tid);
            kh.store(sm.Kh, j, tid);
        });
        if (i == 7) {
            sm.lam[tid % DK] = lam;
            sm.beta[tid & 63] = beta;
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) load1(c.nchunks - 1, i);
#pragma unroll
    for (int i = 0; i < 8; ++i) load2(c.nchunks - 1, i);
#pragma unroll
    for (int i = 0; i < 8; ++i) store1(i);
#pragma unroll
    for (int i = 0; i < 8; ++i) load1(max(c.nchunks - 2, 0L), i);

    for (long jc = c.nchunks - 1; jc >= 0; --jc) {
        const long widx = (c.cbase + jc) * H + c.h;
        const long nxt = max(jc - 1, 0L), nxt2 = max(jc - 2, 0L);   // the first chunk again at the end
        f32x4_t dO[4], X[4];
        __syncthreads();   // (1)
        TokenCols<TIn, DV>::get(own, dO, lane);
        if constexpr (DK == 128) {   // the chunk gradients add their halves to it
            const int len = (int)min(64L, c.seos - (c.sbos + jc * 64));
            if (c.tile == 0 && tid < len) b.dbeta[(c.sbos + jc * 64 + tid) * H + c.h] = 0.f;
        }
        // this wave's share of dD = Kd dS'^T + P^T dO: its part of the channels, and of the row tiles of P^T dO
#pragma unroll
        for (int t = 0; t < 4; ++t) X[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        TriFrags<true, NHF> pf;
        mul_rows<NJ>(X, sm.Kd, PK, hf * HK, dST, l16, lq, [&](int i) {
            if (i % 2 == 0) store2(i / 2);
            if (i >= 16 - pf.NB) pf.read(sm.PT, hf, i - (16 - pf.NB), l16, lq);
            const int j = i / 4;
            if (i % 4 == 1 && j < NJ)
                *reinterpret_cast<f32x4_t*>(b.dstates + (widx * DV + col) * DK + hf * HK + 16 * j + 4 * lq) = dST[j];
        });
        {
            f32x4_t y[2];
            pf.mul(dO, hf, y);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int k = 0; k < pf.TILES; ++k)
                    if (pf.tile(hf, k) == t) X[t] += y[k];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) sm.ex[wave][t][lane] = X[t];
        __syncthreads();   // (2)
        // dS'^T Diag(lam) + Qh^T dO on the wave's channels
#pragma unroll
        for (int j = 0; j < NJ; ++j) dST[j] *= *reinterpret_cast<const f32x4_t*>(&sm.lam[hf * HK + 16 * j + 4 * lq]);
        TriFrags<true, NHF> tf;
        mul_cols<NJ>(dST, sm.Qh, PK, hf * HK, dO, l16, lq, [&](int i) {
            if (i % 2 == 0) load2(nxt, i / 2);
            if (i < 4) X[i] = join<NCG, NHF>(sm, cg, i, lane);   // dD
            if (i >= 16 - tf.NB) tf.read(sm.PT + kTriFloats, hf, i - (16 - tf.NB), l16, lq);
        });
        __syncthreads();   // (3)
        // Y = T^T dD on the wave's row tiles
        {
            f32x4_t y[2];
            tf.mul(X, hf, y);
            float* dst = b.ymat + (widx * 64 + 4 * lq) * DV + col;
#pragma unroll
            for (int k = 0; k < tf.TILES; ++k) {
                const int t = tf.tile(hf, k);
                sm.ex2[cg][t][lane] = y[k];
#pragma unroll
                for (int i = 0; i < 4; ++i) dst[(16 * t + i) * DV] = y[k][i];
            }
        }
        __syncthreads();   // (4)
#pragma unroll
        for (int t = 0; t < 4; ++t)   // -dR
            X[t] = -(*reinterpret_cast<const f32x4_t*>(&sm.beta[16 * t + 4 * lq]) * sm.ex2[cg][t][lane]);
        mul_cols<NJ>(dST, sm.Kh, PK, hf * HK, X, l16, lq, [&](int i) {
            if (i % 2 == 0) store1(i / 2);
            else load1(nxt2, i / 2);
        });
    }
    finish();
}

// The reverse walks are the longer ones and come first.
template <typename TIn, int DK, int DV, int NCG, int NHF>
__global__ __launch_bounds__(64 * NHF * NCG) void kda_bwd_walk_kernel(KdaBwdProblem b) {
    __shared__ union Smem {
        __device__ Smem() {}
        KdaRevSmem<DK, NCG, NHF> back;
        KdaStateSmem<DK, NCG, NHF> states;
    } sm;
    constexpr int TILES = DV / (16 * NCG);
    const long half = gridDim.x / 2;
    if (blockIdx.x < half) walk_back<TIn, DK, DV, NCG, NHF>(b, sm.back, chain_of<TILES>(b.f, blockIdx.x, half), threadIdx.x);
    else walk_states<TIn, DK, DV, NCG, NHF>(b, sm.states, chain_of<TILES>(b.f, blockIdx.x - half, half), threadIdx.x);
}

// ------------------------------------------------------------------- gradients of each chunk
// One work-group of four waves per (chunk, head, 64 of the d_k channels), a wave per 16 channels; two work-groups fit a CU, so that
// one's loads and vector work hide behind the other's products (one of eight waves for all 128 channels, alone on its CU:
// 395 us for the training shape, of which the matrix cores were busy for 146). D, Y and dO pass through LDS in
// slices of 32 columns, the next one's loads in flight. Two register layouts of a wave's [64 rows, 16 channels]: the accumulator layout
// (rows 16 t + 4 lq + m) of the products, and the block layout (lane (lq, l16) has rows 16 lq .. 16 lq + 15 of its
// channel), in which the decays are formed, the pairs inside a block are summed and the gradients are formed. An accumulator
// goes to the block layout through a private LDS tile.
//
// The products over d_v (dO D^T, Y D^T, dO S, Y S, D dS') run on the bf16 matrix core at fp32's accuracy: an fp32 operand
// is split into three bf16 planes, x = x0 + x1 + x2 (24 significant bits), and a product takes the six plane products down to
// 2^-24 of it: 00, 01, 10, 11, 02, 20 (a bf16 dO is one plane by itself and takes three). Six 16x16x32 products are 96
// cycles where the fp32 core takes 256.
constexpr int kPlane = 64 * 32;   // elements of one plane of a slice (see plane_at)
template <int OP>                 // planes of dO: 1 (bf16 inputs) or 3
struct alignas(16) KdaGradSmem {
    static constexpr int PC = 68;
    union {
        struct { uint16_t D[3][kPlane], Y[3][kPlane], dO[OP][kPlane]; } in;
        float turn[4][64 * 16];
        float out[2][64 * 64];        // gradients on their way out (see out_at)
    };
    float dP[64 * PC];                // see tri_at
    float dA[64 * PC];
    float beta[64];
    float yv[64];
    float part[4][64];
};

// Element (r, c) of a plane, c a multiple of four: rows of 64 bytes whose 16-byte pieces are permuted. A 16-byte LDS read
// serves lanes 0-3, 12-15, 20-27 together, then 4-11, 16-19, 28-31 (and the same of the upper half): rows 0-3 and 12-15
// of one piece with rows 4-11 of the next. With rows 8-15 of each 16 flipped by 3 these fall into different banks.
__device__ __forceinline__ int plane_at(int r, int c) { return r * 32 + (((c >> 3) ^ ((r >> 3) & 1) * 3) << 3) + (c & 4); }
// Pairs of fp32 values (a, b) as three bf16 planes: in w[0], w[1], w[2] the pair's roundings and those of the two remainders.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&w)[3]) {
    w[0] = pack_bf16x2(a, b);
    a -= bf16_lo_half(w[0]);
    b -= bf16_hi_half(w[0]);
    w[1] = pack_bf16x2(a, b);
    w[2] = pack_bf16x2(a - bf16_lo_half(w[1]), b - bf16_hi_half(w[1]));
}
template <int NP>
struct Planes { uint4 w[NP]; };   // eight values of each plane
__device__ __forceinline__ Planes<3> split8(const float (&x)[8]) {
    uint32_t a[3], b[3], c[3], d[3];
    split_pair(x[0], x[1], a);
    split_pair(x[2], x[3], b);
    split_pair(x[4], x[5], c);
    split_pair(x[6], x[7], d);
    Planes<3> r;
#pragma unroll
    for (int i = 0; i < 3; ++i) r.w[i] = make_uint4(a[i], b[i], c[i], d[i]);
    return r;
}
template <int NP>
__device__ __forceinline__ Planes<NP> read_planes(const uint16_t (*m)[kPlane], int r, int c) {
    Planes<NP> x;
#pragma unroll
    for (int i = 0; i < NP; ++i) x.w[i] = *reinterpret_cast<const uint4*>(&m[i][plane_at(r, c)]);
    return x;
}
// Product i = 0 .. 5 of acc += x y at fp32's accuracy, the smallest first (x of one plane has three of them).
template <int NX>
__device__ __forceinline__ void mul_plane(f32x4_t& acc, const Planes<NX>& x, const Planes<3>& y, int i) {
    constexpr int px[6] = {2, 0, 1, 1, 0, 0}, py[6] = {0, 2, 1, 0, 1, 0};
    if (px[i] < NX) acc = mfma_bf16(x.w[px[i] < NX ? px[i] : 0], y.w[py[i]], acc);
}

// Element (r, i) of dP and dA. They are read by rows (pieces of one row), by columns (16 columns of the row s of all four
// row blocks at once) and by diagonal blocks (a piece of the row s of all four), so the column blocks of row block b are
// permuted by f(b), a permutation for which b ^ f(b) is one as well: either way the four blocks sit in different banks.
template <int PC>
__device__ __forceinline__ int tri_at(int r, int i) {
    const int b = r >> 4, f = ((b << 1) ^ ((b >> 1) * 3)) & 3;
    return r * PC + (i ^ (16 * f));
}
// Row r of a turning tile [64, 16]: written four rows 4 lq + m at a time and read four rows 16 lq + r at a time, so both
// pick the 16 banks of a row.
__device__ __forceinline__ int turn_at(int r) { return ((r & ~3) | ((r ^ (r >> 2) ^ (r >> 4)) & 3)) * 16; }
// 2^x (0 below fp32's range).
__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }
// Element (r, c) of an output tile: a wave writes 16 columns of four row blocks at once.
template <int W>
__device__ __forceinline__ int out_at(int r, int c) { return r * W + (c ^ (16 * ((r >> 4) & 3))); }

// Orders a wave's own LDS writes before its reads of what other lanes wrote.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename TIn, typename TG, int DK, int DV>
__global__ __launch_bounds__(256, 2) void kda_bwd_grad_kernel(KdaBwdProblem b) {
    constexpr int NH = DK / 64, NS = DV / 32, EB = (int)sizeof(TIn), OP = EB == 2 ? 1 : 3;
    using SM = KdaGradSmem<OP>;
    constexpr int PC = SM::PC;
    __shared__ SM sm;
    const ChunkProblem& p = b.f;
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = p.H;
    // the channel halves of a unit read the same D, Y, dO: eight work-groups apart, on one XCD (see chain_of)
    const long blk = blockIdx.x, full = (gridDim.x / (8 * NH)) * (8 * NH);
    const long unit = blk < full ? blk / (8 * NH) * 8 + blk % 8 : blk / NH;
    const int half = (int)(blk < full ? blk / 8 % NH : blk % NH);
    const int c0 = 64 * half, ch = c0 + 16 * wave + l16;
    long bos;
    int len;
    if (!locate_chunk(p, unit / H, bos, len)) return;   // packed: past the last chunk
    const int h = (int)(unit % H);

    // a slice's pieces of four columns (two per thread), raw; inputs through resources that end at the chunk's last token
    const long vb = (bos * H + h) * DV;
    const unsigned vrows = (unsigned)((len - 1) * H * DV + DV);
    const auto gres = make_rsrc(static_cast<const TIn*>(b.d_o) + vb, vrows * EB);
    const auto vres = make_rsrc(static_cast<const TIn*>(p.v) + vb, vrows * EB);
    f32x4_t dpc[2], ypc[2];
    u32x4_t gpc[2], vpc[2];
    float sn[8], dn[8];   // the lane's rows 32 sl + 8 lq + e of S and dS'
    const float* sp = p.states + unit * DV * DK + ch;
    const float* dp = b.dstates + unit * DV * DK + ch;
    auto piece = [](__amdgpu_buffer_rsrc_t r, int o) {
        if constexpr (EB == 2) {
            const u32x2_t x = __builtin_amdgcn_raw_buffer_load_b64(r, o, 0, 0);
            return u32x4_t{x[0], x[1], 0u, 0u};
        } else {
            return __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
        }
    };
    auto load = [&](int sl) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int i = tid + 256 * n, r = i / 8, cc = 32 * sl + 4 * (i % 8);
            dpc[n] = *reinterpret_cast<const f32x4_t*>(b.delta + (unit * 64 + r) * DV + cc);
            ypc[n] = *reinterpret_cast<const f32x4_t*>(b.ymat + (unit * 64 + r) * DV + cc);
            gpc[n] = piece(gres, (r * H * DV + cc) * EB);
            vpc[n] = piece(vres, (r * H * DV + cc) * EB);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sn[e] = sp[(32 * sl + 8 * lq + e) * DK];
            dn[e] = dp[(32 * sl + 8 * lq + e) * DK];
        }
    };
    load(0);
    float bt[2];   // beta of the thread's two piece rows
    {
        const auto br = make_rsrc(p.beta + bos * H + h, (unsigned)(((len - 1) * H + 1) * 4));
#pragma unroll
        for (int n = 0; n < 2; ++n) bt[n] = buf_in<float>(br, ((tid + 256 * n) / 8) * H * 4);
        if (tid % 8 == 0) sm.beta[tid / 8] = bt[0], sm.beta[tid / 8 + 32] = bt[1];
    }
    auto widen = [](u32x4_t x) {
        if constexpr (EB == 2) return f32x4_t{bf16_lo_half(x[0]), bf16_hi_half(x[0]), bf16_lo_half(x[1]), bf16_hi_half(x[1])};
        else return __builtin_bit_cast(f32x4_t, x);
    };

    // dP = dO D^T and dA = -Y D^T (job w + 4 n: lower tile number job / 2, of dP or dA in turn), dO S, Y S and D dS' on the
    // wave's channels, colsum(S dS'), Y . V, all summed slice by slice; dV = beta Y on the way
    f32x4_t aq[4], ay[4], ad[4], tri[5];
    float sds = 0.f, yv[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t) aq[t] = ay[t] = ad[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 5; ++n) tri[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto tile_row = [](int tile) { return tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3; };
    // a wave's jobs alternate between dP and dA, since dA takes twice dP's products: job w + 4 n is one of dA where
    // w + n is odd
    auto tri_jobs = [&](auto parity) {
#pragma unroll
        for (int n = 0; n < 5; ++n) {
            constexpr int par = decltype(parity)::value;
            const int tile = (wave + 4 * n) >> 1, I = tile_row(tile), J = tile - I * (I + 1) / 2;
            const auto y = read_planes<3>(sm.in.D, 16 * J + l16, 8 * lq);
            if ((par + n) & 1) {
                const auto x = read_planes<3>(sm.in.Y, 16 * I + l16, 8 * lq);
#pragma unroll
                for (int i = 0; i < 6; ++i) mul_plane<3>(tri[n], x, y, i);
            } else {
                const auto x = read_planes<OP>(sm.in.dO, 16 * I + l16, 8 * lq);
#pragma unroll
                for (int i = 0; i < 6; ++i) mul_plane<OP>(tri[n], x, y, i);
            }
        }
    };
    auto tri_store = [&](auto parity) {
#pragma unroll
        for (int n = 0; n < 5; ++n) {
            constexpr int par = decltype(parity)::value;
            const int tile = (wave + 4 * n) >> 1, I = tile_row(tile), J = tile - I * (I + 1) / 2;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int r = 16 * I + 4 * lq + m, i = 16 * J + l16;
                if ((par + n) & 1) sm.dA[tri_at<PC>(r, i)] = i < r ? -tri[n][m] : 0.f;
                else sm.dP[tri_at<PC>(r, i)] = i <= r ? tri[n][m] : 0.f;
            }
        }
    };
    auto put = [](uint16_t (*m)[kPlane], int at, const f32x4_t& x) {
        uint32_t a[3], c[3];
        split_pair(x[0], x[1], a);
        split_pair(x[2], x[3], c);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(&m[i][at]) = make_uint2(a[i], c[i]);
    };
#pragma unroll 1
    for (int sl = 0; sl < NS; ++sl) {
        __syncthreads();   // the previous slice is dead
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int i = tid + 256 * n, r = i / 8, cc = 4 * (i % 8);
            const f32x4_t y = ypc[n], v = widen(vpc[n]);
            const int at = plane_at(r, cc);
            put(sm.in.D, at, dpc[n]);
            put(sm.in.Y, at, y);
            if constexpr (OP == 1) *reinterpret_cast<uint2*>(&sm.in.dO[0][at]) = make_uint2(gpc[n][0], gpc[n][1]);
            else put(sm.in.dO, at, widen(gpc[n]));
            yv[n] += y[0] * v[0] + y[1] * v[1] + y[2] * v[2] + y[3] * v[3];
            if (half == 0 && r < len)
                kb_out4(static_cast<TG*>(b.dv) + vb + (long)r * H * DV + 32 * sl + cc,
                        make_float4(bt[n] * y[0], bt[n] * y[1], bt[n] * y[2], bt[n] * y[3]));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sds += sn[i] * dn[i];
        const Planes<3> s = split8(sn), d = split8(dn);
        __syncthreads();
        load(min(sl + 1, NS - 1));   // the last slice again at the end
        if (wave & 1) tri_jobs(std::integral_constant<int, 1>{});
        else tri_jobs(std::integral_constant<int, 0>{});
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const auto o = read_planes<OP>(sm.in.dO, 16 * t + l16, 8 * lq);
            const auto y = read_planes<3>(sm.in.Y, 16 * t + l16, 8 * lq), x = read_planes<3>(sm.in.D, 16 * t + l16, 8 * lq);
#pragma unroll
            for (int i = 0; i < 6; ++i) {   // three chains of products side by side
                mul_plane<3>(ay[t], y, s, i);
                mul_plane<3>(ad[t], x, d, i);
                mul_plane<OP>(aq[t], o, s, i);
            }
        }
    }
    pin();
    // k, q, g of the lane's rows and channel: only now, their registers are the slices' until here
    float k[16], q[16], gm[16];
    const long base = (bos * H + h) * DK;
    {
        const unsigned rows = (unsigned)((len - 1) * H * DK + DK);
        const auto kr = make_rsrc(static_cast<const TIn*>(p.k) + base, rows * EB);
        const auto qr = make_rsrc(static_cast<const TIn*>(p.q) + base, rows * EB);
        const auto gr = make_rsrc(p.g + base, rows * 4);
        const int o0 = 16 * lq * H * DK + ch;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int o = o0 + r * H * DK;
            k[r] = buf_in<TIn>(kr, o * EB);
            q[r] = buf_in<TIn>(qr, o * EB);
            gm[r] = buf_in<float>(gr, o * 4);
        }
    }
    if (wave & 1) tri_store(std::integral_constant<int, 1>{});
    else tri_store(std::integral_constant<int, 0>{});
    // zeros in the upper tiles (I, J) = (0, 1), (0, 2), (0, 3), (1, 2), (1, 3), (2, 3)
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const int job = wave + 4 * n, tile = job >> 1, I = tile < 3 ? 0 : tile < 5 ? 1 : 2, J = tile < 3 ? tile + 1 : tile < 5 ? tile - 1 : 3;
        float* out = (job & 1) ? sm.dA : sm.dP;
#pragma unroll
        for (int m = 0; m < 4; ++m) out[tri_at<PC>(16 * I + 4 * lq + m, 16 * J + l16)] = 0.f;
    }
    sds += __shfl_xor(sds, 16, 64);
    sds += __shfl_xor(sds, 32, 64);
#pragma unroll
    for (int n = 0; n < 2; ++n) {   // a row's eight pieces are consecutive lanes
        float x = yv[n];
        x += dpp_f32<0xB1>(x);
        x += dpp_f32<0x4E>(x);
        x += dpp_f32<0x141>(x);
        if (tid % 8 == 0) sm.yv[tid / 8 + 32 * n] = x;
    }
    __syncthreads();   // dP and dA are whole; D, Y, dO are dead

    // Decays as products of the tokens' own, a[r] = e^{g_r}, each factor at most 1, so that what passes between two tokens never
    // depends on the decays outside of them (differences of gamma summed over the chunk cost 2e-4 of dq among tokens
    // of g = -104, whose sums run into thousands). es holds one of two runs of them within the lane's block, formed anew for
    // each use (registers): from before the block through row r, or from behind row r through the block's end.
    float a[16], es[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) a[r] = exp2_raw(gm[r] * 1.44269504f);   // 2^x is one instruction
    auto through = [&]() {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            hold(a[r]);
            es[r] = r > 0 ? es[r > 0 ? r - 1 : 0] * a[r] : a[r];
        }
    };
    auto behind = [&]() {
        es[15] = 1.f;
#pragma unroll
        for (int r = 14; r >= 0; --r) {
            hold(a[r + 1]);
            es[r] = es[r + 1] * a[r + 1];
        }
    };
    through();
    // decays over whole blocks
    const float t0 = __shfl(es[15], l16, 64), t1 = __shfl(es[15], 16 + l16, 64), t2 = __shfl(es[15], 32 + l16, 64),
                t3 = __shfl(es[15], 48 + l16, 64);
    const float above = (lq > 0 ? t0 : 1.f) * (lq > 1 ? t1 : 1.f) * (lq > 2 ? t2 : 1.f);    // the blocks before the lane's
    const float below = (lq < 3 ? t3 : 1.f) * (lq < 2 ? t2 : 1.f) * (lq < 1 ? t1 : 1.f);    // and behind it

    float* turn = sm.turn[wave];
    auto to_block = [&](const f32x4_t (&x)[4], float (&y)[16]) {
        wave_lds_fence();
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int m = 0; m < 4; ++m) turn[turn_at(16 * t + 4 * lq + m) + l16] = x[t][m];
        wave_lds_fence();
#pragma unroll
        for (int r = 0; r < 16; ++r) y[r] = turn[turn_at(16 * lq + r) + l16];
    };
    float dq[16], l[16], ar[16], w[16];   // ar: with e^{gamma_last - gamma} (D dS') of the row in it
    float kx = lq == 0 ? t0 * t1 * t2 * t3 * sds : 0.f;   // summed over the four blocks at the end
    hold(kx);   // formed here, not there
    to_block(aq, w);
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[r] = above * es[r] * w[r];
    to_block(ay, w);
#pragma unroll
    for (int r = 0; r < 16; ++r) l[r] = -(above * es[r]) * w[r];
    to_block(ad, w);
    behind();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        ar[r] = es[r] * below * w[r];
        kx += k[r] * ar[r];
    }

    // pairs of different blocks. Rows of block I against all rows before it, through the border before
    // block I: step s takes row s of every block (lane lq its own), blocks I and later as zeros.
#pragma unroll
    for (int t = 0; t < 4; ++t) aq[t] = ay[t] = ad[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    {
        f32x4_t vp[2], va[2];   // this step's operands and the next one's: step n has block I = 1 + n / 4, rows 4 (n % 4) ..
        auto read = [&](int n) {
            const int o = tri_at<PC>(16 * (1 + n / 4) + l16, 16 * lq + 4 * (n % 4));
            vp[n & 1] = *reinterpret_cast<const f32x4_t*>(&sm.dP[o]);
            va[n & 1] = *reinterpret_cast<const f32x4_t*>(&sm.dA[o]);
        };
        read(0);
        float gap = 0.f;   // the decay over the blocks between the lane's and block I; 0 for the block itself and those behind it
#pragma unroll
        for (int n = 0; n < 12; ++n) {
            if (n + 1 < 12) read(n + 1);
            pin();
            const int I = 1 + n / 4;
            if (n % 4 == 0) gap = lq == I - 1 ? 1.f : gap * (I == 2 ? t1 : t2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int s = 4 * (n % 4) + e;
                const float kb = k[s] * (es[s] * gap);
                aq[I] = mfma4(vp[n & 1][e], kb, aq[I]);
                ay[I] = mfma4(va[n & 1][e], kb, ay[I]);
            }
        }
    }
    // Columns of block J against all rows behind it, through the border behind block J.
    through();
    {
        f32x4_t vp[2], va[2], bt4[2];   // step n has block J = 2 - n / 4, rows 4 (n % 4) .. of every block
        auto read = [&](int n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int o = tri_at<PC>(16 * lq + 4 * (n % 4) + e, 16 * (2 - n / 4) + l16);
                vp[n & 1][e] = sm.dP[o];
                va[n & 1][e] = sm.dA[o];
            }
            bt4[n & 1] = *reinterpret_cast<const f32x4_t*>(&sm.beta[16 * lq + 4 * (n % 4)]);
        };
        read(0);
        float gap = 0.f;   // over the blocks between block J and the lane's
#pragma unroll
        for (int n = 0; n < 12; ++n) {
            if (n + 1 < 12) read(n + 1);
            pin();
            const int J = 2 - n / 4;
            if (n % 4 == 0) gap = lq == J + 1 ? 1.f : gap * (J == 1 ? t2 : t1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = 4 * (n % 4) + i;
                const float e = es[s] * gap;
                ad[J] = mfma4(vp[n & 1][i], q[s] * e, ad[J]);
                ad[J] = mfma4(va[n & 1][i], bt4[n & 1][i] * k[s] * e, ad[J]);
            }
        }
    }
    to_block(aq, w);
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[r] += es[r] * w[r];
    to_block(ay, w);
#pragma unroll
    for (int r = 0; r < 16; ++r) l[r] += es[r] * w[r];
    to_block(ad, w);
    behind();
#pragma unroll
    for (int r = 0; r < 16; ++r) ar[r] += es[r] * w[r];

    // pairs inside the lane's block: w[i] holds e^{gamma_r - gamma_i}, decayed row by row
    f32x4_t vp[2][4], va[2][4];   // rows r and r + 1 of the lane's diagonal blocks
    auto read = [&](int r) {
        const int o = tri_at<PC>(16 * lq + r, 16 * lq);
#pragma unroll
        for (int i4 = 0; 4 * i4 < r; ++i4) {
            vp[r & 1][i4] = *reinterpret_cast<const f32x4_t*>(&sm.dP[o + 4 * i4]);
            va[r & 1][i4] = *reinterpret_cast<const f32x4_t*>(&sm.dA[o + 4 * i4]);
        }
    };
    read(0);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        if (r + 1 < 16) read(r + 1);
        pin();
        const float bk = sm.beta[16 * lq + r] * k[r];
        w[r] = 1.f;
#pragma unroll
        for (int i = 0; i < r; ++i) {
            const float p1 = vp[r & 1][i / 4][i % 4], p2 = va[r & 1][i / 4][i % 4];
            w[i] *= a[r];
            const float ke = w[i] * k[i];
            dq[r] += p1 * ke;
            l[r] += p2 * ke;
            ar[i] += (p1 * q[r] + p2 * bk) * w[i];
        }
        // The row's sums are formed here, not at their use at the end. Without this the compiler moved all of them there and
        // spilled some 800 registers, and that build had the sums of rows 14 and 15 wrong for a chunk of 16 tokens, the same on
        // every run, for a reason that was not found.
        hold(dq[r]);
        hold(l[r]);
#pragma unroll
        for (int i = 0; i < r; ++i) hold(ar[i]);
    }
    // gradients; a token's pair with itself has no decay, so it stays out of w (its two parts there would cancel)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const float bl = sm.beta[16 * lq + r] * l[r];
        w[r] = q[r] * dq[r] + k[r] * (bl - ar[r]);
        const float db = row16_sum(k[r] * l[r]);
        if (l16 == 0) sm.part[wave][16 * lq + r] = db;
        const float own_pair = sm.dP[tri_at<PC>(16 * lq + r, 16 * lq + r)];
        dq[r] += own_pair * k[r];
        l[r] = bl + ar[r] + own_pair * q[r];   // dk
    }
    kx += __shfl_xor(kx, 16, 64);
    kx += __shfl_xor(kx, 32, 64);
#pragma unroll
    for (int r = 14; r >= 0; --r) w[r] += w[r + 1];
    const float b1 = __shfl(w[0], 16 + l16, 64), b2 = __shfl(w[0], 32 + l16, 64), b3 = __shfl(w[0], 48 + l16, 64);
    const float tail = kx + (lq < 3 ? b3 : 0.f) + (lq < 2 ? b2 : 0.f) + (lq < 1 ? b1 : 0.f);
    __syncthreads();   // every wave is done with its turning tile
    auto store_rows = [&](const float* tile, auto* dst) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int i = tid + 256 * n, r = i / 16, cc = 4 * (i % 16);
            if (r < len) kb_out4(dst + base + (long)r * H * DK + c0 + cc, *reinterpret_cast<const float4*>(&tile[out_at<64>(r, cc)]));
        }
    };
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int o = out_at<64>(16 * lq + r, 16 * wave + l16);
        sm.out[0][o] = dq[r];
        sm.out[1][o] = l[r];
    }
    __syncthreads();
    store_rows(sm.out[0], static_cast<TG*>(b.dq));
    store_rows(sm.out[1], static_cast<TG*>(b.dk));
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r) sm.out[0][out_at<64>(16 * lq + r, 16 * wave + l16)] = w[r] + tail;
    __syncthreads();
    store_rows(sm.out[0], b.dg);
    if (tid < len) {
        float s = (half == 0 ? sm.yv[tid] : 0.f) + (sm.part[0][tid] + sm.part[1][tid]) + (sm.part[2][tid] + sm.part[3][tid]);
        float* dst = b.dbeta + (bos + tid) * H + h;
        // two halves add to the zero that the reverse walk left: one addition each, whose order does not matter
        if constexpr (NH == 1) *dst = s;
        else atomicAdd(dst, s);
    }
}

// -------------------------------------------------------------------- launchers
KdaBwdLayout kda_bwd_workspace_layout(int B, int T, int H, int dk, int dv, int N, int varlen) {
    auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
    KdaBwdLayout w{};
    w.fwd = kda_workspace_layout(B, T, H, dk, N, varlen, 4);
    const size_t units = (size_t)w.fwd.nc_bound * H;
    w.off_states = al(w.fwd.total);
    w.off_dstates = al(w.off_states + units * dv * dk * 4);
    w.off_delta = al(w.off_dstates + units * dv * dk * 4);
    w.off_y = al(w.off_delta + units * 64 * dv * 4);
    w.total = units ? w.off_y + units * 64 * dv * 4 : w.fwd.total;
    return w;
}

// The rule by the number of work-groups of 32 columns. Those (2 x 2 waves, a SIMD each) step a chunk in about 6 us, those of
// 64 columns (4 x 2 waves) in about 10, moving half the operators per column, those of 16 (1 x 4 waves) in about 5, moving
// twice as many. The narrower ones win as long as all of them run at once. The whole pass, dk = dv = 128, bf16:
//   pairs x chunks   16 columns   32    64
//    4 x 64             322      398   596
//   16 x 64             470      542   740
//   18 x 64             659      570   768
//   32 x 32             454      381   476
//   64 x 32             910      714   667
// Packed sequences mostly differ in length, so the longest one's time counts up to twice as many of 32 columns (64 pairs,
// 331 .. 1345 tokens: 393 us, with 64 columns 406); those of 16 keep their limit (16 pairs: 157 us against 183, 32: 245, 231).
constexpr long kShortWalks = 128, kNarrowWalks = 256;

template <typename TIn, int DK, int DV>
static hipError_t kda_bwd_launch(const KdaBwdProblem& b, hipStream_t s) {
    const ChunkProblem& p = b.f;
    const long pairs = (long)p.N * p.H, units = p.nc_bound * p.H;
    if (pairs == 0) return hipSuccess;
    auto walk = [&](auto kern, int columns, int threads) {
        return launch(kern, dim3((unsigned)(2 * pairs * (DV / columns))), dim3(threads), s, b);
    };
    const long groups = 2 * pairs * (DV / 32);   // work-groups of 32 columns
    const hipError_t e = groups <= kShortWalks ? walk(kda_bwd_walk_kernel<TIn, DK, DV, 1, 4>, 16, 256)
                         : groups <= (p.cu_seqlens ? 2 : 1) * kNarrowWalks ? walk(kda_bwd_walk_kernel<TIn, DK, DV, 2, 2>, 32, 256)
                                                                         : walk(kda_bwd_walk_kernel<TIn, DK, DV, 4, 2>, 64, 512);
    if (e != hipSuccess || units == 0) return e;
    const dim3 grid((unsigned)(units * (DK / 64)));
    return b.grad_bf16 ? launch(kda_bwd_grad_kernel<TIn, uint16_t, DK, DV>, grid, dim3(256), s, b)
                       : launch(kda_bwd_grad_kernel<TIn, float, DK, DV>, grid, dim3(256), s, b);
}

template <typename TIn>
static hipError_t kda_bwd_dispatch(const KdaBwdProblem& b, hipStream_t s) {
    if (b.f.dk == 64)
        return b.f.dv == 64 ? kda_bwd_launch<TIn, 64, 64>(b, s) : kda_bwd_launch<TIn, 64, 128>(b, s);
    return b.f.dv == 64 ? kda_bwd_launch<TIn, 128, 64>(b, s) : kda_bwd_launch<TIn, 128, 128>(b, s);
}

hipError_t launch_kda_chunk_bwd(const KdaBwdProblem& b, hipStream_t s) {
    hipError_t e = launch_chunk_base(b.f, s);
    if (e == hipSuccess) e = launch_kda_prepare_f32(b.f, s);
    if (e != hipSuccess) return e;
    return b.f.bf16 ? kda_bwd_dispatch<uint16_t>(b, s) : kda_bwd_dispatch<float>(b, s);
}

}  // namespace gdn
