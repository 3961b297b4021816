// Gated linear recurrence per channel: a scan over long sequences, its gradients, and its form on a pool of states, for gfx950.
//
// Per sequence and channel, a_t = exp(g_t):
//     h_t = a_t h_{t-1} + b_t,   b_t = x_t, or (blend) (1 - a_t) x_t.
// Backward, with D_t the gradient reaching h_t and E_t = a_t D_t what it passes on to h_{t-1}:
//     D_t = dh_t + E_{t+1},   E_{len+1} = dhT,   dx = D or (1 - a) D,   dg = E_t h_{t-1} or E_t (h_{t-1} - x_t),   dh0 = E_1.
// Four operations an element against 8 (forward) or 14 (backward) bytes in bf16: bound by bytes, if the sequence is cut. A run of tokens
// maps the state entering it to the one leaving it by h -> e^G h + H, G the sum of its gates, and such maps compose, so every thread first
// forms the map of its few tokens (8 channels wide, as loaded, in registers), the maps of a tile of 256 tokens (or 32) x 64 channels are
// joined in LDS, and with the state entering the tile known each thread runs its tokens again from registers: inputs are read once,
// outputs written once.
// Where a gate is slow, e^G in fp32 has lost the digits of 1 - e^G, and a product of such numbers drifts with the length (32768 blended tokens of
// g = -1e-6 and a constant input: 1.5e-3 off). So maps go by sums of gates, and where G > -1/2 by K = 1 - e^G: h + (H - K h).
// The state entering a tile comes from the tiles before it, in the same launch, as in the published single-pass scan with decoupled look-back (D. Merrill,
// M. Garland, 2016): a tile publishes its own map as soon as it has it, and its
// final state once it knows what enters. One that waits reads the four tiles before it and goes on from the last
// final state through the maps behind it. It always takes the same sums in the same order, wherever it finds the state, so the
// bits do not depend on timing. Tiles are numbered by a ticket drawn at the start of a work-group, and a tile waits for
// lower tickets only, whose work-groups run already and publish their maps without waiting: every wait ends. The words that pass
// between work-groups are single relaxed atomics at device scope that hold their own mark (all ones: not there yet), so nothing has to be
// fenced. Where sequences are short, one work-group walks a sequence's tiles instead and keeps the state itself. The backward pass takes the
// tiles the other way; the states entering them are kept by the forward one.
#include "gdn_block.h"
#include "gdn_row.h"

namespace gdn {

constexpr uint32_t kNotYet = 0xffffffffu;
constexpr int kLookBack = 4;

// 1 - e^g for g in (-1/2, 1/2): the series to g^9 / 9! (the rest is below 2^-27 of it).
__device__ __forceinline__ float complement(float g) {
    float s = 1.f / 362880.f;
    s = __fmaf_rn(s, g, 1.f / 40320.f);
    s = __fmaf_rn(s, g, 1.f / 5040.f);
    s = __fmaf_rn(s, g, 1.f / 720.f);
    s = __fmaf_rn(s, g, 1.f / 120.f);
    s = __fmaf_rn(s, g, 1.f / 24.f);
    s = __fmaf_rn(s, g, 1.f / 6.f);
    s = __fmaf_rn(s, g, 0.5f);
    s = __fmaf_rn(s, g, 1.f);
    return -g * s;
}
// 1 - e^g, a = e^g: 1 - a loses the digits of a small difference.
__device__ __forceinline__ float one_minus_exp(float g, float a) {
    const float k = complement(g);   // always: a branch here costs registers and spills
    return fabsf(g) < 0.5f ? k : 1.f - a;
}
// The factor of a map as one number, with the digits that matter: e^G, or where that is near 1 minus its distance to 1. decay(0) = 1: what is infinite
// stays so where nothing decays.
__device__ __forceinline__ float decay(float G) {
    const float k = complement(G), a = __expf(G);
    return ((G < 0.f) & (G > -0.5f)) ? -k : a;
}
// One map applied. (Chosen before the sum, which shortens the chains of maps: 1 x 262144 x 64 204 us otherwise, 192 so.)
__device__ __forceinline__ float apply(float q, float h, float H) {
    return __fmaf_rn(q, h, H) + (__float_as_int(q) < 0 ? h : 0.f);
}

// a value that is never the mark (any NaN becomes the ordinary one)
__device__ __forceinline__ float publishable(float x) { return x == x ? x : __uint_as_float(0x7fc00000u); }
__device__ __forceinline__ void publish_map(uint64_t* p, float q, float H) {
    const uint64_t w = (uint64_t)__float_as_uint(publishable(H)) << 32 | __float_as_uint(publishable(q));
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(float* p, float h) {
    __hip_atomic_store(reinterpret_cast<uint32_t*>(p), __float_as_uint(publishable(h)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What leaves the tile before this one, for column `col` (within a row) of every lane. step: the distance of the tile before it in rows
// (-1 forward, 1 backward); before: the number of tiles before it in its sequence (>= 1).
__device__ __forceinline__ float enter_from(const ScanProblem& p, long row, int step, int before, unsigned col) {
    const long pitch = (long)p.ncb * kScanChannels;
    const int depth = min(before, kLookBack);
    for (;;) {
        float c = 0.f;
        bool ok = false;
        uint32_t state[kLookBack];
        uint64_t map[kLookBack];
#pragma unroll
        for (int j = 0; j < kLookBack; ++j) {
            const long at = (row + (long)step * (min(j, depth - 1) + 1)) * pitch;
            state[j] = __hip_atomic_load(reinterpret_cast<uint32_t*>(p.pref) + at + col, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            map[j] = __hip_atomic_load(p.agg + at + col, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int j = kLookBack - 1; j >= 0; --j) {
            if (j < depth) {
                const bool here = state[j] != kNotYet, mapped = (uint32_t)map[j] != kNotYet;
                const float through = apply(__uint_as_float((uint32_t)map[j]), c, __uint_as_float((uint32_t)(map[j] >> 32)));
                c = here ? __uint_as_float(state[j]) : through;
                ok = here || (ok && mapped);
            }
        }
        if (__all(ok)) return c;
        __builtin_amdgcn_s_sleep(1);
    }
}

// The rows of tiles of this call; where one work-group walks a whole sequence, its sequences.
__device__ __forceinline__ long scan_rows(const ScanProblem& p) {
    if (!p.ticket) return p.N;
    return p.base ? min((long)p.base[p.N], p.rows) : p.rows;
}

// A tile's place: sequence, number within it, first token, tokens.
struct ScanTile {
    int n, s, last, t0, len;   // last: the number of its sequence's last tile
    int begin, end;            // the sequence's tokens
    long row;                  // of the carries
    // on to tile `to` of the same sequence
    __device__ __forceinline__ void move(const ScanProblem& p, int to) {
        row += to - s;
        s = to;
        t0 = begin + s * p.tile;
        len = max(0, min(end - t0, p.tile));
    }
};
// walk: row is a sequence, and the tile its first or (back) its last. The tiles of sequence n then begin at row n + begin / tile.
__device__ __forceinline__ ScanTile scan_tile(const ScanProblem& p, long row, long rows, bool back) {
    ScanTile k;
    const bool walk = !p.ticket;
    const int per = max(1, (p.T + p.tile - 1) / p.tile);
    k.s = 0;
    if (walk) {
        k.n = (int)row;
    } else if (!p.cu_seqlens) {
        k.n = (int)(row / per);
        k.s = (int)(row - (long)k.n * per);
    } else {
        int lo = 0, hi = p.N;   // the last n with base[n] <= row
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.base[mid] <= row) lo = mid; else hi = mid;
        }
        k.n = lo;
        k.s = (int)(row - p.base[lo]);
    }
    if (p.cu_seqlens) {
        k.begin = min(max(p.cu_seqlens[k.n], 0), p.tokens);
        k.end = min(max(p.cu_seqlens[k.n + 1], k.begin), p.tokens);
    } else {
        k.begin = k.n * p.T;
        k.end = k.begin + p.T;
    }
    k.last = max(0, (k.end - k.begin - 1) / p.tile);
    if (p.base) k.last = (int)min((long)k.last, rows - 1 - (row - k.s));   // none waits for a tile that is not run
    k.row = !walk ? row - k.s : !p.cu_seqlens ? row * per : row + k.begin / p.tile;
    const int at = walk && back ? k.last : k.s;
    k.s = 0;
    k.move(p, at);
    return k;
}

// A work-group's channel block, and its row of tiles: in chained calls the ticket drawn from the block's own counter (one counter for all, and
// 1,024 work-groups queue 5 us for it). Rows shift by one channel block each, so that the L2 of one XCD, which takes every eighth
// work-group, does not see the same few channels of every row (32768 x 2048: 113 us without, 106 with it).
struct ScanPlace {
    int cb;
    long row;
};
__device__ __forceinline__ ScanPlace scan_place(const ScanProblem& p) {
    const unsigned id = blockIdx.x, row = id / (unsigned)p.ncb;
    return ScanPlace{(int)((id + row) % (unsigned)p.ncb), (long)row};
}
constexpr int kTicketWords = 16;   // a counter to itself in 64 bytes
__device__ __forceinline__ long draw_row(const ScanProblem& p, const ScanPlace& place, int* lds) {
    if (!p.ticket) return place.row;
    if (threadIdx.x == 0)
        *lds = __hip_atomic_fetch_add(p.ticket + kTicketWords * place.cb, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*lds);   // one for all: rows and addresses stay scalar
}

// Lays the tiles of packed sequences out, by one work-group: K sequences a thread at a time.
template <int K>
__device__ __forceinline__ void lay_tiles_out(const ScanProblem& p, int* sum) {
    int before = 0;
    for (int n0 = 0; n0 < p.N; n0 += 256 * K) {
        const int n = n0 + K * threadIdx.x;
        int cu[K + 1], tiles[K], mine = 0;
#pragma unroll
        for (int i = 0; i <= K; ++i) cu[i] = p.cu_seqlens[min(n + i, p.N)];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int lo = min(max(cu[i], 0), p.tokens), hi = min(max(cu[i + 1], lo), p.tokens);
            tiles[i] = n + i < p.N ? max(1, (hi - lo + p.tile - 1) / p.tile) : 0;
            mine += tiles[i];
        }
        mine = (int)min((long)mine, p.rows);   // fewer than 2^23: the sums fit
        __syncthreads();
        sum[threadIdx.x] = mine;
        __syncthreads();
        for (int d = 1; d < 256; d *= 2) {
            const int add = (int)threadIdx.x >= d ? sum[threadIdx.x - d] : 0;
            __syncthreads();
            sum[threadIdx.x] += add;
            __syncthreads();
        }
        // offsets that fall can count more tiles than there are rows: those past the last row are not run
        long first = (long)before + sum[threadIdx.x] - mine;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if (n + i < p.N) p.base[n + i] = (int)min(first, p.rows);
            first += tiles[i];
        }
        before = (int)min((long)before + sum[255], p.rows);
    }
    if (threadIdx.x == 0) p.base[p.N] = before;
}

// Clears the marks and the tickets, and lays the tiles of packed sequences out: 16 sequences a thread where they are many (a call on 8192
// sequences 340 -> 311 us), one where they are few (8 sequences, both directions 55.5 -> 53.5).
__global__ __launch_bounds__(256) void scan_setup_kernel(ScanProblem p) {
    __shared__ int sum[256];
    const long words = p.rows * p.ncb * kScanChannels;   // agg: 2 a word, pref: 1
    const long at = (long)blockIdx.x * 256 + threadIdx.x, step = (long)gridDim.x * 256;
    uint4* a = reinterpret_cast<uint4*>(p.agg);
    uint4* b = reinterpret_cast<uint4*>(p.pref);
    const uint4 mark = make_uint4(kNotYet, kNotYet, kNotYet, kNotYet);
    for (long i = at; i < words / 2; i += step) a[i] = mark;
    for (long i = at; i < words / 4; i += step) b[i] = mark;
    if (blockIdx.x != 0) return;
    for (int i = threadIdx.x; i < p.ncb; i += 256) p.ticket[kTicketWords * i] = 0;
    if (!p.base) return;
    if (p.N <= 512) lay_tiles_out<1>(p, sum);
    else lay_tiles_out<16>(p, sum);
}

constexpr int R = 4;   // tokens per thread
// as Raw8's hide(), for what is computed from them
__device__ __forceinline__ void hide(Raw8<float>& r) {
    asm volatile("" : "+v"(r.a.x), "+v"(r.a.y), "+v"(r.a.z), "+v"(r.a.w), "+v"(r.b.x), "+v"(r.b.y), "+v"(r.b.z), "+v"(r.b.w));
}
constexpr int scan_threads(int TOK) { return 8 * TOK / R; }
// A wave's threads form the maps of eight groups, and as lanes of one channel each they join them; the first wave joins the waves' maps, and hands
// every wave what enters it. What all waves read of another is written between the two barriers of a tile or by it alone, so that a
// work-group that walks needs no third one.
constexpr int kGroups = 8;
__device__ __forceinline__ void wave_fence() {   // between LDS writes of some lanes and reads of others of the same wave
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// TOK: tokens of a tile; TOK / R groups of 8 lanes, 8 channels a lane. 32768 x 2048 in bf16, blended: 101 us, 5.3 TB/s (1.5 us of it for factors
// with the digits of slow gates).
template <typename TX, typename TH, int TOK, bool BLEND, bool NT>
__global__ __launch_bounds__(scan_threads(TOK), 4) void scan_fwd_kernel(ScanProblem p) {
    constexpr int G = TOK / R, W = G / kGroups;
    __shared__ float2 maps[G][kScanChannels];    // of every group: G, then the state entering it; H
    __shared__ float sums[W][kScanChannels];     // of every wave's groups together: G
    __shared__ float2 waves[W][kScanChannels];   // factor and H
    __shared__ float enter[W][kScanChannels];    // the state entering it
    __shared__ int ticket;
    const long rows = scan_rows(p);
    const ScanPlace place = scan_place(p);
    const int cb = place.cb;
    const long row = draw_row(p, place, &ticket);
    if (row >= rows) return;
    ScanTile tile = scan_tile(p, row, rows, false);
    float state = 0.f;   // walking, a lane of the first wave's channel: what leaves the tile
    for (;;) {
        unsigned thread = threadIdx.x;
        asm volatile("" : "+v"(thread));   // what is computed from it is not kept from one tile to the next
        const int l = thread & 7, grp = thread >> 3;
        const unsigned c = (unsigned)(cb * kScanChannels + 8 * l);
        const bool in = c < (unsigned)p.D;
        // offsets within a tile fit 32 bits (256 tokens of at most 2^20 channels); only x may lie further apart
        const unsigned at0 = (unsigned)(grp * R) * p.D + c;
        Raw8<TX> xr[R];
        Raw8<float> gr[R];
        const long first = (long)tile.t0 * p.D;
        const int mine = min(max(tile.len - grp * R, 0), R);   // this thread's tokens
        // every thread loads: tokens past the end the last one again, channels past the end the first ones, put out of action below. (A branch
        // around each load, and the compiler waits for it before the next.)
        const unsigned cl = in ? c : 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            xr[i].zero();
            gr[i].zero();
        }
        if (tile.len > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int t = min(grp * R + i, tile.len - 1);
                gr[i].load(p.g + first + ((unsigned)t * (unsigned)p.D + cl));
                xr[i].load(static_cast<const TX*>(p.x) + (tile.t0 + t) * p.x_row + cl);
            }
        }
        float a[R][8], b[BLEND ? R : 1][8], S[8], H[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) S[e] = H[e] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {   // tokens past the end: g = 0, x = 0, the state as it is
            float x[8];
            gr[i].get(a[i]);
            xr[i].get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = i < mine ? a[i][e] : 0.f;
                x[e] = i < mine ? x[e] : 0.f;
                a[i][e] = __expf(g);
                if constexpr (BLEND) {
                    x[e] *= one_minus_exp(g, a[i][e]);
                    b[i][e] = x[e];
                }
                H[e] = __fmaf_rn(a[i][e], H[e], x[e]);
                S[e] += g;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) maps[grp][8 * l + e] = make_float2(S[e], H[e]);
        wave_fence();
        const int wave = __builtin_amdgcn_readfirstlane(thread >> 6), ch = thread & 63, g0 = kGroups * wave;
        float qk[kGroups], hk[kGroups];
        {
            float St = 0.f, Ht = 0.f;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                const float2 m = maps[g0 + k][ch];
                qk[k] = decay(m.x);
                hk[k] = m.y;
                Ht = apply(qk[k], Ht, m.y);
                St += m.x;
            }
            sums[wave][ch] = St;
            waves[wave][ch] = make_float2(decay(St), Ht);
        }
        __syncthreads();
        if (wave == 0) {
            const unsigned col = (unsigned)(cb * kScanChannels + ch);
            const bool real = col < (unsigned)p.D;
            float St = 0.f, Ht = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const float2 m = waves[k][ch];
                Ht = apply(m.x, Ht, m.y);
                St += sums[k][ch];
            }
            const float q = decay(St);
            const long at = row * p.ncb * kScanChannels + col;
            float h = state;
            if (tile.s == 0) {
                if (p.h0 && real) h = p.h0[(long)tile.n * p.D + col];
            } else if (p.ticket) {
                publish_map(p.agg + at, q, Ht);
                h = enter_from(p, row, -1, tile.s, col);
            }
            state = apply(q, h, Ht);
            if (p.ticket && tile.s < tile.last) publish_state(p.pref + at, state);
            // blended, the map's: the last tokens' own factors would add their rounding to it, call by call
            if (BLEND && p.hT && real && tile.s == tile.last) p.hT[(long)tile.n * p.D + col] = state;
            if (p.carries && real) p.carries[tile.row * p.D + col] = h;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                enter[k][ch] = h;
                h = apply(waves[k][ch].x, h, waves[k][ch].y);
            }
        }
        __syncthreads();
        {
            float h = enter[wave][ch];
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                maps[g0 + k][ch].x = h;
                h = apply(qk[k], h, hk[k]);
            }
        }
        wave_fence();
        if constexpr (!BLEND) {
#pragma unroll
            for (int i = 0; i < R; ++i) xr[i].hide();
        }
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = maps[grp][8 * l + e].x;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float x[8];
            if constexpr (!BLEND) xr[i].get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = __fmaf_rn(a[i][e], h[e], BLEND ? b[i][e] : i < mine ? x[e] : 0.f);
            if (in && i < mine) store8<NT>(static_cast<TH*>(p.h) + first + (at0 + i * p.D), h);
        }
        // the state behind the sequence's last token (or the one it began with, where it has none)
        if (!BLEND && p.hT && in && tile.s == tile.last && (mine > 0 ? grp * R + mine == tile.len : grp == 0 && tile.len == 0))
            store8<false>(p.hT + (long)tile.n * p.D + c, h);
        if (p.ticket || tile.s == tile.last) break;
        tile.move(p, tile.s + 1);
    }
}

// Two work-groups per CU at 128 registers a thread for bf16 x. Blended, a and 1 - a together do not fit: both are formed again from g, and the
// gradient's part of a tile's map is summed forward, so that a is not kept for it either (4 x 2048 x 2048 in bf16 60 us; with both kept and one
// work-group per CU 64, half the size 29 and 34). fp32 x spills even so and has one work-group per CU (us, one and two: blended 4 x 2048 x 2048 84 and
// 102; plain 80 and 84, 1 x 262144 x 64 194 and 238, 64 packed sequences of 128 x 2048 90 and 85). bf16 x with an fp32 h spills 7 registers without
// blend and keeps two (4 x 2048 x 2048 64 and 64, packed 70 and 79; 1 x 262144 x 64 232 and 190).
template <typename TX, typename TH, int TOK, bool BLEND, bool NT>
__global__ __launch_bounds__(scan_threads(TOK), sizeof(TX) == 4 ? 2 : 4) void scan_bwd_kernel(ScanProblem p) {
    constexpr int G = TOK / R, W = G / kGroups;
    // of every group: G, then its factor; H, then the state entering it; the gradient's part of its map, then the gradient entering it
    __shared__ float mQ[G][kScanChannels], mH[G][kScanChannels], mE[G][kScanChannels];
    // of every wave's groups together: G, factor, H, the gradient's part
    __shared__ float wS[W][kScanChannels], wQ[W][kScanChannels], wH[W][kScanChannels], wE[W][kScanChannels];
    __shared__ float enter[W][kScanChannels];   // the gradient entering it
    __shared__ int ticket;
    const long rows = scan_rows(p);
    const ScanPlace place = scan_place(p);
    const int cb = place.cb;
    const long row = rows - 1 - draw_row(p, place, &ticket);   // the last tiles first
    if (row < 0) return;
    ScanTile tile = scan_tile(p, row, rows, true);
    float back = 0.f;   // walking: what leaves the tile, as in the forward pass
    for (;;) {
        unsigned thread = threadIdx.x;
        asm volatile("" : "+v"(thread));   // what is computed from it is not kept from one tile to the next
        const int l = thread & 7, grp = thread >> 3;
        const unsigned c = (unsigned)(cb * kScanChannels + 8 * l);
        const bool in = c < (unsigned)p.D;
        const unsigned at0 = (unsigned)(grp * R) * p.D + c;
        Raw8<TX> xr[R];
        Raw8<TH> dr[R];
        Raw8<float> gr[R];
        const long first = (long)tile.t0 * p.D;
        const int mine = min(max(tile.len - grp * R, 0), R);
        const unsigned cl = in ? c : 0;   // loads as in the forward pass
#pragma unroll
        for (int i = 0; i < R; ++i) {
            xr[i].zero();
            dr[i].zero();
            gr[i].zero();
        }
        if (tile.len > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int t = min(grp * R + i, tile.len - 1);
                const unsigned at = (unsigned)t * (unsigned)p.D + cl;
                gr[i].load(p.g + first + at);
                xr[i].load(static_cast<const TX*>(p.x) + (tile.t0 + t) * p.x_row + cl);
                dr[i].load(static_cast<const TH*>(p.dh) + first + at);
            }
        }
        float a[BLEND ? 1 : R][8], A[8], S[8], H[8], E[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) A[e] = 1.f, S[e] = H[e] = E[e] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float g[8], x[8], d[8];
            gr[i].get(g);
            xr[i].get(x);
            dr[i].get(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (i >= mine) g[e] = x[e] = d[e] = 0.f;
                const float at = __expf(g[e]);
                if constexpr (BLEND) x[e] *= one_minus_exp(g[e], at);
                else a[i][e] = at;
                H[e] = __fmaf_rn(at, H[e], x[e]);
                S[e] += g[e];
                if constexpr (BLEND) {
                    A[e] *= at;
                    E[e] = __fmaf_rn(A[e], d[e], E[e]);
                }
            }
        }
        if constexpr (!BLEND) {
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                float d[8];
                dr[i].get(d);
#pragma unroll
                for (int e = 0; e < 8; ++e) E[e] = a[i][e] * ((i < mine ? d[e] : 0.f) + E[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mQ[grp][8 * l + e] = S[e];
            mH[grp][8 * l + e] = H[e];
            mE[grp][8 * l + e] = E[e];
        }
        wave_fence();
        const int wave = __builtin_amdgcn_readfirstlane(thread >> 6), ch = thread & 63, g0 = kGroups * wave;
        const unsigned col = (unsigned)(cb * kScanChannels + ch);
        float h = col < (unsigned)p.D ? p.carries[tile.row * p.D + col] : 0.f;
        {
            float St = 0.f, Ht = 0.f, Et = 0.f;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                const float m = mQ[g0 + k][ch], q = decay(m);
                mQ[g0 + k][ch] = q;
                Ht = apply(q, Ht, mH[g0 + k][ch]);
                St += m;
            }
#pragma unroll
            for (int k = kGroups - 1; k >= 0; --k) Et = apply(mQ[g0 + k][ch], Et, mE[g0 + k][ch]);
            wS[wave][ch] = St;
            wQ[wave][ch] = decay(St);
            wH[wave][ch] = Ht;
            wE[wave][ch] = Et;
        }
        __syncthreads();
        if (wave == 0) {   // what comes from the tiles behind this one
            float St = 0.f, Et = 0.f;
#pragma unroll
            for (int k = W - 1; k >= 0; --k) {
                Et = apply(wQ[k][ch], Et, wE[k][ch]);
                St += wS[k][ch];
            }
            const float q = decay(St);
            const long at = row * p.ncb * kScanChannels + col;
            float d = back;
            if (tile.s == tile.last) {
                if (p.dhT && col < (unsigned)p.D) d = p.dhT[(long)tile.n * p.D + col];
            } else if (p.ticket) {
                publish_map(p.agg + at, q, Et);
                d = enter_from(p, row, 1, tile.last - tile.s, col);
            }
            back = apply(q, d, Et);
            if (p.ticket && tile.s > 0) publish_state(p.pref + at, back);
#pragma unroll
            for (int k = W - 1; k >= 0; --k) {
                enter[k][ch] = d;
                d = apply(wQ[k][ch], d, wE[k][ch]);
            }
        }
        // the states entering the groups
        for (int k = 0; k < wave; ++k) h = apply(wQ[k][ch], h, wH[k][ch]);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const float m = mH[g0 + k][ch];
            mH[g0 + k][ch] = h;
            h = apply(mQ[g0 + k][ch], h, m);
        }
        __syncthreads();
        {
            float d = enter[wave][ch];
#pragma unroll
            for (int k = kGroups - 1; k >= 0; --k) {
                const float m = mE[g0 + k][ch];
                mE[g0 + k][ch] = d;
                d = apply(mQ[g0 + k][ch], d, m);
            }
        }
        wave_fence();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            xr[i].hide();
            dr[i].hide();
            if constexpr (BLEND) hide(gr[i]);
        }
        // backward over the tokens for D, which takes the place of dh, then forward for the states
        float D[R][8], hs[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) E[e] = mE[grp][8 * l + e];
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            float g[8];
            gr[i].get(g);
            dr[i].get(D[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                D[i][e] = (i < mine ? D[i][e] : 0.f) + E[e];
                E[e] = (BLEND ? __expf(i < mine ? g[e] : 0.f) : a[i][e]) * D[i][e];
            }
        }
        if (p.dh0 && in && tile.s == 0 && grp == 0) store8<false>(p.dh0 + (long)tile.n * p.D + c, E);
#pragma unroll
        for (int i = 0; i < R; ++i)
            if constexpr (BLEND) hide(gr[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) hs[e] = mH[grp][8 * l + e];
#pragma unroll
        for (int i = 0; i < R; ++i) {   // tokens past the end are the last ones: what becomes of the state there meets nobody
            float g[8], x[8];
            gr[i].get(g);
            xr[i].get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float at = BLEND ? __expf(g[e]) : a[i][e], Et = at * D[i][e];
                if constexpr (BLEND) {
                    const float keep = one_minus_exp(g[e], at);
                    g[e] = Et * (hs[e] - x[e]);
                    D[i][e] *= keep;
                    x[e] *= keep;
                } else {
                    g[e] = Et * hs[e];
                }
                hs[e] = __fmaf_rn(at, hs[e], x[e]);
            }
            if (in && i < mine) {
                store8<NT>(static_cast<TX*>(p.dx) + first + (at0 + i * p.D), D[i]);
                store8<NT>(p.dg + first + (at0 + i * p.D), g);
            }
        }
        if (p.ticket || tile.s == 0) break;
        tile.move(p, tile.s - 1);
    }
}

// Runs of tokens on a pool of states: a lane walks its sequence's tokens for four channels. Tokens come four at a time, so that a run waits for memory once
// in four (24 runs of 5 tokens, 2048 channels: 4.9 us).
template <typename TX, typename TH, bool BLEND>
__global__ __launch_bounds__(64) void scan_update_kernel(ScanProblem p, int cblocks) {
    const int n = blockIdx.x / cblocks;
    const long c = ((long)(blockIdx.x % cblocks) * 64 + threadIdx.x) * 4;
    if (c >= p.D) return;
    int t0 = n, t1 = n + 1;
    if (p.cu_seqlens) {   // offsets outside [0, tokens] or falling ones are clamped
        t0 = min(max(p.cu_seqlens[n], 0), p.tokens);
        t1 = min(max(p.cu_seqlens[n + 1], t0), p.tokens);
    }
    if (t0 >= t1) return;
    const int slot = p.slots[n];
    TH* hp = static_cast<TH*>(p.h) + c;
    float h[4] = {0.f, 0.f, 0.f, 0.f};
    if (slot < 0 || slot >= p.n_slots) {   // a padded entry: zeros for its tokens, no state touched
        for (int t = t0; t < t1; ++t) store4c(hp + (long)t * p.D, h);
        return;
    }
    Raw4<float> state;
    state.load(p.pool + (long)slot * p.D + c);
    state.get(h);
    constexpr int TB = 4;
    for (int tb = t0; tb < t1; tb += TB) {
        Raw4<TX> xr[TB];
        Raw4<float> gr[TB];
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const long t = min(tb + i, t1 - 1);
            xr[i].load(static_cast<const TX*>(p.x) + t * p.x_row + c);
            gr[i].load(p.g + t * p.D + c);
        }
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const int t = tb + i;
            if (t < t1) {
                float x[4], g[4];
                xr[i].get(x);
                gr[i].get(g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float q = decay(g[e]);
                    h[e] = apply(q, h[e], BLEND ? one_minus_exp(g[e], q) * x[e] : x[e]);
                }
                store4c(hp + (long)t * p.D, h);
                if (p.out_slots) {
                    const int to = p.out_slots[t];
                    if (to >= 0 && to < p.n_slots) store4c(p.pool + (long)to * p.D + c, h);
                }
            }
        }
    }
    if (!p.out_slots) store4c(p.pool + (long)slot * p.D + c, h);
}

// Tiles of 256 tokens, or of 32 where that leaves most of them empty: rows of at most 32 tokens, and sequences of fewer than 128 (on average, where
// they are packed) in calls that fill the device (8192 tokens of 2048 channels forward, in tiles of 256 and 32: sequences of 16 tokens 235 and 48 us, of
// 64 68 and 37, of 128 44 and 39, of 256 33 and 41). In small calls one tile a sequence saves the pass that clears the marks. Empty sequences count in the
// average, since their number is all that the host knows: one of 32768 x 2048 alone 102 us, beside 255 empty ones 219, beside 256, in tiles of 32, 300.
// Where no sequence can have more than two tiles (four of 32 tokens) one work-group walks them all, which saves that pass and the wait for other
// work-groups (1 x 512 x 2048, a call: 14.6 and 10.6 us, backward 17.3 and 13.5; 128 x 64 x 2048 in tiles of 32: 32.1 and 29.7, 51.7 and 47.3), as long as
// the device holds all of them at once (64 x 512 x 2048: 98 and 103, backward 183 and 205). Three tiles gain no more (8 x 700 x 1024: 16.5 and
// 16.3, backward 21.1 and 23.6), but packed sequences are as a rule far shorter than all of them together: there the call may have four, which goes
// before tiles of 32 (40 sequences of 25 tokens, 512 channels: 15.2 passed on, 11.1 walked, backward 17.4 and 14.0).
ScanLayout scan_layout(int tokens, int T, int N, int D, int varlen) {
    ScanLayout w{};
    const long ncb = ((long)D + kScanChannels - 1) / kScanChannels;
    const int longest = varlen ? tokens : T;   // the longest that a sequence can be
    const bool brief = longest <= 32 || (tokens >= (varlen ? 257 : 4096) && tokens < 128L * N), at_once = N * ncb <= 512;
    const bool few = varlen && N > 1 && tokens <= 1024 && at_once;
    w.tile = brief && !(few && longest > 32) ? 32 : 256;
    const long per = T > w.tile ? ((long)T + w.tile - 1) / w.tile : 1;
    w.carry_rows = varlen ? (long)N + tokens / (brief ? 32 : 256) : N * per;   // whatever the channels are
    w.rows = varlen ? (long)N + tokens / w.tile : N * per;
    if (w.tile == 32 ? longest <= 128 : longest <= 256 || few || (longest <= 512 && at_once)) return w;
    const size_t cells = (size_t)w.rows * ncb * kScanChannels;
    w.off_base = ((size_t)kTicketWords * 4 * ncb + 255) / 256 * 256;
    w.off_agg = w.off_base + (varlen ? (((size_t)N + 1) * 4 + 255) / 256 * 256 : 0);
    w.off_pref = w.off_agg + cells * 8;
    w.total = w.off_pref + cells * 4;
    return w;
}

// The grid of tiles, with the marks cleared first where tiles pass states on.
static hipError_t scan_setup(const ScanProblem& p, long& tiles, hipStream_t s) {
    tiles = (p.ticket ? p.rows : (long)p.N) * p.ncb;
    if (!p.ticket) return hipSuccess;
    const long blocks = (p.rows * p.ncb * kScanChannels / 2 + 511) / 512;   // two stores of 16 bytes a thread, and one
    return launch(scan_setup_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), s, p);
}

// Outputs go past the caches where they exceed the L2s together.
static bool scan_large(const ScanProblem& p) { return (long)p.tokens * p.D >= 1 << 23; }

template <typename TX, typename TH, bool BLEND>
static hipError_t scan_fwd(const ScanProblem& p, hipStream_t s) {
    long tiles;
    const hipError_t e = scan_setup(p, tiles, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)tiles), block(scan_threads(p.tile));
    if (p.tile == 32) return launch(scan_fwd_kernel<TX, TH, 32, BLEND, false>, grid, block, s, p);
    return scan_large(p) ? launch(scan_fwd_kernel<TX, TH, 256, BLEND, true>, grid, block, s, p)
                         : launch(scan_fwd_kernel<TX, TH, 256, BLEND, false>, grid, block, s, p);
}
template <typename TX, typename TH, bool BLEND>
static hipError_t scan_bwd(const ScanProblem& p, hipStream_t s) {
    long tiles;
    const hipError_t e = scan_setup(p, tiles, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)tiles), block(scan_threads(p.tile));
    if (p.tile == 32) return launch(scan_bwd_kernel<TX, TH, 32, BLEND, false>, grid, block, s, p);
    return scan_large(p) ? launch(scan_bwd_kernel<TX, TH, 256, BLEND, true>, grid, block, s, p)
                         : launch(scan_bwd_kernel<TX, TH, 256, BLEND, false>, grid, block, s, p);
}
template <typename TX, typename TH, bool BLEND>
static hipError_t scan_update(const ScanProblem& p, hipStream_t s) {
    const int cblocks = (p.D + 255) / 256;
    return launch(scan_update_kernel<TX, TH, BLEND>, dim3((unsigned)((long)p.N * cblocks)), dim3(64), s, p, cblocks);
}

hipError_t launch_scan_fwd(const ScanProblem& p, hipStream_t s) {
    if (p.N == 0) return hipSuccess;
    if (!p.bf16) return p.blend ? scan_fwd<float, float, true>(p, s) : scan_fwd<float, float, false>(p, s);
    if (p.h_bf16) return p.blend ? scan_fwd<uint16_t, uint16_t, true>(p, s) : scan_fwd<uint16_t, uint16_t, false>(p, s);
    return p.blend ? scan_fwd<uint16_t, float, true>(p, s) : scan_fwd<uint16_t, float, false>(p, s);
}
hipError_t launch_scan_bwd(const ScanProblem& p, hipStream_t s) {
    if (p.N == 0) return hipSuccess;
    if (!p.bf16) return p.blend ? scan_bwd<float, float, true>(p, s) : scan_bwd<float, float, false>(p, s);
    if (p.h_bf16) return p.blend ? scan_bwd<uint16_t, uint16_t, true>(p, s) : scan_bwd<uint16_t, uint16_t, false>(p, s);
    return p.blend ? scan_bwd<uint16_t, float, true>(p, s) : scan_bwd<uint16_t, float, false>(p, s);
}
hipError_t launch_scan_update(const ScanProblem& p, hipStream_t s) {
    if (p.N == 0 || p.tokens == 0) return hipSuccess;
    if (!p.bf16) return p.blend ? scan_update<float, float, true>(p, s) : scan_update<float, float, false>(p, s);
    if (p.h_bf16) return p.blend ? scan_update<uint16_t, uint16_t, true>(p, s) : scan_update<uint16_t, uint16_t, false>(p, s);
    return p.blend ? scan_update<uint16_t, float, true>(p, s) : scan_update<uint16_t, float, false>(p, s);
}

}  // namespace gdn
