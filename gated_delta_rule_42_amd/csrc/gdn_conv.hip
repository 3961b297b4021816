// Short causal convolution per channel, its gradients, and its form on a pool of windows, for gfx950.
//
// Per sequence and channel c, with W taps (2 .. 4) and u_t the inputs, those before the sequence from its window (or zero):
//     z_t = b + sum_{k < W} w[W-1-k] u_{t-k},   y_t = z_t, or z_t sigmoid(z_t).
// Backward, with dz_t = dy_t act'(z_t), z computed again:
//     dx_t = sum_{k < W, t+k < len} w[W-1-k] dz_{t+k} + (the gradient of the window left behind, for its W - 1 tokens),
//     dw[W-1-k] = sum_t dz_t u_{t-k},   db = sum_t dz_t,   and the window's gradient as dx continued to t < 0.
// Some ten operations an element against 4 (forward) or 6 (backward) bytes in bf16: bound by bytes. A lane owns V neighbouring channels and
// walks TL tokens, all of whose rows it loads first, so that an input is read from HBM once and W times from registers; the
// W - 1 rows before (and, backward, behind) the tile are read again and come from the caches. Which sequence a token belongs to is
// looked up by one lane per token and broadcast, so that sequences may begin anywhere in a tile.
#include <type_traits>

#include "gdn_block.h"
#include "gdn_row.h"

namespace gdn {

constexpr int V = 4;   // channels of a lane: 8 in bf16 halve the loads but cost a wave per SIMD (41 us against 46 forward, 12.4 against 13.7 on the pool)

// Where token t stands: its sequence, its position there, the tokens from it to the sequence's end (0: no sequence covers it).
struct Token {
    int n, pos, rem;
};
__device__ __forceinline__ Token locate_token(const ConvProblem& p, int t) {
    Token k{0, 0, 0};
    if (t < 0 || t >= p.tokens) return k;
    if (!p.cu_seqlens) {
        k.n = t / p.T;
        k.pos = t - k.n * p.T;
        k.rem = p.T - k.pos;
        return k;
    }
    int lo = 0, hi = p.N;   // the last n with cu[n] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_seqlens[mid] <= t) lo = mid; else hi = mid;
    }
    const int b = min(max(p.cu_seqlens[lo], 0), p.tokens), e = min(max(p.cu_seqlens[lo + 1], b), p.tokens);
    if (t >= b && t < e) {
        k.n = lo;
        k.pos = t - b;
        k.rem = e - t;
    }
    return k;
}
// The tokens t0 .. t0 + count - 1 of a wave's tile, looked up by a lane each. What every token asks for are bits of masks, which all
// lanes share; the sequence is kept in LDS for the few tokens that need it.
template <int W>
struct TileTokens {
    uint64_t covered, starts, ends[W - 1];   // ends[r]: the tokens with r + 1 to go
    const int* seq;
    int pos0;                                // the first token's position
    __device__ __forceinline__ TileTokens(const ConvProblem& p, long t0, int count, int* lds) {
        const int lane = threadIdx.x & 63;
        const Token k = locate_token(p, lane < count && t0 + lane < p.tokens ? (int)(t0 + lane) : -1);   // -1: none
        covered = __ballot(k.rem > 0);
        starts = __ballot(k.rem > 0 && k.pos == 0);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) ends[r] = __ballot(k.rem == r + 1);
        lds[lane] = k.n;
        seq = lds;
        pos0 = __builtin_amdgcn_readfirstlane(k.pos);   // all lanes are here
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __device__ __forceinline__ bool is(uint64_t mask, int i) const { return (mask >> i) & 1; }
};

// A lane's taps, w[v][j] of its channels.
template <int W>
__device__ __forceinline__ void load_taps(const float* weight, long c, float (&w)[V][W]) {
    float f[V * W];
#pragma unroll
    for (int i = 0; i < V * W; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(weight + c * W + i);
        f[i] = a.x; f[i + 1] = a.y; f[i + 2] = a.z; f[i + 3] = a.w;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) w[v][j] = f[v * W + j];
}

__device__ __forceinline__ void load_bias(const float* bias, long c, float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = 0.f;
    if (bias) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const float4 a = *reinterpret_cast<const float4*>(bias + c + v);
            b[v] = a.x; b[v + 1] = a.y; b[v + 2] = a.z; b[v + 3] = a.w;
        }
    }
}

__device__ __forceinline__ float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// Row r of sequence n's window (zeros without one).
template <typename T, int W>
__device__ __forceinline__ void window_row(const ConvProblem& p, const void* window, int n, int r, long c, float (&x)[V]) {
    Raw4<T> raw;
    raw.zero();
    if (window) raw.load(static_cast<const T*>(window) + ((long)n * (W - 1) + r) * p.D + c);
    raw.get(x);
}

// The last W - 1 inputs of sequence n, as they lie in memory.
template <typename T, int W>
__device__ __forceinline__ void leave_window(const ConvProblem& p, int n, long c) {
    int b = n * p.T, e = b + p.T;
    if (p.cu_seqlens) {
        b = min(max(p.cu_seqlens[n], 0), p.tokens);
        e = min(max(p.cu_seqlens[n + 1], b), p.tokens);
    }
    const int len = e - b;
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int pos = len - (W - 1) + r;
        Raw4<T> raw;
        raw.zero();
        if (pos >= 0) raw.load(static_cast<const T*>(p.x) + (long)(b + pos) * p.x_row + c);
        else if (p.window0) raw.load(static_cast<const T*>(p.window0) + ((long)n * (W - 1) + r + len) * p.D + c);
        raw.put(static_cast<T*>(p.windowT) + ((long)n * (W - 1) + r) * p.D + c);
    }
}

// One token of the forward pass from the inputs u[0] .. u[W-1] tokens back.
template <int W, bool SILU>
__device__ __forceinline__ void conv_token(const float (&w)[V][W], const float (&b)[V], const float (&u)[W][V], float (&y)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float z = b[v];
#pragma unroll
        for (int j = W - 1; j >= 0; --j) z += w[v][W - 1 - j] * u[j][v];
        y[v] = SILU ? z * sigmoid_f(z) : z;
    }
}
template <int W>
__device__ __forceinline__ void move_on(float (&u)[W][V]) {
#pragma unroll
    for (int j = W - 1; j > 0; --j)
#pragma unroll
        for (int v = 0; v < V; ++v) u[j][v] = u[j - 1][v];
}

// Work-groups in rows of cblocks, which share tokens; those past the `tiles` rows of tiles leave the windows, a wave per sequence. TL = 6 tokens a wave:
// with fewer the rows before a tile weigh more, with more there are fewer waves (kernels, 4 x 2048 x 6144 bf16, TL 4, 6, 8, 12: 41.5, 38.6, 40.0, 40.5 us; fp32
// 70.7, 69.8, 71.6, 74.7; 8 x 500 x 2048 9.2, 9.0, 9.7, 10.7). Bound by bytes: 5.2 TB/s.
template <typename T, int W, int TL, bool SILU>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvProblem p, int cblocks, int tiles) {
    using Raw = Raw4<T>;
    __shared__ int seq[4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // scalar, and so are tokens and masks
    const unsigned id = blockIdx.y * gridDim.x + blockIdx.x;   // y: past 2^32 threads
    const int by = (int)(id / (unsigned)cblocks), bx = (int)(id - (unsigned)by * (unsigned)cblocks);
    const long c0 = ((long)bx * 64 + lane) * V;
    const bool in = c0 < p.D;
    const long c = in ? c0 : 0;   // lanes past the channels go along with the first ones and store nothing
    const unsigned cb = (unsigned)c * sizeof(T);
    if (by >= tiles) {
        const int n = (by - tiles) * 4 + wave;
        if (p.windowT && n < p.N && in) leave_window<T, W>(p, n, c);
        return;
    }
    const long first = ((long)by * 4 + wave) * TL;
    if (first >= p.tokens) return;
    const int t0 = (int)first;
    // rows outside the tensor: the nearest one, for no token's sake. (A branch around each load, and the compiler waits for it
    // before the next.)
    Raw raw[TL + W - 1];
#pragma unroll
    for (int i = 0; i < TL + W - 1; ++i)
        raw[i].load(at_byte(static_cast<const T*>(p.x) + (long)min(max(t0 - (W - 1) + i, 0), p.tokens - 1) * p.x_row, cb));
    float w[V][W], b[V];
    load_taps<W>(p.weight, c, w);
    load_bias(p.bias, c, b);
    const TileTokens<W> tok(p, t0, TL, seq[wave]);
    T* yp = static_cast<T*>(p.y) + (long)t0 * p.D;
    float u[W][V], y[V];   // u[k]: the input k tokens back
#pragma unroll
    for (int k = 1; k < W; ++k) raw[W - 1 - k].get(u[k]);
    if (tok.covered == (1ull << TL) - 1 && tok.starts == 0 && tok.pos0 >= W - 1) {   // one sequence, away from its beginning
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            raw[i + W - 1].get(u[0]);
            conv_token<W, SILU>(w, b, u, y);
            if (in) store4c(at_byte(yp + (long)i * p.D, cb), y);
            move_on<W>(u);
        }
        return;
    }
    // sequences begin or end here: token by token, rows read again (they are in the caches), in a loop that takes no registers from the
    // way above
#pragma unroll
    for (int k = 1; k < W; ++k)
        if (tok.is(tok.covered, 0) && tok.pos0 < k) window_row<T, W>(p, p.window0, tok.seq[0], W - 1 - k + tok.pos0, c, u[k]);
    const int count = min(TL, p.tokens - t0);
    const T* xp = static_cast<const T*>(p.x) + (long)t0 * p.x_row;
    Raw next;
    next.load(at_byte(xp, cb));
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        next.get(u[0]);
        next.load(at_byte(xp + (long)min(i + 1, count - 1) * p.x_row, cb));
        if (tok.is(tok.covered, i)) {
            if (i > 0 && tok.is(tok.starts, i)) {
#pragma unroll
                for (int j = 1; j < W; ++j) window_row<T, W>(p, p.window0, tok.seq[i], W - 1 - j, c, u[j]);
            }
            conv_token<W, SILU>(w, b, u, y);
            if (in) store4c(at_byte(yp + (long)i * p.D, cb), y);
        }
        move_on<W>(u);
    }
}

// The gradient of sequence n's window: its rows enter the first W - 1 tokens, and those that are still there at the end
// are rows of the window left behind.
template <typename T, int W>
__device__ __forceinline__ void window_gradient(const ConvProblem& p, int n, long c) {
    int b0 = n * p.T, e0 = b0 + p.T;
    if (p.cu_seqlens) {
        b0 = min(max(p.cu_seqlens[n], 0), p.tokens);
        e0 = min(max(p.cu_seqlens[n + 1], b0), p.tokens);
    }
    const int len = e0 - b0;
    float w[V][W], b[V], g[W - 1][V], u[2 * W - 2][V];
    load_taps<W>(p.weight, c, w);
    load_bias(p.bias, c, b);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        window_row<T, W>(p, p.window0, n, r, c, u[r]);
        Raw4<T> raw;
        raw.zero();
        if (r < len) raw.load(static_cast<const T*>(p.x) + (long)(b0 + r) * p.x_row + c);
        raw.get(u[W - 1 + r]);
#pragma unroll
        for (int v = 0; v < V; ++v) g[r][v] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        if (t < len) {
            Raw4<T> raw;
            float dz[V];
            raw.load(static_cast<const T*>(p.dy) + (long)(b0 + t) * p.D + c);
            raw.get(dz);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (p.silu) {
                    float z = b[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) z += w[v][j] * u[t + j][v];
                    const float s = sigmoid_f(z);
                    dz[v] *= s * (1.f + z * (1.f - s));
                }
#pragma unroll
                for (int r = t; r < W - 1; ++r) g[r][v] += w[v][r - t] * dz[v];
            }
        }
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        if (p.dwindowT && r >= len) {
            float d[V];
            window_row<T, W>(p, p.dwindowT, n, r - len, c, d);
#pragma unroll
            for (int v = 0; v < V; ++v) g[r][v] += d[v];
        }
        store4c(static_cast<T*>(p.dwindow0) + ((long)n * (W - 1) + r) * p.D + c, g[r]);
    }
}

// Backward, a wave walks a run of tokens, blocks of BL at a time, the next block's rows in flight while the current one is worked on. It
// carries the last W - 1 inputs and dz; a token's dx is complete W - 1 tokens later, so that a run goes W - 1 tokens past its end (where
// its sequence does). Run lengths are multiples of BL less W - 1: whole blocks. Packed 8053 x 6144 in bf16: 71 us at 4.6 TB/s (a copy of as many
// bytes 5.3), with 40 us of vector instructions close behind (24 an element).
//
// Rows of work-groups below `parts` take four runs each, sum their contributions to dw and db in registers, then over the waves in
// LDS, and write a partial row [D, W], [D] (the gradients themselves if there is only one); those past them take the windows' gradients. No
// atomics: the same inputs give the same bits.
constexpr int kConvBlock = 4;   // BL: with 8 in bf16 two waves fit a SIMD instead of three (packed 8054 x 6144: 85 us against 69)
template <typename T, int W, bool SILU, bool DW>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvProblem p, int cblocks, int parts, int run) {
    constexpr int BL = kConvBlock, H = W - 1;
    __shared__ float part[DW ? 4 : 1][DW ? 64 * V * (W + 1) : 1];
    __shared__ int seq[4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // scalar, and so are tokens and masks
    const int by = (int)(blockIdx.x / (unsigned)cblocks), bx = (int)(blockIdx.x - (unsigned)by * (unsigned)cblocks);
    const long c0 = ((long)bx * 64 + lane) * V;
    const bool in = c0 < p.D;
    const long c = in ? c0 : 0;   // lanes past the channels go along with the first ones and store nothing
    const unsigned cb = (unsigned)c * sizeof(T);
    if (by >= parts) {
        const int n = (by - parts) * 4 + wave;
        if (n < p.N && in) window_gradient<T, W>(p, n, c);
        return;
    }
    float w[V][W], b[V], dw[V][W], db[V];
    load_taps<W>(p.weight, c, w);
    load_bias(p.bias, c, b);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[v][j] = 0.f;
    }
    const long begin = ((long)by * 4 + wave) * run;
    if (begin < p.tokens) {
        const int r0 = (int)begin, r1 = (int)min(begin + run, (long)p.tokens), last = p.tokens - 1;
        const T* xp = static_cast<const T*>(p.x);
        const T* gp = static_cast<const T*>(p.dy);
        T* dxp = static_cast<T*>(p.dx);
        float u[W][V], dz[W][V];   // u[k]: the input k tokens back; dz[k]: k tokens back
        Raw4<T> xr[BL], gr[BL], xn[BL], gn[BL];
#pragma unroll
        for (int i = 0; i < BL; ++i) {   // rows past the tensor: the last one, for no token's sake
            xr[i].load(at_byte(xp + (long)min(r0 + i, last) * p.x_row, cb));
            gr[i].load(at_byte(gp + (long)min(r0 + i, last) * p.D, cb));
        }
#pragma unroll
        for (int k = 1; k < W; ++k) {
            Raw4<T> before;
            before.load(at_byte(xp + (long)max(r0 - k, 0) * p.x_row, cb));
            before.get(u[k]);
#pragma unroll
            for (int v = 0; v < V; ++v) dz[k][v] = 0.f;
        }
        // the tokens base - H .. of masks and seq; every SPAN tokens they are looked up anew
        constexpr int SPAN = (64 - H) / BL * BL;
        int base = r0;
        TileTokens<W> tok(p, (long)r0 - H, 64, seq[wave]);
        if (tok.is(tok.covered, H)) {
            const Token k = locate_token(p, r0);
#pragma unroll
            for (int j = 1; j < W; ++j)
                if (k.pos < j) window_row<T, W>(p, p.window0, k.n, H - j + k.pos, c, u[j]);
        }
        for (int t0 = r0; t0 < r1 + H; t0 += BL) {
            if (t0 - base == SPAN) {
                base = t0;
                tok = TileTokens<W>(p, (long)t0 - H, 64, seq[wave]);
            }
            const int s = t0 - base, own = r1 - t0;   // tokens i < own are the run's own
#pragma unroll
            for (int i = 0; i < BL; ++i) {
                xn[i].load(at_byte(xp + (long)min(t0 + BL + i, last) * p.x_row, cb));
                gn[i].load(at_byte(gp + (long)min(t0 + BL + i, last) * p.D, cb));
            }
            // bits: the H tokens before the block (before the run, whatever they are), then the block's
            const unsigned all = (1u << (H + BL)) - 1, before = (1u << H) - 1;
            const unsigned covered = (unsigned)(tok.covered >> s) | (t0 == r0 ? before : 0u);
            const bool plain = (covered & all) == all && ((unsigned)(tok.starts >> (s + H)) & (all >> H)) == 0 &&
                               ((unsigned)(tok.ends[0] >> s) & (all >> 1)) == 0 && own + H >= BL;
            if (plain) {   // inside one sequence, its end no nearer than this block's: no token needs a look at the masks
#pragma unroll
                for (int i = 0; i < BL; ++i) {
                    float d[V];
                    xr[i].get(u[0]);
                    gr[i].get(d);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if constexpr (SILU) {
                            float z = b[v];
#pragma unroll
                            for (int j = W - 1; j >= 0; --j) z += w[v][W - 1 - j] * u[j][v];
                            const float sg = sigmoid_f(z);
                            d[v] *= sg * (1.f + z * (1.f - sg));
                        }
                        dz[0][v] = d[v];
                    }
                    if (DW && (BL - i > H || i < own)) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            db[v] += d[v];
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[v][W - 1 - j] += d[v] * u[j][v];
                        }
                    }
                    if (i >= H || t0 > r0) {   // the token H back has all of its terms
                        float dx[V];
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            dx[v] = w[v][W - 1] * dz[W - 1][v];
#pragma unroll
                            for (int m = 1; m < W; ++m) dx[v] += w[v][W - 1 - m] * dz[W - 1 - m][v];
                        }
                        if (in) store4c(at_byte(dxp + (long)(t0 + i - H) * p.dx_row, cb), dx);
                    }
                    move_on<W>(u);
                    move_on<W>(dz);
                }
            } else {   // token by token, rows read again (they are in the caches), in a loop that takes no registers from the way above
                Raw4<T> xt, gt;
                xt.load(at_byte(xp + (long)min(t0, last) * p.x_row, cb));
                gt.load(at_byte(gp + (long)min(t0, last) * p.D, cb));
#pragma unroll 1
                for (int i = 0; i < BL; ++i) {
                    const int t = t0 + i, at = s + H + i;   // at: the token's bit
                    float d[V];
                    xt.get(u[0]);
                    gt.get(d);
                    xt.load(at_byte(xp + (long)min(t + 1, last) * p.x_row, cb));
                    gt.load(at_byte(gp + (long)min(t + 1, last) * p.D, cb));
#pragma unroll
                    for (int v = 0; v < V; ++v) dz[0][v] = 0.f;
                    // a token behind the run matters only where the run's last one belongs to the same sequence
                    const bool reach = i < own || (t < r1 + H && !(tok.starts >> (at - (i - own)) & ((2ull << (i - own)) - 1)));
                    if (tok.is(tok.covered, at) && reach) {
                        if (t > r0 && tok.is(tok.starts, at)) {
#pragma unroll
                            for (int j = 1; j < W; ++j) window_row<T, W>(p, p.window0, tok.seq[at], H - j, c, u[j]);
                        }
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            dz[0][v] = d[v];
                            if constexpr (SILU) {
                                float z = b[v];
#pragma unroll
                                for (int j = W - 1; j >= 0; --j) z += w[v][W - 1 - j] * u[j][v];
                                const float sg = sigmoid_f(z);
                                dz[0][v] *= sg * (1.f + z * (1.f - sg));
                            }
                            if (DW && i < own) {
                                db[v] += dz[0][v];
#pragma unroll
                                for (int j = 0; j < W; ++j) dw[v][W - 1 - j] += dz[0][v] * u[j][v];
                            }
                        }
                    }
                    if (t - H >= r0 && t - H < r1 && tok.is(tok.covered, at - H)) {
                        float dx[V];
                        int rem = W;   // tokens of its sequence from it on, W for that or more
#pragma unroll
                        for (int r = 0; r < H; ++r)
                            if (tok.is(tok.ends[r], at - H)) rem = r + 1;
#pragma unroll
                        for (int v = 0; v < V; ++v) dx[v] = w[v][W - 1] * dz[W - 1][v];
#pragma unroll
                        for (int m = 1; m < W; ++m)
                            if (m < rem)
#pragma unroll
                                for (int v = 0; v < V; ++v) dx[v] += w[v][W - 1 - m] * dz[W - 1 - m][v];
                        if (p.dwindowT && rem < W) {
                            float e[V];
                            window_row<T, W>(p, p.dwindowT, tok.seq[at - H], H - rem, c, e);
#pragma unroll
                            for (int v = 0; v < V; ++v) dx[v] += e[v];
                        }
                        if (in) store4c(at_byte(dxp + (long)(t - H) * p.dx_row, cb), dx);
                    }
                    move_on<W>(u);
                    move_on<W>(dz);
                }
            }
#pragma unroll
            for (int i = 0; i < BL; ++i) {
                xr[i] = xn[i];
                gr[i] = gn[i];
            }
        }
    }
    if constexpr (DW) {
        float* mine = part[wave] + lane * V * (W + 1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) mine[v * (W + 1) + j] = dw[v][j];
            mine[v * (W + 1) + W] = db[v];
        }
        __syncthreads();
        float* rw = parts > 1 ? p.partial + (long)by * p.D * (W + 1) : p.dweight;
        float* rb = parts > 1 ? rw + (long)p.D * W : p.dbias;
        for (int i = threadIdx.x; i < 64 * V * (W + 1); i += 256) {
            const int ch = i / (W + 1), j = i % (W + 1);
            const long cc = (long)bx * 64 * V + ch;
            if (cc < p.D) {
                const float a = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
                if (j < W) {
                    if (rw) rw[cc * W + j] = a;
                } else if (rb) {
                    rb[cc] = a;
                }
            }
        }
    }
}

// Runs of tokens on a pool of windows: a lane walks its sequence's tokens for V channels. The window stays as loaded, so its rows
// are moved, never rounded. Tokens come four at a time. 256 sequences of one token, 12288 channels in bf16: 11.9 us, bound by bytes (4.2 TB/s, a
// copy of as many bytes 4.4).
template <typename T, int W>
__global__ __launch_bounds__(256) void conv_update_kernel(ConvProblem p, int cblocks) {
    using Raw = Raw4<T>;
    const int n = blockIdx.x / cblocks;
    const long c = ((long)(blockIdx.x % cblocks) * 256 + threadIdx.x) * V;
    if (c >= p.D) return;
    int t0 = n, t1 = n + 1;
    if (p.cu_seqlens) {   // offsets outside [0, tokens] or falling ones are clamped
        t0 = min(max(p.cu_seqlens[n], 0), p.tokens);
        t1 = min(max(p.cu_seqlens[n + 1], t0), p.tokens);
    }
    if (t0 >= t1) return;
    const int slot = p.slots[n];
    T* yp = static_cast<T*>(p.y) + c;
    float y[V];
    if (slot < 0 || slot >= p.n_slots) {   // a padded entry: zeros for its tokens, no window touched
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = 0.f;
        for (int t = t0; t < t1; ++t) store4c(yp + (long)t * p.D, y);
        return;
    }
    T* pool = static_cast<T*>(p.pool) + c;
    const long slot_size = (long)(W - 1) * p.D;
    Raw u[W];   // u[k]: the input k tokens back
#pragma unroll
    for (int k = 1; k < W; ++k) u[k].load(pool + slot * slot_size + (long)(W - 1 - k) * p.D);
    float w[V][W], b[V];
    load_taps<W>(p.weight, c, w);
    load_bias(p.bias, c, b);
    constexpr int TB = 4;
    for (int tb = t0; tb < t1; tb += TB) {
        Raw x[TB];
#pragma unroll
        for (int i = 0; i < TB; ++i) x[i].load(static_cast<const T*>(p.x) + (long)min(tb + i, t1 - 1) * p.x_row + c);
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const int t = tb + i;
            if (t < t1) {
                u[0] = x[i];
                float f[W][V];
#pragma unroll
                for (int k = 0; k < W; ++k) u[k].get(f[k]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float z = b[v];
#pragma unroll
                    for (int j = W - 1; j >= 0; --j) z += w[v][W - 1 - j] * f[j][v];
                    y[v] = p.silu ? z * sigmoid_f(z) : z;
                }
                store4c(yp + (long)t * p.D, y);
#pragma unroll
                for (int k = W - 1; k > 0; --k) u[k] = u[k - 1];
                if (p.out_slots) {
                    const int to = p.out_slots[t];
                    if (to >= 0 && to < p.n_slots)
#pragma unroll
                        for (int k = 1; k < W; ++k) u[k].put(pool + to * slot_size + (long)(W - 1 - k) * p.D);
                }
            }
        }
    }
    if (!p.out_slots)
#pragma unroll
        for (int k = 1; k < W; ++k) u[k].put(pool + slot * slot_size + (long)(W - 1 - k) * p.D);
}

// f of the number of taps as a constant.
template <typename F>
static hipError_t conv_taps(int W, F f) {
    if (W == 2) return f(std::integral_constant<int, 2>{});
    if (W == 3) return f(std::integral_constant<int, 3>{});
    return f(std::integral_constant<int, 4>{});
}

template <typename T>
static hipError_t conv_fwd(const ConvProblem& p, hipStream_t s) {
    return conv_taps(p.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value, TL = 6;
        const int tiles = (int)(((long)p.tokens + 4 * TL - 1) / (4 * TL));
        const int cblocks = (p.D + 64 * V - 1) / (64 * V);
        const long groups = (long)cblocks * (tiles + (p.windowT ? (p.N + 3) / 4 : 0));
        if (groups == 0) return hipSuccess;
        constexpr long kMost = 1 << 23;   // work-groups along x
        const dim3 grid((unsigned)(groups < kMost ? groups : kMost), (unsigned)((groups + kMost - 1) / kMost)), block(256);
        if (p.silu) return launch(conv_fwd_kernel<T, W, TL, true>, grid, block, s, p, cblocks, tiles);
        return launch(conv_fwd_kernel<T, W, TL, false>, grid, block, s, p, cblocks, tiles);
    });
}

hipError_t launch_conv_fwd(const ConvProblem& p, hipStream_t s) {
    return p.bf16 ? conv_fwd<uint16_t>(p, s) : conv_fwd<float>(p, s);
}

// Tokens of a run of the backward pass: as many waves as the device holds at once (three a SIMD, in fp32 two), whole blocks less W - 1, four
// blocks at least (so that few tokens still spread). Up to some 110 tokens are four runs of up to eight blocks: one partial row, which nobody has to
// sum (100 tokens 18.7 and 16.4 us a call; 230 would take 18.5 and 24).
static int conv_run(int tokens, int D, int W, int bf16) {
    const long cblocks = (D + 64 * V - 1) / (64 * V), most = 4L * kMaxParts;   // at most kMaxParts rows of four runs
    long waves = ((bf16 ? 3 : 2) * 1024L + cblocks - 1) / cblocks;
    waves = waves < most ? waves : most;
    const long len = (tokens + waves - 1) / waves, blocks = (len + W - 1 + kConvBlock - 1) / kConvBlock;
    const long each = ((tokens + 3) / 4 + W - 1 + kConvBlock - 1) / kConvBlock, least = each <= 8 ? each : 4;
    return (int)((blocks > least ? blocks : least) * kConvBlock - (W - 1));
}
static int conv_rows(int tokens, int run) { return (int)(((long)tokens + 4L * run - 1) / (4L * run)); }
// Rows of partial sums of the backward pass (of bf16 calls; fp32 ones have no more).
int conv_parts(int tokens, int D, int W) { return conv_rows(tokens, conv_run(tokens, D, W, 1)); }

template <typename T, int W, bool SILU>
static hipError_t conv_bwd(const ConvProblem& p, hipStream_t s) {
    const bool dw = p.dweight || p.dbias;
    const int run = conv_run(p.tokens, p.D, W, p.bf16), parts = conv_rows(p.tokens, run), cblocks = (p.D + 64 * V - 1) / (64 * V);
    const long groups = (long)cblocks * (parts + (p.dwindow0 ? (p.N + 3) / 4 : 0));
    if (groups > 0) {
        const dim3 grid((unsigned)groups), block(256);
        const hipError_t e = dw ? launch(conv_bwd_kernel<T, W, SILU, true>, grid, block, s, p, cblocks, parts, run)
                                : launch(conv_bwd_kernel<T, W, SILU, false>, grid, block, s, p, cblocks, parts, run);
        if (e != hipSuccess) return e;
    }
    if (!dw || parts == 1) return hipSuccess;
    return launch_column_sum(p.partial, parts, (long)p.D * W, p.D, p.dweight, p.dbias, s);
}

hipError_t launch_conv_bwd(const ConvProblem& p, hipStream_t s) {
    return conv_taps(p.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value;
        if (p.bf16) return p.silu ? conv_bwd<uint16_t, W, true>(p, s) : conv_bwd<uint16_t, W, false>(p, s);
        return p.silu ? conv_bwd<float, W, true>(p, s) : conv_bwd<float, W, false>(p, s);
    });
}

template <typename T>
static hipError_t conv_update(const ConvProblem& p, hipStream_t s) {
    return conv_taps(p.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value;
        const int cblocks = (p.D + 256 * V - 1) / (256 * V);
        return launch(conv_update_kernel<T, W>, dim3((unsigned)((long)p.N * cblocks)), dim3(256), s, p, cblocks);
    });
}

hipError_t launch_conv_update(const ConvProblem& p, hipStream_t s) {
    if (p.N == 0 || p.tokens == 0) return hipSuccess;
    return p.bf16 ? conv_update<uint16_t>(p, s) : conv_update<float>(p, s);
}

}  // namespace gdn
