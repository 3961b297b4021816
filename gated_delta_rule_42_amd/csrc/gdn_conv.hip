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

template <typename T, int V> struct RawOf;
template <typename T> struct RawOf<T, 8> { using type = Raw8<T>; };
template <typename T> struct RawOf<T, 4> { using type = Raw4<T>; };
template <bool NT, typename T> __device__ __forceinline__ void store_v(T* p, const float (&x)[8]) { store8<NT>(p, x); }
template <bool NT, typename T> __device__ __forceinline__ void store_v(T* p, const float (&x)[4]) { store4c<NT>(p, x); }

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
        const Token k = locate_token(p, lane < count && t0 + lane < p.tokens ? (int)(t0 + lane) : -1);
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
template <int V, int W>
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

__device__ __forceinline__ float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// Row r of sequence n's window (zeros without one).
template <typename T, int V, int W>
__device__ __forceinline__ void window_row(const ConvProblem& p, const void* window, int n, int r, long c, float (&x)[V]) {
    typename RawOf<T, V>::type raw;
    raw.zero();
    if (window) raw.load(static_cast<const T*>(window) + ((long)n * (W - 1) + r) * p.D + c);
    raw.get(x);
}

// The last W - 1 inputs of sequence n, as they lie in memory.
template <typename T, int V, int W>
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
        typename RawOf<T, V>::type raw;
        raw.zero();
        if (pos >= 0) raw.load(static_cast<const T*>(p.x) + (long)(b + pos) * p.x_row + c);
        else if (p.window0) raw.load(static_cast<const T*>(p.window0) + ((long)n * (W - 1) + r + len) * p.D + c);
        raw.put(static_cast<T*>(p.windowT) + ((long)n * (W - 1) + r) * p.D + c);
    }
}

// Work-groups in rows of cblocks, which share tokens; those past the `tiles` rows of tiles leave the windows, a wave per sequence.
template <typename T, int V, int W, int TL, bool NT>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvProblem p, int cblocks, int tiles) {
    using Raw = typename RawOf<T, V>::type;
    __shared__ int seq[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int by = (int)(blockIdx.x / (unsigned)cblocks), bx = (int)(blockIdx.x - (unsigned)by * (unsigned)cblocks);
    const long c = ((long)bx * 64 + lane) * V;
    const bool in = c < p.D;
    if (by >= tiles) {
        const int n = (by - tiles) * 4 + wave;
        if (n < p.N && in) leave_window<T, V, W>(p, n, c);
        return;
    }
    const long first = ((long)by * 4 + wave) * TL;
    if (first >= p.tokens) return;
    const int t0 = (int)first;
    const TileTokens<W> tok(p, t0, TL, seq[wave]);
    if (!in) return;
    Raw raw[TL + W - 1];
#pragma unroll
    for (int i = 0; i < TL + W - 1; ++i) {
        const int t = t0 - (W - 1) + i;
        raw[i].zero();
        if (t >= 0 && t < p.tokens) raw[i].load(static_cast<const T*>(p.x) + t * p.x_row + c);
    }
    float w[V][W], b[V];
    load_taps<V, W>(p.weight, c, w);
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = p.bias ? p.bias[c + v] : 0.f;
    float u[W][V];   // u[k]: the input k tokens back
#pragma unroll
    for (int k = 1; k < W; ++k) {
        if (tok.is(tok.covered, 0) && tok.pos0 < k) window_row<T, V, W>(p, p.window0, tok.seq[0], W - 1 - k + tok.pos0, c, u[k]);
        else raw[W - 1 - k].get(u[k]);
    }
#pragma unroll
    for (int i = 0; i < TL; ++i) {
        raw[i + W - 1].get(u[0]);
        if (tok.is(tok.covered, i)) {
            if (i > 0 && tok.is(tok.starts, i)) {
#pragma unroll
                for (int j = 1; j < W; ++j) window_row<T, V, W>(p, p.window0, tok.seq[i], W - 1 - j, c, u[j]);
            }
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float z = b[v];
#pragma unroll
                for (int j = W - 1; j >= 0; --j) z += w[v][W - 1 - j] * u[j][v];
                y[v] = p.silu ? z * sigmoid_f(z) : z;
            }
            store_v<NT>(static_cast<T*>(p.y) + (long)(t0 + i) * p.D + c, y);
        }
#pragma unroll
        for (int j = W - 1; j > 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) u[j][v] = u[j - 1][v];
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
    float w[4][W], g[W - 1][4], u[2 * W - 2][4];
    load_taps<4, W>(p.weight, c, w);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        window_row<T, 4, W>(p, p.window0, n, r, c, u[r]);
        Raw4<T> raw;
        raw.zero();
        if (r < len) raw.load(static_cast<const T*>(p.x) + (long)(b0 + r) * p.x_row + c);
        raw.get(u[W - 1 + r]);
#pragma unroll
        for (int v = 0; v < 4; ++v) g[r][v] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        if (t < len) {
            Raw4<T> raw;
            float dz[4];
            raw.load(static_cast<const T*>(p.dy) + (long)(b0 + t) * p.D + c);
            raw.get(dz);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                if (p.silu) {
                    float z = p.bias ? p.bias[c + v] : 0.f;
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
            float d[4];
            window_row<T, 4, W>(p, p.dwindowT, n, r - len, c, d);
#pragma unroll
            for (int v = 0; v < 4; ++v) g[r][v] += d[v];
        }
        store4c<false>(static_cast<T*>(p.dwindow0) + ((long)n * (W - 1) + r) * p.D + c, g[r]);
    }
}

constexpr int kConvBwdTokens = 16;   // tokens of a wave's tile

// Rows of work-groups below `parts` walk the rows of tiles with that stride, sum their contributions to dw and db in
// registers, then over their four waves in LDS, and write a partial row each [D, W], [D]; those past them take the
// windows' gradients. No atomics: the same inputs give the same bits.
template <typename T, int W, bool DW, bool NT>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvProblem p, int cblocks, int parts) {
    constexpr int TL = kConvBwdTokens, ROWS = TL + W - 1;
    __shared__ float part[DW ? 4 : 1][DW ? 64 * 4 * (W + 1) : 1];
    __shared__ int seq[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int by = (int)(blockIdx.x / (unsigned)cblocks), bx = (int)(blockIdx.x - (unsigned)by * (unsigned)cblocks);
    const long c = ((long)bx * 64 + lane) * 4;
    const bool in = c < p.D;
    if (by >= parts) {
        const int n = (by - parts) * 4 + wave;
        if (n < p.N && in) window_gradient<T, W>(p, n, c);
        return;
    }
    float w[4][W], b[4], dw[4][W], db[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        b[v] = db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) w[v][j] = dw[v][j] = 0.f;
    }
    if (in) {
        load_taps<4, W>(p.weight, c, w);
        if (p.bias)
#pragma unroll
            for (int v = 0; v < 4; ++v) b[v] = p.bias[c + v];
    }
    const long ntiles = ((long)p.tokens + TL - 1) / TL;
    for (long tile = (long)by * 4 + wave; tile < ntiles; tile += (long)parts * 4) {
        const int t0 = (int)(tile * TL);
        const TileTokens<W> tok(p, t0, ROWS, seq[wave]);
        if (!in) continue;
        Raw4<T> xr[ROWS + W - 1], gr[ROWS];   // xr: tokens t0 - (W - 1) .., gr: tokens t0 ..
#pragma unroll
        for (int i = 0; i < ROWS + W - 1; ++i) {
            const long t = (long)t0 - (W - 1) + i;
            xr[i].zero();
            if (t >= 0 && t < p.tokens) xr[i].load(static_cast<const T*>(p.x) + t * p.x_row + c);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long t = (long)t0 + i;
            gr[i].zero();
            if (t < p.tokens) gr[i].load(static_cast<const T*>(p.dy) + t * p.D + c);
        }
        float u[W][4], dz[W][4];   // u[k]: the input k tokens back; dz[k]: k tokens back
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int v = 0; v < 4; ++v) dz[k][v] = 0.f;
#pragma unroll
        for (int k = 1; k < W; ++k) {
            if (tok.is(tok.covered, 0) && tok.pos0 < k) window_row<T, 4, W>(p, p.window0, tok.seq[0], W - 1 - k + tok.pos0, c, u[k]);
            else xr[W - 1 - k].get(u[k]);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
#pragma unroll
            for (int j = W - 1; j > 0; --j)
#pragma unroll
                for (int v = 0; v < 4; ++v) dz[j][v] = dz[j - 1][v];
            xr[i + W - 1].get(u[0]);
            // a token behind the tile matters only where the tile's last one belongs to the same sequence
            if (tok.is(tok.covered, i) && (i < TL || !(tok.starts >> TL & ((2ull << (i - TL)) - 1)))) {
                if (i > 0 && tok.is(tok.starts, i)) {
#pragma unroll
                    for (int j = 1; j < W; ++j) window_row<T, 4, W>(p, p.window0, tok.seq[i], W - 1 - j, c, u[j]);
                }
                gr[i].get(dz[0]);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if (p.silu) {
                        float z = b[v];
#pragma unroll
                        for (int j = W - 1; j >= 0; --j) z += w[v][W - 1 - j] * u[j][v];
                        const float s = sigmoid_f(z);
                        dz[0][v] *= s * (1.f + z * (1.f - s));
                    }
                    if (DW && i < TL) {
                        db[v] += dz[0][v];
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[v][W - 1 - j] += dz[0][v] * u[j][v];
                    }
                }
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) dz[0][v] = 0.f;
            }
            if (i >= W - 1) {   // the token W - 1 back has all of its terms: dz[W - 1] is its own, dz[W - 1 - m] that m tokens on
                const int o = i - (W - 1);
                if (tok.is(tok.covered, o)) {
                    float dx[4];
                    int rem = W;   // tokens of its sequence from it on, W for that or more
#pragma unroll
                    for (int r = 0; r < W - 1; ++r)
                        if (tok.is(tok.ends[r], o)) rem = r + 1;
#pragma unroll
                    for (int v = 0; v < 4; ++v) dx[v] = w[v][W - 1] * dz[W - 1][v];
#pragma unroll
                    for (int m = 1; m < W; ++m)
                        if (m < rem)
#pragma unroll
                            for (int v = 0; v < 4; ++v) dx[v] += w[v][W - 1 - m] * dz[W - 1 - m][v];
                    if (p.dwindowT && rem < W) {
                        float d[4];
                        window_row<T, 4, W>(p, p.dwindowT, tok.seq[o], W - 1 - rem, c, d);
#pragma unroll
                        for (int v = 0; v < 4; ++v) dx[v] += d[v];
                    }
                    store4c<NT>(static_cast<T*>(p.dx) + (long)(t0 + i - (W - 1)) * p.dx_row + c, dx);
                }
            }
#pragma unroll
            for (int j = W - 1; j > 0; --j)
#pragma unroll
                for (int v = 0; v < 4; ++v) u[j][v] = u[j - 1][v];
        }
    }
    if constexpr (DW) {
        float* mine = part[wave] + lane * 4 * (W + 1);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) mine[v * (W + 1) + j] = dw[v][j];
            mine[v * (W + 1) + W] = db[v];
        }
        __syncthreads();
        float* row = p.partial + (long)by * p.D * (W + 1);
        for (int i = threadIdx.x; i < 256 * (W + 1); i += 256) {
            const int ch = i / (W + 1), j = i % (W + 1);
            const long cc = (long)bx * 256 + ch;
            if (cc < p.D) {
                const float a = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
                row[j < W ? cc * W + j : (long)p.D * W + cc] = a;
            }
        }
    }
}

// Runs of tokens on a pool of windows: a lane walks its sequence's tokens for V channels. The window stays as loaded, so its rows
// are moved, never rounded. Tokens come four at a time.
template <typename T, int V, int W>
__global__ __launch_bounds__(256) void conv_update_kernel(ConvProblem p, int cblocks) {
    using Raw = typename RawOf<T, V>::type;
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
        for (int t = t0; t < t1; ++t) store_v<false>(yp + (long)t * p.D, y);
        return;
    }
    T* pool = static_cast<T*>(p.pool) + c;
    const long slot_size = (long)(W - 1) * p.D;
    Raw u[W];   // u[k]: the input k tokens back
#pragma unroll
    for (int k = 1; k < W; ++k) u[k].load(pool + slot * slot_size + (long)(W - 1 - k) * p.D);
    float w[V][W], b[V];
    load_taps<V, W>(p.weight, c, w);
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = p.bias ? p.bias[c + v] : 0.f;
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
                store_v<false>(yp + (long)t * p.D, y);
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

template <typename T, int V>
static hipError_t conv_fwd(const ConvProblem& p, hipStream_t s) {
    return conv_taps(p.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value, TL = 16;
        const int tiles = (int)(((long)p.tokens + 4 * TL - 1) / (4 * TL));
        const int cblocks = (p.D + 64 * V - 1) / (64 * V);
        const long groups = (long)cblocks * (tiles + (p.windowT ? (p.N + 3) / 4 : 0));
        if (groups == 0) return hipSuccess;
        return launch(conv_fwd_kernel<T, V, W, TL, false>, dim3((unsigned)groups), dim3(256), s, p, cblocks, tiles);
    });
}

hipError_t launch_conv_fwd(const ConvProblem& p, hipStream_t s) {
    return p.bf16 ? conv_fwd<uint16_t, 8>(p, s) : conv_fwd<float, 4>(p, s);
}

// Rows of work-groups (and partial rows) of the backward pass: enough to fill the device, but no more than there are rows
// of tiles.
int conv_parts(int tokens, int D) {
    const long rows = ((long)tokens + 4 * kConvBwdTokens - 1) / (4 * kConvBwdTokens);
    const long cblocks = (D + 255) / 256, want = (768 + cblocks - 1) / cblocks;
    const long cap = rows < want ? rows : want;
    return (int)(cap < kMaxParts ? cap : kMaxParts);
}

template <typename T>
static hipError_t conv_bwd(const ConvProblem& p, hipStream_t s) {
    return conv_taps(p.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value;
        const bool dw = p.dweight || p.dbias;
        const int parts = conv_parts(p.tokens, p.D);
        const int cblocks = (p.D + 255) / 256;
        const long groups = (long)cblocks * (parts + (p.dwindow0 ? (p.N + 3) / 4 : 0));
        if (groups > 0) {
            const dim3 grid((unsigned)groups);
            const hipError_t e = dw ? launch(conv_bwd_kernel<T, W, true, false>, grid, dim3(256), s, p, cblocks, parts)
                                    : launch(conv_bwd_kernel<T, W, false, false>, grid, dim3(256), s, p, cblocks, parts);
            if (e != hipSuccess) return e;
        }
        if (!dw) return hipSuccess;
        return launch_column_sum(p.partial, parts, (long)p.D * W, p.D, p.dweight, p.dbias, s);
    });
}

hipError_t launch_conv_bwd(const ConvProblem& p, hipStream_t s) { return p.bf16 ? conv_bwd<uint16_t>(p, s) : conv_bwd<float>(p, s); }

template <typename T, int V>
static hipError_t conv_update(const ConvProblem& p, hipStream_t s) {
    return conv_taps(p.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value;
        const int cblocks = (p.D + 256 * V - 1) / (256 * V);
        return launch(conv_update_kernel<T, V, W>, dim3((unsigned)((long)p.N * cblocks)), dim3(256), s, p, cblocks);
    });
}

hipError_t launch_conv_update(const ConvProblem& p, hipStream_t s) {
    if (p.N == 0 || p.tokens == 0) return hipSuccess;
    return p.bf16 ? conv_update<uint16_t, 8>(p, s) : conv_update<float, 4>(p, s);
}

}  // namespace gdn
