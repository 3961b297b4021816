// Layer norm with the residual sum in the same pass, and its gradients, for gfx950.
//
// Per row of d channels:
//     s = x + r, rounded to the sum's type (or x alone),   m = sum s / d,   v = sum (s - m)^2 / d,
//     xh = (s - m) (v + eps)^(-1/2),   y = w xh + b.
// Backward, with g = w dy and rs = (v + eps)^(-1/2):
//     dx = rs (g - sum g / d - xh sum(g xh) / d) + ds,   dw = sum over rows of dy xh,   db = sum over rows of dy.
// The backward pass has to read s anyway and computes m and v from it again, so nothing but s is kept between the two.
// Both directions are bound by bytes: each row is loaded once, held in registers and written once. Sums are fp32, the variance
// that of the centred values.
//
// A row takes L lanes with P pieces of 8 channels each (channels 8 (lane + L j) + 0..7), so every load and store is
// 16 bytes wide and neighbouring lanes cover whole cache lines. L is 16, 32 or 64 lanes of one wave, whose sums are
// exchanges between lanes, or, for rows past 2048 channels, four or eight waves, which join their sums in LDS.
#include <type_traits>

#include "gdn_block.h"
#include "gdn_row.h"

namespace gdn {

// Sums over the L lanes of a row, of two values at a time. red: two buffers that turn, so that one barrier per sum is enough.
template <int L>
struct RowSums {
    static constexpr int W = L / 64;                     // waves of a row (0: part of one)
    static constexpr int RED = W > 1 ? 2 * 2 * W : 1;    // floats per row group
    float* red;
    int turn = 0;
    __device__ __forceinline__ RowSums(float* r) : red(r) {}
    __device__ __forceinline__ void sum2(float& a, float& b) {
        a = row_sum<(L > 64 ? 64 : L)>(a);
        b = row_sum<(L > 64 ? 64 : L)>(b);
        if constexpr (W > 1) {
            const int wave = (threadIdx.x >> 6) % W;
            float* r = red + 2 * W * turn;
            if ((threadIdx.x & 63) == 0) {
                r[wave] = a;
                r[W + wave] = b;
            }
            __syncthreads();
            a = b = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                a += r[w];
                b += r[W + w];
            }
            turn ^= 1;
        }
    }
    __device__ __forceinline__ float sum(float a) {
        float z = 0.f;
        sum2(a, z);
        return a;
    }
};

// Threads of a forward work-group: four waves, or a row's eight.
constexpr int ln_fwd_threads(int L) { return L > 256 ? L : 256; }

// A row's pieces are in flight together and nothing else is in the way: 8192 x 2048 in bf16 with the residual 23 us, 5.8 TB/s. Weights come from the
// caches once a row (in registers across rows 32768 x 2048 took 100 to 114 us instead of 95).
template <typename TX, typename TS, typename TY, int L, int P>
__global__ __launch_bounds__(ln_fwd_threads(L)) void layer_norm_fwd_kernel(LayerNormProblem p) {
    __shared__ float red[RowSums<L>::RED];
    RowSums<L> rs(red);
    const int l = threadIdx.x % L;
    const long row = ((long)blockIdx.y * gridDim.x + blockIdx.x) * (ln_fwd_threads(L) / L) + threadIdx.x / L;   // y: past 2^32 threads
    const bool ok = row < p.rows;
    const TX* xp = static_cast<const TX*>(p.x) + row * p.x_row;
    const TS* rp = static_cast<const TS*>(p.residual) + row * p.r_row;
    Raw8<TX> xr[P];
    Raw8<TS> rr[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int c = 8 * (l + L * j);
        xr[j].zero();
        if (ok && c < p.d) xr[j].load(xp + c);
    }
    if (p.residual) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int c = 8 * (l + L * j);
            rr[j].zero();
            if (ok && c < p.d) rr[j].load(rp + c);
        }
    }
    float v[P][8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int c = 8 * (l + L * j);
        xr[j].get(v[j]);
        if (p.residual) {
            float t[8];
            rr[j].get(t);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = to_f32(from_f32<TS>(v[j][e] + t[e]));
            if (ok && c < p.d) store8<false>(static_cast<TS*>(p.sum) + row * p.d + c, v[j]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += v[j][e];
    }
    const float inv_d = 1.f / p.d, mean = rs.sum(sum) * inv_d;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const bool in = 8 * (l + L * j) < p.d;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[j][e] = in ? v[j][e] - mean : 0.f;
            sq += v[j][e] * v[j][e];
        }
    }
    const float r = 1.f / sqrtf(rs.sum(sq) * inv_d + p.eps);
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int c = 8 * (l + L * j);
        if (ok && c < p.d) {
            float w[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 1.f, b[e] = 0.f;
            Raw8<float> wr;
            if (p.weight) {
                wr.load(p.weight + c);
                wr.get(w);
            }
            if (p.bias) {
                wr.load(p.bias + c);
                wr.get(b);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * r * w[e] + b[e];
            store8<false>(static_cast<TY*>(p.y) + row * p.d + c, v[j]);
        }
    }
}

constexpr int kLnBwdThreads = 512;   // eight waves

// Rows stay as loaded and are unpacked again for each of the three passes over them (two sums each, then the outputs), which leaves room
// for a lane's weights and sums in registers. Weights read again for every row and pass went through the vector cache at more bytes than the
// rows themselves: 8192 x 2048 38.8 us a call, 32.6 with them in registers.
// AHEAD: the next row is loaded while the current one is worked on, where the registers allow. Rows of several waves wait at barriers and gain most
// (bf16: 4096 x 4096 39 -> 34 us, 2048 x 8192 41 -> 38; fp32: 4096 x 4096 57 -> 53); of the work-groups with eight rows and more only those with
// short rows of bf16 gain (262144 x 64 47 -> 42, 32768 x 512 31 -> 29; 8192 x 2048 31.4 and 32.2, fp32 262144 x 64 49 and 52).
// DW: the gradients of weight and bias too. The grid is then layer_norm_parts work-groups, each of which walks its rows with a
// fixed stride, sums their contributions in registers, then over its row groups in LDS, and writes one partial row
// [2, d] (weight, bias). No atomics: the same inputs give the same bits.
template <typename TS, typename TY, int L, int P, bool DW>
__global__ __launch_bounds__(kLnBwdThreads) void layer_norm_bwd_kernel(LayerNormProblem p) {
    constexpr int RG = kLnBwdThreads / L;
    constexpr bool AHEAD = DW && (L > 64 ? P * (2 * sizeof(TS) + sizeof(TY)) <= 24 : P <= 2 && sizeof(TS) + sizeof(TY) < 8);
    __shared__ float red[RG * RowSums<L>::RED];
    __shared__ float part[DW ? RG * 2 * 8 * L : 1];
    const int l = threadIdx.x % L, grp = threadIdx.x / L;
    RowSums<L> rs(red + grp * RowSums<L>::RED);
    const float inv_d = 1.f / p.d;
    float aw[DW ? P : 1][8], ab[DW ? P : 1][8];
    if constexpr (DW) {
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) aw[j][e] = ab[j][e] = 0.f;
    }
    float w[P][8];
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[j][e] = 1.f;
    if (p.weight) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int c = 8 * (l + L * j);
            Raw8<float> r;
            r.load(p.weight + (c < p.d ? c : 0));
            r.get(w[j]);
        }
    }
    Raw8<TS> xn[AHEAD ? P : 1], tn[AHEAD ? P : 1];
    Raw8<TY> gn[AHEAD ? P : 1];
    // rows and channels past the end load the last row, the first channels, and are put out of action below
    auto load = [&](long row, Raw8<TS> (&x)[P], Raw8<TY> (&g)[P], Raw8<TS> (&t)[P]) {
        const long rl = min(row, p.rows - 1);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int c = 8 * (l + L * j), cl = c < p.d ? c : 0;
            x[j].load(static_cast<const TS*>(p.x) + rl * p.x_row + cl);
            g[j].load(static_cast<const TY*>(p.dy) + rl * p.d + cl);
            t[j].zero();
        }
        if (p.dsum) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int c = 8 * (l + L * j), cl = c < p.d ? c : 0;
                t[j].load(static_cast<const TS*>(p.dsum) + rl * p.d + cl);
            }
        }
    };
    if constexpr (AHEAD) load((long)blockIdx.x * RG + grp, xn, gn, tn);
    for (long row0 = (long)blockIdx.x * RG; row0 < p.rows; row0 += (long)gridDim.x * RG) {
        const long row = row0 + grp;
        const bool ok = row < p.rows;
        Raw8<TS> xr[P], tr[P];
        Raw8<TY> gr[P];
        if constexpr (AHEAD) {
#pragma unroll
            for (int j = 0; j < P; ++j) xr[j] = xn[j], gr[j] = gn[j], tr[j] = tn[j];
            if (row0 + (long)gridDim.x * RG < p.rows) load(row + (long)gridDim.x * RG, xn, gn, tn);
        } else {
            load(row, xr, gr, tr);
        }
        float sum = 0.f, gsum = 0.f;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int c = 8 * (l + L * j);
            float x[8], g[8];
            xr[j].get(x);
            gr[j].get(g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum += c < p.d ? x[e] : 0.f;
                gsum += c < p.d ? g[e] * w[j][e] : 0.f;
            }
            xr[j].hide();
            gr[j].hide();
        }
        rs.sum2(sum, gsum);
        const float mean = sum * inv_d, gm = gsum * inv_d;
        float sq = 0.f, gx = 0.f;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int c = 8 * (l + L * j);
            float x[8], g[8];
            xr[j].get(x);
            gr[j].get(g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = c < p.d ? x[e] - mean : 0.f;
                sq += v * v;
                gx += c < p.d ? g[e] * w[j][e] * v : 0.f;
            }
            xr[j].hide();
            gr[j].hide();
        }
        rs.sum2(sq, gx);
        const float r = 1.f / sqrtf(sq * inv_d + p.eps), k = gx * r * inv_d;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int c = 8 * (l + L * j);
            float x[8], g[8], t[8];
            xr[j].get(x);
            gr[j].get(g);
            tr[j].get(t);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (x[e] - mean) * r;
                if constexpr (DW) {
                    aw[j][e] += ok ? g[e] * xh : 0.f;
                    ab[j][e] += ok ? g[e] : 0.f;
                }
                t[e] += r * (g[e] * w[j][e] - gm - xh * k);
            }
            if (ok && c < p.d) store8<false>(static_cast<TS*>(p.dx) + row * p.d + c, t);
        }
    }
    if constexpr (DW) {
        // piece by piece: the row groups' sums side by side in LDS, then added in their order
#pragma unroll
        for (int j = 0; j < P; ++j) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                part[(grp * 2 + 0) * 8 * L + 8 * l + e] = aw[j][e];
                part[(grp * 2 + 1) * 8 * L + 8 * l + e] = ab[j][e];
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * 8 * L; i += kLnBwdThreads) {
                const int which = i / (8 * L), c = i % (8 * L);
                float a = 0.f;
#pragma unroll
                for (int q = 0; q < RG; ++q) a += part[(q * 2 + which) * 8 * L + c];
                // a single work-group's sums are the gradients
                float* out = gridDim.x > 1 ? p.partial + ((long)blockIdx.x * 2 + which) * p.d : which ? p.dbias : p.dweight;
                if (out && 8 * L * j + c < p.d) out[8 * L * j + c] = a;
            }
        }
    }
}

// A work-group per C columns: C lanes across them and 1024 / C down the rows, joined in LDS. Few columns take 16, for more work-groups
// (4096 columns of 256 rows 4.0 us), many take 64, for whole cache lines.
template <int C>
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* partial, int nparts, long n0, long n1, float* out0, float* out1) {
    constexpr int R = 1024 / C;
    __shared__ float sum[R][C + 1];
    const int lc = threadIdx.x % C, lr = threadIdx.x / C;
    const long n = n0 + n1, c = (long)blockIdx.x * C + lc, at = min(c, n - 1);
    float a = 0.f;
    for (int i0 = lr; i0 < nparts; i0 += 8 * R) {   // eight rows at a time in flight
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = partial[(long)min(i0 + R * j, nparts - 1) * n + at];
#pragma unroll
        for (int j = 0; j < 8; ++j) a += i0 + R * j < nparts ? x[j] : 0.f;
    }
    sum[lr][lc] = a;
    __syncthreads();
#pragma unroll
    for (int m = R / 2; m > 0; m /= 2) {
        if (lr < m) sum[lr][lc] += sum[lr + m][lc];
        __syncthreads();
    }
    if (lr == 0 && c < n) {
        if (c < n0) {
            if (out0) out0[c] = sum[0][lc];
        } else if (out1) {
            out1[c - n0] = sum[0][lc];
        }
    }
}

hipError_t launch_column_sum(const float* partial, int nparts, long n0, long n1, float* out0, float* out1, hipStream_t s) {
    const long n = n0 + n1;
    if (n < 16384) return launch(column_sum_kernel<16>, dim3((unsigned)((n + 15) / 16)), dim3(1024), s, partial, nparts, n0, n1, out0, out1);
    return launch(column_sum_kernel<64>, dim3((unsigned)((n + 63) / 64)), dim3(1024), s, partial, nparts, n0, n1, out0, out1);
}

// Lanes of a row and pieces per lane.
template <typename F>
static hipError_t ln_shape(int d, F f) {
    if (d <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    if (d <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
    if (d <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    if (d <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    if (d <= 2048) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    if (d <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    if (d <= 8192) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{});
}
template <typename TX, typename TS, typename TY>
static hipError_t ln_fwd(const LayerNormProblem& p, hipStream_t s) {
    return ln_shape(p.d, [&](auto lanes, auto pieces) {
        constexpr int L = decltype(lanes)::value, P = decltype(pieces)::value;
        constexpr int NT = ln_fwd_threads(L), RG = NT / L;
        constexpr long kMost = 1 << 22;   // work-groups along x
        const long groups = (p.rows + RG - 1) / RG;
        const dim3 grid((unsigned)(groups < kMost ? groups : kMost), (unsigned)((groups + kMost - 1) / kMost));
        return launch(layer_norm_fwd_kernel<TX, TS, TY, L, P>, grid, dim3(NT), s, p);
    });
}

hipError_t launch_layer_norm_fwd(const LayerNormProblem& p, hipStream_t s) {
    if (p.rows == 0) return hipSuccess;
    if (!p.x_bf16) return p.y_bf16 ? ln_fwd<float, float, uint16_t>(p, s) : ln_fwd<float, float, float>(p, s);
    if (p.s_bf16) return p.y_bf16 ? ln_fwd<uint16_t, uint16_t, uint16_t>(p, s) : ln_fwd<uint16_t, uint16_t, float>(p, s);
    return p.y_bf16 ? ln_fwd<uint16_t, float, uint16_t>(p, s) : ln_fwd<uint16_t, float, float>(p, s);
}

static int ln_lanes(int d) { return d <= 128 ? 16 : d <= 256 ? 32 : d <= 2048 ? 64 : d <= 8192 ? 256 : 512; }

// Work-groups (and partial rows) of the backward pass with gradients of weight and bias: one per CU, but no more than there
// are groups of rows; one for two groups, which saves the launch that sums partial rows.
int layer_norm_parts(long rows, int d) {
    const int rg = kLnBwdThreads / ln_lanes(d);
    const long blocks = (rows + rg - 1) / rg;
    return (int)(blocks == 2 ? 1 : blocks < 256 ? blocks : 256);
}

template <typename TS, typename TY>
static hipError_t ln_bwd(const LayerNormProblem& p, hipStream_t s) {
    return ln_shape(p.d, [&](auto lanes, auto pieces) {
        constexpr int L = decltype(lanes)::value, P = decltype(pieces)::value, RG = kLnBwdThreads / L;
        if (!p.dweight && !p.dbias) {
            if (p.rows == 0) return hipSuccess;
            constexpr long kMost = 1 << 22;   // work-groups, which go on to further rows
            const long groups = (p.rows + RG - 1) / RG;
            return launch(layer_norm_bwd_kernel<TS, TY, L, P, false>, dim3((unsigned)(groups < kMost ? groups : kMost)), dim3(kLnBwdThreads), s, p);
        }
        const int parts = layer_norm_parts(p.rows, p.d);
        if (parts > 0) {
            const hipError_t e = launch(layer_norm_bwd_kernel<TS, TY, L, P, true>, dim3((unsigned)parts), dim3(kLnBwdThreads), s, p);
            if (e != hipSuccess || parts == 1) return e;
        }
        return launch_column_sum(p.partial, parts, p.d, p.d, p.dweight, p.dbias, s);
    });
}

hipError_t launch_layer_norm_bwd(const LayerNormProblem& p, hipStream_t s) {
    if (p.s_bf16) return p.y_bf16 ? ln_bwd<uint16_t, uint16_t>(p, s) : ln_bwd<uint16_t, float>(p, s);
    return p.y_bf16 ? ln_bwd<float, uint16_t>(p, s) : ln_bwd<float, float>(p, s);
}

}  // namespace gdn
