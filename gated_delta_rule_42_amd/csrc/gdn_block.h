// Host-side descriptors of the operators of a recurrent block around the rule: layer norm, short causal convolution,
// gated linear recurrence. Shared by the C ABI layer and their kernel sources.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// out0[c] (c < n0) and out1[c - n0] (n0 <= c < n0 + n1) = the sum over `nparts` rows of partial [nparts, n0 + n1], in a fixed
// order (either output may be NULL). nparts <= kMaxParts.
constexpr int kMaxParts = 1024;
hipError_t launch_column_sum(const float* partial, int nparts, long n0, long n1, float* out0, float* out1, hipStream_t s);

// Layer norm (gdn_layernorm.hip). Strides in elements between rows; a row's channels are contiguous.
struct LayerNormProblem {
    const void* x;               // forward: [rows, d]; backward: the normalised sum, [rows, d]
    const void* residual;        // forward: [rows, d] or NULL
    const float* weight;         // [d] or NULL (ones)
    const float* bias;           // [d] or NULL (zeros)
    void* y;                     // forward: [rows, d], dense
    void* sum;                   // forward: the sum as it is normalised, [rows, d], dense (with residual)
    const void* dy;              // backward: [rows, d], dense
    const void* dsum;            // backward: [rows, d], dense, or NULL
    void* dx;                    // backward: [rows, d], dense
    float* dweight;              // backward: [d] or NULL
    float* dbias;
    float* partial;              // backward with dweight or dbias: [layer_norm_parts, 2, d]
    long rows, x_row, r_row;
    int d;
    int x_bf16, s_bf16, y_bf16;  // types of x, of the sum, of y (and dy)
    float eps;
};
int layer_norm_parts(long rows, int d);
hipError_t launch_layer_norm_fwd(const LayerNormProblem& p, hipStream_t s);
hipError_t launch_layer_norm_bwd(const LayerNormProblem& p, hipStream_t s);

// Short causal convolution per channel (gdn_conv.hip). x, y, the windows and their gradients are of one type.
struct ConvProblem {
    const void* x;               // [tokens, D], token stride x_row
    const float* weight;         // [D, W]
    const float* bias;           // [D] or NULL
    const void* window0;         // [N, W - 1, D] the inputs before each sequence, or NULL (zeros)
    const int32_t* cu_seqlens;   // [N + 1], or NULL: N sequences of T tokens
    void* y;                     // forward: [tokens, D], dense
    void* windowT;               // forward: [N, W - 1, D] the last inputs of each sequence, or NULL
    const void* dy;              // backward: [tokens, D], dense
    const void* dwindowT;        // backward: [N, W - 1, D] or NULL
    void* dx;                    // backward: [tokens, D], token stride dx_row
    void* dwindow0;              // backward: [N, W - 1, D] or NULL
    float* dweight;              // backward: [D, W] or NULL
    float* dbias;                // backward: [D] or NULL
    float* partial;              // backward with dweight or dbias: [conv_parts, D * (W + 1)]
    void* pool;                  // runs on a pool: [n_slots, W - 1, D]
    const int32_t* slots;        // [N]
    const int32_t* out_slots;    // [tokens] or NULL
    long x_row, dx_row;
    int tokens, T, N, D, W, n_slots;
    int bf16, silu;
};
int conv_parts(int tokens, int D, int W);
hipError_t launch_conv_fwd(const ConvProblem& p, hipStream_t s);
hipError_t launch_conv_bwd(const ConvProblem& p, hipStream_t s);
hipError_t launch_conv_update(const ConvProblem& p, hipStream_t s);

// Gated linear recurrence per channel (gdn_scan.hip). A sequence is cut into tiles of `tile` tokens (one tile at least); row r of
// the tiles is tile s of sequence n, r = base[n] + s.
constexpr int kScanChannels = 64;
struct ScanProblem {
    const void* x;               // [tokens, D], token stride x_row
    const float* g;              // [tokens, D], dense
    const float* h0;             // [N, D] or NULL (zeros)
    const int32_t* cu_seqlens;   // [N + 1], or NULL: N sequences of T tokens
    void* h;                     // forward: [tokens, D], dense
    float* hT;                   // forward: [N, D] or NULL
    float* carries;              // [rows, D], the state entering each tile: forward NULL or written, backward read
    const void* dh;              // backward: [tokens, D], dense
    const float* dhT;            // backward: [N, D] or NULL
    void* dx;                    // backward: [tokens, D], dense
    float* dg;                   // backward: [tokens, D], dense
    float* dh0;                  // backward: [N, D] or NULL
    float* pool;                 // runs on a pool: [n_slots, D]
    const int32_t* slots;        // [N]
    const int32_t* out_slots;    // [tokens] or NULL
    // workspace, where tiles pass states on between work-groups (else ticket NULL)
    int32_t* ticket;
    int32_t* base;               // [N + 1] first tile of each sequence (cu_seqlens only)
    uint64_t* agg;               // [rows, 64 ncb] a tile's map of what enters it to what leaves it
    float* pref;                 // [rows, 64 ncb] what leaves a tile
    long x_row, rows;            // rows: an upper bound with cu_seqlens
    int tokens, T, N, D, ncb, tile, n_slots;
    int bf16, h_bf16, blend;     // types of x (and dx), of h (and dh)
};
// Tokens of a tile, rows of tiles (an upper bound with cu_seqlens), and the workspace of a scan.
struct ScanLayout {
    int tile;
    long rows, carry_rows;
    size_t off_base, off_agg, off_pref, total;   // total 0: a work-group walks a sequence's tiles, no workspace
};
ScanLayout scan_layout(int tokens, int T, int N, int D, int varlen);
hipError_t launch_scan_fwd(const ScanProblem& p, hipStream_t s);
hipError_t launch_scan_bwd(const ScanProblem& p, hipStream_t s);
hipError_t launch_scan_update(const ScanProblem& p, hipStream_t s);

}  // namespace gdn
