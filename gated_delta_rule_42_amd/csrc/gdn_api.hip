// C ABI of libgdn.so (declared in include/gdn.h): argument checks, workspace layout and
// kernel dispatch. Every check runs before any HIP call, so a rejected call launches
// nothing and touches no device state.
#include "gdn.h"
#include "gdn_internal.h"

#include <cstdlib>
#include <cstring>
#include <mutex>
#include <vector>

#define GDN_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool head_dim_ok(int d) { return d == 64 || d == 128; }

// Size checks shared by the chunked entry points and their workspace queries (after the dtype,
// chunk and head-dimension checks): B, H >= 1, T >= 0, H <= 32768 (one chunk of one head spans
// 64 token rows of H heads, addressed with 32-bit byte offsets inside the kernels), N = B
// without packed sequences and B = 1, N >= 1 with them, at most 2^40 elements in any token
// tensor and at most 2^30 (sequence, head) pairs. Each product is formed only once its factors
// are known to keep it inside 64 bits.
int shape_check(int B, int T, int H, int dk, int dv, int N, bool varlen) {
    if (B < 1 || H < 1 || H > 32768 || T < 0) return GDN_ERR_SHAPE;
    if (varlen ? (B != 1 || N < 1) : (N != B)) return GDN_ERR_SHAPE;
    const long long tokens = (long long)B * T;   // < 2^62
    if (tokens > (1LL << 40) || tokens * H * (dk > dv ? dk : dv) > (1LL << 40)) return GDN_ERR_SHAPE;
    if ((long long)N * H > (1LL << 30)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

// The forward workspace: the stage-1 regions, then the state records of the long-chain split
struct FwdLayout {
    gdn::WorkspaceLayout w;
    gdn::SegPlan seg;
    size_t off_seg, total;
};
FwdLayout fwd_layout(int B, int T, int H, int dk, int dv, int N, int varlen, int bf16) {
    FwdLayout f;
    f.w = gdn::workspace_layout(B, T, H, dk, N, varlen, bf16 ? 2 : 4);
    f.seg = gdn::segment_plan(T, H, dk, dv, N, bf16);
    f.off_seg = (f.w.total + 255) & ~(size_t)255;
    f.total = f.seg.n > 1 ? f.off_seg + f.seg.bytes : f.w.total;
    return f;
}

// GDN_CHECK=1 in the environment: copy cu_seqlens to the host (this synchronises `stream`) and
// reject offsets that break 0 = cu[0] <= cu[1] <= ... <= cu[N] = T. A debugging aid: without it
// the offsets are a precondition that the kernels only clamp into [0, T]. padded: tokens behind the last sequence
// are allowed (cu[N] <= T).
int debug_check_offsets(const int32_t* cu, int N, int T, hipStream_t s, bool padded = false) {
    const char* env = std::getenv("GDN_CHECK");
    if (!cu || !env || std::strcmp(env, "1") != 0) return GDN_OK;
    std::vector<int32_t> h((size_t)N + 1);
    if (hipMemcpyAsync(h.data(), cu, h.size() * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess)
        return GDN_ERR_HIP;
    if (h[0] != 0 || (padded ? h[(size_t)N] > T : h[(size_t)N] != T)) return GDN_ERR_SHAPE;
    for (int i = 0; i < N; ++i)
        if (h[(size_t)i + 1] < h[(size_t)i]) return GDN_ERR_SHAPE;
    return GDN_OK;
}

// Shared checks of the chunked forward entry points. `need` flags: 1 = q,k,g,beta;
// 2 = v,o. Fills the problem description on success.
int check_chunk(const void* q, const void* k, const void* v, const float* g, const float* beta,
                const float* h0, const void* o, const float* hT, const int32_t* cu, int chunk,
                int B, int T, int H, int dk, int dv, int N, int dtype, int o_dtype,
                const void* ws, size_t ws_bytes, int need, gdn::ChunkProblem* p) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (o_dtype != GDN_F32 && !(o_dtype == GDN_BF16 && dtype == GDN_BF16)) return GDN_ERR_DTYPE;
    if (chunk != 64) return GDN_ERR_UNSUPPORTED;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    const int sc = shape_check(B, T, H, dk, dv, N, cu != nullptr);
    if (sc != GDN_OK) return sc;
    const long long tokens = (long long)B * T;
    if (tokens > 0) {
        if ((need & 1) && (!q || !k || !g || !beta)) return GDN_ERR_NULL;
        if ((need & 2) && (!q || !k || !v || !o)) return GDN_ERR_NULL;
    }
    const void* al16[] = {q, k, v, o, h0, hT};
    for (const void* x : al16)
        if (x && !aligned(x, 16)) return GDN_ERR_ALIGN;
    const void* al4[] = {g, beta, cu};
    for (const void* x : al4)
        if (x && !aligned(x, 4)) return GDN_ERR_ALIGN;
    const FwdLayout f = fwd_layout(B, T, H, dk, dv, N, cu != nullptr, dtype == GDN_BF16);
    const gdn::WorkspaceLayout& w = f.w;
    if (w.nc_bound * H > 0x7fffffffL) return GDN_ERR_SHAPE;
    if (f.total > 0 && (!ws || ws_bytes < f.total)) return GDN_ERR_WORKSPACE;
    if (ws && !aligned(ws, 256)) return GDN_ERR_ALIGN;

    gdn::ChunkProblem& P = *p;
    P.q = q; P.k = k; P.v = v; P.g = g; P.beta = beta; P.h0 = h0;
    P.o = const_cast<void*>(o); P.hT = const_cast<float*>(hT); P.cu_seqlens = cu;
    P.B = B; P.T = T; P.H = H; P.dk = dk; P.dv = dv; P.N = N;
    P.bf16 = dtype == GDN_BF16;
    P.o_bf16 = o_dtype == GDN_BF16;
    P.nc_bound = w.nc_bound;
    P.nc_per_seq = (T + 63) / 64;
    char* base = static_cast<char*>(const_cast<void*>(ws));
    P.chunk_base = cu ? reinterpret_cast<int32_t*>(base + w.off_base) : nullptr;
    P.gates = w.nc_bound ? reinterpret_cast<float*>(base + w.off_gates) : nullptr;
    P.mmat = w.nc_bound ? base + w.off_m : nullptr;
    P.pmat = w.nc_bound ? base + w.off_p : nullptr;
    P.k16 = (w.nc_bound && P.bf16) ? reinterpret_cast<_Float16*>(base + w.off_k16) : nullptr;
    P.q16 = (w.nc_bound && P.bf16) ? reinterpret_cast<_Float16*>(base + w.off_q16) : nullptr;
    P.seg_n = f.seg.n;
    P.seg_len = f.seg.len;
    P.seg_ncp = f.seg.ncp;
    P.segst = f.seg.n > 1 ? reinterpret_cast<float*>(base + f.off_seg) : nullptr;
    return GDN_OK;
}

}  // namespace

GDN_EXPORT int gdn_version(void) { return 100; }

GDN_EXPORT const char* gdn_status_string(int status) {
    switch (status) {
        case GDN_OK: return "ok";
        case GDN_ERR_NULL: return "a required pointer is NULL";
        case GDN_ERR_SHAPE: return "a size is out of range or inconsistent";
        case GDN_ERR_DTYPE: return "unknown dtype code";
        case GDN_ERR_ALIGN: return "a pointer or stride is misaligned (q/k/v/o/states 16 B, gates 4 B, workspace 256 B)";
        case GDN_ERR_UNSUPPORTED: return "unsupported chunk size, head dimension, norm or rotation (chunk 64; d_k, d_v in {64, 128})";
        case GDN_ERR_WORKSPACE: return "workspace missing or smaller than the entry point's ..._workspace_bytes()";
        case GDN_ERR_HIP: return "a HIP launch failed";
        default: return "unknown status";
    }
}

GDN_EXPORT size_t gdn_chunk_fwd_workspace_bytes(int B, int T, int H, int dk, int dv, int N,
                                                int varlen, int chunk, int dtype) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return 0;
    if (chunk != 64 || !head_dim_ok(dk) || !head_dim_ok(dv)) return 0;
    if (shape_check(B, T, H, dk, dv, N, varlen != 0) != GDN_OK) return 0;
    return fwd_layout(B, T, H, dk, dv, N, varlen != 0, dtype == GDN_BF16).total;
}

GDN_EXPORT int gdn_chunk_prepare(const void* q, const void* k, const float* g, const float* beta,
                                 const int32_t* cu_seqlens, int chunk, int B, int T, int H, int dk,
                                 int dv, int N, int dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    gdn::ChunkProblem p{};
    int st = check_chunk(q, k, nullptr, g, beta, nullptr, nullptr, nullptr, cu_seqlens, chunk, B, T,
                         H, dk, dv, N, dtype, GDN_F32, workspace, workspace_bytes, 1, &p);
    if (st != GDN_OK) return st;
    st = debug_check_offsets(cu_seqlens, N, T, static_cast<hipStream_t>(stream));
    if (st != GDN_OK) return st;
    return gdn::launch_chunk_prepare(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK
                                                                                      : GDN_ERR_HIP;
}

GDN_EXPORT int gdn_chunk_propagate(const void* q, const void* k, const void* v, const float* h0,
                                   void* o, float* hT, const int32_t* cu_seqlens, int chunk, int B,
                                   int T, int H, int dk, int dv, int N, int dtype, int o_dtype,
                                   const void* workspace, size_t workspace_bytes, void* stream) {
    gdn::ChunkProblem p{};
    int st = check_chunk(q, k, v, nullptr, nullptr, h0, o, hT, cu_seqlens, chunk, B, T, H, dk, dv,
                         N, dtype, o_dtype, workspace, workspace_bytes, 2, &p);
    if (st != GDN_OK) return st;
    st = debug_check_offsets(cu_seqlens, N, T, static_cast<hipStream_t>(stream));
    if (st != GDN_OK) return st;
    return gdn::launch_chunk_propagate(p, static_cast<hipStream_t>(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

namespace gdn {
// gdn_chunk_fwd's argument checks (host only, no HIP call) for a caller that will supply a
// workspace of gdn_chunk_fwd_workspace_bytes(...) bytes itself: GDN_OK or the status
// gdn_chunk_fwd would return for any argument other than the workspace.
int chunk_fwd_check(const void* q, const void* k, const void* v, const float* g_log_alpha, const float* beta,
                    const float* h0, const void* o, const float* hT, const int32_t* cu_seqlens, int chunk,
                    int B, int T, int H, int dk, int dv, int N, int dtype, int o_dtype) {
    gdn::ChunkProblem p{};
    const int st = check_chunk(q, k, v, g_log_alpha, beta, h0, o, hT, cu_seqlens, chunk, B, T, H, dk, dv, N,
                               dtype, o_dtype, nullptr, 0, 3, &p);
    return st == GDN_ERR_WORKSPACE ? GDN_OK : st;
}

// gdn_chunk_fwd with its arguments as given (also serves entry points that supply their own
// workspace)
int chunk_fwd(const void* q, const void* k, const void* v, const float* g_log_alpha, const float* beta,
              const float* h0, void* o, float* hT, const int32_t* cu_seqlens, int chunk, int B, int T,
              int H, int dk, int dv, int N, int dtype, int o_dtype, void* workspace,
              size_t workspace_bytes, void* stream) {
    gdn::ChunkProblem p{};
    int st = check_chunk(q, k, v, g_log_alpha, beta, h0, o, hT, cu_seqlens, chunk, B, T, H, dk, dv,
                         N, dtype, o_dtype, workspace, workspace_bytes, 3, &p);
    if (st != GDN_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    st = debug_check_offsets(cu_seqlens, N, T, s);
    if (st != GDN_OK) return st;
    if (gdn::fused_wanted(p.N, p.H, p.dk, p.dv, p.bf16))
        return gdn::launch_chunk_fused(p, s) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    if (gdn::launch_chunk_prepare(p, s) != hipSuccess) return GDN_ERR_HIP;
    if (gdn::launch_chunk_propagate(p, s) != hipSuccess) return GDN_ERR_HIP;
    return GDN_OK;
}
}  // namespace gdn

GDN_EXPORT int gdn_chunk_fwd(const void* q, const void* k, const void* v, const float* g_log_alpha,
                             const float* beta, const float* h0, void* o, float* hT,
                             const int32_t* cu_seqlens, int chunk, int B, int T, int H, int dk,
                             int dv, int N, int dtype, int o_dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
    return gdn::chunk_fwd(q, k, v, g_log_alpha, beta, h0, o, hT, cu_seqlens, chunk, B, T, H, dk, dv, N,
                          dtype, o_dtype, workspace, workspace_bytes, stream);
}

GDN_EXPORT int gdn_decode_step(const void* q, const void* k, const void* v, const float* g_log_alpha,
                               const float* beta, float* state, void* o, int N, int H, int dk,
                               int dv, int dtype, int o_dtype, void* stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (o_dtype != GDN_F32 && o_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    if (N < 1 || H < 1 || (long long)N * H > 0x7fffffffLL) return GDN_ERR_SHAPE;
    if (!q || !k || !v || !g_log_alpha || !beta || !state || !o) return GDN_ERR_NULL;
    const void* al16[] = {q, k, v, o, state};
    for (const void* x : al16)
        if (!aligned(x, 16)) return GDN_ERR_ALIGN;
    if (!aligned(g_log_alpha, 4) || !aligned(beta, 4)) return GDN_ERR_ALIGN;
    gdn::DecodeProblem p{q,  k, v,  g_log_alpha, beta,           state,
                         o,  N, H,  dk,          dv,   dtype == GDN_BF16, o_dtype == GDN_BF16};
    return gdn::launch_decode(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK
                                                                                : GDN_ERR_HIP;
}

GDN_EXPORT size_t gdn_chunk_bwd_workspace_bytes(int B, int T, int H, int dk, int dv, int N,
                                                int varlen, int chunk, int dtype) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return 0;
    if (chunk != 64 || !head_dim_ok(dk) || !head_dim_ok(dv)) return 0;
    if (shape_check(B, T, H, dk, dv, N, varlen != 0) != GDN_OK) return 0;
    return gdn::bwd_workspace_layout(B, T, H, dk, dv, N, varlen != 0, dtype == GDN_BF16).total;
}

GDN_EXPORT int gdn_chunk_bwd(const void* q, const void* k, const void* v, const float* g_log_alpha,
                             const float* beta, const float* h0, const void* d_o, const float* dhT,
                             void* dq, void* dk_out, void* dv_out, float* dg, float* dbeta, float* dh0,
                             const int32_t* cu_seqlens, int chunk, int B, int T, int H, int dk, int dv,
                             int N, int dtype, int grad_dtype, void* workspace, size_t workspace_bytes,
                             void* stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (grad_dtype != GDN_F32 && !(grad_dtype == GDN_BF16 && dtype == GDN_BF16)) return GDN_ERR_DTYPE;
    if (chunk != 64) return GDN_ERR_UNSUPPORTED;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    const int sc = shape_check(B, T, H, dk, dv, N, cu_seqlens != nullptr);
    if (sc != GDN_OK) return sc;
    const long long tokens = (long long)B * T;
    if (tokens > 0 && (!q || !k || !v || !g_log_alpha || !beta || !d_o || !dq || !dk_out || !dv_out ||
                       !dg || !dbeta))
        return GDN_ERR_NULL;
    const void* al16[] = {q, k, v, d_o, dq, dk_out, dv_out, h0, dhT, dh0};
    for (const void* x : al16)
        if (x && !aligned(x, 16)) return GDN_ERR_ALIGN;
    const void* al4[] = {g_log_alpha, beta, dg, dbeta, cu_seqlens};
    for (const void* x : al4)
        if (x && !aligned(x, 4)) return GDN_ERR_ALIGN;
    const int bf16 = dtype == GDN_BF16;
    const gdn::BwdLayout w = gdn::bwd_workspace_layout(B, T, H, dk, dv, N, cu_seqlens != nullptr, bf16);
    if (w.fwd.nc_bound * H > 0x7fffffffL) return GDN_ERR_SHAPE;
    if (w.total > 0 && (!workspace || workspace_bytes < w.total)) return GDN_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256)) return GDN_ERR_ALIGN;

    char* base = static_cast<char*>(workspace);
    gdn::BwdProblem b{};
    gdn::ChunkProblem& P = b.f;
    b.q_in = q; b.k_in = k; b.v_in = v; b.do_in = d_o;
    P.q = q;
    P.k = k;
    P.v = v;
    b.do32 = bf16 ? nullptr : static_cast<const float*>(d_o);
    P.g = g_log_alpha; P.beta = beta; P.h0 = h0; P.o = nullptr; P.hT = nullptr;
    P.cu_seqlens = cu_seqlens;
    P.B = B; P.T = T; P.H = H; P.dk = dk; P.dv = dv; P.N = N;
    P.bf16 = bf16; P.o_bf16 = 0;
    P.nc_bound = w.fwd.nc_bound;
    P.nc_per_seq = (T + 63) / 64;
    const bool any = w.fwd.nc_bound > 0;
    P.chunk_base = cu_seqlens ? reinterpret_cast<int32_t*>(base + w.fwd.off_base) : nullptr;
    P.gates = any ? reinterpret_cast<float*>(base + w.fwd.off_gates) : nullptr;
    P.mmat = any ? base + w.fwd.off_m : nullptr;
    P.pmat = any ? base + w.fwd.off_p : nullptr;
    P.tmat = (any && !bf16) ? reinterpret_cast<float*>(base + w.off_t) : nullptr;
    P.tmat16 = (any && bf16) ? reinterpret_cast<_Float16*>(base + w.off_t) : nullptr;
    P.states = (any && !bf16) ? reinterpret_cast<float*>(base + w.off_states) : nullptr;
    P.states16 = (any && bf16) ? reinterpret_cast<_Float16*>(base + w.off_states) : nullptr;
    // bf16: the fp32 Mmat region (not written) holds the fp16 images of Mmat, then of P
    P.mimg16 = (any && bf16) ? reinterpret_cast<_Float16*>(base + w.fwd.off_m) : nullptr;
    P.pimg16 = (any && bf16) ? reinterpret_cast<_Float16*>(base + w.fwd.off_m) + w.fwd.nc_bound * H * 4096 : nullptr;
    // bf16: the fp32 P region (not written) holds the image of P's fp16 rounding remainder
    P.plo16 = (any && bf16) ? reinterpret_cast<_Float16*>(base + w.fwd.off_p) : nullptr;
    P.k16 = (any && bf16) ? reinterpret_cast<_Float16*>(base + w.off_k16) : nullptr;
    P.q16 = (any && bf16) ? reinterpret_cast<_Float16*>(base + w.off_q16) : nullptr;
    b.dstates = any ? reinterpret_cast<float*>(base + w.off_dstates) : nullptr;
    b.dhT = dhT;
    b.dq = dq; b.dk = dk_out; b.dv = dv_out; b.dg = dg; b.dbeta = dbeta; b.dh0 = dh0;
    b.grad_bf16 = grad_dtype == GDN_BF16;
    const int chk = debug_check_offsets(cu_seqlens, N, T, static_cast<hipStream_t>(stream));
    if (chk != GDN_OK) return chk;
    return gdn::launch_chunk_backward(b, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK
                                                                                       : GDN_ERR_HIP;
}

GDN_EXPORT size_t gdn_kda_chunk_fwd_workspace_bytes(int B, int T, int H, int dk, int dv, int N,
                                                    int varlen, int chunk, int dtype) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return 0;
    if (chunk != 64 || !head_dim_ok(dk) || !head_dim_ok(dv)) return 0;
    if (shape_check(B, T, H, dk, dv, N, varlen != 0) != GDN_OK) return 0;
    return gdn::kda_workspace_layout(B, T, H, dk, N, varlen != 0, dtype == GDN_BF16 ? 2 : 4).total;
}

namespace {
// Shared by the channel-wise-decay entry points: beta, or the erase and write gates.
int kda_chunk_fwd(const void* q, const void* k, const void* v, const float* g_log_alpha,
                  const float* beta, const float* erase, const float* write, const float* h0, void* o,
                  float* hT, const int32_t* cu_seqlens, int chunk, int B, int T, int H, int dk, int dv,
                  int N, int dtype, int o_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (o_dtype != GDN_F32 && !(o_dtype == GDN_BF16 && dtype == GDN_BF16)) return GDN_ERR_DTYPE;
    if (chunk != 64) return GDN_ERR_UNSUPPORTED;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    const int sc = shape_check(B, T, H, dk, dv, N, cu_seqlens != nullptr);
    if (sc != GDN_OK) return sc;
    const long long tokens = (long long)B * T;
    if (tokens > 0 && (!q || !k || !v || !g_log_alpha || !o || (!erase && !beta) || (erase && !write)))
        return GDN_ERR_NULL;
    const void* al16[] = {q, k, v, o, h0, hT, g_log_alpha, erase, write};
    for (const void* x : al16)
        if (x && !aligned(x, 16)) return GDN_ERR_ALIGN;
    const void* al4[] = {beta, cu_seqlens};
    for (const void* x : al4)
        if (x && !aligned(x, 4)) return GDN_ERR_ALIGN;
    const gdn::KdaLayout w = gdn::kda_workspace_layout(B, T, H, dk, N, cu_seqlens != nullptr, dtype == GDN_BF16 ? 2 : 4);
    if (w.nc_bound * H > 0x7fffffffL) return GDN_ERR_SHAPE;
    if (w.total > 0 && (!workspace || workspace_bytes < w.total)) return GDN_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256)) return GDN_ERR_ALIGN;
    char* base = static_cast<char*>(workspace);
    gdn::ChunkProblem P{};
    P.q = q; P.k = k; P.v = v; P.g = g_log_alpha; P.beta = beta; P.h0 = h0; P.o = o; P.hT = hT;
    P.cu_seqlens = cu_seqlens;
    P.B = B; P.T = T; P.H = H; P.dk = dk; P.dv = dv; P.N = N;
    P.bf16 = dtype == GDN_BF16;
    P.o_bf16 = o_dtype == GDN_BF16;
    P.nc_bound = w.nc_bound;
    P.nc_per_seq = (T + 63) / 64;
    const bool any = w.nc_bound > 0;
    P.chunk_base = cu_seqlens ? reinterpret_cast<int32_t*>(base + w.off_base) : nullptr;
    P.mmat = any ? base + w.off_m : nullptr;
    P.pmat = any ? base + w.off_p : nullptr;
    P.khat = any ? reinterpret_cast<float*>(base + w.off_kh) : nullptr;
    P.qhat = any ? reinterpret_cast<float*>(base + w.off_qh) : nullptr;
    P.kdec = any ? reinterpret_cast<float*>(base + w.off_kd) : nullptr;
    P.lam = any ? reinterpret_cast<float*>(base + w.off_lam) : nullptr;
    P.erase = erase;
    P.write = erase ? write : nullptr;
    const int chk = debug_check_offsets(cu_seqlens, N, T, static_cast<hipStream_t>(stream));
    if (chk != GDN_OK) return chk;
    return gdn::launch_kda_chunk_fwd(P, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK
                                                                                       : GDN_ERR_HIP;
}
}  // namespace

GDN_EXPORT int gdn_kda_chunk_fwd(const void* q, const void* k, const void* v, const float* g_log_alpha,
                                 const float* beta, const float* h0, void* o, float* hT,
                                 const int32_t* cu_seqlens, int chunk, int B, int T, int H, int dk,
                                 int dv, int N, int dtype, int o_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    return kda_chunk_fwd(q, k, v, g_log_alpha, beta, nullptr, nullptr, h0, o, hT, cu_seqlens, chunk, B, T,
                         H, dk, dv, N, dtype, o_dtype, workspace, workspace_bytes, stream);
}

GDN_EXPORT int gdn_decoupled_chunk_fwd(const void* q, const void* k, const void* v, const float* g_log_alpha,
                                       const float* erase, const float* write, const float* h0, void* o,
                                       float* hT, const int32_t* cu_seqlens, int chunk, int B, int T, int H,
                                       int dk, int dv, int N, int dtype, int o_dtype, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    if (B * (long long)T > 0 && (!erase || !write)) return GDN_ERR_NULL;
    return kda_chunk_fwd(q, k, v, g_log_alpha, nullptr, erase, write, h0, o, hT, cu_seqlens, chunk, B, T,
                         H, dk, dv, N, dtype, o_dtype, workspace, workspace_bytes, stream);
}

GDN_EXPORT size_t gdn_kda_chunk_bwd_workspace_bytes(int B, int T, int H, int dk, int dv, int N, int varlen,
                                                    int chunk, int dtype) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return 0;
    if (chunk != 64 || !head_dim_ok(dk) || !head_dim_ok(dv)) return 0;
    if (shape_check(B, T, H, dk, dv, N, varlen != 0) != GDN_OK) return 0;
    return gdn::kda_bwd_workspace_layout(B, T, H, dk, dv, N, varlen != 0).total;
}

GDN_EXPORT int gdn_kda_chunk_bwd(const void* q, const void* k, const void* v, const float* g_log_alpha,
                                 const float* beta, const float* h0, const void* d_o, const float* dhT,
                                 void* dq, void* dk_out, void* dv_out, float* dg, float* dbeta, float* dh0,
                                 const int32_t* cu_seqlens, int chunk, int B, int T, int H, int dk, int dv,
                                 int N, int dtype, int grad_dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (grad_dtype != GDN_F32 && !(grad_dtype == GDN_BF16 && dtype == GDN_BF16)) return GDN_ERR_DTYPE;
    if (chunk != 64) return GDN_ERR_UNSUPPORTED;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    const int sc = shape_check(B, T, H, dk, dv, N, cu_seqlens != nullptr);
    if (sc != GDN_OK) return sc;
    const long long tokens = (long long)B * T;
    if (tokens > 0 && (!q || !k || !v || !g_log_alpha || !beta || !d_o || !dq || !dk_out || !dv_out || !dg || !dbeta))
        return GDN_ERR_NULL;
    const void* al16[] = {q, k, v, d_o, dq, dk_out, dv_out, h0, dhT, dh0, g_log_alpha, dg};
    for (const void* x : al16)
        if (x && !aligned(x, 16)) return GDN_ERR_ALIGN;
    const void* al4[] = {beta, dbeta, cu_seqlens};
    for (const void* x : al4)
        if (x && !aligned(x, 4)) return GDN_ERR_ALIGN;
    const gdn::KdaBwdLayout w = gdn::kda_bwd_workspace_layout(B, T, H, dk, dv, N, cu_seqlens != nullptr);
    if (w.fwd.nc_bound * H > 0x7fffffffL) return GDN_ERR_SHAPE;
    // two work-groups of 512 threads per (sequence, head, 64 columns), one of 256 per (chunk, head, 64 channels): fewer than
    // 2^32 threads each
    if ((long long)N * H >= 1 << 21 || (long long)w.fwd.nc_bound * H >= 1 << 23) return GDN_ERR_SHAPE;
    if (w.total > 0 && (!workspace || workspace_bytes < w.total)) return GDN_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256)) return GDN_ERR_ALIGN;
    char* base = static_cast<char*>(workspace);
    gdn::KdaBwdProblem b{};
    gdn::ChunkProblem& P = b.f;
    P.q = q; P.k = k; P.v = v; P.g = g_log_alpha; P.beta = beta; P.h0 = h0;
    P.cu_seqlens = cu_seqlens;
    P.B = B; P.T = T; P.H = H; P.dk = dk; P.dv = dv; P.N = N;
    P.bf16 = dtype == GDN_BF16;
    P.nc_bound = w.fwd.nc_bound;
    P.nc_per_seq = (T + 63) / 64;
    P.chunk_base = cu_seqlens ? reinterpret_cast<int32_t*>(base + w.fwd.off_base) : nullptr;
    if (w.fwd.nc_bound > 0) {
        P.tmat = reinterpret_cast<float*>(base + w.fwd.off_m);   // T in the place of Mmat
        P.pmat = base + w.fwd.off_p;
        P.khat = reinterpret_cast<float*>(base + w.fwd.off_kh);
        P.qhat = reinterpret_cast<float*>(base + w.fwd.off_qh);
        P.kdec = reinterpret_cast<float*>(base + w.fwd.off_kd);
        P.lam = reinterpret_cast<float*>(base + w.fwd.off_lam);
        P.states = reinterpret_cast<float*>(base + w.off_states);
        b.dstates = reinterpret_cast<float*>(base + w.off_dstates);
        b.delta = reinterpret_cast<float*>(base + w.off_delta);
        b.ymat = reinterpret_cast<float*>(base + w.off_y);
    }
    b.d_o = d_o; b.dhT = dhT;
    b.dq = dq; b.dk = dk_out; b.dv = dv_out; b.dg = dg; b.dbeta = dbeta; b.dh0 = dh0;
    b.grad_bf16 = grad_dtype == GDN_BF16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int chk = debug_check_offsets(cu_seqlens, N, T, s);
    if (chk != GDN_OK) return chk;
    return gdn::launch_kda_chunk_bwd(b, s) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

GDN_EXPORT int gdn_kda_decode_step(const void* q, const void* k, const void* v, const float* g_log_alpha,
                                   const float* beta, float* state, void* o, int N, int H, int dk,
                                   int dv, int dtype, int o_dtype, void* stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (o_dtype != GDN_F32 && o_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    if (N < 1 || H < 1 || (long long)N * H > 0x7fffffffLL) return GDN_ERR_SHAPE;
    if (!q || !k || !v || !g_log_alpha || !beta || !state || !o) return GDN_ERR_NULL;
    const void* al16[] = {q, k, v, o, state, g_log_alpha};
    for (const void* x : al16)
        if (!aligned(x, 16)) return GDN_ERR_ALIGN;
    if (!aligned(beta, 4)) return GDN_ERR_ALIGN;
    gdn::DecodeProblem p{q,  k, v,  g_log_alpha, beta,           state,
                         o,  N, H,  dk,          dv,   dtype == GDN_BF16, o_dtype == GDN_BF16};
    p.channel_gate = 1;
    return gdn::launch_decode(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK
                                                                                : GDN_ERR_HIP;
}

GDN_EXPORT int gdn_decoupled_decode_step(const void* q, const void* k, const void* v, const float* g_log_alpha,
                                         const float* erase, const float* write, float* state, void* o, int N,
                                         int H, int dk, int dv, int dtype, int o_dtype, void* stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (o_dtype != GDN_F32 && o_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    if (N < 1 || H < 1 || (long long)N * H > 0x7fffffffLL) return GDN_ERR_SHAPE;
    if (!q || !k || !v || !g_log_alpha || !erase || !write || !state || !o) return GDN_ERR_NULL;
    const void* al16[] = {q, k, v, o, state, g_log_alpha, erase, write};
    for (const void* x : al16)
        if (!aligned(x, 16)) return GDN_ERR_ALIGN;
    gdn::DecodeProblem p{q,  k, v,  g_log_alpha, nullptr,        state,
                         o,  N, H,  dk,          dv,   dtype == GDN_BF16, o_dtype == GDN_BF16};
    p.channel_gate = 1;
    p.erase = erase;
    p.write = write;
    return gdn::launch_decode(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK
                                                                                : GDN_ERR_HIP;
}

GDN_EXPORT int gdn_recurrent_fwd(const void* q, const void* k, const void* v, const float* g_log_alpha,
                                 const float* beta, float* states, const int32_t* slots,
                                 const int32_t* cu_seqlens, const int32_t* out_slots, void* o, int T, int N,
                                 int H, int HV, int dk, int dv, int n_slots, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, int channel_gate, int dtype, int o_dtype, void* stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (o_dtype != GDN_F32 && o_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    if (N < 0 || T < 0 || H < 1 || HV < H || HV % H != 0 || HV > 32768 || n_slots < 0) return GDN_ERR_SHAPE;
    if (!cu_seqlens && T != N) return GDN_ERR_SHAPE;
    // a work-group of 256 threads per (sequence, value head, tile of state rows), fewer than 2^32 threads in all
    if ((long long)N * HV >= 1 << 21) return GDN_ERR_SHAPE;
    if (q_stride < 0 || k_stride < 0 || v_stride < 0) return GDN_ERR_SHAPE;
    if (T == 0 || N == 0) return GDN_OK;   // no token: nothing to read or write
    if (!q || !k || !v || !g_log_alpha || !beta || !slots || !o || (!states && n_slots > 0)) return GDN_ERR_NULL;
    const void* al16[] = {q, k, v, o, states};
    for (const void* x : al16)
        if (!aligned(x, 16)) return GDN_ERR_ALIGN;
    const void* al4[] = {beta, slots, cu_seqlens, out_slots};
    for (const void* x : al4)
        if (!aligned(x, 4)) return GDN_ERR_ALIGN;
    if (!aligned(g_log_alpha, channel_gate ? 16 : 4)) return GDN_ERR_ALIGN;
    const int per16 = dtype == GDN_BF16 ? 8 : 4;   // elements of 16 bytes
    if (q_stride % per16 || k_stride % per16 || v_stride % per16) return GDN_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int chk = debug_check_offsets(cu_seqlens, N, T, s, true);
    if (chk != GDN_OK) return chk;
    gdn::RecurrentProblem p{};
    p.q = q; p.k = k; p.v = v; p.g = g_log_alpha; p.beta = beta; p.states = states;
    p.slots = slots; p.cu_seqlens = cu_seqlens; p.out_slots = out_slots; p.o = o;
    p.q_token = q_stride; p.k_token = k_stride; p.v_token = v_stride;
    p.T = T; p.N = N; p.H = H; p.HV = HV; p.dk = dk; p.dv = dv; p.n_slots = n_slots;
    p.bf16 = dtype == GDN_BF16;
    p.o_bf16 = o_dtype == GDN_BF16;
    p.channel_gate = channel_gate != 0;
    return gdn::launch_recurrent(p, s) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

namespace {
// Checks shared by both directions of the q/k norm; fills the shared part of the problem.
int check_norm(const void* q, const void* k, const float* q_weight, const float* k_weight, const int32_t* positions,
               const float* inv_freq, int tokens, int hq, int hk, int d, int64_t q_token, int64_t q_head,
               int64_t k_token, int64_t k_head, int norm, float eps, int rot, int rope, float q_scale,
               float rope_scale, int dtype, int y_dtype, gdn::NormProblem* p) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (y_dtype != GDN_F32 && !(y_dtype == GDN_BF16 && dtype == GDN_BF16)) return GDN_ERR_DTYPE;
    if (norm != GDN_NORM_L2 && norm != GDN_NORM_RMS) return GDN_ERR_UNSUPPORTED;
    if (rope != GDN_ROPE_HALF && rope != GDN_ROPE_INTERLEAVED) return GDN_ERR_UNSUPPORTED;
    if (d < 8 || d > 256 || d % 8) return GDN_ERR_UNSUPPORTED;
    if (rot < 0 || rot > d || rot % (rope == GDN_ROPE_HALF ? 16 : 2)) return GDN_ERR_UNSUPPORTED;
    if (tokens < 0 || hq < 1 || hk < 1 || hq > 32768 || hk > 32768) return GDN_ERR_SHAPE;
    if (!(eps > 0.f)) return GDN_ERR_SHAPE;
    // rows are counted in 32 bits, and a large call's work-groups of 256 threads take 32 rows or more: fewer than 2^32 threads
    if ((long long)tokens * (hq + hk) > (1LL << 28)) return GDN_ERR_SHAPE;
    const int64_t strides[] = {q_token, q_head, k_token, k_head};
    for (int64_t x : strides)
        if (x < 0) return GDN_ERR_SHAPE;
    if (tokens > 0 && (!q || !k || (rot > 0 && (!positions || !inv_freq)))) return GDN_ERR_NULL;
    const void* al16[] = {q, k, q_weight, k_weight};
    for (const void* x : al16)
        if (!aligned(x, 16)) return GDN_ERR_ALIGN;
    if (!aligned(positions, 4) || !aligned(inv_freq, 4)) return GDN_ERR_ALIGN;
    const int per16 = dtype == GDN_BF16 ? 8 : 4;   // elements of 16 bytes
    for (int64_t x : strides)
        if (x % per16) return GDN_ERR_ALIGN;
    p->q = q; p->k = k; p->q_weight = q_weight; p->k_weight = k_weight;
    p->q_token = q_token; p->q_head = q_head; p->k_token = k_token; p->k_head = k_head;
    p->positions = positions; p->inv_freq = inv_freq;
    p->tokens = tokens; p->hq = hq; p->hk = hk; p->d = d; p->rot = rot;
    p->interleaved = rope == GDN_ROPE_INTERLEAVED;
    p->x_bf16 = dtype == GDN_BF16;
    p->y_bf16 = y_dtype == GDN_BF16;
    p->inv_n = norm == GDN_NORM_RMS ? 1.f / d : 1.f;
    p->eps = eps; p->q_scale = q_scale; p->rope_scale = rope_scale;
    return GDN_OK;
}

// Whether two of the rows [d] that start at token * token_stride + head * head_stride share an element (strides >= 0; one of 0
// is how an expanded tensor looks).
bool rows_overlap(int tokens, int heads, int d, int64_t token_stride, int64_t head_stride) {
    if ((tokens > 1 && token_stride < d) || (heads > 1 && head_stride < d)) return true;
    if (tokens <= 1 || heads <= 1) return false;
    using wide = __int128;   // a multiple of a stride can leave 64 bits
    const wide ts = token_stride, hs = head_stride;
    if (ts >= (heads - 1) * hs + d || hs >= (tokens - 1) * ts + d) return false;   // one dimension within the other
    // interleaved: head h's first row against the rows of head 0 that start before and behind it (every other pair of rows is such
    // a pair shifted, or further apart)
    for (int h = 1; h < heads; ++h) {
        const wide t = h * hs / ts, behind = h * hs - t * ts;
        if ((t < tokens && behind < d) || (t + 1 < tokens && ts - behind < d)) return true;
    }
    return false;
}
}  // namespace

GDN_EXPORT int gdn_qk_norm_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                               const int32_t* positions, const float* inv_freq, void* q_out, void* k_out,
                               int tokens, int hq, int hk, int d, int64_t q_token_stride, int64_t q_head_stride,
                               int64_t k_token_stride, int64_t k_head_stride, int norm, float eps, int rot,
                               int rope, float q_scale, float rope_scale, int dtype, int out_dtype, void* stream) {
    gdn::NormProblem p{};
    const int st = check_norm(q, k, q_weight, k_weight, positions, inv_freq, tokens, hq, hk, d, q_token_stride,
                              q_head_stride, k_token_stride, k_head_stride, norm, eps, rot, rope, q_scale, rope_scale,
                              dtype, out_dtype, &p);
    if (st != GDN_OK) return st;
    if (tokens > 0 && (!q_out || !k_out)) return GDN_ERR_NULL;
    if (!aligned(q_out, 16) || !aligned(k_out, 16)) return GDN_ERR_ALIGN;
    p.q_out = q_out;
    p.k_out = k_out;
    return gdn::launch_qk_norm(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

GDN_EXPORT size_t gdn_qk_norm_bwd_workspace_bytes(int tokens, int hq, int hk, int d) {
    if (tokens < 0 || hq < 1 || hk < 1 || hq > 32768 || hk > 32768 || d < 8 || d > 256 || d % 8) return 0;
    if ((long long)tokens * (hq + hk) > (1LL << 28)) return 0;
    return (size_t)gdn::norm_grad_blocks((long)tokens * (hq + hk)) * 2 * d * sizeof(float);
}

GDN_EXPORT int gdn_qk_norm_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                               const float* q_weight, const float* k_weight, const int32_t* positions,
                               const float* inv_freq, void* dq, void* dk, float* dq_weight, float* dk_weight,
                               int tokens, int hq, int hk, int d, int64_t q_token_stride, int64_t q_head_stride,
                               int64_t k_token_stride, int64_t k_head_stride, int64_t dq_token_stride,
                               int64_t dq_head_stride, int64_t dk_token_stride, int64_t dk_head_stride, int norm,
                               float eps, int rot, int rope, float q_scale, float rope_scale, int dtype,
                               int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::NormProblem p{};
    const int st = check_norm(q, k, q_weight, k_weight, positions, inv_freq, tokens, hq, hk, d, q_token_stride,
                              q_head_stride, k_token_stride, k_head_stride, norm, eps, rot, rope, q_scale, rope_scale,
                              dtype, out_dtype, &p);
    if (st != GDN_OK) return st;
    const int64_t strides[] = {dq_token_stride, dq_head_stride, dk_token_stride, dk_head_stride};
    for (int64_t x : strides)
        if (x < 0) return GDN_ERR_SHAPE;
    // rows of an output must not lie over each other: two work-groups would write the same elements
    if (rows_overlap(tokens, hq, d, dq_token_stride, dq_head_stride) || rows_overlap(tokens, hk, d, dk_token_stride, dk_head_stride))
        return GDN_ERR_SHAPE;
    if (tokens > 0 && (!dq_out || !dk_out || !dq || !dk)) return GDN_ERR_NULL;
    const void* al16[] = {dq_out, dk_out, dq, dk};
    for (const void* x : al16)
        if (!aligned(x, 16)) return GDN_ERR_ALIGN;
    for (int64_t x : strides)
        if (x % (p.x_bf16 ? 8 : 4)) return GDN_ERR_ALIGN;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return GDN_ERR_ALIGN;
    if (dq_weight || dk_weight) {
        const size_t need = gdn_qk_norm_bwd_workspace_bytes(tokens, hq, hk, d);
        if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return GDN_ERR_ALIGN;
    }
    p.backward = 1;
    p.dq_in = dq_out; p.dk_in = dk_out; p.dq_out = dq; p.dk_out = dk;
    p.dq_token = dq_token_stride; p.dq_head = dq_head_stride;
    p.dk_token = dk_token_stride; p.dk_head = dk_head_stride;
    p.dqw = dq_weight; p.dkw = dk_weight;
    p.partial = static_cast<float*>(workspace);
    return gdn::launch_qk_norm(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}
