// C-ABI entry points of the short causal convolution, the selective state space scan and the group norm:
// argument validation and dispatch.  Declarations and the contract are in efla.h.
#include <math.h>

#include "api_args.cuh"
#include "conv.cuh"
#include "group_norm.cuh"
#include "ssm.cuh"

using namespace efla;

namespace {

constexpr long long MOST = (1LL << 31) - 1;

bool activation_ok(efla_activation a) { return a == EFLA_ACT_NONE || a == EFLA_ACT_SILU; }

// Whether lead x T x d elements can be counted (the kernels' row indexes and grids fit 31 bits).
efla_status check_rows(const char *what, int B, int T, int D) {
    if (B < 0 || T < 0 || D <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "bad sizes B=%d T=%d %s=%d", B, T, what, D);
    if (D % 8) return api_fail(EFLA_ERR_UNSUPPORTED, "%s=%d must be a multiple of 8", what, D);
    const long long tok = (long long)B * T;
    if (D > (1 << 20) || tok > MOST - 4096 || tok > (1LL << 40) / D || (long long)B > (1LL << 33) / D)
        return api_fail(EFLA_ERR_UNSUPPORTED, "B=%d T=%d %s=%d: more than 2^31-4097 tokens, 2^20 channels or 2^40 elements", B, T, what, D);
    return EFLA_OK;
}

efla_status check_conv(int B, int T, int D, int W, efla_dtype dtype, efla_activation act) {
    const efla_status s = check_rows("D", B, T, D);
    if (s != EFLA_OK) return s;
    if (W < 2 || W > 4) return api_fail(EFLA_ERR_UNSUPPORTED, "W=%d: supported convolution widths are 2, 3, 4", W);
    if (!dtype_ok(dtype)) return api_fail(EFLA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (!activation_ok(act)) return api_fail(EFLA_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    return EFLA_OK;
}

// The number of sequences: B rows, or those of cu_seqlens over one row.
efla_status check_sequences(const int32_t *cu_seqlens, int B, int N, int D) {
    if (N < 0 || (long long)N > (1LL << 33) / D) return api_fail(EFLA_ERR_INVALID_ARG, "bad number of sequences N=%d", N);
    if (cu_seqlens ? B != 1 : N != B)
        return api_fail(EFLA_ERR_INVALID_ARG, cu_seqlens ? "cu_seqlens given with B=%d (must be 1), N=%d"
                                                         : "B=%d, N=%d: N must equal B when cu_seqlens is NULL", B, N);
    return EFLA_OK;
}

efla_status check_ssm(int B, int T, int D, int N, int G, efla_dtype dtype) {
    if (G <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "G=%d must be positive", G);
    const efla_status s = check_rows("D", B, T, D);
    if (s != EFLA_OK) return s;
    if (N != 16 && N != 32 && N != 64 && N != 128)
        return api_fail(EFLA_ERR_UNSUPPORTED, "d_state=%d: supported state sizes are 16, 32, 64, 128", N);
    if (D % G) return api_fail(EFLA_ERR_INVALID_ARG, "D=%d must be a multiple of G=%d", D, G);
    if (!dtype_ok(dtype)) return api_fail(EFLA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    const int vec = 16 / (int)es(dtype);  // (a channel tile begins on 16 bytes)
    if (D / G % vec) return api_fail(EFLA_ERR_UNSUPPORTED, "D=%d: a group's %d channels must be a multiple of %d", D, D / G, vec);
    if (((long long)B + 1) * ssm_fwd_tiles(D, N, G) > MOST / 4 || (long long)B * T > (1LL << 40) / ((long long)G * N))
        return api_fail(EFLA_ERR_UNSUPPORTED, "B=%d T=%d D=%d G=%d: too many rows of channels", B, T, D, G);
    return EFLA_OK;
}

efla_status check_group_norm(int rows, int L, int C, int groups, efla_dtype dtype, efla_activation act, float eps) {
    if (groups <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "groups=%d must be positive", groups);
    const efla_status s = check_rows("C", rows, L, C);
    if (s != EFLA_OK) return s;
    if (C % groups) return api_fail(EFLA_ERR_INVALID_ARG, "C=%d must be a multiple of groups=%d", C, groups);
    if (!dtype_ok(dtype)) return api_fail(EFLA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (!activation_ok(act)) return api_fail(EFLA_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    if (!(eps >= 0.f) || !isfinite(eps)) return api_fail(EFLA_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", eps);
    if ((long long)rows * C > MOST * 4) return api_fail(EFLA_ERR_UNSUPPORTED, "rows=%d C=%d: too many rows of channels", rows, C);
    return EFLA_OK;
}

// Segments of a scan without training: their length (0: uncut) and number for N sequences of T / N tokens on average.
void scan_segments(int T, int D, int d_state, int N, bool packed, int &seg, int &slots) {
    seg = ssm_segment(N, packed && N > 0 ? (int)(((long long)T + N - 1) / N) : T, D, d_state, packed && N > 1);
    slots = !seg ? N : packed ? T / seg + N : N * ssm_pieces(T, seg);
}
size_t scan_bytes(int D, int d_state, int seg, int slots) { return seg ? (size_t)slots * D * (d_state + 1) * sizeof(float) : 0; }

}  // namespace

extern "C" {

efla_status efla_causal_conv(const void *x, const float *w, const float *bias, const void *state0,
                             const int32_t *cu_seqlens, void *y, void *state_T, int B, int T, int D, int W, int N,
                             efla_dtype dtype, efla_activation activation, efla_stream_t stream) {
    efla_status s = check_conv(B, T, D, W, dtype, activation);
    if (s != EFLA_OK) return s;
    if ((s = check_sequences(cu_seqlens, B, N, D)) != EFLA_OK) return s;
    const size_t xb = (size_t)B * T * D * es(dtype), st = (size_t)N * (W - 1) * D * es(dtype);
    s = check_args({{"x", x, xb, IN}, {"w", w, (size_t)D * W * 4, IN}, {"bias", bias, (size_t)D * 4, IN_OPT},
                    {"state0", state0, st, IN_OPT}, {"cu_seqlens", cu_seqlens, cu_seqlens ? ((size_t)N + 1) * 4 : 0, IN_OPT},
                    {"y", y, xb, OUT}, {"state_T", state_T, st, OUT_OPT}});
    if (s != EFLA_OK) return s;
    if (N == 0) return api_ok();
    ConvArgs a{};
    a.x = x, a.w = w, a.bias = bias, a.state0 = state0, a.cu_seqlens = cu_seqlens, a.y = y, a.state_T = state_T;
    a.B = B, a.T = T, a.D = D, a.W = W, a.N = N, a.dtype = dtype, a.silu = activation == EFLA_ACT_SILU;
    a.stream = reinterpret_cast<cudaStream_t>(stream), a.status = device_status_ptr();
    if (!a.status) return api_fail(EFLA_ERR_CUDA, "cannot resolve the device status word");
    return launched(launch_conv(a), "convolution kernel launch");
}

efla_status efla_causal_conv_bwd_workspace(int B, int T, int D, int W, size_t *bytes) {
    if (!bytes) return api_fail(EFLA_ERR_INVALID_ARG, "bytes must be non-NULL");
    const efla_status s = check_conv(B, T, D, W, EFLA_F32, EFLA_ACT_NONE);
    if (s != EFLA_OK) return s;
    const int parts = conv_bwd_runs(B, T, D, W).parts;
    *bytes = (size_t)parts * D * (W + 1) * sizeof(float);
    return api_ok();
}

efla_status efla_causal_conv_bwd(const void *x, const float *w, const float *bias, const void *state0, const void *dy,
                                 const void *dstate_T, void *dx, float *dw, float *dbias, void *dstate0, int B, int T,
                                 int D, int W, efla_dtype dtype, efla_activation activation, void *workspace,
                                 size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_conv(B, T, D, W, dtype, activation);
    if (s != EFLA_OK) return s;
    size_t need = 0;
    if ((s = efla_causal_conv_bwd_workspace(B, T, D, W, &need)) != EFLA_OK) return s;
    if ((s = need_workspace(workspace, workspace_bytes, need)) != EFLA_OK) return s;
    const size_t xb = (size_t)B * T * D * es(dtype), st = (size_t)B * (W - 1) * D * es(dtype), wb = (size_t)D * W * 4, bb = (size_t)D * 4;
    s = check_args({{"x", x, xb, IN}, {"w", w, wb, IN}, {"bias", bias, bb, IN_OPT}, {"state0", state0, st, IN_OPT},
                    {"dy", dy, xb, IN}, {"dstate_T", dstate_T, st, IN_OPT}, {"dx", dx, xb, OUT}, {"dw", dw, wb, OUT},
                    {"dbias", dbias, bb, OUT_OPT}, {"dstate0", dstate0, st, OUT_OPT}, {"workspace", workspace, need, OUT_OPT}});
    if (s != EFLA_OK) return s;
    ConvArgs a{};
    a.x = x, a.w = w, a.bias = bias, a.state0 = state0, a.dy = dy, a.dstate_T = dstate_T;
    a.dx = dx, a.dw = dw, a.dbias = dbias, a.dstate0 = dstate0, a.ws = static_cast<float *>(workspace);
    a.B = B, a.T = T, a.D = D, a.W = W, a.N = B, a.dtype = dtype, a.silu = activation == EFLA_ACT_SILU;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_conv_bwd(a), "convolution backward launch");
}

efla_status efla_causal_conv_step(const void *x, const float *w, const float *bias, void *state, void *y, int B, int D,
                                  int W, efla_dtype dtype, efla_activation activation, efla_stream_t stream) {
    efla_status s = check_conv(B, 1, D, W, dtype, activation);
    if (s != EFLA_OK) return s;
    const size_t xb = (size_t)B * D * es(dtype);
    s = check_args({{"x", x, xb, IN}, {"w", w, (size_t)D * W * 4, IN}, {"bias", bias, (size_t)D * 4, IN_OPT},
                    {"state", state, xb * (W - 1), OUT}, {"y", y, xb, OUT}});
    if (s != EFLA_OK) return s;
    if (B == 0) return api_ok();
    ConvArgs a{};
    a.x = x, a.w = w, a.bias = bias, a.state0 = state, a.state_T = state, a.y = y;
    a.B = B, a.T = 1, a.D = D, a.W = W, a.N = B, a.dtype = dtype, a.silu = activation == EFLA_ACT_SILU;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_conv_step(a), "convolution step launch");
}

efla_status efla_ssm_scan_workspace(int B, int T, int D, int d_state, int G, int N, int packed, size_t *bytes) {
    if (!bytes) return api_fail(EFLA_ERR_INVALID_ARG, "bytes must be non-NULL");
    efla_status s = check_ssm(B, T, D, d_state, G, EFLA_F32);
    if (s != EFLA_OK) return s;
    if (N < 0 || (long long)N > (1LL << 33) / D || (packed ? B != 1 : N != B))
        return api_fail(EFLA_ERR_INVALID_ARG, "bad number of sequences N=%d", N);
    int seg, slots;
    scan_segments(T, D, d_state, N, packed != 0, seg, slots);
    *bytes = scan_bytes(D, d_state, seg, slots);
    return api_ok();
}

efla_status efla_ssm_scan(const void *x, const void *dt, const float *A_log, const void *Bm, const void *Cm,
                          const float *D_skip, const float *dt_bias, const void *z, const float *S0,
                          const int32_t *cu_seqlens, void *y, float *S_T, int B, int T, int D, int d_state, int G,
                          int N, efla_dtype dtype, void *workspace, size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_ssm(B, T, D, d_state, G, dtype);
    if (s != EFLA_OK) return s;
    if ((s = check_sequences(cu_seqlens, B, N, D)) != EFLA_OK) return s;
    if ((long long)N * ssm_fwd_tiles(D, d_state, G) > MOST) return api_fail(EFLA_ERR_UNSUPPORTED, "N=%d D=%d: too many sequences of channels", N, D);
    int seg, slots;
    scan_segments(T, D, d_state, N, cu_seqlens != nullptr, seg, slots);
    const size_t need = scan_bytes(D, d_state, seg, slots);
    if ((s = need_workspace(workspace, workspace_bytes, need)) != EFLA_OK) return s;
    const size_t tok = (size_t)B * T, xb = tok * D * es(dtype), bb = tok * G * d_state * es(dtype), st = (size_t)N * D * d_state * 4;
    s = check_args({{"x", x, xb, IN}, {"dt", dt, xb, IN}, {"A_log", A_log, (size_t)D * d_state * 4, IN}, {"B", Bm, bb, IN},
                    {"C", Cm, bb, IN}, {"D_skip", D_skip, (size_t)D * 4, IN_OPT}, {"dt_bias", dt_bias, (size_t)D * 4, IN_OPT},
                    {"z", z, xb, IN_OPT}, {"S0", S0, st, IN_OPT},
                    {"cu_seqlens", cu_seqlens, cu_seqlens ? ((size_t)N + 1) * 4 : 0, IN_OPT}, {"y", y, xb, OUT},
                    {"S_T", S_T, st, OUT_OPT, {"S0"}}, {"workspace", workspace, need, OUT_OPT}});
    if (s != EFLA_OK) return s;
    if (N == 0) return api_ok();
    SsmArgs a{};
    a.x = x, a.dt = dt, a.z = z, a.A_log = A_log, a.Dskip = D_skip, a.dt_bias = dt_bias, a.Bm = Bm, a.Cm = Cm, a.S0 = S0;
    a.cu_seqlens = cu_seqlens, a.y = y, a.S_T = S_T, a.B = B, a.T = T, a.D = D, a.N = d_state, a.G = G, a.nseq = N;
    a.dtype = dtype, a.stream = reinterpret_cast<cudaStream_t>(stream), a.status = device_status_ptr();
    if (!a.status) return api_fail(EFLA_ERR_CUDA, "cannot resolve the device status word");
    a.seg = seg, a.slots = slots;
    a.state = static_cast<float *>(workspace);
    a.sum = seg ? a.state + (size_t)slots * D * d_state : nullptr;
    return launched(launch_ssm_scan(a), "scan kernel launch");
}

efla_status efla_ssm_bwd_workspace(int B, int T, int D, int d_state, int G, size_t *bytes) {
    if (!bytes) return api_fail(EFLA_ERR_INVALID_ARG, "bytes must be non-NULL");
    const efla_status s = check_ssm(B, T, D, d_state, G, EFLA_F32);
    if (s != EFLA_OK) return s;
    *bytes = ssm_ws(B, T, D, d_state, G).bytes;
    return api_ok();
}

static SsmArgs train_args(const void *x, const void *dt, const float *A_log, const void *Bm, const void *Cm, const float *D_skip,
                          const float *dt_bias, const void *z, const float *S0, int B, int T, int D, int d_state, int G,
                          efla_dtype dtype, const SsmWs &w, void *workspace, efla_stream_t stream) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    SsmArgs a{};
    a.x = x, a.dt = dt, a.z = z, a.A_log = A_log, a.Dskip = D_skip, a.dt_bias = dt_bias, a.Bm = Bm, a.Cm = Cm, a.S0 = S0;
    a.B = B, a.T = T, a.D = D, a.N = d_state, a.G = G, a.nseq = B, a.dtype = dtype;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    a.seg = w.seg, a.slots = w.slots;
    a.state = reinterpret_cast<float *>(ws + w.state), a.sum = reinterpret_cast<float *>(ws + w.sum);
    a.keep = reinterpret_cast<float *>(ws + w.keep);
    return a;
}

efla_status efla_ssm_scan_train(const void *x, const void *dt, const float *A_log, const void *Bm, const void *Cm,
                                const float *D_skip, const float *dt_bias, const void *z, const float *S0, void *y,
                                float *S_T, int B, int T, int D, int d_state, int G, efla_dtype dtype, void *workspace,
                                size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_ssm(B, T, D, d_state, G, dtype);
    if (s != EFLA_OK) return s;
    const SsmWs w = ssm_ws(B, T, D, d_state, G);
    if ((s = need_workspace(workspace, workspace_bytes, w.bytes)) != EFLA_OK) return s;
    const size_t tok = (size_t)B * T, xb = tok * D * es(dtype), bb = tok * G * d_state * es(dtype), st = (size_t)B * D * d_state * 4;
    s = check_args({{"x", x, xb, IN}, {"dt", dt, xb, IN}, {"A_log", A_log, (size_t)D * d_state * 4, IN}, {"B", Bm, bb, IN},
                    {"C", Cm, bb, IN}, {"D_skip", D_skip, (size_t)D * 4, IN_OPT}, {"dt_bias", dt_bias, (size_t)D * 4, IN_OPT},
                    {"z", z, xb, IN_OPT}, {"S0", S0, st, IN_OPT}, {"y", y, xb, OUT}, {"S_T", S_T, st, OUT_OPT, {"S0"}},
                    {"workspace", workspace, w.bytes, OUT_OPT}});
    if (s != EFLA_OK) return s;
    if (B == 0) return api_ok();
    SsmArgs a = train_args(x, dt, A_log, Bm, Cm, D_skip, dt_bias, z, S0, B, T, D, d_state, G, dtype, w, workspace, stream);
    a.y = y, a.S_T = S_T;
    return launched(launch_ssm_scan(a), "scan kernel launch");
}

efla_status efla_ssm_scan_bwd(const void *x, const void *dt, const float *A_log, const void *Bm, const void *Cm,
                              const float *D_skip, const float *dt_bias, const void *z, const float *S0, const void *dy,
                              const float *dS_T, void *dx, void *ddt, float *dA_log, void *dB, void *dC, float *dD,
                              float *ddt_bias, void *dz, float *dS0, int B, int T, int D, int d_state, int G,
                              efla_dtype dtype, int saved, void *workspace, size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_ssm(B, T, D, d_state, G, dtype);
    if (s != EFLA_OK) return s;
    if ((dz && !z) || (z && !dz && (size_t)B * T > 0)) return api_fail(EFLA_ERR_INVALID_ARG, "dz must be given exactly where z is");
    const SsmWs w = ssm_ws(B, T, D, d_state, G);
    if ((s = need_workspace(workspace, workspace_bytes, w.bytes)) != EFLA_OK) return s;
    const size_t tok = (size_t)B * T, xb = tok * D * es(dtype), bb = tok * G * d_state * es(dtype), st = (size_t)B * D * d_state * 4;
    const size_t ab = (size_t)D * d_state * 4, db = (size_t)D * 4;
    s = check_args({{"x", x, xb, IN}, {"dt", dt, xb, IN}, {"A_log", A_log, ab, IN}, {"B", Bm, bb, IN}, {"C", Cm, bb, IN},
                    {"D_skip", D_skip, db, IN_OPT}, {"dt_bias", dt_bias, db, IN_OPT}, {"z", z, xb, IN_OPT},
                    {"S0", S0, st, IN_OPT}, {"dy", dy, xb, IN}, {"dS_T", dS_T, st, IN_OPT}, {"dx", dx, xb, OUT},
                    {"ddt", ddt, xb, OUT}, {"dA_log", dA_log, ab, OUT}, {"dB", dB, bb, OUT}, {"dC", dC, bb, OUT},
                    {"dD", dD, db, OUT_OPT}, {"ddt_bias", ddt_bias, db, OUT_OPT}, {"dz", dz, xb, OUT_OPT},
                    {"dS0", dS0, st, OUT_OPT}, {"workspace", workspace, w.bytes, OUT_OPT}});
    if (s != EFLA_OK) return s;
    SsmBwdArgs a{};
    a.f = train_args(x, dt, A_log, Bm, Cm, D_skip, dt_bias, z, S0, B, T, D, d_state, G, dtype, w, workspace, stream);
    if (!saved && B > 0 && T > 0) {  // the forward for the states it keeps
        const cudaError_t e = launch_ssm_scan(a.f);
        if (e != cudaSuccess) return launched(e, "scan kernel launch");
    }
    a.f.seg = w.bwd_seg, a.f.slots = w.bwd_slots;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.dy = dy, a.dS_T = dS_T, a.dx = dx, a.ddt = ddt, a.dz = dz, a.dB = dB, a.dC = dC;
    a.dA_log = dA_log, a.dD = dD, a.ddt_bias = ddt_bias, a.dS0 = dS0;
    a.part = reinterpret_cast<float *>(ws + w.part), a.sums = reinterpret_cast<float *>(ws + w.sums);
    a.sums2 = reinterpret_cast<float *>(ws + w.sums2);
    return launched(launch_ssm_bwd(a), "scan backward launch");
}

efla_status efla_ssm_step(const void *x, const void *dt, const float *A_log, const void *Bm, const void *Cm,
                          const float *D_skip, const float *dt_bias, const void *z, float *S, void *y, int B, int D,
                          int d_state, int G, efla_dtype dtype, efla_stream_t stream) {
    efla_status s = check_ssm(B, 1, D, d_state, G, dtype);
    if (s != EFLA_OK) return s;
    const size_t xb = (size_t)B * D * es(dtype), bb = (size_t)B * G * d_state * es(dtype);
    s = check_args({{"x", x, xb, IN}, {"dt", dt, xb, IN}, {"A_log", A_log, (size_t)D * d_state * 4, IN}, {"B", Bm, bb, IN},
                    {"C", Cm, bb, IN}, {"D_skip", D_skip, (size_t)D * 4, IN_OPT}, {"dt_bias", dt_bias, (size_t)D * 4, IN_OPT},
                    {"z", z, xb, IN_OPT}, {"S", S, (size_t)B * D * d_state * 4, OUT}, {"y", y, xb, OUT}});
    if (s != EFLA_OK) return s;
    if (B == 0) return api_ok();
    SsmArgs a{};
    a.x = x, a.dt = dt, a.z = z, a.A_log = A_log, a.Dskip = D_skip, a.dt_bias = dt_bias, a.Bm = Bm, a.Cm = Cm, a.S0 = S, a.S_T = S;
    a.y = y, a.B = B, a.T = 1, a.D = D, a.N = d_state, a.G = G, a.nseq = B, a.dtype = dtype;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_ssm_step(a), "scan step launch");
}

efla_status efla_group_norm_workspace(int rows, int L, int C, int groups, efla_dtype dtype, int backward, size_t *bytes) {
    if (!bytes) return api_fail(EFLA_ERR_INVALID_ARG, "bytes must be non-NULL");
    const efla_status s = check_group_norm(rows, L, C, groups, dtype, EFLA_ACT_NONE, 0.f);
    if (s != EFLA_OK) return s;
    *bytes = (size_t)rows * L > 0 ? gn_ws(rows, L, C, groups, dtype, backward != 0) * sizeof(float) : 0;
    return api_ok();
}

efla_status efla_group_norm(const void *x, const float *w, const float *b, void *y, float *stats, int rows, int L, int C,
                            int groups, efla_dtype dtype, efla_activation activation, float eps, void *workspace,
                            size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_group_norm(rows, L, C, groups, dtype, activation, eps);
    if (s != EFLA_OK) return s;
    size_t need = 0;
    if ((s = efla_group_norm_workspace(rows, L, C, groups, dtype, 0, &need)) != EFLA_OK) return s;
    if ((s = need_workspace(workspace, workspace_bytes, need)) != EFLA_OK) return s;
    const size_t n = (size_t)rows * L * C * es(dtype), cb = (size_t)C * 4;
    s = check_args({{"x", x, n, IN}, {"w", w, cb, IN_OPT}, {"b", b, cb, IN_OPT}, {"y", y, n, OUT, {"x"}},
                    {"stats", stats, (size_t)rows * groups * 8, OUT_OPT}, {"workspace", workspace, need, OUT_OPT}});
    if (s != EFLA_OK) return s;
    if (n == 0)  // no values have no mean: NaN
        return launched(stats && rows > 0 ? cudaMemsetAsync(stats, 0xff, (size_t)rows * groups * 8, reinterpret_cast<cudaStream_t>(stream)) : cudaSuccess,
                        "group norm of no positions");
    GroupNormArgs a{};
    a.x = x, a.w = w, a.b = b, a.y = y, a.stats = stats, a.ws = static_cast<float *>(workspace);
    a.rows = rows, a.L = L, a.C = C, a.G = groups, a.dtype = dtype, a.silu = activation == EFLA_ACT_SILU, a.eps = eps;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_group_norm(a), "group norm launch");
}

efla_status efla_group_norm_bwd(const void *x, const float *w, const float *b, const float *stats, const void *dy,
                                void *dx, float *dw, float *db, int rows, int L, int C, int groups, efla_dtype dtype,
                                efla_activation activation, void *workspace, size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_group_norm(rows, L, C, groups, dtype, activation, 0.f);
    if (s != EFLA_OK) return s;
    size_t need = 0;
    if ((s = efla_group_norm_workspace(rows, L, C, groups, dtype, 1, &need)) != EFLA_OK) return s;
    if ((s = need_workspace(workspace, workspace_bytes, need)) != EFLA_OK) return s;
    const size_t n = (size_t)rows * L * C * es(dtype), cb = (size_t)C * 4;
    s = check_args({{"x", x, n, IN}, {"w", w, cb, IN_OPT}, {"b", b, cb, IN_OPT}, {"stats", stats, n ? (size_t)rows * groups * 8 : 0, IN},
                    {"dy", dy, n, IN}, {"dx", dx, n, OUT}, {"dw", dw, cb, OUT_OPT}, {"db", db, cb, OUT_OPT},
                    {"workspace", workspace, need, OUT_OPT}});
    if (s != EFLA_OK) return s;
    GroupNormArgs a{};
    a.x = x, a.w = w, a.b = b, a.stats = const_cast<float *>(stats), a.dy = dy, a.dx = dx, a.dw = dw, a.db = db;
    a.ws = static_cast<float *>(workspace);
    a.rows = rows, a.L = L, a.C = C, a.G = groups, a.dtype = dtype, a.silu = activation == EFLA_ACT_SILU;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_group_norm_bwd(a), "group norm backward launch");
}

}  // extern "C"
