// C-ABI entry points of the gated delta rule and of the norms around it: argument validation and
// dispatch.  Declarations and the contract are in efla.h.
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "gated.cuh"
#include "mixer_norm.cuh"

using namespace efla;

namespace {

size_t es(efla_dtype t) { return t == EFLA_BF16 ? 2 : 4; }
bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(efla_dtype t) { return t == EFLA_BF16 || t == EFLA_F32; }

enum Role { IN, IN_OPT, OUT, OUT_OPT };
struct Arg {
    const char *name;
    const void *p;
    size_t bytes;
    Role role;
    const char *may_be[2] = {nullptr, nullptr};  // an output may be exactly the inputs of these names
};

// Whether output o may lie where x does: x is an input that o's contract names, at the same address.
bool may_share(const Arg &o, const Arg &x) {
    if (x.p != o.p || x.bytes != o.bytes || (x.role != IN && x.role != IN_OPT)) return false;
    for (const char *name : o.may_be)
        if (name && strcmp(name, x.name) == 0) return true;
    return false;
}

// Every non-optional argument with bytes > 0 present, every pointer 16-byte aligned, no output
// overlapping any other argument than an input it may be.
efla_status check_args(std::initializer_list<Arg> args) {
    for (const Arg &a : args) {
        if (!a.p && a.bytes > 0 && (a.role == IN || a.role == OUT))
            return api_fail(EFLA_ERR_INVALID_ARG, "%s must be non-NULL", a.name);
        if (reinterpret_cast<uintptr_t>(a.p) & 15u)
            return api_fail(EFLA_ERR_INVALID_ARG, "%s=%p is not 16-byte aligned", a.name, a.p);
    }
    for (const Arg &o : args) {
        if ((o.role != OUT && o.role != OUT_OPT) || !o.p || o.bytes == 0) continue;
        const uintptr_t o0 = reinterpret_cast<uintptr_t>(o.p), o1 = o0 + o.bytes;
        for (const Arg &x : args) {
            if (&x == &o || !x.p || x.bytes == 0 || may_share(o, x)) continue;
            const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.p), x1 = x0 + x.bytes;
            if (o0 < x1 && x0 < o1) return api_fail(EFLA_ERR_INVALID_ARG, "output %s overlaps %s", o.name, x.name);
        }
    }
    return EFLA_OK;
}

efla_status check_sizes(int B, int T, int Hk, int H, int dk, int dv, efla_dtype in, efla_dtype out, efla_update u) {
    if (B < 0 || T < 0 || H <= 0 || Hk <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "bad sizes B=%d T=%d H_k=%d H=%d", B, T, Hk, H);
    if (H % Hk) return api_fail(EFLA_ERR_INVALID_ARG, "H=%d must be a multiple of H_k=%d", H, Hk);
    if (dk <= 0 || dv <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "d_k=%d d_v=%d must be positive", dk, dv);
    if (!dim_ok(dk) || !dim_ok(dv))
        return api_fail(EFLA_ERR_UNSUPPORTED, "d_k=%d d_v=%d: supported head sizes are 32, 64, 128", dk, dv);
    if (!dtype_ok(in) || !dtype_ok(out)) return api_fail(EFLA_ERR_INVALID_ARG, "unknown dtype (in=%d, o=%d)", (int)in, (int)out);
    if (u != EFLA_UPDATE_EXACT && u != EFLA_UPDATE_EULER) return api_fail(EFLA_ERR_INVALID_ARG, "unknown update rule %d", (int)u);
    // (launch grids count units x slabs of 32 columns, and units x chunks, in 31 bits; a product of three
    // sizes may pass 64)
    constexpr long long MOST = (1LL << 31) - 1;
    const long long tok = (long long)B * T;
    if (tok > MOST || tok * H > MOST || (long long)B * H > MOST / 4)
        return api_fail(EFLA_ERR_UNSUPPORTED, "B=%d T=%d H=%d: more than 2^31-1 token-heads, or 2^29-1 heads of sequences", B, T, H);
    return EFLA_OK;
}

efla_status launched(cudaError_t e, const char *what) {
    if (e != cudaSuccess) return api_fail(EFLA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
    return api_ok();
}

efla_status need_workspace(const void *ws, size_t have, size_t need) {
    if (need > 0 && (!ws || have < need))
        return api_fail(EFLA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu at %p)", need, ws ? have : (size_t)0, ws);
    return EFLA_OK;
}

cudaError_t run_fwd(const GatedFwdArgs &a, const char **why) {
    if (gated_tc(a.in_dtype)) return launch_gated_chunk_tc(a, why);
    *why = "gated chunk kernel launch";
    return launch_gated_chunk_simt(a);
}

}  // namespace

extern "C" {

efla_status efla_gated_fwd_chunked(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                   const float *S0, const int32_t *cu_seqlens, void *o, float *S_T, int B, int T,
                                   int H_k, int H, int d_k, int d_v, int N, efla_dtype in_dtype, efla_dtype o_dtype,
                                   efla_update update, efla_stream_t stream) {
    efla_status s = check_sizes(B, T, H_k, H, d_k, d_v, in_dtype, o_dtype, update);
    if (s != EFLA_OK) return s;
    if (N < 0 || (long long)N * H > ((1LL << 31) - 1) / 4) return api_fail(EFLA_ERR_INVALID_ARG, "bad number of sequences N=%d", N);
    if (cu_seqlens ? B != 1 : N != B)
        return api_fail(EFLA_ERR_INVALID_ARG, cu_seqlens ? "cu_seqlens given with B=%d (must be 1), N=%d"
                                                         : "B=%d, N=%d: N must equal B when cu_seqlens is NULL", B, N);
    const size_t tok = (size_t)B * T, kb = tok * H_k * d_k * es(in_dtype), st = (size_t)N * H * d_k * d_v * 4;
    s = check_args({{"q", q, kb, IN}, {"k", k, kb, IN}, {"v", v, tok * H * d_v * es(in_dtype), IN}, {"g", g, tok * H * 4, IN},
                    {"beta", beta, tok * H * 4, IN}, {"S0", S0, st, IN_OPT},
                    {"cu_seqlens", cu_seqlens, cu_seqlens ? ((size_t)N + 1) * 4 : 0, IN_OPT},
                    {"o", o, tok * H * d_v * es(o_dtype), OUT}, {"S_T", S_T, st, OUT_OPT, {"S0"}}});
    if (s != EFLA_OK) return s;
    if (N == 0) return api_ok();
    GatedFwdArgs a{q, k, v, g, beta, S0, cu_seqlens, o, S_T, B, T, H_k, H, d_k, d_v, N, in_dtype, o_dtype,
                   update == EFLA_UPDATE_EULER, reinterpret_cast<cudaStream_t>(stream), device_status_ptr()};
    if (!a.status) return api_fail(EFLA_ERR_CUDA, "cannot resolve the device status word");
    const char *why = nullptr;
    const cudaError_t e = run_fwd(a, &why);
    return launched(e, why);
}

efla_status efla_gated_bwd_workspace(int B, int T, int H_k, int H, int d_k, int d_v, efla_dtype in_dtype, size_t *bytes) {
    if (!bytes) return api_fail(EFLA_ERR_INVALID_ARG, "bytes must be non-NULL");
    const efla_status s = check_sizes(B, T, H_k, H, d_k, d_v, in_dtype, in_dtype, EFLA_UPDATE_EULER);
    if (s != EFLA_OK) return s;
    *bytes = gated_ws(B, T, H_k, H, d_k, d_v, in_dtype).bytes;
    return api_ok();
}

efla_status efla_gated_fwd_chunked_train(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                         const float *S0, void *o, float *S_T, int B, int T, int H_k, int H, int d_k,
                                         int d_v, efla_dtype in_dtype, efla_update update, void *workspace,
                                         size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_sizes(B, T, H_k, H, d_k, d_v, in_dtype, in_dtype, update);
    if (s != EFLA_OK) return s;
    const size_t need = gated_ws(B, T, H_k, H, d_k, d_v, in_dtype).bytes;
    if ((s = need_workspace(workspace, workspace_bytes, need)) != EFLA_OK) return s;
    const size_t tok = (size_t)B * T, kb = tok * H_k * d_k * es(in_dtype), vb = tok * H * d_v * es(in_dtype);
    const size_t st = (size_t)B * H * d_k * d_v * 4;
    s = check_args({{"q", q, kb, IN}, {"k", k, kb, IN}, {"v", v, vb, IN}, {"g", g, tok * H * 4, IN},
                    {"beta", beta, tok * H * 4, IN}, {"S0", S0, st, IN_OPT}, {"o", o, vb, OUT}, {"S_T", S_T, st, OUT_OPT, {"S0"}},
                    {"workspace", workspace, need, OUT_OPT}});
    if (s != EFLA_OK) return s;
    if (B == 0) return api_ok();
    GatedFwdArgs a{q, k, v, g, beta, S0, nullptr, o, S_T, B, T, H_k, H, d_k, d_v, B, in_dtype, in_dtype,
                   update == EFLA_UPDATE_EULER, reinterpret_cast<cudaStream_t>(stream), device_status_ptr(),
                   T > 0 ? workspace : nullptr};
    if (!a.status) return api_fail(EFLA_ERR_CUDA, "cannot resolve the device status word");
    const char *why = nullptr;
    const cudaError_t e = run_fwd(a, &why);
    return launched(e, why);
}

efla_status efla_gated_bwd_chunked(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                   const float *S0, const void *dO, const float *dS_T, void *dq, void *dk, void *dv,
                                   float *dg, float *dbeta, float *dS0, int B, int T, int H_k, int H, int d_k, int d_v,
                                   efla_dtype in_dtype, efla_update update, int saved, void *workspace,
                                   size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_sizes(B, T, H_k, H, d_k, d_v, in_dtype, in_dtype, update);
    if (s != EFLA_OK) return s;
    const size_t need = gated_ws(B, T, H_k, H, d_k, d_v, in_dtype).bytes;
    if ((s = need_workspace(workspace, workspace_bytes, need)) != EFLA_OK) return s;
    const size_t tok = (size_t)B * T, kb = tok * H_k * d_k * es(in_dtype), vb = tok * H * d_v * es(in_dtype);
    const size_t st = (size_t)B * H * d_k * d_v * 4, gb = tok * H * 4;
    s = check_args({{"q", q, kb, IN}, {"k", k, kb, IN}, {"v", v, vb, IN}, {"g", g, gb, IN}, {"beta", beta, gb, IN},
                    {"S0", S0, st, IN_OPT}, {"dO", dO, vb, IN}, {"dS_T", dS_T, st, IN_OPT}, {"dq", dq, kb, OUT},
                    {"dk", dk, kb, OUT}, {"dv", dv, vb, OUT}, {"dg", dg, gb, OUT}, {"dbeta", dbeta, gb, OUT},
                    {"dS0", dS0, st, OUT_OPT}, {"workspace", workspace, need, OUT_OPT}});
    if (s != EFLA_OK) return s;
    if (B == 0) return api_ok();
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    int *status = device_status_ptr();
    if (!status) return api_fail(EFLA_ERR_CUDA, "cannot resolve the device status word");
    const int euler = update == EFLA_UPDATE_EULER;
    if (T > 0 && !saved) {  // the forward for its chunk states (no outputs)
        GatedFwdArgs f{q, k, v, g, beta, S0, nullptr, nullptr, nullptr, B, T, H_k, H, d_k, d_v, B, in_dtype, in_dtype,
                       euler, cs, status, workspace};
        const char *why = nullptr;
        const cudaError_t e = run_fwd(f, &why);
        if (e != cudaSuccess) return launched(e, why);
    }
    GatedBwdArgs a{q, k, v, g, beta, S0, dO, dS_T, dq, dk, dv, dg, dbeta, dS0, B, T, H_k, H, d_k, d_v, in_dtype,
                   euler, cs, status, workspace};
    const char *why = "gated backward kernel launch";
    const cudaError_t e = gated_tc(in_dtype) && T > 0 ? launch_gated_bwd_tc(a, &why) : launch_gated_bwd_simt(a);
    return launched(e, why);
}

static efla_status decode(const void *q, const void *k, const void *v, const float *g, const float *beta, float *S, void *o,
                          int B, int m, int H_k, int H, int d_k, int d_v, efla_dtype in_dtype, efla_dtype o_dtype,
                          efla_update update, efla_stream_t stream, bool step) {
    efla_status s = check_sizes(B, m, H_k, H, d_k, d_v, in_dtype, o_dtype, update);
    if (s != EFLA_OK) return s;
    const size_t tok = (size_t)B * m, kb = tok * H_k * d_k * es(in_dtype), gb = tok * H * 4;
    s = check_args({{"q", q, kb, IN}, {"k", k, kb, IN}, {"v", v, tok * H * d_v * es(in_dtype), IN}, {"g", g, gb, IN},
                    {"beta", beta, gb, IN}, {"S", S, (size_t)B * H * d_k * d_v * 4, OUT},
                    {"o", o, tok * H * d_v * es(o_dtype), OUT}});
    if (s != EFLA_OK) return s;
    if (tok == 0) return api_ok();
    GatedDecodeArgs a{q, k, v, g, beta, S, o, B, m, H_k, H, d_k, d_v, in_dtype, o_dtype, update == EFLA_UPDATE_EULER,
                      reinterpret_cast<cudaStream_t>(stream)};
    if (step) return launched(launch_gated_decode_step(a), "gated decode kernel launch");
    const char *why = "gated decode-tokens kernel launch";
    const cudaError_t e = gated_tc(in_dtype) && d_k == 128 && d_v == 128 ? launch_gated_decode_tokens_tc(a, &why) : launch_gated_decode_tokens(a);
    return launched(e, why);
}

efla_status efla_gated_decode_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                   float *S, void *o, int B, int H_k, int H, int d_k, int d_v, efla_dtype in_dtype,
                                   efla_dtype o_dtype, efla_update update, efla_stream_t stream) {
    return decode(q, k, v, g, beta, S, o, B, 1, H_k, H, d_k, d_v, in_dtype, o_dtype, update, stream, true);
}

efla_status efla_gated_decode_tokens(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                     float *S, void *o, int B, int m, int H_k, int H, int d_k, int d_v,
                                     efla_dtype in_dtype, efla_dtype o_dtype, efla_update update,
                                     efla_stream_t stream) {
    return decode(q, k, v, g, beta, S, o, B, m, H_k, H, d_k, d_v, in_dtype, o_dtype, update, stream, false);
}

static efla_status check_prep(long long tokens, int H_k, int H, int d_k, efla_dtype dtype, float scale, float eps) {
    if (tokens < 0 || H_k <= 0 || H <= 0)
        return api_fail(EFLA_ERR_INVALID_ARG, "bad sizes tokens=%lld H_k=%d H=%d", tokens, H_k, H);
    if (d_k <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "d_k=%d must be positive", d_k);
    if (!dim_ok(d_k)) return api_fail(EFLA_ERR_UNSUPPORTED, "d_k=%d: supported head sizes are 32, 64, 128", d_k);
    if (!dtype_ok(dtype)) return api_fail(EFLA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (!isfinite(scale) || !(eps >= 0.f) || !isfinite(eps))
        return api_fail(EFLA_ERR_INVALID_ARG, "scale=%g must be finite and eps=%g finite and >= 0", scale, eps);
    if (tokens > (1LL << 31) / H || tokens > (1LL << 31) / H_k)
        return api_fail(EFLA_ERR_UNSUPPORTED, "tokens=%lld times the heads exceeds 2^31", tokens);
    return EFLA_OK;
}

efla_status efla_gated_prep(const void *q, const void *k, const void *a, const void *b, const float *A_log,
                            const float *dt_bias, void *q_out, void *k_out, float *g, float *beta, long long tokens,
                            int H_k, int H, int d_k, efla_dtype dtype, float scale, float eps, efla_stream_t stream) {
    efla_status s = check_prep(tokens, H_k, H, d_k, dtype, scale, eps);
    if (s != EFLA_OK) return s;
    const size_t n = (size_t)tokens, kb = n * H_k * d_k * es(dtype), ab = n * H * es(dtype), gb = n * H * 4;
    s = check_args({{"q", q, kb, IN}, {"k", k, kb, IN}, {"a", a, ab, IN}, {"b", b, ab, IN}, {"A_log", A_log, (size_t)H * 4, IN},
                    {"dt_bias", dt_bias, (size_t)H * 4, IN}, {"q_out", q_out, kb, OUT, {"q"}}, {"k_out", k_out, kb, OUT, {"k"}},
                    {"g", g, gb, OUT}, {"beta", beta, gb, OUT}});
    if (s != EFLA_OK) return s;
    MixerPrepArgs p{};
    p.q = q, p.k = k, p.a = a, p.b = b, p.A_log = A_log, p.dt_bias = dt_bias;
    p.q_out = q_out, p.k_out = k_out, p.g_out = g, p.beta_out = beta;
    p.tokens = tokens, p.Hk = H_k, p.H = H, p.d = d_k, p.dtype = dtype, p.scale = scale, p.eps = eps;
    p.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_mixer_prep(p, false), "gated prep kernel launch");
}

efla_status efla_gated_prep_bwd_workspace(long long tokens, int H, size_t *bytes) {
    if (!bytes) return api_fail(EFLA_ERR_INVALID_ARG, "bytes must be non-NULL");
    if (tokens < 0 || H <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "bad sizes tokens=%lld H=%d", tokens, H);
    *bytes = tokens ? (size_t)mixer_prep_parts(tokens) * 2 * H * sizeof(float) : 0;
    return api_ok();
}

efla_status efla_gated_prep_bwd(const void *q, const void *k, const void *a, const void *b, const float *A_log,
                                const float *dt_bias, const void *dq_out, const void *dk_out, const float *dg,
                                const float *dbeta, void *dq, void *dk, void *da, void *db, float *dA_log,
                                float *ddt_bias, long long tokens, int H_k, int H, int d_k, efla_dtype dtype,
                                float scale, float eps, void *workspace, size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_prep(tokens, H_k, H, d_k, dtype, scale, eps);
    if (s != EFLA_OK) return s;
    size_t need = 0;
    if ((s = efla_gated_prep_bwd_workspace(tokens, H, &need)) != EFLA_OK) return s;
    if ((s = need_workspace(workspace, workspace_bytes, need)) != EFLA_OK) return s;
    const size_t n = (size_t)tokens, kb = n * H_k * d_k * es(dtype), ab = n * H * es(dtype), gb = n * H * 4, hb = (size_t)H * 4;
    s = check_args({{"q", q, kb, IN}, {"k", k, kb, IN}, {"a", a, ab, IN}, {"b", b, ab, IN}, {"A_log", A_log, hb, IN},
                    {"dt_bias", dt_bias, hb, IN}, {"dq_out", dq_out, kb, IN}, {"dk_out", dk_out, kb, IN}, {"dg", dg, gb, IN},
                    {"dbeta", dbeta, gb, IN}, {"dq", dq, kb, OUT}, {"dk", dk, kb, OUT}, {"da", da, ab, OUT},
                    {"db", db, ab, OUT}, {"dA_log", dA_log, hb, OUT}, {"ddt_bias", ddt_bias, hb, OUT},
                    {"workspace", workspace, need, OUT_OPT}});
    if (s != EFLA_OK) return s;
    MixerPrepArgs p{};
    p.q = q, p.k = k, p.a = a, p.b = b, p.A_log = A_log, p.dt_bias = dt_bias;
    p.dq_in = dq_out, p.dk_in = dk_out, p.dg_in = dg, p.dbeta_in = dbeta;
    p.dq_out = dq, p.dk_out = dk, p.da_out = da, p.db_out = db, p.dA_log = dA_log, p.ddt_bias = ddt_bias;
    p.ws = static_cast<float *>(workspace);
    p.tokens = tokens, p.Hk = H_k, p.H = H, p.d = d_k, p.dtype = dtype, p.scale = scale, p.eps = eps;
    p.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_mixer_prep(p, true), "gated prep backward launch");
}

static efla_status check_norm(long long rows, int d, efla_dtype dtype, float eps) {
    if (rows < 0 || d <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "bad sizes rows=%lld d=%d", rows, d);
    if (!dim_ok(d)) return api_fail(EFLA_ERR_UNSUPPORTED, "d=%d: supported head sizes are 32, 64, 128", d);
    if (!dtype_ok(dtype)) return api_fail(EFLA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (!(eps >= 0.f) || !isfinite(eps)) return api_fail(EFLA_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", eps);
    if (rows > (1LL << 33)) return api_fail(EFLA_ERR_UNSUPPORTED, "rows=%lld too large", rows);
    return EFLA_OK;
}

efla_status efla_norm_gate(const void *o, const void *z, const float *w, void *y, long long rows, int d,
                           efla_dtype dtype, float eps, efla_stream_t stream) {
    efla_status s = check_norm(rows, d, dtype, eps);
    if (s != EFLA_OK) return s;
    const size_t n = (size_t)rows * d * es(dtype);
    s = check_args({{"o", o, n, IN}, {"z", z, n, IN}, {"w", w, (size_t)d * 4, IN}, {"y", y, n, OUT, {"o", "z"}}});
    if (s != EFLA_OK) return s;
    NormGateArgs p{};
    p.o = o, p.z = z, p.w = w, p.y = y, p.rows = rows, p.d = d, p.dtype = dtype, p.eps = eps;
    p.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_norm_gate(p, false), "norm-gate kernel launch");
}

efla_status efla_norm_gate_bwd_workspace(int d, size_t *bytes) {
    if (!bytes) return api_fail(EFLA_ERR_INVALID_ARG, "bytes must be non-NULL");
    if (d <= 0) return api_fail(EFLA_ERR_INVALID_ARG, "d=%d must be positive", d);
    *bytes = (size_t)NORM_GATE_PARTS * d * sizeof(float);
    return api_ok();
}

efla_status efla_norm_gate_bwd(const void *o, const void *z, const float *w, const void *dy, void *d_o, void *d_z,
                               float *d_w, long long rows, int d, efla_dtype dtype, float eps, void *workspace,
                               size_t workspace_bytes, efla_stream_t stream) {
    efla_status s = check_norm(rows, d, dtype, eps);
    if (s != EFLA_OK) return s;
    size_t need = 0;
    if ((s = efla_norm_gate_bwd_workspace(d, &need)) != EFLA_OK) return s;
    if ((s = need_workspace(workspace, workspace_bytes, need)) != EFLA_OK) return s;
    const size_t n = (size_t)rows * d * es(dtype), wb = (size_t)d * 4;
    s = check_args({{"o", o, n, IN}, {"z", z, n, IN}, {"w", w, wb, IN}, {"dy", dy, n, IN}, {"d_o", d_o, n, OUT},
                    {"d_z", d_z, n, OUT}, {"d_w", d_w, wb, OUT}, {"workspace", workspace, need, OUT_OPT}});
    if (s != EFLA_OK) return s;
    NormGateArgs p{};
    p.o = o, p.z = z, p.w = w, p.dy = dy, p.do_ = d_o, p.dz = d_z, p.dw = d_w, p.rows = rows, p.d = d, p.dtype = dtype;
    p.eps = eps, p.ws = static_cast<float *>(workspace), p.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_norm_gate(p, true), "norm-gate backward launch");
}

}  // extern "C"
