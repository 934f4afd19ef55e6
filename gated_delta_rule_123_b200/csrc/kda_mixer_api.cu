// extern "C" entry points of the selective mixer's operators: host-side argument
// validation, then launches on the caller's stream.  Declared and documented in
// include/kda.h.
#include "kda_scan.cuh"

namespace kda {

static bool bad_dtype(int dtype) { return dtype != KDA_BF16 && dtype != KDA_FP32; }
// Pointers of the element type are aligned to it.
static bool aligned_es(const void* p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == KDA_BF16 ? 1u : 3u)) == 0;
}
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// Row and column counts leave room for the kernels' rounding up in 32 bits.
static bool too_long(int a, int b, int c = 0) { return a > 0x7fffff00 || b > 0x7fffff00 || c > 0x7fffff00; }
// (the launchers of the norm, the convolution and the scan leave the runtime's error here to be taken)
static int launched(int rc) {
    return rc == KDA_OK ? KDA_OK : fail(rc, cudaGetErrorString(cudaGetLastError()));
}
// Token axis checks shared by the convolution and the scan: sequence count and tokens.
static int check_tokens(const int32_t* cu, int num_seqs, int B, int T, int* nseq, int* tokens) {
    if (B < 0 || T < 0) return fail(KDA_ERR_INVALID_ARG, "negative size");
    if (cu) {
        if (B != 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens requires B == 1");
        if (num_seqs < 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens requires num_seqs >= 1");
        if (!aligned4(cu)) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens must be 4-byte aligned");
    } else if (num_seqs != 0) {
        return fail(KDA_ERR_INVALID_ARG, "num_seqs must be 0 for dense input");
    }
    if ((long long)B * T > 0x7fffff00ll) return fail(KDA_ERR_UNSUPPORTED, "more than 2^31 tokens");
    *nseq = cu ? num_seqs : B;
    *tokens = B * T;
    return KDA_OK;
}
static int check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return KDA_OK;
    if (!ws || have < need) return fail(KDA_ERR_WORKSPACE, "workspace NULL or smaller than the matching query");
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    return KDA_OK;
}
// A new state from an old one, for calls without tokens.
static int pass_state(void* out, const void* in, size_t bytes, cudaStream_t s) {
    if (!out || bytes == 0 || out == in) return KDA_OK;
    const cudaError_t e = in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(out, 0, bytes, s);
    return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
}
static int zero_out(void* out, size_t bytes, cudaStream_t s) { return pass_state(out, nullptr, bytes, s); }

static int check_scan(const kda_scan_params* w) {
    if (!w) return fail(KDA_ERR_INVALID_ARG, "NULL parameters");
    if (w->channels < 0 || w->groups < 1 || w->state < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes");
    if (w->channels % w->groups) return fail(KDA_ERR_INVALID_ARG, "channels must be a multiple of groups");
    if (w->state > 32) return fail(KDA_ERR_UNSUPPORTED, "more than 32 states per channel");
    if (w->channels > 0 && !w->A) return fail(KDA_ERR_INVALID_ARG, "NULL A");
    if (!aligned4(w->A) || !aligned4(w->D) || !aligned4(w->dt_bias))
        return fail(KDA_ERR_INVALID_ARG, "fp32 pointers must be 4-byte aligned");
    return KDA_OK;
}

}  // namespace kda

extern "C" {

int kda_layer_norm_fwd(const void* x, long long ldx, const float* weight, const float* bias, void* y, long long ldy,
                       float* mean, float* rstd, int M, int N, int dtype, float eps, void* stream) {
    t_last_error[0] = 0;
    if (bad_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "dtype must be KDA_BF16 or KDA_FP32");
    if (M < 0 || N < 1) return fail(KDA_ERR_INVALID_ARG, "M must not be negative and N must be positive");
    if (too_long(M, N)) return fail(KDA_ERR_UNSUPPORTED, "more than 2^31 - 256 rows or columns");
    if (M == 0) return KDA_OK;
    if (!x || !y) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (ldx < N || ldy < N) return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    if (!aligned_es(x, dtype) || !aligned_es(y, dtype) || !aligned4(weight) || !aligned4(bias) || !aligned4(mean) ||
        !aligned4(rstd))
        return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (x == y) return fail(KDA_ERR_INVALID_ARG, "y must not alias x");
    return launched(launch_layer_norm_fwd(x, ldx, weight, bias, y, ldy, mean, rstd, M, N, dtype, eps,
                                          static_cast<cudaStream_t>(stream)));
}

size_t kda_layer_norm_bwd_workspace(int M, int N) {
    return M <= 0 || N <= 0 ? 0 : layer_norm_bwd_workspace_bytes(M, N);
}

int kda_layer_norm_bwd(const void* dy, long long lddy, const void* x, long long ldx, const float* weight,
                       const float* mean, const float* rstd, void* dx, long long lddx, float* dweight, float* dbias,
                       int M, int N, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    t_last_error[0] = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (bad_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "dtype must be KDA_BF16 or KDA_FP32");
    if (M < 0 || N < 1) return fail(KDA_ERR_INVALID_ARG, "M must not be negative and N must be positive");
    if (too_long(M, N)) return fail(KDA_ERR_UNSUPPORTED, "more than 2^31 - 256 rows or columns");
    if (!aligned4(weight) || !aligned4(mean) || !aligned4(rstd) || !aligned4(dweight) || !aligned4(dbias))
        return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (M == 0) {
        const int rc = zero_out(dweight, size_t(N) * 4, s);
        return rc != KDA_OK ? rc : zero_out(dbias, size_t(N) * 4, s);
    }
    if (!dy || !x || !mean || !rstd || !dx) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (lddy < N || ldx < N || lddx < N) return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    if (!aligned_es(dy, dtype) || !aligned_es(x, dtype) || !aligned_es(dx, dtype))
        return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (dx == dy || dx == x) return fail(KDA_ERR_INVALID_ARG, "dx must not alias dy or x");
    if (dweight || dbias) {
        const int rc = check_workspace(workspace, workspace_bytes, layer_norm_bwd_workspace_bytes(M, N));
        if (rc != KDA_OK) return rc;
    }
    return launched(launch_layer_norm_bwd(dy, lddy, x, ldx, weight, mean, rstd, dx, lddx, dweight, dbias, M, N, dtype,
                                          workspace, s));
}

int kda_linear_act_bf16(const void* x, int ldx, const void* W, int ldw, const float* bias, const void* residual,
                        int ldr, void* y, int ldy, void* pre, int ldp, int M, int N, int K, int act, void* stream) {
    t_last_error[0] = 0;
    if (M < 0 || N < 0 || K < 0) return fail(KDA_ERR_INVALID_ARG, "negative size");
    if (too_long(M, N, K)) return fail(KDA_ERR_UNSUPPORTED, "more than 2^31 - 256 rows or columns");
    if (act < KDA_ACT_NONE || act > KDA_ACT_SOFTPLUS) return fail(KDA_ERR_INVALID_ARG, "unknown activation");
    if ((long long)M * N == 0) return KDA_OK;
    if (K == 0) return fail(KDA_ERR_UNSUPPORTED, "K must be positive");
    if (!x || !W || !y) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (ldx < K || ldw < K || ldy < N || (residual && ldr < N) || (pre && ldp < N))
        return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    if (!aligned16(x) || !aligned16(W) || !aligned16(y) || ldx % 8 || ldw % 8 || ldy % 8 ||
        (pre && (!aligned16(pre) || ldp % 8)))
        return fail(KDA_ERR_INVALID_ARG, "pointers and row strides must be 16-byte aligned");
    if (!aligned_es(residual, KDA_BF16) || !aligned4(bias))
        return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (y == x || y == W || y == residual || (pre && (pre == x || pre == W || pre == residual || pre == y)))
        return fail(KDA_ERR_INVALID_ARG, "outputs must not alias inputs or each other");
    const char* why = "";
    const int rc = launch_linear_act(x, ldx, W, ldw, bias, residual, ldr, y, ldy, pre, ldp, M, N, K, act,
                                     static_cast<cudaStream_t>(stream), &why);
    return rc == KDA_OK ? KDA_OK : fail(rc, why);
}

size_t kda_linear_act_bwd_workspace(int M, int N) {
    return M <= 0 || N <= 0 ? 0 : linear_act_bwd_workspace_bytes(M, N);
}

int kda_linear_act_bwd_bf16(const void* dy, int lddy, const void* x, int ldx, const void* W, int ldw, const void* pre,
                            int ldp, void* dx, int lddx, void* dW, int lddw, float* dbias, int M, int N, int K, int act,
                            void* workspace, size_t workspace_bytes, void* stream) {
    t_last_error[0] = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M < 0 || N < 0 || K < 0) return fail(KDA_ERR_INVALID_ARG, "negative size");
    if (too_long(M, N, K)) return fail(KDA_ERR_UNSUPPORTED, "more than 2^31 - 256 rows or columns");
    if (act < KDA_ACT_NONE || act > KDA_ACT_SOFTPLUS) return fail(KDA_ERR_INVALID_ARG, "unknown activation");
    if (!aligned4(dbias)) return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (K == 0 && (long long)M * N != 0) return fail(KDA_ERR_UNSUPPORTED, "K must be positive");
    if ((dx && lddx < K) || (dW && lddw < K)) return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    if (M == 0 || N == 0) {  // sums over nothing
        cudaError_t e = cudaSuccess;
        if (dx && M > 0 && K > 0) e = cudaMemset2DAsync(dx, size_t(lddx) * 2, 0, size_t(K) * 2, M, s);
        if (e == cudaSuccess && dW && N > 0 && K > 0) e = cudaMemset2DAsync(dW, size_t(lddw) * 2, 0, size_t(K) * 2, N, s);
        if (e == cudaSuccess && dbias && N > 0) e = cudaMemsetAsync(dbias, 0, size_t(N) * 4, s);
        return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, cudaGetErrorString(e));
    }
    if (!dy || (dW && !x) || (dx && !W) || (act != KDA_ACT_NONE && !pre))
        return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (lddy < N || (dW && ldx < K) || (dx && ldw < K) || (act != KDA_ACT_NONE && ldp < N))
        return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    if ((dW && (!aligned16(x) || ldx % 8 || !aligned16(dW) || lddw % 8)) ||
        (dx && (!aligned16(W) || ldw % 8 || !aligned16(dx) || lddx % 8)))
        return fail(KDA_ERR_INVALID_ARG, "pointers and row strides must be 16-byte aligned");
    if (!aligned_es(dy, KDA_BF16) || (act != KDA_ACT_NONE && !aligned_es(pre, KDA_BF16)))
        return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    for (const void* o : {static_cast<const void*>(dx), static_cast<const void*>(dW)})
        if (o && (o == dy || o == x || o == W || o == pre)) return fail(KDA_ERR_INVALID_ARG, "outputs must not alias inputs");
    if (dx && dx == dW) return fail(KDA_ERR_INVALID_ARG, "outputs must not alias each other");
    const int wc = check_workspace(workspace, workspace_bytes, linear_act_bwd_workspace_bytes(M, N));
    if (wc != KDA_OK) return wc;
    const char* why = "";
    const int rc = launch_linear_act_bwd(dy, lddy, x, ldx, W, ldw, act == KDA_ACT_NONE ? nullptr : pre, ldp, dx, lddx,
                                         dW, lddw, dbias, M, N, K, act, workspace, s, &why);
    return rc == KDA_OK ? KDA_OK : fail(rc, why);
}

int kda_short_conv_fwd(const void* x, long long ldx, const void* w, const float* bias, void* y, long long ldy,
                       const void* conv_state_in, void* conv_state_out, const int32_t* cu_seqlens, int num_seqs, int B,
                       int T, int C, int width, int dtype, int silu, void* stream) {
    t_last_error[0] = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int nseq = 0, tokens = 0;
    if (bad_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "dtype must be KDA_BF16 or KDA_FP32");
    if (C < 0) return fail(KDA_ERR_INVALID_ARG, "negative size");
    if (width < 2 || width > 4) return fail(KDA_ERR_UNSUPPORTED, "width must be 2, 3 or 4");
    const int tc = check_tokens(cu_seqlens, num_seqs, B, T, &nseq, &tokens);
    if (tc != KDA_OK) return tc;
    if (C == 0 || nseq == 0) return KDA_OK;
    if (!aligned_es(x, dtype) || !aligned_es(w, dtype) || !aligned_es(y, dtype) || !aligned4(bias) ||
        !aligned_es(conv_state_in, dtype) || !aligned_es(conv_state_out, dtype))
        return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (tokens == 0)
        return pass_state(conv_state_out, conv_state_in, size_t(nseq) * (width - 1) * C * (dtype == KDA_BF16 ? 2 : 4), s);
    if (!x || !w || !y) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (ldx < C || ldy < C) return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    if (y == x || y == w) return fail(KDA_ERR_INVALID_ARG, "y must not alias x or w");
    return launched(launch_short_conv_fwd(x, ldx, w, bias, y, ldy, conv_state_in, conv_state_out, cu_seqlens, nseq, T,
                                          tokens, C, width, dtype, silu != 0, s));
}

size_t kda_short_conv_bwd_workspace(int tokens, int C, int width) {
    return tokens <= 0 || C <= 0 || width < 2 || width > 4 ? 0 : short_conv_bwd_workspace_bytes(tokens, C, width);
}

int kda_short_conv_bwd(const void* dy, long long lddy, const void* x, long long ldx, const void* w, const float* bias,
                       const void* conv_state_in, const void* d_conv_state_out, void* dx, long long lddx, void* dw,
                       float* dbias, void* d_conv_state_in, const int32_t* cu_seqlens, int num_seqs, int B, int T,
                       int C, int width, int dtype, int silu, void* workspace, size_t workspace_bytes, void* stream) {
    t_last_error[0] = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int nseq = 0, tokens = 0;
    const int es = dtype == KDA_BF16 ? 2 : 4;
    if (bad_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "dtype must be KDA_BF16 or KDA_FP32");
    if (C < 0) return fail(KDA_ERR_INVALID_ARG, "negative size");
    if (width < 2 || width > 4) return fail(KDA_ERR_UNSUPPORTED, "width must be 2, 3 or 4");
    const int tc = check_tokens(cu_seqlens, num_seqs, B, T, &nseq, &tokens);
    if (tc != KDA_OK) return tc;
    if (C == 0) return KDA_OK;
    const void* ps[] = {dy, x, w, conv_state_in, d_conv_state_out, dx, dw, d_conv_state_in};
    for (const void* q : ps)
        if (!aligned_es(q, dtype)) return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (!aligned4(bias) || !aligned4(dbias)) return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (tokens == 0) {
        int rc = pass_state(d_conv_state_in, d_conv_state_out, size_t(nseq) * (width - 1) * C * es, s);
        if (rc == KDA_OK) rc = zero_out(dw, size_t(C) * width * es, s);
        return rc == KDA_OK ? zero_out(dbias, size_t(C) * 4, s) : rc;
    }
    if (!dy || !x || !w || !dx) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (lddy < C || ldx < C || lddx < C) return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    if (dx == dy || dx == x || dx == w || (d_conv_state_in && d_conv_state_in == d_conv_state_out))
        return fail(KDA_ERR_INVALID_ARG, "outputs must not alias inputs");
    const int wc = check_workspace(workspace, workspace_bytes, short_conv_bwd_workspace_bytes(tokens, C, width));
    if (wc != KDA_OK) return wc;
    return launched(launch_short_conv_bwd(dy, lddy, x, ldx, w, bias, conv_state_in, d_conv_state_out, dx, lddx, dw,
                                          dbias, d_conv_state_in, cu_seqlens, nseq, T, tokens, C, width, dtype,
                                          silu != 0, workspace, s));
}

int kda_short_conv_step(const void* x, long long ldx, const void* w, const float* bias, void* conv_state, void* y,
                        long long ldy, int B, int C, int width, int dtype, int silu, void* stream) {
    t_last_error[0] = 0;
    if (bad_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "dtype must be KDA_BF16 or KDA_FP32");
    if (B < 0 || C < 0) return fail(KDA_ERR_INVALID_ARG, "negative size");
    if (width < 2 || width > 4) return fail(KDA_ERR_UNSUPPORTED, "width must be 2, 3 or 4");
    if ((long long)B * C == 0) return KDA_OK;
    if ((long long)B * C > (1ll << 37)) return fail(KDA_ERR_UNSUPPORTED, "too many sequences and channels");
    if (!x || !w || !conv_state || !y) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (ldx < C || ldy < C) return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    if (!aligned_es(x, dtype) || !aligned_es(w, dtype) || !aligned_es(conv_state, dtype) || !aligned_es(y, dtype) ||
        !aligned4(bias))
        return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (y == x || y == w || y == conv_state || conv_state == x)
        return fail(KDA_ERR_INVALID_ARG, "x, y and conv_state must not alias each other");
    return launched(launch_short_conv_step(x, ldx, w, bias, conv_state, y, ldy, B, C, width, dtype, silu != 0,
                                           static_cast<cudaStream_t>(stream)));
}

size_t kda_selective_scan_fwd_workspace(int B, int T, int channels, int groups, int state, int num_seqs) {
    if (B <= 0 || T <= 0 || channels <= 0 || groups <= 0 || state <= 0 || state > 32 || channels % groups || num_seqs < 0)
        return 0;
    return selective_scan_fwd_workspace_bytes(B, T, channels, groups, state, num_seqs);
}

int kda_selective_scan_fwd(const void* u, long long ldu, const void* dt, long long lddt, const void* B, long long ldb,
                           const void* C, long long ldc, const void* z, long long ldz, const kda_scan_params* params,
                           const float* initial_state, float* final_state, void* y, long long ldy,
                           const int32_t* cu_seqlens, int num_seqs, int batch, int T, int dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
    t_last_error[0] = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int nseq = 0, tokens = 0;
    if (bad_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "dtype must be KDA_BF16 or KDA_FP32");
    int rc = check_scan(params);
    if (rc != KDA_OK) return rc;
    rc = check_tokens(cu_seqlens, num_seqs, batch, T, &nseq, &tokens);
    if (rc != KDA_OK) return rc;
    const int D = params->channels, N = params->state, G = params->groups;
    if (D == 0 || nseq == 0) return KDA_OK;
    if (!aligned4(initial_state) || !aligned4(final_state))
        return fail(KDA_ERR_INVALID_ARG, "fp32 pointers must be 4-byte aligned");
    if (tokens == 0) return pass_state(final_state, initial_state, size_t(nseq) * D * N * 4, s);
    if (!u || !dt || !B || !C || !y) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (ldu < D || lddt < D || ldy < D || (z && ldz < D) || ldb < (long long)G * N || ldc < (long long)G * N)
        return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    const void* ps[] = {u, dt, B, C, z, y};
    for (const void* q : ps)
        if (!aligned_es(q, dtype)) return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (y == u || y == dt || y == B || y == C || y == z) return fail(KDA_ERR_INVALID_ARG, "y must not alias an input");
    if (!cu_seqlens && batch > 65535) return fail(KDA_ERR_UNSUPPORTED, "more than 65535 rows: pack them (cu_seqlens)");
    rc = check_workspace(workspace, workspace_bytes, selective_scan_fwd_workspace_bytes(batch, T, D, G, N, num_seqs));
    if (rc != KDA_OK) return rc;
    scan::SArgs a{};
    a.u = u; a.ldu = ldu; a.dt = dt; a.lddt = lddt; a.Bm = B; a.ldb = ldb; a.Cm = C; a.ldc = ldc; a.z = z; a.ldz = ldz;
    a.A = params->A; a.skip = params->D; a.bias = params->dt_bias; a.softplus = params->dt_softplus != 0;
    a.h0 = initial_state; a.hT = final_state; a.y = y; a.ldy = ldy;
    a.cu = cu_seqlens; a.nseq = nseq; a.seq_len = T; a.ntok = tokens; a.D = D; a.G = G; a.N = N; a.Dg = D / G;
    return launched(launch_selective_scan_fwd(a, batch, T, dtype, workspace, s));
}

size_t kda_selective_scan_bwd_workspace(int B, int T, int channels, int groups, int state, int num_seqs) {
    if (B <= 0 || T <= 0 || channels <= 0 || groups <= 0 || state <= 0 || state > 32 || channels % groups || num_seqs < 0)
        return 0;
    return selective_scan_bwd_workspace_bytes(B, T, channels, groups, state, num_seqs > 0);
}

int kda_selective_scan_bwd(const void* dy, long long lddy, const void* u, long long ldu, const void* dt, long long lddt,
                           const void* B, long long ldb, const void* C, long long ldc, const void* z, long long ldz,
                           const kda_scan_params* params, const float* initial_state, const float* d_final_state,
                           void* du, long long lddu, void* ddt, long long ldddt, void* dB, long long lddb, void* dC,
                           long long lddc, void* dz, long long lddz, float* dA, float* dD, float* ddt_bias,
                           float* d_initial_state, const int32_t* cu_seqlens, int num_seqs, int batch, int T, int dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
    t_last_error[0] = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int nseq = 0, tokens = 0;
    if (bad_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "dtype must be KDA_BF16 or KDA_FP32");
    int rc = check_scan(params);
    if (rc != KDA_OK) return rc;
    rc = check_tokens(cu_seqlens, num_seqs, batch, T, &nseq, &tokens);
    if (rc != KDA_OK) return rc;
    const int D = params->channels, N = params->state, G = params->groups;
    if (D == 0) return KDA_OK;
    const float* fs[] = {initial_state, d_final_state, dA, dD, ddt_bias, d_initial_state};
    for (const float* q : fs)
        if (!aligned4(q)) return fail(KDA_ERR_INVALID_ARG, "fp32 pointers must be 4-byte aligned");
    if (!dA) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (tokens == 0) {
        rc = pass_state(d_initial_state, d_final_state, size_t(nseq) * D * N * 4, s);
        if (rc == KDA_OK) rc = zero_out(dA, size_t(D) * N * 4, s);
        if (rc == KDA_OK) rc = zero_out(dD, size_t(D) * 4, s);
        return rc == KDA_OK ? zero_out(ddt_bias, size_t(D) * 4, s) : rc;
    }
    if (!dy || !u || !dt || !B || !C || !du || !ddt || !dB || !dC || (z && !dz))
        return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    const long long GN = (long long)G * N;
    if (lddy < D || ldu < D || lddt < D || (z && (ldz < D || lddz < D)) || ldb < GN || ldc < GN || lddu < D ||
        ldddt < D || lddb < GN || lddc < GN)
        return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    const void* in[] = {dy, u, dt, B, C, z};
    const void* out[] = {du, ddt, dB, dC, z ? dz : nullptr};
    for (const void* q : in)
        if (!aligned_es(q, dtype)) return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    for (int i = 0; i < 5; ++i) {
        if (!aligned_es(out[i], dtype)) return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
        for (const void* q : in)
            if (out[i] && out[i] == q) return fail(KDA_ERR_INVALID_ARG, "outputs must not alias inputs");
        for (int j = 0; j < i; ++j)
            if (out[i] && out[i] == out[j]) return fail(KDA_ERR_INVALID_ARG, "outputs must not alias each other");
    }
    if (d_initial_state && (d_initial_state == d_final_state || d_initial_state == initial_state))
        return fail(KDA_ERR_INVALID_ARG, "d_initial_state must not alias an input");
    if (!cu_seqlens && batch > 65535) return fail(KDA_ERR_UNSUPPORTED, "more than 65535 rows: pack them (cu_seqlens)");
    rc = check_workspace(workspace, workspace_bytes, selective_scan_bwd_workspace_bytes(batch, T, D, G, N, cu_seqlens != nullptr));
    if (rc != KDA_OK) return rc;
    scan::SArgs a{};
    a.u = u; a.ldu = ldu; a.dt = dt; a.lddt = lddt; a.Bm = B; a.ldb = ldb; a.Cm = C; a.ldc = ldc; a.z = z; a.ldz = ldz;
    a.dy = dy; a.lddy = lddy;
    a.A = params->A; a.skip = params->D; a.bias = params->dt_bias; a.softplus = params->dt_softplus != 0;
    a.h0 = initial_state; a.dhT = d_final_state; a.dh0 = d_initial_state;
    a.du = du; a.lddu = lddu; a.ddt = ddt; a.ldddt = ldddt; a.dz = z ? dz : nullptr; a.lddz = lddz;
    a.cu = cu_seqlens; a.nseq = nseq; a.seq_len = T; a.ntok = tokens; a.D = D; a.G = G; a.N = N; a.Dg = D / G;
    const scan::BwdOut o{dB, dC, lddb, lddc, dA, dD, ddt_bias};
    return launched(launch_selective_scan_bwd(a, o, batch, T, dtype, workspace, s));
}

int kda_selective_scan_step(const void* u, long long ldu, const void* dt, long long lddt, const void* B, long long ldb,
                            const void* C, long long ldc, const void* z, long long ldz, const kda_scan_params* params,
                            float* state, void* y, long long ldy, int batch, int dtype, void* stream) {
    t_last_error[0] = 0;
    if (bad_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "dtype must be KDA_BF16 or KDA_FP32");
    const int rc = check_scan(params);
    if (rc != KDA_OK) return rc;
    if (batch < 0) return fail(KDA_ERR_INVALID_ARG, "negative size");
    const int D = params->channels, N = params->state, G = params->groups;
    if ((long long)batch * D == 0) return KDA_OK;
    if ((long long)batch * D > (1ll << 36)) return fail(KDA_ERR_UNSUPPORTED, "too many sequences and channels");
    if (!u || !dt || !B || !C || !state || !y) return fail(KDA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (ldu < D || lddt < D || ldy < D || (z && ldz < D) || ldb < (long long)G * N || ldc < (long long)G * N)
        return fail(KDA_ERR_INVALID_ARG, "row stride smaller than the row");
    const void* ps[] = {u, dt, B, C, z, y};
    for (const void* q : ps)
        if (!aligned_es(q, dtype)) return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their element type");
    if (!aligned4(state)) return fail(KDA_ERR_INVALID_ARG, "fp32 pointers must be 4-byte aligned");
    if (y == u || y == dt || y == B || y == C || y == z || y == state)
        return fail(KDA_ERR_INVALID_ARG, "y must not alias an input");
    scan::SArgs a{};
    a.u = u; a.ldu = ldu; a.dt = dt; a.lddt = lddt; a.Bm = B; a.ldb = ldb; a.Cm = C; a.ldc = ldc; a.z = z; a.ldz = ldz;
    a.A = params->A; a.skip = params->D; a.bias = params->dt_bias; a.softplus = params->dt_softplus != 0;
    a.y = y; a.ldy = ldy; a.rows = batch; a.D = D; a.G = G; a.N = N; a.Dg = D / G;
    return launched(launch_selective_scan_step(a, state, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
