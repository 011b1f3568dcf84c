// sad_features_api.cu -- the C ABI of the feature-field calls (include/sad.h):
// argument checks, status codes and messages.  Nothing is launched before
// every check has passed.
#include <cstdarg>
#include <cstdio>

#include "sad.h"
#include "sad_features.h"

namespace {

// one message per host thread: the calls share no context
thread_local char g_message[256] = "";

int bad(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_message, sizeof(g_message), fmt, ap);
    va_end(ap);
    return code;
}

int status(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return SAD_OK;
    return bad(SAD_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

cudaStream_t cs(sad_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int element_bytes(int dtype) { return dtype == SAD_F32 ? 4 : dtype == SAD_BF16 || dtype == SAD_F16 ? 2 : 0; }

int check_type(int dtype) {
    if (!element_bytes(dtype)) return bad(SAD_ERR_UNSUPPORTED, "unknown element type %d", dtype);
    return SAD_OK;
}

// T rows of K slots: n = T K pairs are counted in 31 bits
int check_pairs(int64_t T, int K) {
    if (T < 0) return bad(SAD_ERR_INVALID_ARG, "n_rows = %lld is negative", (long long)T);
    if (K < 1) return bad(SAD_ERR_INVALID_ARG, "K = %d is below 1", K);
    if (K > SAD_K) return bad(SAD_ERR_UNSUPPORTED, "K = %d exceeds %d", K, SAD_K);
    if (T > (int64_t)(0x7fffffff / K)) return bad(SAD_ERR_CAPACITY, "%lld rows x %d slots exceed 2^31 pairs", (long long)T, K);
    return SAD_OK;
}

int check_rows(const char *name, int dtype, const void *p, int64_t ld, int D) {
    if (!p) return bad(SAD_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, element_bytes(dtype))) return bad(SAD_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    if (ld < D) return bad(SAD_ERR_INVALID_ARG, "%s: %lld elements between rows of %d", name, (long long)ld, D);
    // the kernels count a row's bytes in 32 bits
    if (ld >= (1ll << 30)) return bad(SAD_ERR_INVALID_ARG, "%s: row distance %lld is too large", name, (long long)ld);
    return SAD_OK;
}

int check_words(const char *name, const void *p, bool required = true) {
    if (!p && required) return bad(SAD_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, 4)) return bad(SAD_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
    return SAD_OK;
}

int check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return SAD_OK;
    if (!ws) return bad(SAD_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned(ws, 16)) return bad(SAD_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    if (have < need) return bad(SAD_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", have, need);
    return SAD_OK;
}

int check_sites(int E) {
    if (E < 1 || E >= (1 << 30)) return bad(SAD_ERR_INVALID_ARG, "n_sites = %d outside [1, 2^30)", E);
    return SAD_OK;
}

int check_width(int D) {
    if (D < 1) return bad(SAD_ERR_INVALID_ARG, "D = %d is below 1", D);
    if (D >= (1 << 30)) return bad(SAD_ERR_UNSUPPORTED, "D = %d exceeds 2^30", D);
    return SAD_OK;
}

#define TRY(expr)                  \
    do {                           \
        const int r_ = (expr);     \
        if (r_ != SAD_OK) return r_; \
    } while (0)

}  // namespace

extern "C" {

const char *sad_feature_error(void) { return g_message; }

int sad_route_workspace_bytes(int64_t n_rows, int K, int n_sites, size_t *bytes) {
    if (!bytes) return bad(SAD_ERR_INVALID_ARG, "bytes is NULL");
    TRY(check_pairs(n_rows, K));
    TRY(check_sites(n_sites));
    *bytes = sad::route_workspace_bytes(n_rows, K, n_sites);
    return SAD_OK;
}

int sad_route(const int32_t *ids, int64_t n_rows, int K, int n_sites, int32_t *offsets, int32_t *order,
              int32_t *place, void *workspace, size_t workspace_bytes, sad_stream_t stream) {
    TRY(check_pairs(n_rows, K));
    TRY(check_sites(n_sites));
    TRY(check_words("ids", ids, n_rows > 0));
    TRY(check_words("offsets", offsets));
    TRY(check_words("order", order, n_rows > 0));
    TRY(check_words("place", place, n_rows > 0));
    TRY(check_workspace(workspace, workspace_bytes, sad::route_workspace_bytes(n_rows, K, n_sites)));
    return status(sad::launch_route(ids, n_rows, K, n_sites, offsets, order, place, workspace, cs(stream)), "route");
}

int sad_dispatch(int dtype, const void *x, int64_t ldx, const float *weights, const int32_t *place, int64_t n_rows,
                 int K, int D, void *xs, int64_t ldxs, sad_stream_t stream) {
    TRY(check_type(dtype));
    TRY(check_pairs(n_rows, K));
    TRY(check_width(D));
    if (n_rows == 0) return SAD_OK;
    TRY(check_rows("x", dtype, x, ldx, D));
    TRY(check_rows("xs", dtype, xs, ldxs, D));
    TRY(check_words("weights", weights, false));
    TRY(check_words("place", place));
    return status(sad::launch_spread(dtype, {x, ldx}, place, n_rows * K, weights, {nullptr, 0}, n_rows, K, D,
                                     {xs, ldxs}, nullptr, cs(stream)),
                  "dispatch");
}

int sad_dispatch_backward(int dtype, const void *dxs, int64_t lddxs, const void *x, int64_t ldx,
                          const float *weights, const int32_t *place, int64_t n_rows, int K, int D, void *dx,
                          int64_t lddx, float *dweights, sad_stream_t stream) {
    TRY(check_type(dtype));
    TRY(check_pairs(n_rows, K));
    TRY(check_width(D));
    if (n_rows == 0) return SAD_OK;
    TRY(check_rows("dxs", dtype, dxs, lddxs, D));
    TRY(check_rows("dx", dtype, dx, lddx, D));
    if (dweights) TRY(check_rows("x", dtype, x, ldx, D));
    TRY(check_words("weights", weights, false));
    TRY(check_words("place", place));
    TRY(check_words("dweights", dweights, false));
    return status(sad::launch_gather(dtype, {dxs, lddxs}, place, n_rows * K, weights, {x, ldx}, n_rows, K, D,
                                     {dx, lddx}, dweights, cs(stream)),
                  "dispatch backward");
}

int sad_combine(int dtype, const void *y, int64_t ldy, const float *weights, const int32_t *place, int64_t n_rows,
                int K, int D, void *out, int64_t ldout, sad_stream_t stream) {
    TRY(check_type(dtype));
    TRY(check_pairs(n_rows, K));
    TRY(check_width(D));
    if (n_rows == 0) return SAD_OK;
    TRY(check_rows("y", dtype, y, ldy, D));
    TRY(check_rows("out", dtype, out, ldout, D));
    TRY(check_words("weights", weights, false));
    TRY(check_words("place", place));
    return status(sad::launch_gather(dtype, {y, ldy}, place, n_rows * K, weights, {nullptr, 0}, n_rows, K, D,
                                     {out, ldout}, nullptr, cs(stream)),
                  "combine");
}

int sad_combine_backward(int dtype, const void *dout, int64_t lddout, const void *y, int64_t ldy,
                         const float *weights, const int32_t *place, int64_t n_rows, int K, int D, void *dy,
                         int64_t lddy, float *dweights, sad_stream_t stream) {
    TRY(check_type(dtype));
    TRY(check_pairs(n_rows, K));
    TRY(check_width(D));
    if (n_rows == 0) return SAD_OK;
    TRY(check_rows("dout", dtype, dout, lddout, D));
    TRY(check_rows("dy", dtype, dy, lddy, D));
    if (dweights) TRY(check_rows("y", dtype, y, ldy, D));
    TRY(check_words("weights", weights, false));
    TRY(check_words("place", place));
    TRY(check_words("dweights", dweights, false));
    return status(sad::launch_spread(dtype, {dout, lddout}, place, n_rows * K, weights, {y, ldy}, n_rows, K, D,
                                     {dy, lddy}, dweights, cs(stream)),
                  "combine backward");
}

int sad_blend(int dtype, const void *F, int64_t ldf, int n_sites, const int32_t *ids, const float *weights,
              int64_t n_rows, int K, int D, void *out, int64_t ldout, sad_stream_t stream) {
    TRY(check_type(dtype));
    TRY(check_pairs(n_rows, K));
    TRY(check_sites(n_sites));
    TRY(check_width(D));
    if (n_rows == 0) return SAD_OK;
    TRY(check_rows("F", dtype, F, ldf, D));
    TRY(check_rows("out", dtype, out, ldout, D));
    TRY(check_words("ids", ids));
    TRY(check_words("weights", weights));
    return status(sad::launch_gather(dtype, {F, ldf}, ids, n_sites, weights, {nullptr, 0}, n_rows, K, D,
                                     {out, ldout}, nullptr, cs(stream)),
                  "blend");
}

int sad_blend_workspace_bytes(int64_t n_rows, int K, int n_sites, int D, size_t *bytes) {
    if (!bytes) return bad(SAD_ERR_INVALID_ARG, "bytes is NULL");
    TRY(check_pairs(n_rows, K));
    TRY(check_sites(n_sites));
    TRY(check_width(D));
    *bytes = sad::segment_workspace_bytes(n_rows, K, n_sites, D);
    return SAD_OK;
}

int sad_blend_backward(int dtype, const void *dout, int64_t lddout, const void *F, int64_t ldf, int n_sites,
                       const int32_t *ids, const float *weights, const int32_t *offsets, const int32_t *order,
                       int64_t n_rows, int K, int D, float *dF, float *dweights, void *workspace,
                       size_t workspace_bytes, sad_stream_t stream) {
    TRY(check_type(dtype));
    TRY(check_pairs(n_rows, K));
    TRY(check_sites(n_sites));
    TRY(check_width(D));
    if (n_rows > 0) {
        TRY(check_rows("dout", dtype, dout, lddout, D));
        TRY(check_words("weights", weights));
        if (dweights) {
            TRY(check_rows("F", dtype, F, ldf, D));
            TRY(check_words("ids", ids));
            TRY(check_words("dweights", dweights));
        }
    }
    if (dF) {
        TRY(check_words("dF", dF));
        if (n_rows > 0) {
            TRY(check_words("offsets", offsets));
            TRY(check_words("order", order));
        }
        TRY(check_workspace(workspace, workspace_bytes, sad::segment_workspace_bytes(n_rows, K, n_sites, D)));
    }
    cudaError_t e = cudaSuccess;
    if (dF && n_rows == 0) e = cudaMemsetAsync(dF, 0, sizeof(float) * (size_t)n_sites * D, cs(stream));
    if (n_rows > 0 && dweights)
        e = sad::launch_gather(dtype, {F, ldf}, ids, n_sites, nullptr, {dout, lddout}, n_rows, K, D, {nullptr, 0},
                               dweights, cs(stream));
    if (e == cudaSuccess && n_rows > 0 && dF)
        e = sad::launch_segment_sums(dtype, {dout, lddout}, weights, offsets, order, n_rows, K, n_sites, D, dF,
                                     workspace, cs(stream));
    return status(e, "blend backward");
}

int sad_layer_norm(int dtype, const void *x, int64_t ldx, const float *gamma, const float *beta, float eps,
                   int64_t n_rows, int D, void *y, int64_t ldy, float *mean, float *rstd, sad_stream_t stream) {
    TRY(check_type(dtype));
    if (n_rows < 0 || n_rows > 0x7fffffff) return bad(SAD_ERR_INVALID_ARG, "n_rows = %lld outside [0, 2^31)", (long long)n_rows);
    if (D < 1) return bad(SAD_ERR_INVALID_ARG, "D = %d is below 1", D);
    if (D > SAD_NORM_MAX_D) return bad(SAD_ERR_UNSUPPORTED, "D = %d exceeds %d", D, SAD_NORM_MAX_D);
    if (!(eps >= 0.0f)) return bad(SAD_ERR_INVALID_ARG, "eps must be >= 0");
    if (n_rows == 0) return SAD_OK;
    TRY(check_rows("x", dtype, x, ldx, D));
    TRY(check_rows("y", dtype, y, ldy, D));
    TRY(check_words("gamma", gamma, false));
    TRY(check_words("beta", beta, false));
    TRY(check_words("mean", mean, false));
    TRY(check_words("rstd", rstd, false));
    if (x == y && ldx != ldy) return bad(SAD_ERR_INVALID_ARG, "y is x with another row distance");
    return status(sad::launch_layer_norm(dtype, {x, ldx}, gamma, beta, eps, n_rows, D, {y, ldy}, mean, rstd, cs(stream)),
                  "layer norm");
}

int sad_layer_norm_workspace_bytes(int64_t n_rows, int D, size_t *bytes) {
    if (!bytes) return bad(SAD_ERR_INVALID_ARG, "bytes is NULL");
    if (n_rows < 0 || n_rows > 0x7fffffff) return bad(SAD_ERR_INVALID_ARG, "n_rows = %lld outside [0, 2^31)", (long long)n_rows);
    if (D < 1) return bad(SAD_ERR_INVALID_ARG, "D = %d is below 1", D);
    if (D > SAD_NORM_MAX_D) return bad(SAD_ERR_UNSUPPORTED, "D = %d exceeds %d", D, SAD_NORM_MAX_D);
    *bytes = sad::layer_norm_workspace_bytes(n_rows, D);
    return SAD_OK;
}

int sad_layer_norm_backward(int dtype, const void *dy, int64_t lddy, const void *x, int64_t ldx, const float *gamma,
                            const float *mean, const float *rstd, int64_t n_rows, int D, void *dx, int64_t lddx,
                            float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes,
                            sad_stream_t stream) {
    TRY(check_type(dtype));
    if (n_rows < 0 || n_rows > 0x7fffffff) return bad(SAD_ERR_INVALID_ARG, "n_rows = %lld outside [0, 2^31)", (long long)n_rows);
    if (D < 1) return bad(SAD_ERR_INVALID_ARG, "D = %d is below 1", D);
    if (D > SAD_NORM_MAX_D) return bad(SAD_ERR_UNSUPPORTED, "D = %d exceeds %d", D, SAD_NORM_MAX_D);
    if (!dgamma != !dbeta) return bad(SAD_ERR_INVALID_ARG, "dgamma and dbeta are given together or not at all");
    TRY(check_words("dgamma", dgamma, false));
    TRY(check_words("dbeta", dbeta, false));
    if (n_rows == 0) {
        cudaError_t e = cudaSuccess;
        if (dgamma) e = cudaMemsetAsync(dgamma, 0, sizeof(float) * (size_t)D, cs(stream));
        if (dgamma && e == cudaSuccess) e = cudaMemsetAsync(dbeta, 0, sizeof(float) * (size_t)D, cs(stream));
        return status(e, "layer norm backward");
    }
    TRY(check_rows("dy", dtype, dy, lddy, D));
    TRY(check_rows("x", dtype, x, ldx, D));
    TRY(check_rows("dx", dtype, dx, lddx, D));
    TRY(check_words("gamma", gamma, false));
    TRY(check_words("mean", mean));
    TRY(check_words("rstd", rstd));
    if (dx == dy && lddx != lddy) return bad(SAD_ERR_INVALID_ARG, "dx is dy with another row distance");
    if (dgamma) TRY(check_workspace(workspace, workspace_bytes, sad::layer_norm_workspace_bytes(n_rows, D)));
    return status(sad::launch_layer_norm_backward(dtype, {dy, lddy}, {x, ldx}, gamma, mean, rstd, n_rows, D,
                                                  {dx, lddx}, dgamma, dbeta, workspace, cs(stream)),
                  "layer norm backward");
}

int sad_distill(int dtype, const void *logits, int64_t ld, const int32_t *teacher_ids, const float *teacher_logits,
                const float *row_weight, int64_t n_rows, int V, int M, float tau, float *loss, void *dlogits,
                int64_t lddlogits, sad_stream_t stream) {
    TRY(check_type(dtype));
    if (n_rows < 0 || n_rows > 0x7fffffff) return bad(SAD_ERR_INVALID_ARG, "n_rows = %lld outside [0, 2^31)", (long long)n_rows);
    if (V < 1 || V >= (1 << 30)) return bad(SAD_ERR_INVALID_ARG, "V = %d outside [1, 2^30)", V);
    if (M < 1) return bad(SAD_ERR_INVALID_ARG, "M = %d is below 1", M);
    if (M > SAD_DISTILL_MAX_M) return bad(SAD_ERR_UNSUPPORTED, "M = %d exceeds %d", M, SAD_DISTILL_MAX_M);
    // 1 / tau has to be a normal number too
    if (!(tau >= 1e-30f && tau <= 1e30f)) return bad(SAD_ERR_INVALID_ARG, "tau must lie in [1e-30, 1e30]");
    if (n_rows == 0) return SAD_OK;
    TRY(check_rows("logits", dtype, logits, ld, V));
    if (dlogits) TRY(check_rows("dlogits", dtype, dlogits, lddlogits, V));
    if (dlogits == logits && ld != lddlogits) return bad(SAD_ERR_INVALID_ARG, "dlogits is logits with another row distance");
    TRY(check_words("teacher_ids", teacher_ids));
    TRY(check_words("teacher_logits", teacher_logits));
    TRY(check_words("row_weight", row_weight, false));
    TRY(check_words("loss", loss));
    return status(sad::launch_distill(dtype, {logits, ld}, teacher_ids, teacher_logits, row_weight, n_rows, V, M, tau,
                                      loss, {dlogits, lddlogits}, cs(stream)),
                  "distill");
}

}  // extern "C"
