// sad_features.h -- host-side launchers of the feature-field kernels
// (internal).  Arguments are checked by the C ABI (sad_features_api.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace sad {

// a row matrix: rows of D elements, ld elements apart
struct RowsIn {
    const void *p;
    long long ld;
};
struct RowsOut {
    void *p;
    long long ld;
};

size_t route_workspace_bytes(long long n_rows, int K, int E);
cudaError_t launch_route(const int32_t *ids, long long n_rows, int K, int E, int32_t *offsets, int32_t *order,
                         int32_t *place, void *ws, cudaStream_t st);

// out[t] = sum_k w rows[at[t][k]] (out.p NULL: not wanted), dots[t][k] =
// <rows[at], other[t]> (dots NULL: not wanted); at[] outside [0, n_at) is an
// empty slot
cudaError_t launch_gather(int dtype, RowsIn rows, const int32_t *at, long long n_at, const float *w, RowsIn other,
                          long long T, int K, int D, RowsOut out, float *dots, cudaStream_t st);
// to[at[t][k]] = w x[t], dots[t][k] = <rows[at], x[t]> (dots NULL: not wanted)
cudaError_t launch_spread(int dtype, RowsIn x, const int32_t *at, long long n_at, const float *w, RowsIn rows,
                          long long T, int K, int D, RowsOut to, float *dots, cudaStream_t st);
// dF[e] = sum over e's pairs of w dout[pair / K]
size_t segment_workspace_bytes(long long n_rows, int K, int E, int D);
cudaError_t launch_segment_sums(int dtype, RowsIn dout, const float *w, const int32_t *offsets, const int32_t *order,
                                long long T, int K, int E, int D, float *dF, void *ws, cudaStream_t st);

size_t layer_norm_workspace_bytes(long long n_rows, int D);
cudaError_t launch_layer_norm(int dtype, RowsIn x, const float *gamma, const float *beta, float eps, long long T,
                              int D, RowsOut y, float *mean, float *rstd, cudaStream_t st);
cudaError_t launch_layer_norm_backward(int dtype, RowsIn dy, RowsIn x, const float *gamma, const float *mean,
                                       const float *rstd, long long T, int D, RowsOut dx, float *dgamma, float *dbeta,
                                       void *ws, cudaStream_t st);

cudaError_t launch_distill(int dtype, RowsIn z, const int32_t *tid, const float *tl, const float *rw, long long T,
                           int V, int M, float tau, float *loss, RowsOut dz, cudaStream_t st);

}  // namespace sad
