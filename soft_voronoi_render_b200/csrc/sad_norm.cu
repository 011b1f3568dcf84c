// sad_norm.cu -- layer norm of rows, forward and backward, with the gradients
// of its scale and shift.
//
// Forward, per row: mean, variance about that mean, y = (x - mean) rstd gamma
// + beta.  Backward, with g = dy gamma and h = (x - mean) rstd: dx = rstd (g -
// mean(g) - h mean(g h)), dgamma = sum over rows of dy h, dbeta = sum of dy.
// Floor: x and y once forward; dy, x and dx once backward.
#include "sad_features.h"
#include "sad_rows.cuh"

namespace sad {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int SUM_BLOCKS = 148;  // row runs of the dgamma, dbeta sums

// sum over the block, the same bits in every thread
__device__ __forceinline__ float block_sum(float v, float *scratch) {
    v = group_sum<32>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < WARPS; ++q) s += scratch[q];
    return s;
}

// a block per row; the row is read from L1 or L2 after the first time
template <typename T>
__global__ void __launch_bounds__(THREADS) norm_kernel(const T *x, long long ldx, const float *__restrict__ gamma,
                                                       const float *__restrict__ beta, float eps, int D, T *y,
                                                       long long ldy, float *__restrict__ mean,
                                                       float *__restrict__ rstd) {
    __shared__ float scratch[WARPS];
    const long long r = blockIdx.x;
    const T *row = x + r * ldx;
    float s = 0.0f;
    for (int c = threadIdx.x; c < D; c += THREADS) s += to_f32<T>(row[c]);
    const float m = block_sum(s, scratch) / (float)D;
    s = 0.0f;
    for (int c = threadIdx.x; c < D; c += THREADS) {
        const float d = to_f32<T>(row[c]) - m;
        s = fmaf(d, d, s);
    }
    const float rs = 1.0f / sqrtf(block_sum(s, scratch) / (float)D + eps);
    for (int c = threadIdx.x; c < D; c += THREADS) {
        const float h = (to_f32<T>(row[c]) - m) * rs;
        y[r * ldy + c] = from_f32<T>(fmaf(h, gamma ? gamma[c] : 1.0f, beta ? beta[c] : 0.0f));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[r] = m;
        if (rstd) rstd[r] = rs;
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) norm_dx_kernel(const T *dy, long long lddy,
                                                          const T *__restrict__ x, long long ldx,
                                                          const float *__restrict__ gamma,
                                                          const float *__restrict__ mean,
                                                          const float *__restrict__ rstd, int D, T *dx,
                                                          long long lddx) {
    __shared__ float scratch[WARPS];
    const long long r = blockIdx.x;
    const float m = mean[r], rs = rstd[r];
    float a = 0.0f, b = 0.0f;
    for (int c = threadIdx.x; c < D; c += THREADS) {
        const float g = to_f32<T>(dy[r * lddy + c]) * (gamma ? gamma[c] : 1.0f);
        a += g;
        b = fmaf(g, (to_f32<T>(x[r * ldx + c]) - m) * rs, b);
    }
    a = block_sum(a, scratch) / (float)D;
    b = block_sum(b, scratch) / (float)D;
    for (int c = threadIdx.x; c < D; c += THREADS) {
        const float g = to_f32<T>(dy[r * lddy + c]) * (gamma ? gamma[c] : 1.0f);
        const float h = (to_f32<T>(x[r * ldx + c]) - m) * rs;
        dx[r * lddx + c] = from_f32<T>(rs * (g - a - h * b));
    }
}

// partial sums over a run of rows, a thread per column
template <typename T>
__global__ void __launch_bounds__(THREADS) norm_sums_kernel(const T *__restrict__ dy, long long lddy,
                                                            const T *__restrict__ x, long long ldx,
                                                            const float *__restrict__ mean,
                                                            const float *__restrict__ rstd, long long n, int D,
                                                            float *__restrict__ partial) {
    const int c = blockIdx.x * THREADS + threadIdx.x;
    if (c >= D) return;
    float g = 0.0f, b = 0.0f;
    for (long long r = blockIdx.y; r < n; r += SUM_BLOCKS) {
        const float v = to_f32<T>(dy[r * lddy + c]);
        b += v;
        g = fmaf(v, (to_f32<T>(x[r * ldx + c]) - mean[r]) * rstd[r], g);
    }
    partial[(size_t)(2 * blockIdx.y) * D + c] = g;
    partial[(size_t)(2 * blockIdx.y + 1) * D + c] = b;
}

__global__ void __launch_bounds__(THREADS) norm_final_kernel(const float *__restrict__ partial, int D,
                                                             float *__restrict__ dgamma, float *__restrict__ dbeta) {
    const int c = blockIdx.x * THREADS + threadIdx.x;
    if (c >= D) return;
    float g = 0.0f, b = 0.0f;
    for (int q = 0; q < SUM_BLOCKS; ++q) {
        g += partial[(size_t)(2 * q) * D + c];
        b += partial[(size_t)(2 * q + 1) * D + c];
    }
    dgamma[c] = g;
    dbeta[c] = b;
}

template <typename T>
cudaError_t backward(RowsIn dy, RowsIn x, const float *gamma, const float *mean, const float *rstd, long long n,
                     int D, RowsOut dx, float *dgamma, float *dbeta, float *partial, cudaStream_t st) {
    const T *dyp = static_cast<const T *>(dy.p), *xp = static_cast<const T *>(x.p);
    // the sums first: dx may take the place of dy
    if (dgamma) {
        const unsigned cols = (unsigned)((D + THREADS - 1) / THREADS);
        norm_sums_kernel<T><<<dim3(cols, SUM_BLOCKS), THREADS, 0, st>>>(dyp, dy.ld, xp, x.ld, mean, rstd, n, D,
                                                                        partial);
        norm_final_kernel<<<cols, THREADS, 0, st>>>(partial, D, dgamma, dbeta);
    }
    norm_dx_kernel<T><<<(unsigned)n, THREADS, 0, st>>>(dyp, dy.ld, xp, x.ld, gamma, mean, rstd, D,
                                                       static_cast<T *>(dx.p), dx.ld);
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward(RowsIn x, const float *gamma, const float *beta, float eps, long long n, int D, RowsOut y,
                    float *mean, float *rstd, cudaStream_t st) {
    norm_kernel<T><<<(unsigned)n, THREADS, 0, st>>>(static_cast<const T *>(x.p), x.ld, gamma, beta, eps, D,
                                                    static_cast<T *>(y.p), y.ld, mean, rstd);
    return cudaGetLastError();
}

}  // namespace

size_t layer_norm_workspace_bytes(long long n_rows, int D) {
    (void)n_rows;
    return sizeof(float) * 2 * SUM_BLOCKS * (size_t)D;
}

cudaError_t launch_layer_norm(int dtype, RowsIn x, const float *gamma, const float *beta, float eps, long long T,
                              int D, RowsOut y, float *mean, float *rstd, cudaStream_t st) {
    if (dtype == 0) return forward<float>(x, gamma, beta, eps, T, D, y, mean, rstd, st);
    if (dtype == 1) return forward<__nv_bfloat16>(x, gamma, beta, eps, T, D, y, mean, rstd, st);
    return forward<__half>(x, gamma, beta, eps, T, D, y, mean, rstd, st);
}

cudaError_t launch_layer_norm_backward(int dtype, RowsIn dy, RowsIn x, const float *gamma, const float *mean,
                                       const float *rstd, long long T, int D, RowsOut dx, float *dgamma, float *dbeta,
                                       void *ws, cudaStream_t st) {
    float *p = static_cast<float *>(ws);
    if (dtype == 0) return backward<float>(dy, x, gamma, mean, rstd, T, D, dx, dgamma, dbeta, p, st);
    if (dtype == 1) return backward<__nv_bfloat16>(dy, x, gamma, mean, rstd, T, D, dx, dgamma, dbeta, p, st);
    return backward<__half>(dy, x, gamma, mean, rstd, T, D, dx, dgamma, dbeta, p, st);
}

}  // namespace sad
