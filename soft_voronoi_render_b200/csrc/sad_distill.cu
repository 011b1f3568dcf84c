// sad_distill.cu -- distillation from a teacher's top logits: the divergence
// of the student's softmax from the teacher's over the M classes that it
// hands out, and the gradient of the student's logits.
//
// With q = softmax(teacher / tau) over the counting entries and p =
// softmax(z / tau): loss = rw tau^2 sum_m q_m (ln q_m - ln p[id_m]) and dz_v =
// rw tau (p_v - sum of q_m over id_m = v).  Floor: z once in, dz once out.
#include "sad_features.h"
#include "sad_rows.cuh"

namespace sad {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int M_MAX = 128;

// maximum in which a NaN wins, so that a row of NaN does not pass for an empty one
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float block_reduce_sum(float v, float *scratch) {
    v = group_sum<32>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < WARPS; ++q) s += scratch[q];
    return s;
}

__device__ __forceinline__ float block_reduce_max(float v, float *scratch) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = scratch[0];
#pragma unroll
    for (int q = 1; q < WARPS; ++q) s = max_nan(s, scratch[q]);
    return s;
}

// a block per row; the row is read again for the sum and for the gradient
template <typename T>
__global__ void __launch_bounds__(THREADS) distill_kernel(const T *z, long long ldz, const int32_t *__restrict__ tid,
                                                          const float *__restrict__ tl,
                                                          const float *__restrict__ rw, int V, int M, float tau,
                                                          float *__restrict__ loss, T *dz, long long lddz) {
    __shared__ float scratch[WARPS];
    __shared__ int32_t id[M_MAX];
    __shared__ float q[M_MAX], zid[M_MAX];
    constexpr float INF = __builtin_huge_valf();
    const long long t = blockIdx.x;
    const T *row = z + t * ldz;
    const float it = 1.0f / tau;
    const float weight = rw ? rw[t] : 1.0f;
    const int m = threadIdx.x;

    // the teacher's side: q over the counting entries
    float l = -INF;
    if (m < M) {
        id[m] = tid[t * M + m];
        if ((uint32_t)id[m] < (uint32_t)V) {
            l = tl[t * M + m] * it;
            zid[m] = to_f32<T>(row[id[m]]) * it;
        }
    }
    const bool counts = l != -INF;  // a NaN logit of a valid class counts, and shows
    const float tmax = block_reduce_max(l, scratch);
    const float e = counts ? expf(l - tmax) : 0.0f;
    const float tsum = block_reduce_sum(e, scratch);
    const bool any = __syncthreads_or(counts);

    // the student's side: the largest logit and the sum of exponentials
    float big = -INF;
    for (int c = threadIdx.x; c < V; c += THREADS) big = max_nan(big, to_f32<T>(row[c]) * it);
    big = block_reduce_max(big, scratch);
    if (!any || weight == 0.0f || big == -INF) {
        if (threadIdx.x == 0) loss[t] = 0.0f;
        if (dz)
            for (int c = threadIdx.x; c < V; c += THREADS) dz[t * lddz + c] = from_f32<T>(0.0f);
        return;
    }
    float s = 0.0f;
    for (int c = threadIdx.x; c < V; c += THREADS) s += expf(to_f32<T>(row[c]) * it - big);
    s = block_reduce_sum(s, scratch);

    float part = 0.0f, qm = 0.0f;
    if (counts) {
        qm = e / tsum;
        // ln q - ln p with both maxima taken out first
        if (qm != 0.0f) part = qm * ((l - tmax) - logf(tsum) - (zid[m] - big) + logf(s));
    }
    if (m < M) {
        q[m] = qm;
        if (!counts) id[m] = -1;
    }
    part = block_reduce_sum(part, scratch);
    if (threadIdx.x == 0) loss[t] = weight * tau * tau * part;
    if (!dz) return;
    const float scale = weight * tau, is = 1.0f / s;
    for (int c = threadIdx.x; c < V; c += THREADS)
        dz[t * lddz + c] = from_f32<T>(scale * (expf(to_f32<T>(row[c]) * it - big) * is));
    __syncthreads();
    // the teacher's classes, from p in float32; an id listed twice gets the
    // same value from each of its entries
    if (m < M && counts) {
        float sum = 0.0f;
        for (int k = 0; k < M; ++k)
            if (id[k] == id[m]) sum += q[k];
        dz[t * lddz + id[m]] = from_f32<T>(scale * (expf(zid[m] - big) * is - sum));
    }
}

template <typename T>
cudaError_t distill(RowsIn z, const int32_t *tid, const float *tl, const float *rw, long long n, int V, int M,
                    float tau, float *loss, RowsOut dz, cudaStream_t st) {
    distill_kernel<T><<<(unsigned)n, THREADS, 0, st>>>(static_cast<const T *>(z.p), z.ld, tid, tl, rw, V, M, tau, loss,
                                                       static_cast<T *>(dz.p), dz.ld);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_distill(int dtype, RowsIn z, const int32_t *tid, const float *tl, const float *rw, long long T,
                           int V, int M, float tau, float *loss, RowsOut dz, cudaStream_t st) {
    if (dtype == 0) return distill<float>(z, tid, tl, rw, T, V, M, tau, loss, dz, st);
    if (dtype == 1) return distill<__nv_bfloat16>(z, tid, tl, rw, T, V, M, tau, loss, dz, st);
    return distill<__half>(z, tid, tl, rw, T, V, M, tau, loss, dz, st);
}

}  // namespace sad
