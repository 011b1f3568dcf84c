// sad_exchange.cu -- rows out to their experts and back with weights
// (dispatch, combine), rows shared by an expert's pairs (blend), and their
// gradients.
//
//   gather   out[t] = sum_k w_tk R[at_tk]     combine, blend, dispatch's dx
//            dots[t][k] = <R[at_tk], G[t]>    every gradient of the weights
//   spread   S[at_tk] = w_tk x[t]             dispatch, combine's dy
//   segments dF[e] = sum_{j of e} w_j G[t_j]  blend's dF
//
// All three move rows; the arithmetic is one multiply-add per element moved.
#include "sad_features.h"
#include "sad_rows.cuh"

namespace sad {

namespace {

constexpr int THREADS = 256;
constexpr int K_MAX = 8;

// a group of 32 lanes per row
template <typename T, int VEC, bool SUM, bool DOT>
__global__ void __launch_bounds__(THREADS) gather_kernel(const T *__restrict__ R, long long ldr,
                                                         const int32_t *__restrict__ at, uint32_t n_at,
                                                         const float *__restrict__ w, const T *__restrict__ G,
                                                         long long ldg, long long n_rows, int K, int D,
                                                         T *__restrict__ out, long long ldo,
                                                         float *__restrict__ dots) {
    const int lane = threadIdx.x & 31;
    const long long t = ((long long)blockIdx.x * THREADS + threadIdx.x) >> 5;
    if (t >= n_rows) return;
    uint32_t id[K_MAX];
    float wt[K_MAX], dot[K_MAX];
#pragma unroll
    for (int k = 0; k < K_MAX; ++k) {
        id[k] = k < K ? (uint32_t)at[t * K + k] : 0xffffffffu;
        wt[k] = SUM && id[k] < n_at ? (w ? w[t * K + k] : 1.0f) : 0.0f;
        dot[k] = 0.0f;
    }
    for (int c = lane * VEC; c < D; c += 32 * VEC) {
        float acc[VEC] = {}, g[VEC] = {};
        if (DOT) {
            const Pack<T, VEC> p = load_pack<T, VEC>(G + t * ldg + c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) g[i] = p.get(i);
        }
#pragma unroll
        for (int k = 0; k < K_MAX; ++k) {
            if (id[k] >= n_at) continue;
            const Pack<T, VEC> p = load_pack<T, VEC>(R + (long long)id[k] * ldr + c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (SUM) acc[i] = fmaf(wt[k], p.get(i), acc[i]);
                if (DOT) dot[k] = fmaf(p.get(i), g[i], dot[k]);
            }
        }
        if (SUM) {
            Pack<T, VEC> p;
#pragma unroll
            for (int i = 0; i < VEC; ++i) p.set(i, acc[i]);
            store_pack<T, VEC>(out + t * ldo + c, p);
        }
    }
    if (DOT) {
#pragma unroll
        for (int k = 0; k < K_MAX; ++k) {
            const float s = group_sum<32>(dot[k]);
            if (lane == 0 && k < K) dots[t * K + k] = s;
        }
    }
}

template <typename T, int VEC, bool DOT>
__global__ void __launch_bounds__(THREADS) spread_kernel(const T *__restrict__ X, long long ldx,
                                                         const int32_t *__restrict__ at, uint32_t n_at,
                                                         const float *__restrict__ w, const T *__restrict__ R,
                                                         long long ldr, long long n_rows, int K, int D,
                                                         T *__restrict__ S, long long lds,
                                                         float *__restrict__ dots) {
    const int lane = threadIdx.x & 31;
    const long long t = ((long long)blockIdx.x * THREADS + threadIdx.x) >> 5;
    if (t >= n_rows) return;
    uint32_t id[K_MAX];
    float wt[K_MAX], dot[K_MAX];
#pragma unroll
    for (int k = 0; k < K_MAX; ++k) {
        id[k] = k < K ? (uint32_t)at[t * K + k] : 0xffffffffu;
        wt[k] = id[k] < n_at ? (w ? w[t * K + k] : 1.0f) : 0.0f;
        dot[k] = 0.0f;
    }
    for (int c = lane * VEC; c < D; c += 32 * VEC) {
        const Pack<T, VEC> x = load_pack<T, VEC>(X + t * ldx + c);
#pragma unroll
        for (int k = 0; k < K_MAX; ++k) {
            if (id[k] >= n_at) continue;
            Pack<T, VEC> p;
            if (DOT) {
                p = load_pack<T, VEC>(R + (long long)id[k] * ldr + c);
#pragma unroll
                for (int i = 0; i < VEC; ++i) dot[k] = fmaf(p.get(i), x.get(i), dot[k]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) p.set(i, wt[k] * x.get(i));
            store_pack<T, VEC>(S + (long long)id[k] * lds + c, p);
        }
    }
    if (DOT) {
#pragma unroll
        for (int k = 0; k < K_MAX; ++k) {
            const float s = group_sum<32>(dot[k]);
            if (lane == 0 && k < K) dots[t * K + k] = s;
        }
    }
}

// a warp per site
template <typename T, int VEC>
__global__ void __launch_bounds__(THREADS) segment_kernel(const T *__restrict__ G, long long ldg,
                                                          const float *__restrict__ w,
                                                          const int32_t *__restrict__ offsets,
                                                          const int32_t *__restrict__ order, uint32_t n, int K, int E,
                                                          int D, float *__restrict__ dF) {
    const int lane = threadIdx.x & 31;
    const long long e = ((long long)blockIdx.x * THREADS + threadIdx.x) >> 5;
    if (e >= E) return;
    const uint32_t lo = min((uint32_t)offsets[e], n), hi = min((uint32_t)offsets[e + 1], n);
    for (int c = lane * VEC; c < D; c += 32 * VEC) {
        float acc[VEC] = {};
        for (uint32_t s = lo; s < hi; ++s) {
            const uint32_t j = (uint32_t)order[s];
            if (j >= n) continue;
            const float wj = w[j];
            const Pack<T, VEC> p = load_pack<T, VEC>(G + (long long)(j / K) * ldg + c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = fmaf(wj, p.get(i), acc[i]);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) dF[e * D + c + i] = acc[i];
    }
}

// rows can be read 16 bytes at a time: base and row distance on 16-byte
// boundaries (D need not be: the caller adds that)
bool wide(const void *p, long long ld, int bytes) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * bytes & 15) == 0);
}

unsigned warp_blocks(long long rows) { return (unsigned)((rows + THREADS / 32 - 1) / (THREADS / 32)); }

template <typename T, int VEC>
cudaError_t gather(RowsIn rows, const int32_t *at, long long n_at, const float *w, RowsIn other, long long n, int K,
                   int D, RowsOut out, float *dots, cudaStream_t st) {
    const T *r = static_cast<const T *>(rows.p), *g = static_cast<const T *>(other.p);
    T *o = static_cast<T *>(out.p);
    const unsigned blocks = warp_blocks(n);
    if (o && dots)
        gather_kernel<T, VEC, true, true><<<blocks, THREADS, 0, st>>>(r, rows.ld, at, (uint32_t)n_at, w, g, other.ld,
                                                                      n, K, D, o, out.ld, dots);
    else if (o)
        gather_kernel<T, VEC, true, false><<<blocks, THREADS, 0, st>>>(r, rows.ld, at, (uint32_t)n_at, w, g, other.ld,
                                                                       n, K, D, o, out.ld, dots);
    else
        gather_kernel<T, VEC, false, true><<<blocks, THREADS, 0, st>>>(r, rows.ld, at, (uint32_t)n_at, w, g, other.ld,
                                                                       n, K, D, o, out.ld, dots);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t spread(RowsIn x, const int32_t *at, long long n_at, const float *w, RowsIn rows, long long n, int K,
                   int D, RowsOut to, float *dots, cudaStream_t st) {
    const T *xp = static_cast<const T *>(x.p), *r = static_cast<const T *>(rows.p);
    T *o = static_cast<T *>(to.p);
    const unsigned blocks = warp_blocks(n);
    if (dots)
        spread_kernel<T, VEC, true><<<blocks, THREADS, 0, st>>>(xp, x.ld, at, (uint32_t)n_at, w, r, rows.ld, n, K, D,
                                                                o, to.ld, dots);
    else
        spread_kernel<T, VEC, false><<<blocks, THREADS, 0, st>>>(xp, x.ld, at, (uint32_t)n_at, w, r, rows.ld, n, K, D,
                                                                 o, to.ld, dots);
    return cudaGetLastError();
}

template <typename T>
cudaError_t gather_typed(RowsIn rows, const int32_t *at, long long n_at, const float *w, RowsIn other, long long n,
                         int K, int D, RowsOut out, float *dots, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (D % V == 0 && wide(rows.p, rows.ld, sizeof(T)) && (!dots || wide(other.p, other.ld, sizeof(T))) &&
        wide(out.p, out.ld, sizeof(T)))
        return gather<T, V>(rows, at, n_at, w, other, n, K, D, out, dots, st);
    return gather<T, 1>(rows, at, n_at, w, other, n, K, D, out, dots, st);
}

template <typename T>
cudaError_t spread_typed(RowsIn x, const int32_t *at, long long n_at, const float *w, RowsIn rows, long long n, int K,
                         int D, RowsOut to, float *dots, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (D % V == 0 && wide(x.p, x.ld, sizeof(T)) && (!dots || wide(rows.p, rows.ld, sizeof(T))) &&
        wide(to.p, to.ld, sizeof(T)))
        return spread<T, V>(x, at, n_at, w, rows, n, K, D, to, dots, st);
    return spread<T, 1>(x, at, n_at, w, rows, n, K, D, to, dots, st);
}

template <typename T>
cudaError_t segments_typed(RowsIn g, const float *w, const int32_t *offsets, const int32_t *order, long long n_rows,
                           int K, int E, int D, float *dF, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const T *p = static_cast<const T *>(g.p);
    const uint32_t n = (uint32_t)(n_rows * K);
    if (D % V == 0 && wide(g.p, g.ld, sizeof(T)))
        segment_kernel<T, V><<<warp_blocks(E), THREADS, 0, st>>>(p, g.ld, w, offsets, order, n, K, E, D, dF);
    else
        segment_kernel<T, 1><<<warp_blocks(E), THREADS, 0, st>>>(p, g.ld, w, offsets, order, n, K, E, D, dF);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gather(int dtype, RowsIn rows, const int32_t *at, long long n_at, const float *w, RowsIn other,
                          long long T, int K, int D, RowsOut out, float *dots, cudaStream_t st) {
    if (dtype == 0) return gather_typed<float>(rows, at, n_at, w, other, T, K, D, out, dots, st);
    if (dtype == 1) return gather_typed<__nv_bfloat16>(rows, at, n_at, w, other, T, K, D, out, dots, st);
    return gather_typed<__half>(rows, at, n_at, w, other, T, K, D, out, dots, st);
}

cudaError_t launch_spread(int dtype, RowsIn x, const int32_t *at, long long n_at, const float *w, RowsIn rows,
                          long long T, int K, int D, RowsOut to, float *dots, cudaStream_t st) {
    if (dtype == 0) return spread_typed<float>(x, at, n_at, w, rows, T, K, D, to, dots, st);
    if (dtype == 1) return spread_typed<__nv_bfloat16>(x, at, n_at, w, rows, T, K, D, to, dots, st);
    return spread_typed<__half>(x, at, n_at, w, rows, T, K, D, to, dots, st);
}

size_t segment_workspace_bytes(long long n_rows, int K, int E, int D) {
    (void)n_rows, (void)K, (void)E, (void)D;
    return 0;
}

cudaError_t launch_segment_sums(int dtype, RowsIn dout, const float *w, const int32_t *offsets, const int32_t *order,
                                long long T, int K, int E, int D, float *dF, void *ws, cudaStream_t st) {
    (void)ws;
    if (dtype == 0) return segments_typed<float>(dout, w, offsets, order, T, K, E, D, dF, st);
    if (dtype == 1) return segments_typed<__nv_bfloat16>(dout, w, offsets, order, T, K, E, D, dF, st);
    return segments_typed<__half>(dout, w, offsets, order, T, K, E, D, dF, st);
}

}  // namespace sad
