// sad_distill.cu -- distillation from a teacher's top logits: the divergence
// of the student's softmax from the teacher's over the M classes that it
// hands out, and the gradient of the student's logits.
//
// With q = softmax(teacher / tau) over the counting entries and p =
// softmax(z / tau): loss = rw tau^2 sum_m q_m (ln q_m - ln p[id_m]) and dz_v =
// rw tau (p_v - sum of q_m over id_m = v).  Exponentials are taken to base 2
// of z log2(e) / tau, about the row's maximum, in float32.
//
// Bound by memory where rows are read and written once; the exponentials (16
// a clock on a multiprocessor) come next.  Short rows (up to 8 pieces of at
// most 16 bytes for each lane of a group of L <= 32) stay in registers,
// several rows a warp.  Longer rows are shared by a block, which keeps its
// part in shared memory from the first pass (running maximum and sum of every
// thread) to the second (gradient); a row beyond 100 KB, or one of few rows,
// by a cluster of up to eight blocks that join maxima and sums through
// distributed shared memory.  Rows start at any element: the pieces begin at
// the row's first 16-byte boundary, and the elements before and behind them
// are taken one by one.
#include <cooperative_groups.h>

#include "sad_features.h"
#include "sad_rows.cuh"

namespace sad {

namespace {

namespace cg = cooperative_groups;

constexpr int SMS = 148;
constexpr int M_MAX = 128;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// maximum in which a NaN wins, so that a row of NaN does not pass for an empty one
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 2^x, within 2 ulp, below the normal range 0 (far under the rounding of any
// sum that it enters)
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float minus_infinity() { return __int_as_float(0xff800000); }

// A maximum to subtract: 0 for a row, or part of one, of nothing but -infinity
__device__ __forceinline__ float finite_max(float m) { return m == minus_infinity() ? 0.0f : m; }

__device__ __forceinline__ float lanes_sum(float v, int L) {
    for (int o = L >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float lanes_max(float v, int L) {
    for (int o = L >> 1; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The teacher's side of a row, by a group of L lanes; entries m of the row in
// shared memory.
struct Teacher {
    int32_t *id;  // -1: does not count
    float *q;     // first the logit (base 2), then the probability
    float *zid;   // the student's logit of the class (base 2)
    float max, sum;
    bool any;
};

template <typename T>
__device__ __forceinline__ void teacher_load(Teacher &t, const int32_t *__restrict__ tid, const float *__restrict__ tl,
                                             const T *row, int V, int M, float k, bool in, int lane, int L) {
    float big = minus_infinity();
    bool any = false;
    for (int m = lane; m < M; m += L) {
        int32_t id = in ? __ldg(tid + m) : -1;
        float l = minus_infinity(), z = 0.0f;
        if ((uint32_t)id < (uint32_t)V) {
            l = __ldg(tl + m) * k;
            z = to_f32<T>(row[id]) * k;
        }
        if (l == minus_infinity()) id = -1;  // a NaN logit of a valid class counts, and shows
        any = any || id >= 0;
        big = max_nan(big, l);
        t.id[m] = id;
        t.q[m] = l;
        t.zid[m] = z;
    }
    t.max = big;
    t.any = any;
}

__device__ __forceinline__ void teacher_softmax(Teacher &t, int M, int lane, int L) {
    t.max = lanes_max(t.max, L);
    int any = t.any;
    for (int o = L >> 1; o; o >>= 1) any |= __shfl_xor_sync(0xffffffffu, any, o);
    t.any = any;
    float s = 0.0f;
    const float m0 = finite_max(t.max);
    for (int m = lane; m < M; m += L) s += exp2_fast(t.q[m] - m0);
    t.sum = lanes_sum(s, L);
}

// the row's divergence (before rw tau^2), given the student's maximum and sum;
// leaves q in shared memory
__device__ __forceinline__ float teacher_loss(Teacher &t, int M, int lane, int L, float big, float sum) {
    const float is = 1.0f / t.sum, lt = log2f(t.sum), ls = log2f(sum);
    const float m0 = finite_max(t.max);
    float part = 0.0f;
    for (int m = lane; m < M; m += L) {
        float q = 0.0f;
        if (t.id[m] >= 0) {
            const float l = t.q[m] - m0;
            q = exp2_fast(l) * is;
            // ln q - ln p with both maxima taken out first
            if (q != 0.0f) part = fmaf(q, (l - lt) - ((t.zid[m] - big) - ls), part);
        }
        t.q[m] = q;
    }
    return lanes_sum(part, L) * LN2;
}

// gradient of entry m's class, all of its entries counted
__device__ __forceinline__ float teacher_grad(const Teacher &t, int M, int m, float big, float inv_sum, float scale) {
    const int32_t id = t.id[m];
    float q = 0.0f;
    for (int j = 0; j < M; ++j)
        if (t.id[j] == id) q += t.q[j];
    return scale * (exp2_fast(t.zid[m] - big) * inv_sum - q);
}

// ---------------------------------------------------------------------------
// short rows
// ---------------------------------------------------------------------------
constexpr int GROUP_THREADS = 256;

template <typename T, int VEC, int NV, bool GRAD>
__global__ void __launch_bounds__(GROUP_THREADS) distill_group_kernel(
    const T *z, long long ldz, const int32_t *__restrict__ tid, const float *__restrict__ tl,
    const float *__restrict__ rw, long long n, int V, int M, float tau, int log_l, float *__restrict__ loss, T *dz,
    long long lddz) {
    extern __shared__ float teacher_space[];
    const int L = 1 << log_l, lane = threadIdx.x & (L - 1), group = threadIdx.x >> log_l;
    const int c0 = lane * VEC, step = L * VEC;
    const long long t = ((long long)blockIdx.x * GROUP_THREADS + threadIdx.x) >> log_l;
    const bool in = t < n;
    const float k = LOG2E / tau;
    const T *row = z + t * ldz;
    Pack<T, VEC> p[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in && c0 + i * step < V) p[i] = load_pack<T, VEC>(row + c0 + i * step);
    const float weight = in ? (rw ? __ldg(rw + t) : 1.0f) : 0.0f;
    Teacher te;
    float *space = teacher_space + (size_t)group * M * 3;
    te.id = reinterpret_cast<int32_t *>(space);
    te.q = space + M;
    te.zid = space + 2 * M;
    teacher_load<T>(te, tid + t * M, tl + t * M, row, V, M, k, in, lane, L);
    teacher_softmax(te, M, lane, L);

    float e[NV * VEC];
    float big = minus_infinity();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool on = in && c0 + i * step < V;
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            e[i * VEC + q] = on ? p[i].get(q) * k : minus_infinity();
            big = max_nan(big, e[i * VEC + q]);
        }
    }
    big = lanes_max(big, L);
    const bool live = te.any && weight != 0.0f && big != minus_infinity();
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        e[i] = exp2_fast(e[i] - big);
        sum += e[i];
    }
    sum = lanes_sum(sum, L);
    const float part = teacher_loss(te, M, lane, L, big, sum);
    if (lane == 0 && in) loss[t] = live ? weight * tau * tau * part : 0.0f;
    if (!GRAD) return;
    const float scale = weight * tau, is = 1.0f / sum, f = scale * is;
    T *out = dz + t * lddz;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * step;
        if (!in || c >= V) continue;
        float g[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) g[q] = live ? e[i * VEC + q] * f : 0.0f;
        Pack<T, VEC> o;
        o.set(g);
        store_pack<T, VEC>(out + c, o);
    }
    __syncwarp();
    // the teacher's classes once more, from float32: an id listed twice gets
    // the same value from each of its entries
    if (live)
        for (int m = lane; m < M; m += L)
            if (te.id[m] >= 0) out[te.id[m]] = from_f32<T>(teacher_grad(te, M, m, big, is, scale));
}

// ---------------------------------------------------------------------------
// long rows: a block or a cluster each
// ---------------------------------------------------------------------------
constexpr int LONG_THREADS = 512;

template <typename T, bool GRAD, bool CACHE>
__global__ void __launch_bounds__(LONG_THREADS) distill_long_kernel(
    const T *z, long long ldz, const int32_t *__restrict__ tid, const float *__restrict__ tl,
    const float *__restrict__ rw, int V, int M, float tau, int each, float *__restrict__ loss, T *dz,
    long long lddz) {
    constexpr int VEC = 16 / sizeof(T), UNROLL = 4;
    extern __shared__ uint4 cache[];
    __shared__ int32_t s_id[M_MAX];
    __shared__ float s_q[M_MAX], s_zid[M_MAX];
    __shared__ float s_max[LONG_THREADS / 32], s_sum[LONG_THREADS / 32];
    __shared__ float block_max, block_sum, t_any;
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const long long t = blockIdx.x / ranks;
    const T *row = z + t * ldz;
    const float k = LOG2E / tau;
    const float weight = rw ? __ldg(rw + t) : 1.0f;

    // elements before the first 16-byte boundary, whole pieces, elements behind
    const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
    const int pieces = (V - head) / VEC, tail = V - head - pieces * VEC;
    const int first = min(rank * each, pieces), last = min(first + each, pieces);
    const uint4 *body = reinterpret_cast<const uint4 *>(row + head);

    Teacher te{s_id, s_q, s_zid, 0.0f, 0.0f, false};
    if (warp == 0) {
        teacher_load<T>(te, tid + t * M, tl + t * M, row, V, M, k, true, lane, 32);
        teacher_softmax(te, M, lane, 32);
        if (lane == 0) t_any = te.any ? 1.0f : 0.0f;
    }

    // each thread's running maximum and sum of exponentials about it
    float big = minus_infinity(), sum = 0.0f;
    auto take = [&](const float *a, int count) {
        float m = big;
        for (int i = 0; i < count; ++i) m = max_nan(m, a[i]);
        const float m0 = finite_max(m);
        sum *= exp2_fast(big - m0);  // big = -inf: sum is 0
        for (int i = 0; i < count; ++i) sum += exp2_fast(a[i] - m0);
        big = m;
    };
    // one of the elements outside the pieces, for one thread of the first block
    const int edge = rank ? V : (int)threadIdx.x < head ? (int)threadIdx.x
                              : (int)threadIdx.x < head + tail ? V - tail + (int)threadIdx.x - head : V;
    float edge_z = 0.0f;
    if (edge < V) {
        edge_z = to_f32<T>(row[edge]) * k;
        take(&edge_z, 1);
    }
    for (int c = first + threadIdx.x; c < last; c += UNROLL * blockDim.x) {
        Pack<T, VEC> p[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (c + u * (int)blockDim.x < last)
                p[u] = load_pack<T, VEC>(reinterpret_cast<const T *>(body + c + u * blockDim.x));
        float a[UNROLL * VEC];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const bool on = c + u * (int)blockDim.x < last;
            if (GRAD && CACHE && on) cache[c + u * blockDim.x - first] = *reinterpret_cast<const uint4 *>(&p[u]);
#pragma unroll
            for (int q = 0; q < VEC; ++q) a[u * VEC + q] = on ? p[u].get(q) * k : minus_infinity();
        }
        float m = big;
#pragma unroll
        for (int i = 0; i < UNROLL * VEC; ++i) m = max_nan(m, a[i]);
        const float m0 = finite_max(m);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < UNROLL * VEC; ++i) s += exp2_fast(a[i] - m0);
        sum = fmaf(sum, exp2_fast(big - m0), s);
        big = m;
    }

    // joined over the warps, then over the cluster
    {
        const float m = lanes_max(big, 32);
        const float s = lanes_sum(sum * exp2_fast(big - finite_max(m)), 32);
        if (lane == 0) s_max[warp] = m, s_sum[warp] = s;
    }
    __syncthreads();
    {
        const float wm = lane < warps ? s_max[lane] : minus_infinity(), ws = lane < warps ? s_sum[lane] : 0.0f;
        big = lanes_max(wm, 32);
        sum = lanes_sum(ws * exp2_fast(wm - finite_max(big)), 32);
    }
    if (ranks > 1) {
        if (threadIdx.x == 0) block_max = big, block_sum = sum;
        cluster.sync();
        const float wm = lane < ranks ? *cluster.map_shared_rank(&block_max, lane) : minus_infinity();
        const float ws = lane < ranks ? *cluster.map_shared_rank(&block_sum, lane) : 0.0f;
        big = lanes_max(wm, 32);
        sum = lanes_sum(ws * exp2_fast(wm - finite_max(big)), 32);
        cluster.sync();  // no block leaves, or writes a class that another still reads, before all have read
    }
    const bool live = t_any != 0.0f && weight != 0.0f && big != minus_infinity();
    if (warp == 0) {
        const float part = teacher_loss(te, M, lane, 32, big, sum);
        if (lane == 0 && rank == 0) loss[t] = live ? weight * tau * tau * part : 0.0f;
    }
    if (!GRAD) return;
    const float scale = weight * tau, is = 1.0f / sum, f = scale * is;
    T *out = dz + t * lddz;
    const bool same_phase = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row)) & 15) == 0;
    if (edge < V) out[edge] = from_f32<T>(live ? exp2_fast(edge_z - big) * f : 0.0f);
    for (int c = first + threadIdx.x; c < last; c += UNROLL * blockDim.x) {
        Pack<T, VEC> p[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int at = c + u * (int)blockDim.x;
            if (at < last)
                p[u] = load_pack<T, VEC>(reinterpret_cast<const T *>(CACHE ? cache + at - first : body + at));
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int at = c + u * (int)blockDim.x;
            if (at >= last) continue;
            float g[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) g[q] = live ? exp2_fast(fmaf(p[u].get(q), k, -big)) * f : 0.0f;
            T *to = out + head + (long long)at * VEC;
            if (same_phase) {
                Pack<T, VEC> o;
                o.set(g);
                store_pack<T, VEC>(to, o);
            } else {
#pragma unroll
                for (int q = 0; q < VEC; ++q) to[q] = from_f32<T>(g[q]);
            }
        }
    }
    __syncthreads();
    // the teacher's classes in this block's part, from float32
    if (live && threadIdx.x < M && s_id[threadIdx.x] >= 0) {
        const int id = s_id[threadIdx.x];
        const int piece = id < head || id >= V - tail ? -1 : (id - head) / VEC;
        if (piece < 0 ? rank == 0 : (piece >= first && piece < last))
            out[id] = from_f32<T>(teacher_grad(te, M, threadIdx.x, big, is, scale));
    }
}

// the piece that a row at any of the n row starts can be read in
int row_piece(const void *p, long long ld, int V, int bytes) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * bytes) | (uintptr_t)((long long)V * bytes);
    return (all & 15) == 0 ? 16 : (all & 7) == 0 ? 8 : (all & 3) == 0 ? 4 : bytes;
}

struct Args {
    const int32_t *tid;
    const float *tl, *rw;
    long long n;
    int V, M;
    float tau;
    float *loss;
};

template <typename T, int VEC, int NV>
cudaError_t group_launch(RowsIn z, RowsOut dz, const Args &a, int log_l, cudaStream_t st) {
    const int groups = GROUP_THREADS >> log_l;
    const unsigned blocks = (unsigned)((a.n + groups - 1) / groups);
    const size_t shared = sizeof(float) * 3 * groups * a.M;
    const T *zp = static_cast<const T *>(z.p);
    T *dzp = static_cast<T *>(dz.p);
    if (dzp)
        distill_group_kernel<T, VEC, NV, true><<<blocks, GROUP_THREADS, shared, st>>>(
            zp, z.ld, a.tid, a.tl, a.rw, a.n, a.V, a.M, a.tau, log_l, a.loss, dzp, dz.ld);
    else
        distill_group_kernel<T, VEC, NV, false><<<blocks, GROUP_THREADS, shared, st>>>(
            zp, z.ld, a.tid, a.tl, a.rw, a.n, a.V, a.M, a.tau, log_l, a.loss, dzp, dz.ld);
    return cudaGetLastError();
}

constexpr int GROUP_PIECES = 8;  // a lane, at most

template <typename T, int VEC> cudaError_t group_shape(RowsIn z, RowsOut dz, const Args &a, cudaStream_t st) {
    const int pieces = (a.V + VEC - 1) / VEC;
    // the lanes that leave the fewest idle, the fewest on a tie; enough of
    // them that the groups' teachers fit 48 KB
    int log_l = 5, best = 1 << 30;
    for (int l = 0; l <= 5; ++l) {
        const int each = (pieces + (1 << l) - 1) >> l;
        if (each > GROUP_PIECES || (GROUP_THREADS >> l) * a.M * 12 > 48 * 1024) continue;
        if ((each << l) < best) {
            best = each << l;
            log_l = l;
        }
    }
    const int each = (pieces + (1 << log_l) - 1) >> log_l;
    return each <= 2   ? group_launch<T, VEC, 2>(z, dz, a, log_l, st)
           : each <= 4 ? group_launch<T, VEC, 4>(z, dz, a, log_l, st)
                       : group_launch<T, VEC, GROUP_PIECES>(z, dz, a, log_l, st);
}

template <typename T> cudaError_t long_launch(RowsIn z, RowsOut dz, const Args &a, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    const int pieces = (a.V + VEC - 1) / VEC;
    constexpr int FIT = 100 * 1024 / 16, MOST = 200 * 1024 / 16;  // pieces in shared memory: two blocks, or one
    // blocks of a cluster: what shared memory asks for, and more while there
    // are multiprocessors without a row and 8 KB for each block
    int ranks = 1;
    while (ranks < 8 && (pieces > ranks * FIT || (a.n * ranks * 2 <= SMS && pieces >= ranks * 2 * LONG_THREADS)))
        ranks *= 2;
    const int each = (pieces + ranks - 1) / ranks;
    const bool cached = each <= MOST;
    const int threads = each <= 256 ? 128 : each <= 1024 ? 256 : LONG_THREADS;
    const size_t shared = dz.p && cached ? (size_t)each * 16 : 0;
    auto kernel = !dz.p ? distill_long_kernel<T, false, true>
                        : cached ? distill_long_kernel<T, true, true> : distill_long_kernel<T, true, false>;
    cudaError_t e = cudaSuccess;
    if (shared > 40 * 1024)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (e != cudaSuccess) return e;
    // rows beyond what one grid takes in blocks follow in further launches
    const long long rows_each = 0x7fffffffll / ranks;
    for (long long r = 0; r < a.n && e == cudaSuccess; r += rows_each) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim = {(unsigned)ranks, 1, 1};
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((a.n - r < rows_each ? a.n - r : rows_each) * ranks));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = shared;
        cfg.stream = st;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const T *>(z.p) + r * z.ld, z.ld, a.tid + r * a.M,
                               a.tl + r * a.M, a.rw ? a.rw + r : nullptr, a.V, a.M, a.tau, each, a.loss + r,
                               dz.p ? static_cast<T *>(dz.p) + r * dz.ld : nullptr, dz.ld);
    }
    return e;
}

template <typename T> cudaError_t distill(RowsIn z, RowsOut dz, const Args &a, cudaStream_t st) {
    int b = row_piece(z.p, z.ld, a.V, sizeof(T));
    if (dz.p) b = b < row_piece(dz.p, dz.ld, a.V, sizeof(T)) ? b : row_piece(dz.p, dz.ld, a.V, sizeof(T));
    if ((long long)a.V * (int)sizeof(T) > 32ll * GROUP_PIECES * b) return long_launch<T>(z, dz, a, st);
    if (b == 16) return group_shape<T, 16 / sizeof(T)>(z, dz, a, st);
    if (b == 8) return group_shape<T, 8 / sizeof(T)>(z, dz, a, st);
    if (b == 4) return group_shape<T, 4 / sizeof(T)>(z, dz, a, st);
    return group_shape<T, 1>(z, dz, a, st);
}

}  // namespace

cudaError_t launch_distill(int dtype, RowsIn z, const int32_t *tid, const float *tl, const float *rw, long long T,
                           int V, int M, float tau, float *loss, RowsOut dz, cudaStream_t st) {
    const Args a{tid, tl, rw, T, V, M, tau, loss};
    if (dtype == 0) return distill<float>(z, dz, a, st);
    if (dtype == 1) return distill<__nv_bfloat16>(z, dz, a, st);
    return distill<__half>(z, dz, a, st);
}

}  // namespace sad
