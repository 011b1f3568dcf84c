// sad_distill.cu -- distillation from a teacher's top logits: the divergence
// of the student's softmax from the teacher's over the M classes that it
// hands out, and the gradient of the student's logits.
//
// With q = softmax(teacher / tau) over the counting entries and p =
// softmax(z / tau): loss = rw tau^2 sum_m q_m (ln q_m - ln p[id_m]) and dz_v =
// rw tau (p_v - sum of q_m over id_m = v).  Exponentials are taken to base 2
// of (z - max) log2(e) / tau in float32.  The row's maximum is subtracted before
// the product is rounded: what all logits have in common leaves no trace, and no
// tau makes the rounding of z log2(e) / tau count.
//
// Bound by memory where rows are read and written once; the exponentials (16
// a clock on a multiprocessor, two an element with the gradient of a long
// row) come next.  Rows start at any element: the 16-byte pieces begin at the
// row's first boundary, and the elements before and behind them, its edges,
// are taken one by one.  Short rows (up to 8 pieces for each lane of a group
// of L <= 32) stay in registers, several rows a warp.  Longer rows are shared
// by a block: a first pass for the running maximum and sum of every thread, a
// second for the gradient, which reads the block's part from shared memory (up
// to 48 KB) or again from the L2; a row beyond 100 KB, or one of few rows, by a
// cluster of up to eight blocks that join maxima and sums through distributed
// shared memory.
//
// Measured (copy rate 6,540 GB/s), with the gradient: 393,216 x 150 f32 103 us
// (0.74 of it; a third of its instructions are the teacher's side of rows of
// 150), 4096 x 50,001 bf16 172 us (0.73; the part in shared memory, two blocks
// a multiprocessor, took 205 where this took 172), 1 x 128,000 bf16 7 us;
// loss only 74, 80 and 6 us.  The teacher's side of a short row goes by M^2:
// 393,216 x 100 f32 88 us with M = 8, 611 with 32, 1,982 with 64.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>

#include "sad_features.h"
#include "sad_rows.cuh"

namespace sad {

namespace {

namespace cg = cooperative_groups;
using std::max;
using std::min;

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

// 1 / x, within 1 ulp
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float minus_infinity() { return __int_as_float(0xff800000); }

// A maximum to subtract: 0 for a row, or part of one, of nothing but -infinity
__device__ __forceinline__ float finite_max(float m) { return m == minus_infinity() ? 0.0f : m; }

__device__ __forceinline__ float lanes_sum(float v, int L) {
    for (int o = L >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// two at a time
__device__ __forceinline__ void lanes_sum(float &a, float &b, int L) {
    for (int o = L >> 1; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, a, o), v = __shfl_xor_sync(0xffffffffu, b, o);
        a += u;
        b += v;
    }
}
__device__ __forceinline__ void lanes_max(float &a, float &b, int L) {
    for (int o = L >> 1; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, a, o), v = __shfl_xor_sync(0xffffffffu, b, o);
        a = max_nan(a, u);
        b = max_nan(b, v);
    }
}
__device__ __forceinline__ float lanes_max(float v, int L) {
    for (int o = L >> 1; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The teacher's side of a row, by a group of L lanes; entries m of the row in
// shared memory.
struct Teacher {
    int32_t *id;  // -1: does not count
    float *q;     // first the logit, then the probability
    float *zid;   // the student's logit of the class
    float max, sum;  // the largest logit, -infinity where no entry counts
};

template <typename T>
__device__ __forceinline__ void teacher_load(Teacher &t, const int32_t *__restrict__ tid, const float *__restrict__ tl,
                                             const T *row, int V, int M, bool in, int lane, int L) {
    float big = minus_infinity();
    for (int m = lane; m < M; m += L) {
        int32_t id = in ? __ldg(tid + m) : -1;
        float l = minus_infinity(), z = 0.0f;
        if ((uint32_t)id < (uint32_t)V) {
            l = __ldg(tl + m);
            z = to_f32<T>(row[id]);
        }
        if (l == minus_infinity()) id = -1;  // a NaN logit of a valid class counts, and shows
        big = max_nan(big, l);
        t.id[m] = id;
        t.q[m] = l;
        t.zid[m] = z;
    }
    t.max = big;
}

// a lane's share of the sum of exponentials about t.max
__device__ __forceinline__ float teacher_sum(const Teacher &t, int M, float k, int lane, int L) {
    float s = 0.0f;
    const float m0 = finite_max(t.max);
    for (int m = lane; m < M; m += L) s += exp2_fast((t.q[m] - m0) * k);
    return s;
}

// The row's loss, given scale = rw tau and the student's maximum and sum; leaves
// q in shared memory.  tau^2 (ln q - ln p) is tau times the logits' distances
// from their maxima plus tau^2 ln of the sums' quotient: the distances stay
// unscaled, and half of them is summed, so that a class masked by the lowest
// float gives a large loss and no infinity.
__device__ __forceinline__ float teacher_loss(Teacher &t, int M, float k, float tau, float scale, int lane, int L,
                                              float big, float sum) {
    const float is = reciprocal(t.sum);
    const float m0 = finite_max(t.max);
    float part = 0.0f;
    for (int m = lane; m < M; m += L) {
        float q = 0.0f;
        if (t.id[m] >= 0) {
            const float l = t.q[m] - m0;
            q = exp2_fast(l * k) * is;
            if (q != 0.0f) part = fmaf(0.5f * q, l + (big - t.zid[m]), part);
        }
        t.q[m] = q;
    }
    part = lanes_sum(part, L);
    return 2.0f * scale * fmaf(0.5f * LN2 * tau, log2f(sum * is), part);
}

// gradient of entry m's class, all of its entries counted
__device__ __forceinline__ float teacher_grad(const Teacher &t, int M, float k, int m, float big, float inv_sum,
                                              float scale) {
    const int32_t id = t.id[m];
    float q = 0.0f;
#pragma unroll 4
    for (int j = 0; j < M; ++j)
        if (t.id[j] == id) q += t.q[j];
    return scale * (exp2_fast((t.zid[m] - big) * k) * inv_sum - q);
}

// the largest of a piece's elements and m, as loaded; 16-bit ones in pairs
template <typename T, int VEC> __device__ __forceinline__ float piece_max(const Pack<T, VEC> &p, float m) {
    if constexpr (sizeof(T) == 2 && VEC == 8) {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        T2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const T2 *>(&p.w[i]);
        const T2 a = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
        return max_nan(m, max_nan(to_f32<T>(a.x), to_f32<T>(a.y)));
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) m = max_nan(m, p.get(q));
        return m;
    }
}

// e = 2^((z - big) k) of a piece
template <typename T, int VEC>
__device__ __forceinline__ void piece_exp(const Pack<T, VEC> &p, float k, float big, float (&e)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int q = 0; q < VEC; q += 2) {
            both(mul_two(add_two(two(p.get(q), p.get(q + 1)), two(-big, -big)), two(k, k)), e[q], e[q + 1]);
            e[q] = exp2_fast(e[q]);
            e[q + 1] = exp2_fast(e[q + 1]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) e[q] = exp2_fast((p.get(q) - big) * k);
    }
}

// s += the elements of e
template <int VEC> __device__ __forceinline__ void piece_add(const float (&e)[VEC], Two &s) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int q = 0; q < VEC; q += 2) s = add_two(s, two(e[q], e[q + 1]));
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) s = add_two(s, two(e[q], 0.0f));
    }
}

// to[] = e f, as one piece where `to` is on a boundary
template <typename T, int VEC>
__device__ __forceinline__ void store_scaled(T *to, const float (&e)[VEC], float f, bool whole) {
    float g[VEC];
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int q = 0; q < VEC; q += 2) both(mul_two(two(e[q], e[q + 1]), two(f, f)), g[q], g[q + 1]);
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) g[q] = e[q] * f;
    }
    if (whole) {
        Pack<T, VEC> o;
        o.set(g);
        store_pack<T, VEC>(to, o);
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) to[q] = from_f32<T>(g[q]);
    }
}

// Where a row's pieces of VEC elements lie: `head` elements before the first,
// `pieces` of them, `tail` elements behind
template <typename T, int VEC> struct Cut {
    int head, pieces, tail;
    __device__ __forceinline__ Cut(const T *row, int V, bool edges) {
        head = edges ? min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T))) : 0;
        pieces = (V - head) / VEC;
        tail = V - head - pieces * VEC;
    }
    // the q-th of the row's elements outside the pieces, V if there are fewer
    __device__ __forceinline__ int edge(int q, int V) const {
        return q < head ? q : q < head + tail ? V - tail + q - head : V;
    }
    // the piece of element id, -1 for an edge
    __device__ __forceinline__ int piece_of(int id, int V) const {
        return id < head || id >= V - tail ? -1 : (id - head) / VEC;
    }
};

__device__ __forceinline__ bool same_boundaries(const void *a, const void *b) {
    return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// ---------------------------------------------------------------------------
// short rows
// ---------------------------------------------------------------------------
constexpr int GROUP_THREADS = 256;

template <typename T, int VEC, int NV, bool EDGES, bool GRAD>
__global__ void __launch_bounds__(GROUP_THREADS) distill_group_kernel(
    const T *z, long long ldz, const int32_t *__restrict__ tid, const float *__restrict__ tl,
    const float *__restrict__ rw, long long n, int V, int M, float tau, int log_l, float *__restrict__ loss, T *dz,
    long long lddz) {
    extern __shared__ float teacher_space[];
    const int L = 1 << log_l, lane = threadIdx.x & (L - 1), group = threadIdx.x >> log_l;
    const long long t = ((long long)blockIdx.x * GROUP_THREADS + threadIdx.x) >> log_l;
    const bool in = t < n;
    const float k = LOG2E / tau;
    const T *row = z + t * ldz;
    const Cut<T, VEC> cut(row, V, EDGES);
    const int pieces = in ? cut.pieces : 0;
    Pack<T, VEC> p[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (lane + i * L < pieces) p[i] = load_pack<T, VEC>(row + cut.head + (lane + i * L) * VEC);
    const int edge = EDGES && in ? cut.edge(lane, V) : V;
    float edge_z = minus_infinity();
    if (EDGES && edge < V) edge_z = to_f32<T>(row[edge]);
    const float weight = in ? (rw ? __ldg(rw + t) : 1.0f) : 0.0f;
    Teacher te;
    float *space = teacher_space + (size_t)group * M * 3;
    te.id = reinterpret_cast<int32_t *>(space);
    te.q = space + M;
    te.zid = space + 2 * M;
    teacher_load<T>(te, tid + t * M, tl + t * M, row, V, M, in, lane, L);

    float big = EDGES ? edge_z : minus_infinity();
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (lane + i * L < pieces) big = piece_max(p[i], big);
    lanes_max(big, te.max, L);
    const bool live = te.max != minus_infinity() && weight != 0.0f && big != minus_infinity();
    if (!live) {  // the row may hold anything: take 0 for it
#pragma unroll
        for (int i = 0; i < NV; ++i) p[i].clear();
        edge_z = 0.0f;
        big = 0.0f;
    }
    float e[NV][VEC];
    Two sums = two(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (lane + i * L < pieces) {
            piece_exp(p[i], k, big, e[i]);
            piece_add(e[i], sums);
        }
    }
    float sum, other;
    both(sums, sum, other);
    sum += other;
    const float edge_e = EDGES && edge < V ? exp2_fast((edge_z - big) * k) : 0.0f;
    sum += edge_e;
    te.sum = teacher_sum(te, M, k, lane, L);
    lanes_sum(sum, te.sum, L);
    const float scale = weight * tau;
    const float part = teacher_loss(te, M, k, tau, scale, lane, L, big, sum);
    if (lane == 0 && in) loss[t] = live ? part : 0.0f;
    if (!GRAD) return;
    const float is = reciprocal(sum), f = live ? scale * is : 0.0f;
    T *out = dz + t * lddz;
    const bool whole = !EDGES || same_boundaries(out, row);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (lane + i * L < pieces) store_scaled(out + cut.head + (lane + i * L) * VEC, e[i], f, whole);
    if (EDGES && edge < V) out[edge] = from_f32<T>(edge_e * f);
    __syncwarp();
    // the teacher's classes once more, from float32: an id listed twice gets
    // the same value from each of its entries
    if (live)
        for (int m = lane; m < M; m += L)
            if (te.id[m] >= 0) out[te.id[m]] = from_f32<T>(teacher_grad(te, M, k, m, big, is, scale));
}

// ---------------------------------------------------------------------------
// long rows: a block or a cluster each
// ---------------------------------------------------------------------------
constexpr int LONG_THREADS = 256;

// The last warp has the teacher's side: its chain of loads (ids, then the
// student's logits of them) and its sums over repeated ids run beside the row.
template <typename T, bool GRAD, bool CACHE>
__global__ void __launch_bounds__(LONG_THREADS + 32, 4) distill_long_kernel(
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
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int B = blockDim.x - 32, warps = B >> 5;  // of the row
    const bool has_teacher = warp == warps;
    const long long t = blockIdx.x / ranks;
    const T *row = z + t * ldz;
    const float k = LOG2E / tau;
    const float weight = rw ? __ldg(rw + t) : 1.0f;
    const Cut<T, VEC> cut(row, V, true);
    const int first = min(rank * each, cut.pieces), last = has_teacher ? first : min(first + each, cut.pieces);
    const T *body = row + cut.head;

    Teacher te{s_id, s_q, s_zid, 0.0f, 0.0f};
    if (has_teacher) {
        teacher_load<T>(te, tid + t * M, tl + t * M, row, V, M, true, lane, 32);
        te.max = lanes_max(te.max, 32);
        te.sum = lanes_sum(teacher_sum(te, M, k, lane, 32), 32);
        if (lane == 0) t_any = te.max != minus_infinity() ? 1.0f : 0.0f;
    }

    // each thread's running maximum (as loaded) and sum of exponentials about
    // it; one thread of the first block takes an edge each
    const int edge = rank || has_teacher ? V : cut.edge(threadIdx.x, V);
    float big = minus_infinity(), sum = 0.0f;
    if (edge < V) {
        big = to_f32<T>(row[edge]);
        sum = big == minus_infinity() ? 0.0f : exp2_fast((big - big) * k);  // 1, or NaN
    }
    const float edge_z = big;
    for (int c = first + threadIdx.x; c < last; c += UNROLL * B) {
        Pack<T, VEC> p[UNROLL];
        float m = big;
        // whole steps, and the last one, whose missing pieces repeat the first
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int at = c + u * B;
            p[u] = load_pack<T, VEC>(body + (long long)(at < last ? at : c) * VEC);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int at = c + u * B;
            if (GRAD && CACHE && at < last) cache[at - first] = *reinterpret_cast<const uint4 *>(&p[u]);
            m = piece_max(p[u], m);
        }
        const float m0 = finite_max(m);
        Two s = two(sum * exp2_fast((big - m0) * k), 0.0f);  // exactly sum where the maximum stays
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (c + u * B < last) {
                float e[VEC];
                piece_exp(p[u], k, m0, e);
                piece_add(e, s);
            }
        }
        float other;
        both(s, sum, other);
        sum += other;
        big = m;
    }

    // joined over the warps, then over the cluster
    {
        const float m = lanes_max(big, 32);
        const float s = lanes_sum(big == minus_infinity() ? 0.0f : sum * exp2_fast((big - finite_max(m)) * k), 32);
        if (lane == 0 && !has_teacher) s_max[warp] = m, s_sum[warp] = s;
    }
    __syncthreads();
    {
        const float wm = lane < warps ? s_max[lane] : minus_infinity(), ws = lane < warps ? s_sum[lane] : 0.0f;
        big = lanes_max(wm, 32);
        sum = lanes_sum(wm == minus_infinity() ? 0.0f : ws * exp2_fast((wm - finite_max(big)) * k), 32);
    }
    if (ranks > 1) {
        if (threadIdx.x == 0) block_max = big, block_sum = sum;
        cluster.sync();
        const float wm = lane < ranks ? *cluster.map_shared_rank(&block_max, lane) : minus_infinity();
        const float ws = lane < ranks ? *cluster.map_shared_rank(&block_sum, lane) : 0.0f;
        big = lanes_max(wm, 32);
        sum = lanes_sum(wm == minus_infinity() ? 0.0f : ws * exp2_fast((wm - finite_max(big)) * k), 32);
        cluster.sync();  // no block leaves before all have read its shared memory
    }
    const bool live = t_any != 0.0f && weight != 0.0f && big != minus_infinity();
    const float scale = weight * tau, is = reciprocal(sum), f = scale * is;
    if (has_teacher) {
        const float part = teacher_loss(te, M, k, tau, scale, lane, 32, big, sum);
        if (lane == 0 && rank == 0) loss[t] = live ? part : 0.0f;
        if (GRAD) {
            __syncwarp();
            for (int m = lane; m < M; m += 32) s_zid[m] = teacher_grad(te, M, k, m, big, is, scale);
        }
    }
    if (!GRAD) return;
    T *out = dz + t * lddz, *out_body = out + cut.head;
    const bool whole = same_boundaries(out, row);
    if (edge < V) out[edge] = from_f32<T>(live ? exp2_fast((edge_z - big) * k) * f : 0.0f);
    if (live) {
        for (int c = first + threadIdx.x; c < last; c += UNROLL * B) {
            Pack<T, VEC> p[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int at = c + u * B < last ? c + u * B : c;
                if (CACHE) p[u] = *reinterpret_cast<const Pack<T, VEC> *>(cache + at - first);
                else p[u] = load_pack<T, VEC>(body + (long long)at * VEC);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int at = c + u * B;
                float e[VEC];
                piece_exp(p[u], k, big, e);
                if (at < last) store_scaled(out_body + (long long)at * VEC, e, f, whole);
            }
        }
    } else {
        const float zero[VEC] = {};
        for (int c = first + threadIdx.x; c < last; c += B) store_scaled(out_body + (long long)c * VEC, zero, 0.0f, whole);
    }
    __syncthreads();
    // the teacher's classes in this block's part, from float32
    const int end = min(first + each, cut.pieces);
    if (live)
        for (int m = threadIdx.x; m < M; m += blockDim.x) {
            if (s_id[m] < 0) continue;
            const int piece = cut.piece_of(s_id[m], V);
            if (piece < 0 ? rank == 0 : (piece >= first && piece < end)) out[s_id[m]] = from_f32<T>(s_zid[m]);
        }
}

// whether every row begins and ends on a 16-byte boundary
bool whole_rows(const void *p, long long ld, int V, int bytes) { return piece_bytes(p, ld, V, bytes) == 16; }

struct Args {
    const int32_t *tid;
    const float *tl, *rw;
    long long n;
    int V, M;
    float tau;
    float *loss;
};

template <typename T, int VEC, int NV, bool EDGES>
cudaError_t group_launch(RowsIn z, RowsOut dz, const Args &a, int log_l, cudaStream_t st) {
    const int groups = GROUP_THREADS >> log_l;
    const unsigned blocks = (unsigned)((a.n + groups - 1) / groups);
    const size_t shared = sizeof(float) * 3 * groups * a.M;
    const T *zp = static_cast<const T *>(z.p);
    T *dzp = static_cast<T *>(dz.p);
    if (dzp)
        distill_group_kernel<T, VEC, NV, EDGES, true><<<blocks, GROUP_THREADS, shared, st>>>(
            zp, z.ld, a.tid, a.tl, a.rw, a.n, a.V, a.M, a.tau, log_l, a.loss, dzp, dz.ld);
    else
        distill_group_kernel<T, VEC, NV, EDGES, false><<<blocks, GROUP_THREADS, shared, st>>>(
            zp, z.ld, a.tid, a.tl, a.rw, a.n, a.V, a.M, a.tau, log_l, a.loss, dzp, dz.ld);
    return cudaGetLastError();
}

constexpr int GROUP_PIECES = 8;  // a lane, at most

template <typename T, int VEC, bool EDGES> cudaError_t group_shape(RowsIn z, RowsOut dz, const Args &a, cudaStream_t st) {
    const int pieces = EDGES ? max(1, a.V / VEC) : (a.V + VEC - 1) / VEC;
    // the lanes that leave the fewest idle, the most on a tie (the gradient
    // keeps a register for every element: 65,536 x 1000 bf16 in 72 us with 32
    // lanes, 82 with 16); enough for every edge, and that the groups' teachers
    // fit 48 KB
    const int least = EDGES ? 2 * (VEC - 1) : 1;
    int log_l = 5, best = 1 << 30;
    for (int l = 0; l <= 5; ++l) {
        const int each = (pieces + (1 << l) - 1) >> l;
        if ((1 << l) < least || each > GROUP_PIECES || (GROUP_THREADS >> l) * a.M * 12 > 48 * 1024) continue;
        if ((each << l) <= best) {
            best = each << l;
            log_l = l;
        }
    }
    switch ((pieces + (1 << log_l) - 1) >> log_l) {
        case 1: return group_launch<T, VEC, 1, EDGES>(z, dz, a, log_l, st);
        case 2: return group_launch<T, VEC, 2, EDGES>(z, dz, a, log_l, st);
        case 3: return group_launch<T, VEC, 3, EDGES>(z, dz, a, log_l, st);
        case 4: return group_launch<T, VEC, 4, EDGES>(z, dz, a, log_l, st);
        case 5: return group_launch<T, VEC, 5, EDGES>(z, dz, a, log_l, st);
        case 6: return group_launch<T, VEC, 6, EDGES>(z, dz, a, log_l, st);
        default: return group_launch<T, VEC, GROUP_PIECES, EDGES>(z, dz, a, log_l, st);
    }
}

template <typename T> cudaError_t long_launch(RowsIn z, RowsOut dz, const Args &a, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    const int pieces = (a.V + VEC - 1) / VEC;
    constexpr int FIT = 100 * 1024 / 16, CACHED = 48 * 1024 / 16;
    // blocks of a cluster: what keeps the rows in work within half of the L2,
    // for the second pass, and more while there are multiprocessors without a
    // row and 4 KB for each block
    int ranks = 1;
    while (ranks < 8 && (pieces > ranks * FIT || (a.n * ranks * 2 <= SMS && pieces >= ranks * 2 * LONG_THREADS)))
        ranks *= 2;
    const int each = (pieces + ranks - 1) / ranks;
    const bool cached = each <= CACHED;
    // eight pieces a thread, two rounds of loads: with more threads a block of
    // short rows waits for its reductions most of the time
    const int threads = min(LONG_THREADS, max(64, (each + 255) / 256 * 32)) + 32;
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
    constexpr int VEC = 16 / sizeof(T);
    if (a.V > 32 * GROUP_PIECES * VEC) return long_launch<T>(z, dz, a, st);
    const bool whole = whole_rows(z.p, z.ld, a.V, sizeof(T)) && (!dz.p || whole_rows(dz.p, dz.ld, a.V, sizeof(T)));
    if (whole) return group_shape<T, VEC, false>(z, dz, a, st);
    // in pieces with edges, but element by element where the edges' lanes
    // would outnumber the pieces
    if (a.V > 8 * VEC) return group_shape<T, VEC, true>(z, dz, a, st);
    return group_shape<T, 1, false>(z, dz, a, st);
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
