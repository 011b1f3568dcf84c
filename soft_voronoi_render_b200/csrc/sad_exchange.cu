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
//
// gather and spread: a group of L <= 32 lanes takes one row, reads its K ids
// and weights, and has all K rows' loads in flight at once, a piece (16 bytes,
// or what the alignment allows) each, then its next pieces; shape_of says how
// many lanes.  Where there are few wide rows the warps of a block share one.
// The K dot products are summed over the group by halving: each step of the
// butterfly also halves the number of sums a lane keeps, 7 + log2(L / 8)
// shuffles instead of 8 log2 L.  16-bit elements are widened and multiplied in
// pairs.
//
// Measured (copy rate 6,540 GB/s): 16,384 x 8 rows of 2048 bf16, bound by
// memory: dispatch 99 us (0.94 of it), combine 87 (1.06), combine's backward
// 171 (1.02), dispatch's 106 (0.97).  Blend of 2048 x 2048 x 32 bf16 168 us
// (0.50): every row of F is read for about 256 pixels, 2.1 GB through the L1;
// its dot products 192 us.  768 x 512 x 64 f16 33 us.
#include <algorithm>

#include "sad_features.h"
#include "sad_rows.cuh"

namespace sad {

using std::max;
using std::min;

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int K_MAX = 8;

// row r of a matrix with `bytes` from row to row, column c: one multiply-add
template <typename T> __device__ __forceinline__ const T *at_row(const T *base, uint32_t r, uint32_t bytes, int c) {
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(base + c) + (unsigned long long)r * bytes);
}

// acc += w p
template <typename T, int VEC>
__device__ __forceinline__ void add_scaled(const Pack<T, VEC> &p, float w, Two (&acc)[(VEC + 1) / 2]) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2)
        acc[i / 2] = fma_two(two(p.get(i), VEC > 1 ? p.get(i + (VEC > 1)) : 0.0f), two(w, w), acc[i / 2]);
}
// acc += p g
template <typename T, int VEC>
__device__ __forceinline__ void add_product(const Pack<T, VEC> &p, const Pack<T, VEC> &g, Two &acc) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2)
        acc = fma_two(two(p.get(i), VEC > 1 ? p.get(i + (VEC > 1)) : 0.0f),
                      two(g.get(i), VEC > 1 ? g.get(i + (VEC > 1)) : 0.0f), acc);
}

// the K ids and weights of row t; ids beyond K are empty slots
template <bool FULL>
__device__ __forceinline__ void load_slots(const int32_t *__restrict__ at, const float *__restrict__ w, long long t,
                                           int K, bool in, uint32_t (&id)[K_MAX], float (&wt)[K_MAX]) {
    if (FULL) {  // K = 8, 16-byte aligned lists
        int4 a = make_int4(-1, -1, -1, -1), b = a;
        float4 u = make_float4(1.0f, 1.0f, 1.0f, 1.0f), v = u;
        if (in) {
            const int4 *p = reinterpret_cast<const int4 *>(at) + t * 2;
            a = __ldg(p);
            b = __ldg(p + 1);
            if (w) {
                const float4 *q = reinterpret_cast<const float4 *>(w) + t * 2;
                u = __ldg(q);
                v = __ldg(q + 1);
            }
        }
        id[0] = a.x, id[1] = a.y, id[2] = a.z, id[3] = a.w, id[4] = b.x, id[5] = b.y, id[6] = b.z, id[7] = b.w;
        wt[0] = u.x, wt[1] = u.y, wt[2] = u.z, wt[3] = u.w, wt[4] = v.x, wt[5] = v.y, wt[6] = v.z, wt[7] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < K_MAX; ++k) {
            const bool on = in && k < K;
            id[k] = on ? (uint32_t)__ldg(at + t * K + k) : 0xffffffffu;
            wt[k] = on && w ? __ldg(w + t * K + k) : 1.0f;
        }
    }
}

// sums v[0..7] over the L lanes of a group; afterwards lane `first + i` slots
// belong to this lane: v[i], i < count, is the sum of slot first + i
__device__ __forceinline__ void group_sums(float (&v)[K_MAX], int L, int lane, int &first, int &count) {
    first = 0;
    count = K_MAX;
    int o = L >> 1;
#pragma unroll
    for (int half = K_MAX / 2; half; half >>= 1) {
        if (o) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
            first += up ? half : 0;
            count = half;
            o >>= 1;
        }
    }
    for (; o; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
}

// Where a lane works: its row t, the column of its first piece and the
// distance to its next.  ROW_PER_BLOCK: all warps share row blockIdx.x.
template <int VEC, bool ROW_PER_BLOCK> struct Lanes {
    int L, lane;       // lanes of a group, this one's number in it
    long long t;
    bool in;
    int c0, step;
    __device__ __forceinline__ Lanes(int log_l, long long n_rows) {
        if (ROW_PER_BLOCK) {
            L = 32;
            lane = threadIdx.x & 31;
            t = blockIdx.x;
            c0 = threadIdx.x * VEC;
            step = THREADS * VEC;
        } else {
            L = 1 << log_l;
            lane = threadIdx.x & (L - 1);
            t = ((long long)blockIdx.x * THREADS + threadIdx.x) >> log_l;
            c0 = lane * VEC;
            step = L * VEC;
        }
        in = t < n_rows;
    }
};

// writes the dot products of the group's row; dot[k] of empty slots is 0
template <bool FULL, bool ROW_PER_BLOCK>
__device__ __forceinline__ void finish_dots(float (&dot)[K_MAX], int L, int lane, long long t, bool in, int K,
                                            float *__restrict__ dots) {
    int first, count;
    group_sums(dot, L, lane, first, count);
    if (ROW_PER_BLOCK) {
        __shared__ float part[WARPS][K_MAX];
        // 32 lanes: 8 slots over 4 lanes each, one sum a lane
        if ((lane & 3) == 0) part[threadIdx.x >> 5][first] = dot[0];
        __syncthreads();
        if (threadIdx.x < K) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < WARPS; ++q) s += part[q][threadIdx.x];
            dots[t * K + threadIdx.x] = s;
        }
        return;
    }
    // of the lanes that hold the same sum (L > 8) the first writes
    if (!in || (L > 8 && (lane & (L / 8 - 1)))) return;
    if constexpr (FULL) {  // 32 bytes a row, aligned
        float *to = dots + t * K_MAX + first;
        if (count == 1) *to = dot[0];
        else if (count == 2) *reinterpret_cast<float2 *>(to) = make_float2(dot[0], dot[1]);
        else *reinterpret_cast<float4 *>(to) = make_float4(dot[0], dot[1], dot[2], dot[3]);
        if (count == 8) *reinterpret_cast<float4 *>(to + 4) = make_float4(dot[4], dot[5], dot[6], dot[7]);
    } else {
#pragma unroll
        for (int i = 0; i < K_MAX; ++i)
            if (i < count && first + i < K) dots[t * K + first + i] = dot[i];
    }
}

// Empty slots are rows of zeros with weight 0, so that nothing branches
// between the rows but the loads themselves.
template <typename T, int VEC, bool FULL, bool SUM, bool DOT, bool ROW_PER_BLOCK>
__global__ void __launch_bounds__(THREADS, SUM && DOT ? 3 : SUM || VEC * sizeof(T) < 16 ? 4 : 5) gather_kernel(const T *__restrict__ R, uint32_t ldr,
                                                            const int32_t *__restrict__ at, uint32_t n_at,
                                                            const float *__restrict__ w, const T *__restrict__ G,
                                                            uint32_t ldg, long long n_rows, int K, int D, int log_l, int turns,
                                                            T *__restrict__ out, uint32_t ldo,
                                                            float *__restrict__ dots) {
    const Lanes<VEC, ROW_PER_BLOCK> me(log_l, n_rows);
    uint32_t id[K_MAX];
    float wt[K_MAX], dot[K_MAX];
    Two dots2[K_MAX];
    load_slots<FULL>(at, SUM ? w : nullptr, me.t, K, me.in, id, wt);
#pragma unroll
    for (int k = 0; k < K_MAX; ++k) {
        if (id[k] >= n_at) wt[k] = 0.0f;
        dots2[k] = two(0.0f, 0.0f);
    }
    if (me.in) {
        // Where a group's load is less than a line, neighbouring groups begin at
        // different pieces: rows of F lie on 64 or 128 bytes, and the same piece
        // of each falls on the same banks (2048 x 2048 x 32 bf16: 186 us; 168 so).
        constexpr bool TURNS = VEC * sizeof(T) == 16 && !ROW_PER_BLOCK;
        int c = TURNS ? me.c0 + (int)(me.t & turns) * me.step : me.c0;
        if (TURNS && c >= D) c = me.c0;
        for (int at = me.c0; at < D; at += me.step, c = !TURNS || c + me.step < D ? c + me.step : me.c0) {
            Pack<T, VEC> p[K_MAX];
#pragma unroll
            for (int k = 0; k < K_MAX; ++k) {
                p[k].clear();
                if (id[k] < n_at) p[k] = load_pack<T, VEC>(at_row(R, id[k], ldr, c));
            }
            Two acc[(VEC + 1) / 2];
#pragma unroll
            for (int i = 0; i < (VEC + 1) / 2; ++i) acc[i] = two(0.0f, 0.0f);
            Pack<T, VEC> g;
            if (DOT) g = load_pack<T, VEC>(at_row(G, (uint32_t)me.t, ldg, c));
#pragma unroll
            for (int k = 0; k < K_MAX; ++k) {
                if (SUM) add_scaled(p[k], wt[k], acc);
                if (DOT) add_product(p[k], g, dots2[k]);
            }
            if (SUM) {
                float f[VEC + 1];
#pragma unroll
                for (int i = 0; i < VEC; i += 2) both(acc[i / 2], f[i], f[i + 1]);
                float v[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = f[i];
                Pack<T, VEC> o;
                o.set(v);
                store_pack<T, VEC>(const_cast<T *>(at_row(out, (uint32_t)me.t, ldo, c)), o);
            }
        }
    }
    if (DOT) {
#pragma unroll
        for (int k = 0; k < K_MAX; ++k) {
            float other;
            both(dots2[k], dot[k], other);
            dot[k] = id[k] < n_at ? dot[k] + other : 0.0f;  // G may hold infinities
        }
        finish_dots<FULL, ROW_PER_BLOCK>(dot, me.L, me.lane, me.t, me.in, K, dots);
    }
}

template <typename T, int VEC, bool FULL, bool DOT, bool ROW_PER_BLOCK>
__global__ void __launch_bounds__(THREADS) spread_kernel(const T *__restrict__ X, uint32_t ldx,
                                                         const int32_t *__restrict__ at, uint32_t n_at,
                                                         const float *__restrict__ w, const T *__restrict__ R,
                                                         uint32_t ldr, long long n_rows, int K, int D, int log_l,
                                                         T *__restrict__ S, uint32_t lds,
                                                         float *__restrict__ dots) {
    const Lanes<VEC, ROW_PER_BLOCK> me(log_l, n_rows);
    uint32_t id[K_MAX];
    float wt[K_MAX], dot[K_MAX] = {};
    load_slots<FULL>(at, w, me.t, K, me.in, id, wt);
    if (me.in) {
        for (int c = me.c0; c < D; c += me.step) {
            Pack<T, VEC> p[K_MAX];
            if (DOT) {
#pragma unroll
                for (int k = 0; k < K_MAX; ++k)
                    if (id[k] < n_at) p[k] = load_pack<T, VEC>(at_row(R, id[k], ldr, c));
            }
            const Pack<T, VEC> x = load_pack<T, VEC>(at_row(X, (uint32_t)me.t, ldx, c));
#pragma unroll
            for (int k = 0; k < K_MAX; ++k) {
                // a branch here only with the products: 172 us against 224 for the
                // 16384 x 8 x 2048 bf16 backward, but 105 against 100 without
                if (DOT && id[k] >= n_at) continue;
                float f[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if (DOT) dot[k] = fmaf(p[k].get(i), x.get(i), dot[k]);
                    f[i] = wt[k] * x.get(i);
                }
                Pack<T, VEC> o;
                o.set(f);
                if (DOT || id[k] < n_at) store_pack<T, VEC>(const_cast<T *>(at_row(S, id[k], lds, c)), o);
            }
        }
    }
    if (DOT) {
#pragma unroll
        for (int k = 0; k < K_MAX; ++k) dot[k] = id[k] < n_at ? dot[k] : 0.0f;
        finish_dots<FULL, ROW_PER_BLOCK>(dot, me.L, me.lane, me.t, me.in, K, dots);
    }
}

// ---------------------------------------------------------------------------
// segment sums
//
// Near rows (is_far says which): the sorted pairs are cut into chunks
// of C positions, a warp each, whatever the experts' shares are.  A warp walks
// its chunk's runs of one expert; a run that is all of its expert's pairs goes
// to dF, one that is cut at the chunk's start or end to one of the chunk's two
// partial rows, which join_kernel adds up in order.  Experts without pairs are
// skipped by a search, so the cost goes by the runs: 32 rows x 8 pairs over
// 131,072 sites x 32 f32 take 247 us, 1,024 rows 243, the 128 runs of a chunk one
// after another; 512 x 256 rows of 2,000 sites 29 us (f16, 64 columns).
//
// Far rows: every row of dout is read once for each of its K pairs, and where
// ids are in no order over the rows (sites over an image) experts side by
// side in the list would read it from memory K times.  So the work is cut at
// the experts, in pieces of at most C positions, and the pieces are taken in
// the order of their first pair's row, counted into BUCKETS parts of the rows
// (2048 x 2048 x 32 bf16: 784 us for 3.2 GB by chunks in their own order, 588
// us for 1.9 GB with chunks, cut anywhere, in the order of the rows, 376 us
// with pieces: 3.3 GB from the L2, a third of it sectors of which one weight
// is wanted).  The order within a part is not fixed, and no result depends on
// it.
// ---------------------------------------------------------------------------

// acc[] = sum of w_j G[j / K] over the sorted positions a ... b - 1, columns c
// ... of the group: 32 pairs a step, their rows by 32 / L groups side by side.
// The ids of the pairs two steps ahead and the weights of the next are loaded
// while the rows of a step are on their way.
template <typename T, int VEC, int NP>
__device__ __forceinline__ void sum_run(const T *__restrict__ G, uint32_t ldg, const float *__restrict__ w,
                                        const int32_t *__restrict__ order, uint32_t n, uint32_t K, uint32_t a,
                                        uint32_t b, int c, int D, int log_l, float (&acc)[NP][VEC + 1]) {
    const int L = 1 << log_l, S = 32 >> log_l;
    const int lane = threadIdx.x & 31, sub = lane >> log_l;
    const int step = VEC << log_l;
    constexpr int U = NP == 1 ? 4 : 2;  // rows of a group on their way
    Two acc2[NP][(VEC + 1) / 2];
#pragma unroll
    for (int v = 0; v < NP; ++v) {
#pragma unroll
        for (int i = 0; i < (VEC + 1) / 2; ++i) acc2[v][i] = two(0.0f, 0.0f);
    }
    auto pair_at = [&](uint32_t s) { return s + lane < b ? (uint32_t)__ldg(order + s + lane) : 0xffffffffu; };
    auto weight_of = [&](uint32_t j) { return j < n ? __ldg(w + j) : 0.0f; };
    uint32_t j = pair_at(a), j_next = pair_at(a + 32);
    float wj = weight_of(j);
    for (uint32_t s = a; s < b; s += 32) {
        const uint32_t row = j < n ? j / K : 0;
        const uint32_t left = min(b - s, 32u);
        const uint32_t j_ahead = pair_at(s + 64);
        float w_next = 0.0f;
        for (uint32_t q = 0; q < left; q += U * S) {
            Pack<T, VEC> p[U][NP];
            float wq[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t at = q + u * S + sub;
                const uint32_t r = __shfl_sync(0xffffffffu, row, at & 31);
                wq[u] = __shfl_sync(0xffffffffu, wj, at & 31);
                const T *from = at_row(G, r, ldg, c);
#pragma unroll
                for (int v = 0; v < NP; ++v) {
                    p[u][v].clear();
                    if (at < left && c + v * step < D) p[u][v] = load_pack<T, VEC>(from + v * step);
                }
            }
            if (q == 0) w_next = weight_of(j_next);
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int v = 0; v < NP; ++v) add_scaled(p[u][v], wq[u], acc2[v]);  // 0 beyond the run
            }
        }
        j = j_next;
        wj = w_next;
        j_next = j_ahead;
    }
#pragma unroll
    for (int v = 0; v < NP; ++v) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) both(acc2[v][i / 2], acc[v][i], acc[v][i + 1]);
        for (int o = L; o < 32; o <<= 1) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[v][i] += __shfl_xor_sync(0xffffffffu, acc[v][i], o);
        }
    }
}

// pieces a lane: one of 16 bytes, or eight smaller ones (a row of 41 elements
// on 32 lanes left most of them idle in its second part)
template <typename T, int VEC> constexpr int lane_pieces() { return VEC * sizeof(T) == 16 ? 1 : 8; }

// to[i] = acc[i], by the first group; `to` may start anywhere on 4 bytes
template <int VEC> __device__ __forceinline__ void store_sums(float *to, const float (&acc)[VEC + 1]) {
    constexpr int W = VEC % 4 ? VEC : 4;
#pragma unroll
    for (int i = 0; i < VEC; i += W) {
        Pack<float, W> f;
#pragma unroll
        for (int v = 0; v < W; ++v) f.v[v] = acc[i + v];
        if (W == 4 && (reinterpret_cast<uintptr_t>(to + i) & 15) == 0) store_pack<float, W>(to + i, f);
        else
            for (int v = 0; v < W; ++v) to[i + v] = f.v[v];
    }
}

// the last e in [lo, E) with offsets[e] <= s, for offsets[lo] <= s < offsets[E]:
// by a warp, 32 probes a step.  (Offsets that do not ascend give some e of the
// range: every step cuts it to a 32nd.)
__device__ __forceinline__ int expert_at(const int32_t *__restrict__ offsets, int lo, int E, uint32_t s) {
    int hi = E;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + step * (1 + (int)(threadIdx.x & 31));
        const bool below = at < hi && (uint32_t)__ldg(offsets + at) <= s;
        lo += step * __popc(__ballot_sync(0xffffffffu, below));
        hi = min(hi, lo + step);
    }
    return lo;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(THREADS, 4) chunk_kernel(const T *__restrict__ G, uint32_t ldg,
                                                        const float *__restrict__ w,
                                                        const int32_t *__restrict__ offsets,
                                                        const int32_t *__restrict__ order, uint32_t n, int K, int E,
                                                        int D, int log_l, uint32_t C, uint32_t chunks,
                                                        float *__restrict__ dF, float *__restrict__ partial,
                                                        int32_t *__restrict__ cut_expert) {
    const int lane = threadIdx.x & 31, in_row = lane & ((1 << log_l) - 1);
    const uint32_t chunk = (uint32_t)(((long long)blockIdx.x * THREADS + threadIdx.x) >> 5);
    if (chunk >= chunks) return;
    const uint32_t total = min((uint32_t)__ldg(offsets + E), n);
    const uint32_t lo = chunk * C;
    if (lane == 0 && blockIdx.y == 0) cut_expert[chunk] = -1;
    if (lo >= total) return;
    const uint32_t hi = min(lo + C, total);
    const int first = expert_at(offsets, 0, E, lo);
    constexpr int NP = lane_pieces<T, VEC>();
    const int step = VEC << log_l, wide = NP * step;
    for (int slab = blockIdx.y * wide; slab < D; slab += gridDim.y * wide) {
        const int c = slab + in_row * VEC;
        int e = first;
        uint32_t a = lo;
        while (a < hi && e < E) {
            const uint32_t end = min((uint32_t)__ldg(offsets + e + 1), total);
            if (end <= a) {  // no pairs: on to the expert of position a, which may be far
                e = max(e + 1, expert_at(offsets, e, E, a));
                continue;
            }
            const uint32_t b = min(end, hi);
            float acc[NP][VEC + 1];
            sum_run<T, VEC, NP>(G, ldg, w, order, n, (uint32_t)K, a, b, c, D, log_l, acc);
            const uint32_t from = (uint32_t)__ldg(offsets + e);
            const bool whole = from == a && end == b;
            // the expert that starts in this chunk and goes on behind it
            if (lane == 0 && slab == 0 && from >= lo && end > b) cut_expert[chunk] = e;
            float *to = whole ? dF + (long long)e * D : partial + ((size_t)2 * chunk + (a == lo ? 0 : 1)) * D;
#pragma unroll
            for (int v = 0; v < NP; ++v)
                if (lane >> log_l == 0 && c + v * step < D) store_sums<VEC>(to + c + v * step, acc[v]);
            a = b;
            ++e;
        }
    }
}

// Sums rows(q), q = from ... last, of D columns into to[]: by one warp, or
// (many rows) by all warps of the block, a run of the rows each.
template <typename F>
__device__ __forceinline__ void sum_rows_warp(F row, uint32_t from, uint32_t last, int D, float *__restrict__ to) {
    for (int c = threadIdx.x & 31; c < D; c += 32) {
        float s = 0.0f;
#pragma unroll 4
        for (uint32_t q = from; q <= last; ++q) s += __ldg(row(q) + c);
        to[c] = s;
    }
}
template <typename F>
__device__ __forceinline__ void sum_rows_block(F row, uint32_t from, uint32_t last, int D, float *__restrict__ to,
                                               float (*part)[33]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t each = (last - from + WARPS) / WARPS, q0 = from + warp * each, q1 = min(q0 + each, last + 1);
    for (int c0 = 0; c0 < D; c0 += 32) {
        const int c = c0 + lane;
        float s = 0.0f;
        if (c < D) {
#pragma unroll 8
            for (uint32_t q = q0; q < q1; ++q) s += __ldg(row(q) + c);
        }
        part[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && c < D) {
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < WARPS; ++q) sum += part[q][lane];
            to[c] = sum;
        }
        __syncthreads();
    }
}

// For each chunk's expert that starts in it and goes on behind it: the sum of
// that expert's partial rows, from this chunk's to the one that it ends in.
// A warp a chunk; experts of more than LONG chunks are left to the block.
constexpr uint32_t LONG = 32;
__global__ void __launch_bounds__(THREADS) join_kernel(const int32_t *__restrict__ offsets,
                                                       const int32_t *__restrict__ cut_expert, uint32_t n, int E,
                                                       int D, uint32_t C, uint32_t chunks,
                                                       const float *__restrict__ partial, float *__restrict__ dF) {
    __shared__ uint32_t long_chunk[WARPS];
    __shared__ float part[WARPS][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto span = [&](uint32_t chunk, int &e, uint32_t &last, int &slot) {
        e = __ldg(cut_expert + chunk);
        if (e < 0) return;
        const uint32_t end = min((uint32_t)__ldg(offsets + e + 1), n);
        last = min((end - 1) / C, chunks - 1);
        slot = (uint32_t)__ldg(offsets + e) != chunk * C;  // where its first run was put
    };
    const uint32_t chunk = blockIdx.x * WARPS + warp;
    int e = -1, slot = 0;
    uint32_t last = 0;
    if (chunk < chunks) span(chunk, e, last, slot);
    const bool later = e >= 0 && last - chunk >= LONG;
    if (lane == 0) long_chunk[warp] = later ? chunk : 0xffffffffu;
    auto row = [&](uint32_t q) { return partial + ((size_t)2 * q + (q == chunk ? slot : 0)) * D; };
    if (e >= 0 && !later) sum_rows_warp(row, chunk, last, D, dF + (long long)e * D);
    __syncthreads();
    for (int k = 0; k < WARPS; ++k) {
        const uint32_t from = long_chunk[k];
        if (from == 0xffffffffu) continue;
        span(from, e, last, slot);
        auto row_of = [&](uint32_t q) { return partial + ((size_t)2 * q + (q == from ? slot : 0)) * D; };
        sum_rows_block(row_of, from, last, D, dF + (long long)e * D, part);
    }
}

// Far rows: pieces of at most C positions of one expert.  Piece k of an expert
// of several has partial row 2 (from / C) + 1 for k = 0 and 2 (from / C + k)
// else: experts of more than C positions are more than C apart, so no two
// share a row.
__device__ __forceinline__ size_t piece_row(uint32_t from, uint32_t k, uint32_t C) {
    return k ? 2 * ((size_t)(from / C) + k) : 2 * (size_t)(from / C) + 1;
}

// (none where the offsets do not ascend, as those of a route do)
__device__ __forceinline__ uint32_t pieces_of(uint32_t from, uint32_t end, uint32_t C) {
    return end > from ? (end - from + C - 1) / C : 0;
}

// The order in which pieces are taken: a count of each part of the rows, its
// scan, and the pieces put into their part's places.  `per` experts a block:
// fewer where few experts have many pieces.
constexpr int BUCKETS = 4096;
template <bool PLACE>
__global__ void __launch_bounds__(THREADS) turn_kernel(const int32_t *__restrict__ offsets,
                                                       const int32_t *__restrict__ order, uint32_t n, int E, int per,
                                                       uint32_t C, uint32_t *__restrict__ count, uint32_t most,
                                                       uint2 *__restrict__ turn) {
    // a thread takes an expert, and all of them share those of many pieces
    __shared__ uint32_t s_from[THREADS], s_pieces[THREADS];
    const long long e0 = (long long)blockIdx.x * per, e = e0 + threadIdx.x;
    uint32_t from = 0, pieces = 0;
    if (threadIdx.x < per && e < E) {
        from = min((uint32_t)__ldg(offsets + e), n);
        pieces = pieces_of(from, min((uint32_t)__ldg(offsets + e + 1), n), C);
    }
    auto put = [&](uint32_t expert, uint32_t a, uint32_t k) {
        const uint32_t at = a + k * C;
        if (at >= n) return;
        const uint32_t j = (uint32_t)__ldg(order + at);
        const uint32_t b = j < n ? (uint32_t)((unsigned long long)j * BUCKETS / n) : BUCKETS - 1;
        const uint32_t t = atomicAdd(count + b, 1u);
        if (PLACE && t < most) turn[t] = make_uint2(expert, k);
    };
    if (pieces) put((uint32_t)e, from, 0);
    s_from[threadIdx.x] = from;
    s_pieces[threadIdx.x] = pieces;
    if (!__syncthreads_or(pieces > 1)) return;
    for (int l = 0; l < per; ++l)
        for (uint32_t k = 1 + threadIdx.x; k < s_pieces[l]; k += THREADS) put((uint32_t)(e0 + l), s_from[l], k);
}
// count[b] = pieces of the parts before b; count[BUCKETS] = all
__global__ void __launch_bounds__(1024) turn_scan_kernel(uint32_t *__restrict__ count) {
    __shared__ uint32_t warp_total[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint4 v = reinterpret_cast<uint4 *>(count)[threadIdx.x];
    const uint32_t mine = v.x + v.y + v.z + v.w;
    uint32_t s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) warp_total[warp] = s;
    __syncthreads();
    uint32_t before = s - mine;
    for (int q = 0; q < warp; ++q) before += warp_total[q];
    const uint4 o = make_uint4(before, before + v.x, before + v.x + v.y, before + v.x + v.y + v.z);
    reinterpret_cast<uint4 *>(count)[threadIdx.x] = o;
    if (threadIdx.x == 1023) count[BUCKETS] = before + mine;
}
static_assert(BUCKETS == 4 * 1024, "turn_scan_kernel takes four counts a thread");

template <typename T, int VEC>
__global__ void __launch_bounds__(THREADS, 4) piece_kernel(const T *__restrict__ G, uint32_t ldg,
                                                        const float *__restrict__ w,
                                                        const int32_t *__restrict__ offsets,
                                                        const int32_t *__restrict__ order, uint32_t n, int K, int E,
                                                        int D, int log_l, uint32_t C,
                                                        const uint32_t *__restrict__ count, uint32_t most,
                                                        const uint2 *__restrict__ turn, float *__restrict__ dF,
                                                        float *__restrict__ partial) {
    const int lane = threadIdx.x & 31, in_row = lane & ((1 << log_l) - 1);
    const uint32_t t = (uint32_t)(((long long)blockIdx.x * THREADS + threadIdx.x) >> 5);
    if (t >= min(__ldg(count + BUCKETS), most)) return;
    const uint2 piece = __ldg(turn + t);
    if (piece.x >= (uint32_t)E) return;
    const uint32_t from = min((uint32_t)__ldg(offsets + piece.x), n), end = min((uint32_t)__ldg(offsets + piece.x + 1), n);
    if (piece.y >= pieces_of(from, end, C)) return;
    const uint32_t a = from + piece.y * C, b = min(a + C, end);
    const bool whole = end - from <= C;
    constexpr int NP = lane_pieces<T, VEC>();
    const int step = VEC << log_l, wide = NP * step;
    for (int slab = blockIdx.y * wide; slab < D; slab += gridDim.y * wide) {
        const int c = slab + in_row * VEC;
        float acc[NP][VEC + 1];
        sum_run<T, VEC, NP>(G, ldg, w, order, n, (uint32_t)K, a, b, c, D, log_l, acc);
        float *to = whole ? dF + (long long)piece.x * D : partial + piece_row(from, piece.y, C) * D;
#pragma unroll
        for (int v = 0; v < NP; ++v)
            if (lane >> log_l == 0 && c + v * step < D) store_sums<VEC>(to + c + v * step, acc[v]);
    }
}

// the partial rows of every expert of several pieces, by a warp, or by the
// block where they are many; `per` experts a block
__global__ void __launch_bounds__(THREADS) piece_join_kernel(const int32_t *__restrict__ offsets, uint32_t n, int E,
                                                             int per, int D, uint32_t C,
                                                             const float *__restrict__ partial,
                                                             float *__restrict__ dF) {
    __shared__ uint32_t s_from[THREADS], s_pieces[THREADS];
    __shared__ float part[WARPS][33];
    const int warp = threadIdx.x >> 5;
    const long long e0 = (long long)blockIdx.x * per, e = e0 + threadIdx.x;
    // a thread an expert first: most have no partial rows
    uint32_t from = 0, pieces = 0;
    if (threadIdx.x < per && e < E) {
        from = min((uint32_t)__ldg(offsets + e), n);
        pieces = pieces_of(from, min((uint32_t)__ldg(offsets + e + 1), n), C);
    }
    s_from[threadIdx.x] = from;
    s_pieces[threadIdx.x] = pieces;
    if (!__syncthreads_or(pieces > 1)) return;
    auto rows_of = [&](uint32_t f) { return [=](uint32_t k) { return partial + piece_row(f, k, C) * D; }; };
    for (int l = warp; l < per; l += WARPS)
        if (s_pieces[l] > 1 && s_pieces[l] <= LONG)
            sum_rows_warp(rows_of(s_from[l]), 0u, s_pieces[l] - 1, D, dF + (e0 + l) * D);
    for (int l = 0; l < per; ++l)
        if (s_pieces[l] > LONG) sum_rows_block(rows_of(s_from[l]), 0u, s_pieces[l] - 1, D, dF + (e0 + l) * D, part);
}

int ceil_log2(int v) {
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}

// lanes for a row of D elements in pieces of VEC, at most a warp
int group_log(int D, int vec) {
    const int pieces = (D + vec - 1) / vec;
    return pieces >= 32 ? 5 : ceil_log2(pieces);
}

// a row distance below 2^30 elements, in bytes
template <typename T> uint32_t row_bytes(long long ld) { return (uint32_t)(ld * (long long)sizeof(T)); }

struct Shape {
    unsigned blocks;
    int log_l;
    int turns;  // 2^k - 1: pieces that neighbouring groups begin at
    bool row_per_block;
};

// A group loops over its row's pieces.  With fewer lanes a row's ids, weights
// and dot products are handled fewer times over, with more the loads of a row
// lie closer.  16-byte pieces: gathers up to four a lane, two lanes at the
// least (1024 x 1024 x 64 f32: 86 us, 104 with two a lane, 147 with one; 2048 x
// 2048 x 32 bf16: 168 us with two lanes, 192 with one, 212 with four), spreads
// two (65,536 x 8 of 256 bf16: 51 us, 55 with four); smaller ones, up to eight
// a lane while a group's load has 16 bytes (768 x 512 x 41 f32: 84 us, 168 with
// 32 lanes).  Few rows get all the lanes that a row has pieces for, and wide
// ones a block.
Shape shape_of(long long n, int D, int vec, int bytes, bool gathers) {
    Shape s;
    s.log_l = group_log(D, vec);
    s.row_per_block = D > 32 * vec && n < 148 * 8;
    const int pieces = (D + vec - 1) / vec;
    const int fewest = vec * bytes == 16 ? max(1, s.log_l - (gathers ? 2 : 1))
                                         : min(5, max(ceil_log2(16 / (vec * bytes)), ceil_log2((pieces + 7) / 8)));
    while (!s.row_per_block && pieces <= 256 && s.log_l > fewest && (n << (s.log_l - 1)) / 32 >= 148 * 64) --s.log_l;
    s.turns = 0;  // used with 16-byte pieces
    while ((vec * bytes << s.log_l) < 128 && (2 * s.turns + 2) << s.log_l <= pieces) s.turns = 2 * s.turns + 1;
    const long long per_block = s.row_per_block ? 1 : THREADS >> s.log_l;
    s.blocks = (unsigned)((n + per_block - 1) / per_block);
    return s;
}

template <typename T, int VEC, bool FULL, bool SUM, bool DOT>
void gather_launch(const Shape &s, const T *R, long long ld_rows, const int32_t *at, uint32_t n_at, const float *w,
                   const T *G, long long ld_other, long long n, int K, int D, T *out, long long ld_out, float *dots,
                   cudaStream_t st) {
    const uint32_t ldr = row_bytes<T>(ld_rows), ldg = row_bytes<T>(ld_other), ldo = row_bytes<T>(ld_out);
    if (s.row_per_block)
        gather_kernel<T, VEC, FULL, SUM, DOT, true><<<s.blocks, THREADS, 0, st>>>(R, ldr, at, n_at, w, G, ldg, n, K, D,
                                                                                  5, 0, out, ldo, dots);
    else
        gather_kernel<T, VEC, FULL, SUM, DOT, false><<<s.blocks, THREADS, 0, st>>>(R, ldr, at, n_at, w, G, ldg, n, K,
                                                                                   D, s.log_l, s.turns, out, ldo, dots);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, int VEC>
cudaError_t gather(RowsIn rows, const int32_t *at, long long n_at, const float *w, RowsIn other, long long n, int K,
                   int D, RowsOut out, float *dots, cudaStream_t st) {
    const T *r = static_cast<const T *>(rows.p), *g = static_cast<const T *>(other.p);
    T *o = static_cast<T *>(out.p);
    const Shape s = shape_of(n, D, VEC, sizeof(T), true);
    const uint32_t m = (uint32_t)n_at;
    const bool full = K == K_MAX && aligned16(at) && aligned16(w) && aligned16(dots);
    if (o && dots) {
        if (full) gather_launch<T, VEC, true, true, true>(s, r, rows.ld, at, m, w, g, other.ld, n, K, D, o, out.ld, dots, st);
        else gather_launch<T, VEC, false, true, true>(s, r, rows.ld, at, m, w, g, other.ld, n, K, D, o, out.ld, dots, st);
    } else if (o) {
        if (full) gather_launch<T, VEC, true, true, false>(s, r, rows.ld, at, m, w, g, 0, n, K, D, o, out.ld, dots, st);
        else gather_launch<T, VEC, false, true, false>(s, r, rows.ld, at, m, w, g, 0, n, K, D, o, out.ld, dots, st);
    } else {
        if (full) gather_launch<T, VEC, true, false, true>(s, r, rows.ld, at, m, w, g, other.ld, n, K, D, o, 0, dots, st);
        else gather_launch<T, VEC, false, false, true>(s, r, rows.ld, at, m, w, g, other.ld, n, K, D, o, 0, dots, st);
    }
    return cudaGetLastError();
}

template <typename T, int VEC, bool FULL, bool DOT>
void spread_launch(const Shape &s, const T *X, long long ld_x, const int32_t *at, uint32_t n_at, const float *w,
                   const T *R, long long ld_rows, long long n, int K, int D, T *S, long long ld_to, float *dots,
                   cudaStream_t st) {
    const uint32_t ldx = row_bytes<T>(ld_x), ldr = row_bytes<T>(ld_rows), lds = row_bytes<T>(ld_to);
    if (s.row_per_block)
        spread_kernel<T, VEC, FULL, DOT, true><<<s.blocks, THREADS, 0, st>>>(X, ldx, at, n_at, w, R, ldr, n, K, D, 5,
                                                                             S, lds, dots);
    else
        spread_kernel<T, VEC, FULL, DOT, false><<<s.blocks, THREADS, 0, st>>>(X, ldx, at, n_at, w, R, ldr, n, K, D,
                                                                              s.log_l, S, lds, dots);
}

template <typename T, int VEC>
cudaError_t spread(RowsIn x, const int32_t *at, long long n_at, const float *w, RowsIn rows, long long n, int K,
                   int D, RowsOut to, float *dots, cudaStream_t st) {
    const T *xp = static_cast<const T *>(x.p), *r = static_cast<const T *>(rows.p);
    T *o = static_cast<T *>(to.p);
    const Shape s = shape_of(n, D, VEC, sizeof(T), false);
    const uint32_t m = (uint32_t)n_at;
    const bool full = K == K_MAX && aligned16(at) && aligned16(w) && aligned16(dots);
    if (dots) {
        if (full) spread_launch<T, VEC, true, true>(s, xp, x.ld, at, m, w, r, rows.ld, n, K, D, o, to.ld, dots, st);
        else spread_launch<T, VEC, false, true>(s, xp, x.ld, at, m, w, r, rows.ld, n, K, D, o, to.ld, dots, st);
    } else {
        if (full) spread_launch<T, VEC, true, false>(s, xp, x.ld, at, m, w, r, 0, n, K, D, o, to.ld, dots, st);
        else spread_launch<T, VEC, false, false>(s, xp, x.ld, at, m, w, r, 0, n, K, D, o, to.ld, dots, st);
    }
    return cudaGetLastError();
}

// calls f<T, VEC> with the piece that all matrices allow
#define BY_PIECE(T, bytes, f, ...)                                        \
    ((bytes) == 16 ? f<T, 16 / sizeof(T)>(__VA_ARGS__)                    \
                   : (bytes) == 4 ? f<T, 4 / sizeof(T)>(__VA_ARGS__) : f<T, 1>(__VA_ARGS__))

template <typename T>
cudaError_t gather_typed(RowsIn rows, const int32_t *at, long long n_at, const float *w, RowsIn other, long long n,
                         int K, int D, RowsOut out, float *dots, cudaStream_t st) {
    int b = piece_bytes(rows.p, rows.ld, D, sizeof(T));
    if (dots) b = min(b, piece_bytes(other.p, other.ld, D, sizeof(T)));
    if (out.p) b = min(b, piece_bytes(out.p, out.ld, D, sizeof(T)));
    return BY_PIECE(T, b, gather, rows, at, n_at, w, other, n, K, D, out, dots, st);
}

template <typename T>
cudaError_t spread_typed(RowsIn x, const int32_t *at, long long n_at, const float *w, RowsIn rows, long long n, int K,
                         int D, RowsOut to, float *dots, cudaStream_t st) {
    int b = min(piece_bytes(x.p, x.ld, D, sizeof(T)), piece_bytes(to.p, to.ld, D, sizeof(T)));
    if (dots) b = min(b, piece_bytes(rows.p, rows.ld, D, sizeof(T)));
    return BY_PIECE(T, b, spread, x, at, n_at, w, rows, n, K, D, to, dots, st);
}

// Near rows, positions per chunk: about an expert's average share, so that
// few experts are cut (a cut costs two partial rows) and few share a warp,
// between 128 (four steps of a warp) and 4096 (an expert with 2^25 pairs then
// leaves 8192 partial rows).  Far rows, positions per piece: twice that share
// and more, so that most experts are whole.  Either way no more than leaves a
// chunk for each of the 32 warps of a multiprocessor: 65,536 x 8 pairs of nine
// experts in 128 chunks of 4096 took 139 us, in 4096 of 128 a tenth.
uint32_t chunk_of(long long n, int E, bool far) {
    long long c = far ? 512 : 128;
    while (c < 4096 && c < n / E * (far ? 2 : 1) && c * 2 <= n / (148 * 32)) c <<= 1;
    return (uint32_t)c;
}

// Far rows: dout beyond half of the L2; and from 2^21 pairs on pieces pay for
// their three small kernels anyway, since whole experts leave no partial rows
// (768 x 512 x 64 f16, 50,000 sites: 141 us against 164 by chunks; 512 x 256,
// 2,000 sites: 100 against 57).
constexpr size_t FAR_BYTES = 64u << 20;
constexpr long long FAR_PAIRS = 1 << 21;
bool is_far(long long n_rows, int K, int D, size_t element) {
    return n_rows * K >= FAR_PAIRS || (size_t)n_rows * D * element > FAR_BYTES;
}

size_t up(size_t v) { return (v + 255) & ~size_t(255); }

// workspace: partial rows, then the experts that chunks cut, or the counts
// and the turns of the pieces
struct Space {
    uint32_t C, chunks, most;  // most: pieces at most
    float *partial;
    int32_t *cut_expert;
    uint32_t *count;
    uint2 *turn;
    size_t bytes;
    Space(void *ws, long long n, int E, int D, bool far) {
        C = chunk_of(n, E, far);
        chunks = (uint32_t)((n + C - 1) / C);
        most = chunks + (uint32_t)min((long long)E, n);
        char *p = static_cast<char *>(ws);
        partial = reinterpret_cast<float *>(p);
        size_t at = up(sizeof(float) * 2 * ((size_t)chunks + 1) * D);
        cut_expert = reinterpret_cast<int32_t *>(p + at);
        count = reinterpret_cast<uint32_t *>(p + at);
        if (!far) {
            bytes = at + up(sizeof(int32_t) * (size_t)chunks);
            return;
        }
        at += up(sizeof(uint32_t) * (BUCKETS + 1));
        turn = reinterpret_cast<uint2 *>(p + at);
        bytes = at + up(sizeof(uint2) * (size_t)most);
    }
};

template <typename T, int VEC>
cudaError_t segments(RowsIn g, const float *w, const int32_t *offsets, const int32_t *order, long long n, int K,
                     int E, int D, float *dF, void *ws, cudaStream_t st) {
    const bool far = is_far(n / K, K, D, sizeof(T));
    const Space s(ws, n, E, D, far);
    const T *G = static_cast<const T *>(g.p);
    constexpr int NP = lane_pieces<T, VEC>();
    const int log_l = group_log(D, NP * VEC), wide = (NP * VEC) << log_l;
    const unsigned slabs = (unsigned)min((D + wide - 1) / wide, 65535);
    const uint32_t m = (uint32_t)n;
    if (!far) {
        const dim3 grid((s.chunks + WARPS - 1) / WARPS, slabs);
        chunk_kernel<T, VEC><<<grid, THREADS, 0, st>>>(G, row_bytes<T>(g.ld), w, offsets, order, m, K, E, D,
                                                       log_l, s.C, s.chunks, dF, s.partial, s.cut_expert);
        if (s.chunks > 1)
            join_kernel<<<(s.chunks + WARPS - 1) / WARPS, THREADS, 0, st>>>(offsets, s.cut_expert, m, E, D, s.C,
                                                                            s.chunks, s.partial, dF);
        return cudaGetLastError();
    }
    const cudaError_t e = cudaMemsetAsync(s.count, 0, sizeof(uint32_t) * (BUCKETS + 1), st);
    if (e != cudaSuccess) return e;
    const int per = E <= 1024 ? 1 : E <= 16384 ? 16 : THREADS;
    const unsigned experts = (unsigned)(((long long)E + per - 1) / per);
    turn_kernel<false><<<experts, THREADS, 0, st>>>(offsets, order, m, E, per, s.C, s.count, s.most, s.turn);
    turn_scan_kernel<<<1, 1024, 0, st>>>(s.count);
    turn_kernel<true><<<experts, THREADS, 0, st>>>(offsets, order, m, E, per, s.C, s.count, s.most, s.turn);
    const dim3 grid((s.most + WARPS - 1) / WARPS, slabs);
    piece_kernel<T, VEC><<<grid, THREADS, 0, st>>>(G, row_bytes<T>(g.ld), w, offsets, order, m, K, E, D,
                                                   log_l, s.C, s.count, s.most, s.turn, dF, s.partial);
    piece_join_kernel<<<experts, THREADS, 0, st>>>(offsets, m, E, per, D, s.C, s.partial, dF);
    return cudaGetLastError();
}

template <typename T>
cudaError_t segments_typed(RowsIn g, const float *w, const int32_t *offsets, const int32_t *order, long long n,
                           int K, int E, int D, float *dF, void *ws, cudaStream_t st) {
    return BY_PIECE(T, piece_bytes(g.p, g.ld, D, sizeof(T)), segments, g, w, offsets, order, n, K, E, D, dF, ws, st);
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
    // of any element type: whether rows are far depends on it
    const long long n = n_rows * K;
    return max(Space(nullptr, n, E, D, false).bytes, is_far(n_rows, K, D, 4) ? Space(nullptr, n, E, D, true).bytes : 0);
}

cudaError_t launch_segment_sums(int dtype, RowsIn dout, const float *w, const int32_t *offsets, const int32_t *order,
                                long long T, int K, int E, int D, float *dF, void *ws, cudaStream_t st) {
    // experts without pairs
    const cudaError_t e = cudaMemsetAsync(dF, 0, sizeof(float) * (size_t)E * D, st);
    if (e != cudaSuccess) return e;
    const long long n = T * K;
    if (dtype == 0) return segments_typed<float>(dout, w, offsets, order, n, K, E, D, dF, ws, st);
    if (dtype == 1) return segments_typed<__nv_bfloat16>(dout, w, offsets, order, n, K, E, D, dF, ws, st);
    return segments_typed<__half>(dout, w, offsets, order, n, K, E, D, dF, ws, st);
}

}  // namespace sad
