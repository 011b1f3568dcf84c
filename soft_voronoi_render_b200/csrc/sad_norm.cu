// sad_norm.cu -- layer norm of rows, forward and backward, with the gradients
// of its scale and shift.
//
// Forward, per row: mean, variance about that mean, y = (x - mean) rstd gamma
// + beta.  The sum's mean carries roundings of the elements' size: a row whose
// spread is small beside its mean (under 1/32 of it) has its mean and variance
// corrected by the mean of its deviations, which leaves roundings of the
// spread's size (4096 x 8192 f32 53 us, 51 without; for every row the wide forms
// took 3 to 7 % longer).
// Backward, with g = dy gamma and h = (x - mean) rstd: dx = rstd (g - mean(g) - h
// mean(g h)), dgamma = sum over rows of dy h, dbeta = sum of dy.
//
// Bound by memory: x and y once forward; dy, x and dx once backward.
//
// Rows of up to 64 pieces of 16 bytes (256 float32, 512 16-bit elements): a
// group of L <= 32 lanes a row, a few pieces a lane.  Wider rows of whole
// pieces: a block a row (two where the registers are there: the second one's
// loads and sums fill the first one's waits); backward, as many blocks as
// stay resident take rows in turn, and every thread copies its own pieces of
// the rows ahead into shared memory asynchronously (cp.async) and reads back
// only what it copied, so the copies need no barrier and two steps, up to 128 KB
// a block, are on their way (none in rows of more than 8192 float32, where one
// step fills the space).  Rows that no 16-byte piece fits (odd sizes, odd
// addresses) go in pieces of 4 bytes or one element through registers.
//
// Backward, a lane also keeps its columns' dgamma and dbeta in registers; the
// groups of a block are joined once at its end, and the blocks' partial rows
// by a second kernel, in a fixed order: a lane adds few rows before the joins
// (42 for 393,216 rows of 64), which keeps the float32 sums close to their
// exact values.
//
// Measured (copy rate 6,540 GB/s): 393,216 x 64 f32 forward 32 us (0.97 of
// it), backward 50 + 4 us (0.86); 8191 x 4096 bf16 forward 27 us (0.75),
// backward 54 + 4 us (0.53, 42 us without dgamma and dbeta): there the sums'
// registers leave 16 warps a multiprocessor, and what they wait for is one
// another's reductions (512 threads of half the columns took 81 us).
#include <algorithm>

#include "sad_features.h"
#include "sad_rows.cuh"

namespace sad {

using std::max;
using std::min;

namespace {

constexpr int THREADS = 256;   // of a block of row groups
constexpr int SMS = 148;

// a lane's pieces of a row, `step` columns apart; columns beyond D are 0
template <typename T, int VEC, int NV> struct RowPart {
    Pack<T, VEC> p[NV];
    __device__ __forceinline__ void load(const T *row, int c0, int step, int D) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (c0 + i * step < D) {
                p[i] = load_pack<T, VEC>(row + c0 + i * step);
            } else {
                p[i].clear();
            }
        }
    }
    // from here on the elements are widened again: kept as float32 they
    // would take twice the registers (243 instead of 96 for 16 pieces)
    __device__ __forceinline__ void stay_packed() {
        if (sizeof(T) * VEC % 4) return;
        uint32_t *w = reinterpret_cast<uint32_t *>(p);
#pragma unroll
        for (int i = 0; i < (int)(NV * VEC * sizeof(T) / 4); ++i) asm volatile("" : "+r"(w[i]));
    }
};

// s / D with inv = 1 / D: the quotient's remainder corrects it
__device__ __forceinline__ float mean_of(float s, float D, float inv) {
    const float m = s * inv;
    return fmaf(fmaf(-m, D, s), inv, m);
}

// whether a row with the sum dd of squared deviations from m has its mean
// corrected, and how: d is the sum of the deviations.  A row of equal elements
// then has exactly that mean.
__device__ __forceinline__ bool is_narrow(float dd, float m, float inv) { return dd * (1024.0f * inv) < m * m; }
__device__ __forceinline__ void correct(float d, float inv, float &m, float &dd) {
    const float e = d * inv;
    m += e;
    dd = fmaxf(fmaf(-e, d, dd), 0.0f);  // (a narrow row's are no NaN)
}

// the most threads of a block that shares a row of at most 16384 elements
constexpr int block_bound(int vec, int nv) { return 16384 / vec / nv < 1024 ? 16384 / vec / nv : 1024; }

__device__ __forceinline__ float lanes_sum(float v, int L) {
    for (int o = L >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// sum over the block, the same bits in every thread; scratch holds a float a
// warp
__device__ __forceinline__ float block_sum(float v, float *scratch) {
    v = group_sum<32>(v);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int q = 0; q < blockDim.x / 32; ++q) s += scratch[q];
    return s;
}

// gamma or beta of a piece (NULL: `other`)
template <int VEC> __device__ __forceinline__ void load_param(const float *__restrict__ p, int c, float other, float (&v)[VEC]) {
    constexpr int W = VEC % 4 == 0 ? 4 : VEC;  // pieces of 4 or 2 come aligned, see aligned_params
#pragma unroll
    for (int q = 0; q < VEC; q += W) {
        Pack<float, W> f;
        if (p) f = *reinterpret_cast<const Pack<float, W> *>(p + c + q);
#pragma unroll
        for (int u = 0; u < W; ++u) v[q + u] = p ? f.v[u] : other;
    }
}

template <typename T, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? block_bound(VEC, NV) : THREADS) norm_kernel(const T *x, long long ldx,
                                                                     const float *__restrict__ gamma,
                                                                     const float *__restrict__ beta, float eps,
                                                                     long long n, int D, int log_l, T *y,
                                                                     long long ldy, float *__restrict__ mean,
                                                                     float *__restrict__ rstd) {
    __shared__ float scratch[3][32];
    const int L = BLOCK ? blockDim.x : 1 << log_l;
    const int lane = threadIdx.x & (BLOCK ? 0xffff : L - 1);
    const int c0 = lane * VEC, step = L * VEC;
    const long long r = BLOCK ? blockIdx.x : ((long long)blockIdx.x * THREADS + threadIdx.x) >> log_l;
    const bool in = r < n;
    RowPart<T, VEC, NV> row;
    row.load(x + r * ldx, c0, step, in ? D : 0);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int q = 0; q < VEC; ++q) s += row.p[i].get(q);
    }
    const float inv = 1.0f / (float)D;
    float m = mean_of(BLOCK ? block_sum(s, scratch[0]) : lanes_sum(s, L), (float)D, inv);
    row.stay_packed();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (c0 + i * step < D) {
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float d = row.p[i].get(q) - m;
                s = fmaf(d, d, s);
            }
        }
    }
    s = BLOCK ? block_sum(s, scratch[1]) : lanes_sum(s, L);
    // a block's threads agree, and a warp's groups go along with any that does
    const bool narrow = is_narrow(s, m, inv);
    if (BLOCK ? narrow : __any_sync(0xffffffffu, narrow)) {
        row.stay_packed();
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (c0 + i * step < D) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) d += row.p[i].get(q) - m;
            }
        }
        d = BLOCK ? block_sum(d, scratch[2]) : lanes_sum(d, L);
        if (narrow) correct(d, inv, m, s);
    }
    // rsqrtf is within 2 ulp
    const float rs = rsqrtf(fmaf(s, inv, eps));
    if (!in) return;
    row.stay_packed();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * step;
        if (c >= D) break;
        float g[VEC], b[VEC];
        load_param<VEC>(gamma, c, 1.0f, g);
        load_param<VEC>(beta, c, 0.0f, b);
        float f[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) f[q] = fmaf((row.p[i].get(q) - m) * rs, g[q], b[q]);
        Pack<T, VEC> o;
        o.set(f);
        store_pack<T, VEC>(y + r * ldy + c, o);
    }
    if (lane == 0) {
        if (mean) mean[r] = m;
        if (rstd) rstd[r] = rs;
    }
}

// SUMS: also the block's sums for dgamma and dbeta, 2 D elements from block to
// block (one block: dgamma and dbeta themselves)
// BLOCK: 0, or the most threads of a block that shares a row
template <typename T, int VEC, int NV, int BLOCK, bool SUMS>
__global__ void __launch_bounds__(BLOCK ? BLOCK : THREADS, BLOCK ? 1 : 2) norm_backward_kernel(
    const T *dy, long long lddy, const T *__restrict__ x, long long ldx, const float *__restrict__ gamma,
    const float *__restrict__ mean, const float *__restrict__ rstd, long long n, int D, int log_l, T *dx,
    long long lddx, float *__restrict__ sum_g, float *__restrict__ sum_b) {
    __shared__ float scratch[2][2][32];
    const int L = BLOCK ? blockDim.x : 1 << log_l;
    const int lane = threadIdx.x & (BLOCK ? 0xffff : L - 1);
    const int c0 = lane * VEC, step = L * VEC;
    const int per_block = BLOCK ? 1 : THREADS >> log_l;
    const float inv = 1.0f / (float)D;
    float dg[SUMS ? NV * VEC : 1] = {}, db[SUMS ? NV * VEC : 1] = {};
    // a block of 1024 has no registers left for the row ahead
    constexpr bool AHEAD = BLOCK < 1024;
    const int mine = BLOCK ? 0 : threadIdx.x >> log_l;
    const long long stride = (long long)gridDim.x * per_block;
    RowPart<T, VEC, NV> g, h, g_next, h_next;
    float m_next = 0.0f, rs_next = 0.0f;
    auto fetch = [&](long long r) {
        const bool in = r < n;
        g_next.load(dy + r * lddy, c0, step, in ? D : 0);
        h_next.load(x + r * ldx, c0, step, in ? D : 0);
        // a row beyond the last has x = m = rs = dy = 0
        m_next = in ? __ldg(mean + r) : 0.0f;
        rs_next = in ? __ldg(rstd + r) : 0.0f;
    };
    long long r0 = (long long)blockIdx.x * per_block;
    if (AHEAD && r0 < n) fetch(r0 + mine);
    int turn = 0;
    for (; r0 < n; r0 += stride, turn ^= 1) {
        const long long r = r0 + mine;
        if (!AHEAD) fetch(r);
        g = g_next;
        h = h_next;
        const float m = m_next, rs = rs_next;
        if (AHEAD && r0 + stride < n) fetch(r + stride);
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c >= D) break;
            float gm[VEC];
            load_param<VEC>(gamma, c, 1.0f, gm);
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const int k = i * VEC + q;
                const float hk = (h.p[i].get(q) - m) * rs, dk = g.p[i].get(q);
                if (SUMS) {
                    dg[k] = fmaf(dk, hk, dg[k]);
                    db[k] += dk;
                }
                a = fmaf(dk, gm[q], a);
                b = fmaf(__fmul_rn(dk, gm[q]), hk, b);
            }
        }
        if (BLOCK) {
            a = group_sum<32>(a);
            b = group_sum<32>(b);
            // two sets of sums in turn: one barrier a row
            if ((threadIdx.x & 31) == 0) {
                scratch[turn][0][threadIdx.x >> 5] = a;
                scratch[turn][1][threadIdx.x >> 5] = b;
            }
            __syncthreads();
            a = b = 0.0f;
            for (int q = 0; q < blockDim.x / 32; ++q) {
                a += scratch[turn][0][q];
                b += scratch[turn][1][q];
            }
        } else {
            a = lanes_sum(a, L);
            b = lanes_sum(b, L);
        }
        a *= inv;
        b *= inv;
        if (r >= n) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c >= D) break;
            float gm[VEC];
            load_param<VEC>(gamma, c, 1.0f, gm);
            float f[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float hk = (h.p[i].get(q) - m) * rs;
                f[q] = rs * fmaf(g.p[i].get(q), gm[q], -fmaf(hk, b, a));
            }
            Pack<T, VEC> o;
            o.set(f);
            store_pack<T, VEC>(dx + r * lddx + c, o);
        }
    }
    if (!SUMS) return;
    sum_g += (size_t)blockIdx.x * 2 * D;
    sum_b += (size_t)blockIdx.x * 2 * D;
    if (BLOCK) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const int c = c0 + i * step + q;
                if (c0 + i * step >= D) break;
                sum_g[c] = dg[i * VEC + q];
                sum_b[c] = db[i * VEC + q];
            }
        }
        return;
    }
    // the warp's groups, then the warps (in order)
    extern __shared__ float join[];  // [warps][D]
    const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        for (int o = L; o < 32; o <<= 1) {
            dg[i] += __shfl_xor_sync(0xffffffffu, dg[i], o);
            db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
        if (wl < L) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                if (c >= D) break;
#pragma unroll
                for (int q = 0; q < VEC; ++q) join[warp * D + c + q] = which ? db[i * VEC + q] : dg[i * VEC + q];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += THREADS) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < THREADS / 32; ++q) s += join[q * D + c];
            (which ? sum_b : sum_g)[c] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// wide rows of whole 16-byte pieces
// ---------------------------------------------------------------------------
constexpr int WIDE_THREADS = 512;

__device__ __forceinline__ void copy_piece(void *shared, const void *global) {
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(shared);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(global) : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until all but the newest N groups have arrived
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One thread's pieces i * blockDim.x + threadIdx.x of ROWS rows of two
// matrices a step: a ring in shared memory of as many steps as 192 KB hold, the
// current one among them: three, or one of eight pieces
template <typename T, int NV, int ROWS> struct Ring {
    static constexpr int VEC = 16 / sizeof(T), STAGES = 12 / (NV * ROWS);
    uint4 *base;  // [STAGES][ROWS][2][NV][blockDim.x]
    int slot = 0;
    static size_t bytes(int threads) { return (size_t)STAGES * ROWS * 2 * NV * threads * 16; }
    __device__ __forceinline__ uint4 *at(int s, int mat, int i) const {
        return base + ((size_t)(s * ROWS * 2 + mat) * NV + i) * blockDim.x + threadIdx.x;
    }
    __device__ __forceinline__ void fetch(int s, int mat, const T *row, int pieces) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c < pieces) copy_piece(at(s, mat, i), row + (size_t)c * VEC);
        }
    }
    __device__ __forceinline__ Pack<T, VEC> get(int mat, int i) const {
        return *reinterpret_cast<const Pack<T, VEC> *>(at(slot, mat, i));
    }
    __device__ __forceinline__ void next() { slot = slot + 1 == STAGES ? 0 : slot + 1; }
};

// The backward kernels write out which products are fused with which sums, so
// that dx has the same bits with and without the sums.

// sums of `mine` over the warps of the block for each of N values, the same
// bits in every thread; one barrier
template <int N>
__device__ __forceinline__ void block_sums(const float (&mine)[N], float (*scratch)[32], float (&all)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float s[N];
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = mine[j];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
    }
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < N; ++j) scratch[j][warp] = s[j];
    }
    __syncthreads();
    // at most 16 warps
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = (lane & 15) < warps ? scratch[j][lane & 15] : 0.0f;
#pragma unroll
    for (int o = 8; o; o >>= 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) all[j] = s[j];
}

// ROWS rows a block, side by side.  Only a thread's last piece may lie beyond
// the row (wide_threads), and nothing branches on it but loads and stores: with
// branches between the pieces the loads of one waited for the sums of another.
template <typename T, int NV, int ROWS>
__global__ void __launch_bounds__(WIDE_THREADS, 2) norm_wide_kernel(const T *x, long long ldx,
                                                                    const float *__restrict__ gamma,
                                                                    const float *__restrict__ beta, float eps,
                                                                    long long n, int D, T *y, long long ldy,
                                                                    float *__restrict__ mean,
                                                                    float *__restrict__ rstd) {
    constexpr int VEC = 16 / sizeof(T);
    __shared__ float scratch[3][ROWS][32];
    const long long r0 = (long long)blockIdx.x * ROWS;
    const int c0 = threadIdx.x * VEC, step = blockDim.x * VEC;
    RowPart<T, VEC, NV> row[ROWS];
    const float inv = 1.0f / (float)D;
    float s[ROWS], m[ROWS], rs[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) row[j].load(x + (r0 + j) * ldx, c0, step, r0 + j < n ? D : 0);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        Two sum = two(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < VEC; q += 2) sum = add_two(sum, pair_at(row[j].p[i], q));
        }
        float other;
        both(sum, s[j], other);
        s[j] += other;
    }
    block_sums<ROWS>(s, scratch[0], m);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        row[j].stay_packed();
        m[j] = mean_of(m[j], (float)D, inv);
        Two sum = two(0.0f, 0.0f);
        const Two mm = two(-m[j], -m[j]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Two part = sum;
#pragma unroll
            for (int q = 0; q < VEC; q += 2) {
                const Two d = add_two(pair_at(row[j].p[i], q), mm);
                part = fma_two(d, d, part);
            }
            if (i < NV - 1 || c0 + i * step < D) sum = part;
        }
        float other;
        both(sum, s[j], other);
        s[j] += other;
    }
    block_sums<ROWS>(s, scratch[1], rs);
    bool narrow = false;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) narrow |= is_narrow(rs[j], m[j], inv);
    if (narrow) {  // the same in every thread
        float d[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            row[j].stay_packed();
            s[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (c0 + i * step < D) {
#pragma unroll
                    for (int q = 0; q < VEC; ++q) s[j] += row[j].p[i].get(q) - m[j];
                }
            }
        }
        block_sums<ROWS>(s, scratch[2], d);
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
            if (is_narrow(rs[j], m[j], inv)) correct(d[j], inv, m[j], rs[j]);
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        row[j].stay_packed();
        rs[j] = rsqrtf(fmaf(rs[j], inv, eps));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = min(c0 + i * step, D - VEC);
        const bool in = i < NV - 1 || c0 + i * step < D;
        float g[VEC], b[VEC];
        load_param<VEC>(gamma, c, 1.0f, g);
        load_param<VEC>(beta, c, 0.0f, b);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            float f[VEC];
            const Two mm = two(-m[j], -m[j]), rr = two(rs[j], rs[j]);
#pragma unroll
            for (int q = 0; q < VEC; q += 2)
                both(fma_two(mul_two(add_two(pair_at(row[j].p[i], q), mm), rr), two(g[q], g[q + 1]), two(b[q], b[q + 1])),
                     f[q], f[q + 1]);
            Pack<T, VEC> o;
            o.set(f);
            if (in && r0 + j < n) store_pack<T, VEC>(y + (r0 + j) * ldy + c, o);
        }
    }
    if (threadIdx.x < ROWS && r0 + threadIdx.x < n) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (j != threadIdx.x) continue;
            if (mean) mean[r0 + j] = m[j];
            if (rstd) rstd[r0 + j] = rs[j];
        }
    }
}

// ROWS rows at a time, blocks in turn
template <typename T, int NV, int ROWS, bool SUMS>
__global__ void __launch_bounds__(WIDE_THREADS) norm_wide_backward_kernel(
    const T *dy, long long lddy, const T *__restrict__ x, long long ldx, const float *__restrict__ gamma,
    const float *__restrict__ mean, const float *__restrict__ rstd, long long n, int D, T *dx, long long lddx,
    float *__restrict__ sum_g, float *__restrict__ sum_b) {
    constexpr int VEC = 16 / sizeof(T);
    using R = Ring<T, NV, ROWS>;
    extern __shared__ uint4 ring_base[];
    __shared__ float scratch[2][2 * ROWS][32];
    const int pieces = D / VEC;
    const long long stride = (long long)gridDim.x * ROWS;
    const float inv = 1.0f / (float)D;
    R ring{ring_base};
    Two dg[SUMS ? NV * VEC / 2 : 1], db[SUMS ? NV * VEC / 2 : 1];
#pragma unroll
    for (int i = 0; i < (SUMS ? NV * VEC / 2 : 1); ++i) dg[i] = db[i] = two(0.0f, 0.0f);
    auto fetch = [&](int s, long long r) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (r + j < n) {
                ring.fetch(s, 2 * j, dy + (r + j) * lddy, pieces);
                ring.fetch(s, 2 * j + 1, x + (r + j) * ldx, pieces);
            }
        }
        copies_end_group();
    };
    // gamma stays in registers where there are enough: read again for every row
    // it is most of what goes through the L1
    constexpr bool KEEP = NV * VEC <= 16;
    float kept[KEEP ? NV * VEC : 1];
    if (KEEP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float gm[VEC];
            load_param<VEC>(gamma, min(i * (int)blockDim.x + (int)threadIdx.x, pieces - 1) * VEC, 1.0f, gm);
#pragma unroll
            for (int q = 0; q < VEC; ++q) kept[i * VEC + q] = gm[q];
        }
    }
    float m_next[ROWS], rs_next[ROWS];
    auto fetch_stats = [&](long long r) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            m_next[j] = r + j < n ? __ldg(mean + r + j) : 0.0f;
            rs_next[j] = r + j < n ? __ldg(rstd + r + j) : 0.0f;
        }
    };
    long long r = (long long)blockIdx.x * ROWS;
#pragma unroll
    for (int s = 0; s < R::STAGES - 1; ++s) fetch(s, r + s * stride);
    fetch_stats(r);
    for (int turn = 0; r < n; r += stride, turn ^= 1) {
        fetch(ring.slot ? ring.slot - 1 : R::STAGES - 1, r + (R::STAGES - 1) * stride);
        float m[ROWS], rs[ROWS], sums[2 * ROWS], all[2 * ROWS];
        Two pairs[2 * ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) m[j] = m_next[j], rs[j] = rs_next[j];
        fetch_stats(r + stride);
        copies_wait<R::STAGES - 1>();
        RowPart<T, VEC, NV> g[ROWS], h[ROWS];
#pragma unroll
        for (int j = 0; j < 2 * ROWS; ++j) pairs[j] = two(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = min(i * (int)blockDim.x + (int)threadIdx.x, pieces - 1);
            const bool in = i < NV - 1 || i * (int)blockDim.x + (int)threadIdx.x < pieces;
            float gm[VEC];
            if (KEEP) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) gm[q] = kept[i * VEC + q];
            } else {
                load_param<VEC>(gamma, c * VEC, 1.0f, gm);
            }
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                g[j].p[i].clear();
                h[j].p[i].clear();
                if (in && r + j < n) {
                    g[j].p[i] = ring.get(2 * j, i);
                    h[j].p[i] = ring.get(2 * j + 1, i);
                }
                const Two mm = two(-m[j], -m[j]), rr = two(rs[j], rs[j]);
#pragma unroll
                for (int q = 0; q < VEC; q += 2) {
                    const int k = (i * VEC + q) / 2;
                    const Two hk = mul_two(add_two(pair_at(h[j].p[i], q), mm), rr), dk = pair_at(g[j].p[i], q);
                    if (SUMS) {
                        dg[k] = fma_two(dk, hk, dg[k]);
                        db[k] = add_two(db[k], dk);
                    }
                    const Two gk = mul_two(dk, two(gm[q], gm[q + 1]));
                    pairs[2 * j] = add_two(pairs[2 * j], gk);
                    pairs[2 * j + 1] = fma_two(gk, hk, pairs[2 * j + 1]);
                }
            }
        }
        ring.next();
#pragma unroll
        for (int j = 0; j < 2 * ROWS; ++j) {
            float other;
            both(pairs[j], sums[j], other);
            sums[j] += other;
        }
        // two sets of scratch in turn: one barrier a step
        block_sums<2 * ROWS>(sums, scratch[turn], all);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            g[j].stay_packed();
            h[j].stay_packed();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = min(i * (int)blockDim.x + (int)threadIdx.x, pieces - 1);
            const bool in = i < NV - 1 || i * (int)blockDim.x + (int)threadIdx.x < pieces;
            float gm[VEC];
            if (KEEP) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) gm[q] = kept[i * VEC + q];
            } else {
                load_param<VEC>(gamma, c * VEC, 1.0f, gm);
            }
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                const float a = all[2 * j] * inv, b = all[2 * j + 1] * inv;
                float f[VEC];
                const Two mm = two(-m[j], -m[j]), rr = two(rs[j], rs[j]), aa = two(-a, -a), bb = two(-b, -b);
#pragma unroll
                for (int q = 0; q < VEC; q += 2) {
                    const Two hk = mul_two(add_two(pair_at(h[j].p[i], q), mm), rr);
                    const Two gk = fma_two(pair_at(g[j].p[i], q), two(gm[q], gm[q + 1]), fma_two(hk, bb, aa));
                    both(mul_two(rr, gk), f[q], f[q + 1]);
                }
                Pack<T, VEC> o;
                o.set(f);
                if (in && r + j < n) store_pack<T, VEC>(dx + (r + j) * lddx + (long long)c * VEC, o);
            }
        }
    }
    if (!SUMS) return;
    sum_g += (size_t)blockIdx.x * 2 * D;
    sum_b += (size_t)blockIdx.x * 2 * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c >= pieces) break;
#pragma unroll
        for (int q = 0; q < VEC; q += 2) {
            const int k = (i * VEC + q) / 2;
            both(dg[k], sum_g[c * VEC + q], sum_g[c * VEC + q + 1]);
            both(db[k], sum_b[c * VEC + q], sum_b[c * VEC + q + 1]);
        }
    }
}

// adds up the blocks' partial rows: 32 columns a block, 32 warps take a run of
// rows each (with eight the loads of 592 rows came in 74 rounds)
constexpr int JOIN_WARPS = 32;
__global__ void __launch_bounds__(JOIN_WARPS * 32) norm_join_kernel(const float *__restrict__ partial, int rows, int D,
                                                                    float *__restrict__ dgamma,
                                                                    float *__restrict__ dbeta) {
    __shared__ float part[JOIN_WARPS][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // of 2 D columns
    float s = 0.0f;
    if (c < 2 * D) {
        const int each = (rows + JOIN_WARPS - 1) / JOIN_WARPS;
        const int q1 = min(rows, (warp + 1) * each);
#pragma unroll 8
        for (int q = warp * each; q < q1; ++q) s += __ldg(partial + (size_t)q * 2 * D + c);
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp || c >= 2 * D) return;
    s = 0.0f;
#pragma unroll
    for (int q = 0; q < JOIN_WARPS; ++q) s += part[q][lane];
    if (c < D) dgamma[c] = s;
    else dbeta[c - D] = s;
}

// How a row is shared out: groups of 2^log_l lanes, or a block of `threads`.
struct Shape {
    bool block;
    int log_l;
    int threads;
    long long blocks;  // for all rows
};

// at most `most` pieces a lane.  Groups: the power of two of lanes that
// leaves the fewest idle, the smaller on a tie (fewer shuffles).
Shape shape_of(long long n, int pieces, int most, bool block) {
    Shape s;
    s.block = block;
    s.log_l = 5;
    if (block) {
        s.threads = ((pieces + most - 1) / most + 31) / 32 * 32;
        s.blocks = n;
        return s;
    }
    int best = 1 << 30;
    for (int l = 0; l <= 5; ++l) {
        const int each = (pieces + (1 << l) - 1) >> l;
        if (each <= most && (each << l) < best) {
            best = each << l;
            s.log_l = l;
        }
    }
    s.threads = THREADS;
    const int per_block = THREADS >> s.log_l;
    s.blocks = (n + per_block - 1) / per_block;
    return s;
}

template <typename T, int VEC, int NV>
void forward_shape(const Shape &s, RowsIn x, const float *gamma, const float *beta, float eps, long long n, int D,
                   RowsOut y, float *mean, float *rstd, cudaStream_t st) {
    const T *xp = static_cast<const T *>(x.p);
    T *yp = static_cast<T *>(y.p);
    if (s.block)
        norm_kernel<T, VEC, NV, true><<<(unsigned)s.blocks, s.threads, 0, st>>>(xp, x.ld, gamma, beta, eps, n, D, 0,
                                                                                yp, y.ld, mean, rstd);
    else
        norm_kernel<T, VEC, NV, false><<<(unsigned)s.blocks, s.threads, 0, st>>>(xp, x.ld, gamma, beta, eps, n, D,
                                                                                 s.log_l, yp, y.ld, mean, rstd);
}

// blocks of a kernel that takes rows in turn: all that stay resident by its
// registers, at most one a row and `most`
int resident_blocks(int registers, int threads, size_t shared, long long rows, long long most) {
    const int warps = threads / 32;
    int per_sm = min(64 / warps, 65536 / ((registers + 7) / 8 * 8 * 32 * warps));
    per_sm = min(per_sm, (int)(227 * 1024 / (shared + 2048)));  // 1 KB of the system's, and the static arrays
    return (int)min(min(rows, most), (long long)SMS * max(per_sm, 1));
}
template <typename F> int registers_of(F kernel) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kernel) == cudaSuccess ? a.numRegs : 128;
}

// wide rows: pieces a thread, two or what 512 threads need
int wide_pieces(int pieces) {
    int nv = 2;
    while (pieces > nv * WIDE_THREADS) nv *= 2;
    return nv;
}
// rows side by side: a second one hides the first one's reductions, where the
// registers of its pieces are there
constexpr int wide_rows(int nv) { return nv == 2 ? 2 : 1; }
// (fewer pieces than nv * threads, never fewer than (nv - 1) * threads)
int wide_threads(int pieces, int nv) { return ((pieces + nv - 1) / nv + 31) / 32 * 32; }

template <typename F> cudaError_t allow_shared(F kernel, size_t bytes) {
    // 48 KB without asking, the kernel's static arrays among them
    return bytes <= 40 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int NV>
cudaError_t forward_wide(RowsIn x, const float *gamma, const float *beta, float eps, long long n, int D, RowsOut y,
                         float *mean, float *rstd, cudaStream_t st) {
    constexpr int ROWS = wide_rows(NV);
    norm_wide_kernel<T, NV, ROWS>
        <<<(unsigned)((n + ROWS - 1) / ROWS), wide_threads(D * (int)sizeof(T) / 16, NV), 0, st>>>(
            static_cast<const T *>(x.p), x.ld, gamma, beta, eps, n, D, static_cast<T *>(y.p), y.ld, mean, rstd);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t forward(RowsIn x, const float *gamma, const float *beta, float eps, long long n, int D, RowsOut y,
                    float *mean, float *rstd, cudaStream_t st) {
    const int pieces = (D + VEC - 1) / VEC;
    if constexpr (VEC * sizeof(T) == 16) {
        if (pieces > 64) {
            constexpr int MOST = sizeof(T) * 2;  // 16384 elements
            const int nv = wide_pieces(pieces);
            return nv == 2   ? forward_wide<T, 2>(x, gamma, beta, eps, n, D, y, mean, rstd, st)
                   : nv == 4 ? forward_wide<T, 4>(x, gamma, beta, eps, n, D, y, mean, rstd, st)
                             : forward_wide<T, MOST>(x, gamma, beta, eps, n, D, y, mean, rstd, st);
        }
        forward_shape<T, VEC, 2>(shape_of(n, pieces, 2, false), x, gamma, beta, eps, n, D, y, mean, rstd, st);
        return cudaGetLastError();
    }
    // fewer rows than four a multiprocessor: as many lanes a row as there are
    const bool few = n < SMS * 4 && pieces > 64;
    // otherwise few lanes: what a row costs beside its elements (430
    // instructions a warp) is shared by the rows of a warp
    const int most = few ? (pieces <= 2048 ? 2 : pieces <= 8192 ? 8 : 16) : pieces <= 128 ? 8 : 16;
    const Shape s = shape_of(n, pieces, most, few || pieces > 512);
    if (most == 2) forward_shape<T, VEC, 2>(s, x, gamma, beta, eps, n, D, y, mean, rstd, st);
    else if (most == 8) forward_shape<T, VEC, 8>(s, x, gamma, beta, eps, n, D, y, mean, rstd, st);
    else forward_shape<T, VEC, 16>(s, x, gamma, beta, eps, n, D, y, mean, rstd, st);
    return cudaGetLastError();
}

// Backward: a lane's elements of a row in groups (32 bytes), and of a block
// that shares a row without 16-byte pieces
template <typename T> constexpr int lane_elems() { return 32 / sizeof(T); }
constexpr int BLOCK_ELEMS = 16;

// Where a backward pass puts its blocks' sums: into dgamma and dbeta where
// there is one block, else into the workspace, for the second kernel
struct Sums {
    float *dgamma, *dbeta, *partial;
    bool wanted() const { return dgamma != nullptr; }
    float *g(int blocks) const { return blocks == 1 ? dgamma : partial; }
    float *b(int blocks, int D) const { return blocks == 1 ? dbeta : partial + D; }
};

// most blocks of a backward pass, a partial row each
long long backward_blocks(int D) { return D <= 1024 ? SMS * 8 : D <= 4096 ? SMS * 4 : SMS * 2; }

template <typename T, int VEC, int NV, int BLOCK>
int backward_shape(const Shape &s, RowsIn dy, RowsIn x, const float *gamma, const float *mean, const float *rstd,
                   long long n, int D, RowsOut dx, Sums sums, cudaStream_t st) {
    const T *dyp = static_cast<const T *>(dy.p), *xp = static_cast<const T *>(x.p);
    auto kernel = sums.wanted() ? norm_backward_kernel<T, VEC, NV, BLOCK, true> : norm_backward_kernel<T, VEC, NV, BLOCK, false>;
    const size_t shared = sums.wanted() && !BLOCK ? sizeof(float) * (THREADS / 32) * D : 0;
    static const int registers[2] = {registers_of(norm_backward_kernel<T, VEC, NV, BLOCK, false>),
                                     registers_of(norm_backward_kernel<T, VEC, NV, BLOCK, true>)};
    const int blocks = resident_blocks(registers[sums.wanted()], s.threads, shared, s.blocks, backward_blocks(D));
    kernel<<<blocks, s.threads, shared, st>>>(dyp, dy.ld, xp, x.ld, gamma, mean, rstd, n, D, s.log_l,
                                              static_cast<T *>(dx.p), dx.ld, sums.g(blocks), sums.b(blocks, D));
    return blocks;
}

template <typename T, int NV>
int backward_wide(RowsIn dy, RowsIn x, const float *gamma, const float *mean, const float *rstd, long long n, int D,
                  RowsOut dx, Sums sums, cudaStream_t st, cudaError_t &e) {
    const int threads = wide_threads(D * (int)sizeof(T) / 16, NV);
    constexpr int ROWS = wide_rows(NV);
    const size_t shared = Ring<T, NV, ROWS>::bytes(threads);
    auto kernel = sums.wanted() ? norm_wide_backward_kernel<T, NV, ROWS, true> : norm_wide_backward_kernel<T, NV, ROWS, false>;
    e = allow_shared(kernel, shared);
    if (e != cudaSuccess) return 0;
    static const int registers[2] = {registers_of(norm_wide_backward_kernel<T, NV, ROWS, false>),
                                     registers_of(norm_wide_backward_kernel<T, NV, ROWS, true>)};
    const int blocks = resident_blocks(registers[sums.wanted()], threads, shared, (n + ROWS - 1) / ROWS,
                                       backward_blocks(D));
    kernel<<<blocks, threads, shared, st>>>(static_cast<const T *>(dy.p), dy.ld, static_cast<const T *>(x.p), x.ld,
                                            gamma, mean, rstd, n, D, static_cast<T *>(dx.p), dx.ld, sums.g(blocks),
                                            sums.b(blocks, D));
    return blocks;
}

template <typename T, int VEC>
cudaError_t backward(RowsIn dy, RowsIn x, const float *gamma, const float *mean, const float *rstd, long long n,
                     int D, RowsOut dx, float *dgamma, float *dbeta, float *partial, cudaStream_t st) {
    const int pieces = (D + VEC - 1) / VEC;
    const Sums p{dgamma, dbeta, partial};
    constexpr bool WHOLE = VEC * sizeof(T) == 16;
    constexpr int NV = lane_elems<T>() / VEC;
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (pieces <= 32 * NV) {
        blocks = backward_shape<T, VEC, NV, 0>(shape_of(n, pieces, NV, false), dy, x, gamma, mean, rstd, n, D, dx, p, st);
    } else if constexpr (WHOLE) {
        constexpr int MOST = sizeof(T) * 2;  // 16384 elements
        const int nv = wide_pieces(pieces);
        blocks = nv == 2   ? backward_wide<T, 2>(dy, x, gamma, mean, rstd, n, D, dx, p, st, e)
                 : nv == 4 ? backward_wide<T, 4>(dy, x, gamma, mean, rstd, n, D, dx, p, st, e)
                           : backward_wide<T, MOST>(dy, x, gamma, mean, rstd, n, D, dx, p, st, e);
    } else {
        constexpr int M = BLOCK_ELEMS / VEC;
        const Shape s = shape_of(n, pieces, M, true);
        blocks = s.threads <= 512 ? backward_shape<T, VEC, M, 512>(s, dy, x, gamma, mean, rstd, n, D, dx, p, st)
                                  : backward_shape<T, VEC, M, 1024>(s, dy, x, gamma, mean, rstd, n, D, dx, p, st);
    }
    if (e != cudaSuccess) return e;
    if (p.wanted() && blocks > 1)
        norm_join_kernel<<<(2 * D + 31) / 32, JOIN_WARPS * 32, 0, st>>>(partial, blocks, D, dgamma, dbeta);
    return cudaGetLastError();
}

// gamma and beta are read in pieces too (NULL is aligned)
bool aligned_params(const float *a, const float *b) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// 16-byte pieces where every matrix allows them, else 4 bytes, else one element
#define BY_PIECE(T, bytes, f, ...)                     \
    ((bytes) == 16 ? f<T, 16 / sizeof(T)>(__VA_ARGS__) \
                   : (bytes) == 4 ? f<T, 4 / sizeof(T)>(__VA_ARGS__) : f<T, 1>(__VA_ARGS__))

template <typename T>
cudaError_t forward_typed(RowsIn x, const float *gamma, const float *beta, float eps, long long n, int D, RowsOut y,
                          float *mean, float *rstd, cudaStream_t st) {
    int b = min(piece_bytes(x.p, x.ld, D, sizeof(T)), piece_bytes(y.p, y.ld, D, sizeof(T)));
    if (!aligned_params(gamma, beta)) b = sizeof(T);
    return BY_PIECE(T, b, forward, x, gamma, beta, eps, n, D, y, mean, rstd, st);
}

template <typename T>
cudaError_t backward_typed(RowsIn dy, RowsIn x, const float *gamma, const float *mean, const float *rstd, long long n,
                           int D, RowsOut dx, float *dgamma, float *dbeta, float *partial, cudaStream_t st) {
    int b = min(min(piece_bytes(x.p, x.ld, D, sizeof(T)), piece_bytes(dy.p, dy.ld, D, sizeof(T))),
                piece_bytes(dx.p, dx.ld, D, sizeof(T)));
    if (!aligned_params(gamma, nullptr)) b = sizeof(T);
    return BY_PIECE(T, b, backward, dy, x, gamma, mean, rstd, n, D, dx, dgamma, dbeta, partial, st);
}

}  // namespace

// a partial row of dgamma and dbeta for each block of the backward pass
size_t layer_norm_workspace_bytes(long long n_rows, int D) {
    return sizeof(float) * 2 * (size_t)D * (size_t)min(backward_blocks(D), max(n_rows, 1ll));
}

cudaError_t launch_layer_norm(int dtype, RowsIn x, const float *gamma, const float *beta, float eps, long long T,
                              int D, RowsOut y, float *mean, float *rstd, cudaStream_t st) {
    if (dtype == 0) return forward_typed<float>(x, gamma, beta, eps, T, D, y, mean, rstd, st);
    if (dtype == 1) return forward_typed<__nv_bfloat16>(x, gamma, beta, eps, T, D, y, mean, rstd, st);
    return forward_typed<__half>(x, gamma, beta, eps, T, D, y, mean, rstd, st);
}

cudaError_t launch_layer_norm_backward(int dtype, RowsIn dy, RowsIn x, const float *gamma, const float *mean,
                                       const float *rstd, long long T, int D, RowsOut dx, float *dgamma, float *dbeta,
                                       void *ws, cudaStream_t st) {
    float *p = static_cast<float *>(ws);
    if (dtype == 0) return backward_typed<float>(dy, x, gamma, mean, rstd, T, D, dx, dgamma, dbeta, p, st);
    if (dtype == 1) return backward_typed<__nv_bfloat16>(dy, x, gamma, mean, rstd, T, D, dx, dgamma, dbeta, p, st);
    return backward_typed<__half>(dy, x, gamma, mean, rstd, T, D, dx, dgamma, dbeta, p, st);
}

}  // namespace sad
