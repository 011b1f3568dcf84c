// sad_route.cu -- rows sorted by expert: a stable radix sort of the T x K
// (id, pair) list that writes the order, its inverse and every expert's
// offset.
//
// Floor: 12 bytes a pair (ids in; order and place out) and 4 a site.  The key
// is the id, or n_sites for an empty slot, so ceil(log2(n_sites + 1)) bits
// are sorted, least significant digit first, in as few passes of at most
// MAX_BITS bits as that takes.  A pass counts each block's digits, scans the
// counts digit by digit, and ranks every item inside its warp by match
// masks, which keeps pairs of one expert in their order without atomics.
#include "sad_features.h"

namespace sad {

namespace {

constexpr int MAX_BITS = 10;
constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int ITEMS = 8;                  // per thread and tile
constexpr int TILE = THREADS * ITEMS;
constexpr int MAX_BLOCKS = 148 * 4;       // a block takes a run of whole tiles

struct Plan {
    int passes, bits;     // digits of `bits` bits
    int blocks;
    long long per_block;  // items, a multiple of TILE
};

Plan make_plan(long long n, int E) {
    int key_bits = 1;
    while ((1ll << key_bits) < (long long)E + 1) ++key_bits;
    Plan p;
    p.passes = (key_bits + MAX_BITS - 1) / MAX_BITS;
    p.bits = (key_bits + p.passes - 1) / p.passes;
    const long long tiles = (n + TILE - 1) / TILE;
    p.blocks = (int)(tiles < MAX_BLOCKS ? (tiles ? tiles : 1) : MAX_BLOCKS);
    const long long tpb = (tiles + p.blocks - 1) / p.blocks;
    p.per_block = (tpb ? tpb : 1) * TILE;
    p.blocks = (int)((n + p.per_block - 1) / p.per_block);
    if (p.blocks < 1) p.blocks = 1;
    return p;
}

size_t up(size_t v) { return (v + 255) & ~size_t(255); }

__device__ __forceinline__ uint32_t key_of(int32_t id, int E) {
    return (uint32_t)id < (uint32_t)E ? (uint32_t)id : (uint32_t)E;
}

// counts[digit][block]
__global__ void __launch_bounds__(THREADS) count_kernel(const int32_t *__restrict__ ids,
                                                        const uint32_t *__restrict__ keys, long long n, int E,
                                                        long long per_block, int shift, int bits,
                                                        uint32_t *__restrict__ counts) {
    extern __shared__ uint32_t hist[];
    const int D = 1 << bits;
    for (int d = threadIdx.x; d < D; d += THREADS) hist[d] = 0;
    __syncthreads();
    const long long lo = blockIdx.x * per_block, hi = min(n, lo + per_block);
    for (long long i = lo + threadIdx.x; i < hi; i += THREADS) {
        const uint32_t k = keys ? keys[i] : key_of(ids[i], E);
        atomicAdd(&hist[k >> shift & (D - 1)], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += THREADS) counts[(size_t)d * gridDim.x + blockIdx.x] = hist[d];
}

// one block per digit: exclusive scan of its row of counts, in place; the
// row's sum goes to totals
__global__ void __launch_bounds__(THREADS) scan_kernel(uint32_t *__restrict__ counts, int blocks,
                                                       uint32_t *__restrict__ totals) {
    __shared__ uint32_t warp_sum[WARPS];
    uint32_t *row = counts + (size_t)blockIdx.x * blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (int b0 = 0; b0 < blocks; b0 += THREADS) {
        const int b = b0 + threadIdx.x;
        const uint32_t v = b < blocks ? row[b] : 0;
        uint32_t s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += t;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        uint32_t before = carry;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += warp_sum[w];
            carry += warp_sum[w];
        }
        if (b < blocks) row[b] = before + s - v;
        __syncthreads();
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// exclusive scan of the D digit totals into base[] by the whole block
__device__ void digit_bases(const uint32_t *__restrict__ totals, int D, uint32_t *base, uint32_t *warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (int d0 = 0; d0 < D; d0 += THREADS) {
        const int d = d0 + threadIdx.x;
        const uint32_t v = d < D ? totals[d] : 0;
        uint32_t s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += t;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        uint32_t before = carry;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += warp_sum[w];
            carry += warp_sum[w];
        }
        if (d < D) base[d] = before + s - v;
        __syncthreads();
    }
}

// moves every item to its digit's place.  The first pass reads ids (the pair
// is the index); the last writes order and place instead of keys and pairs.
__global__ void __launch_bounds__(THREADS) move_kernel(const int32_t *__restrict__ ids,
                                                       const uint32_t *__restrict__ keys,
                                                       const uint32_t *__restrict__ pairs, long long n, int E,
                                                       long long per_block, int shift, int bits,
                                                       const uint32_t *__restrict__ counts,
                                                       const uint32_t *__restrict__ totals,
                                                       uint32_t *__restrict__ keys_out,
                                                       uint32_t *__restrict__ pairs_out,
                                                       int32_t *__restrict__ order, int32_t *__restrict__ place,
                                                       int32_t *__restrict__ offsets) {
    extern __shared__ uint32_t smem[];
    __shared__ uint32_t warp_sum[WARPS];
    const int D = 1 << bits;
    uint32_t *base = smem;            // [D] next global position of each digit
    uint32_t *wc = smem + D;          // [WARPS][D] counts, then starts, of each warp's items
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    digit_bases(totals, D, base, warp_sum);
    // one pass sorts on the whole key: the digits' bases are the offsets
    if (offsets && blockIdx.x == 0)
        for (int d = threadIdx.x; d <= E; d += THREADS) offsets[d] = (int32_t)base[d];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += THREADS) base[d] += counts[(size_t)d * gridDim.x + blockIdx.x];
    const long long lo = blockIdx.x * per_block, hi = min(n, lo + per_block);
    for (long long t0 = lo; t0 < hi; t0 += TILE) {
        for (int d = threadIdx.x; d < D * WARPS; d += THREADS) wc[d] = 0;
        __syncthreads();
        uint32_t key[ITEMS], pair[ITEMS], rank[ITEMS];
        uint32_t *mine = wc + warp * D;
#pragma unroll
        for (int q = 0; q < ITEMS; ++q) {
            const long long i = t0 + warp * (32 * ITEMS) + q * 32 + lane;
            const bool in = i < hi;
            key[q] = in ? (keys ? keys[i] : key_of(ids[i], E)) : 0xffffffffu;
            pair[q] = in ? (pairs ? pairs[i] : (uint32_t)i) : 0;
            const uint32_t d = key[q] >> shift & (D - 1);
            const unsigned peers = __match_any_sync(0xffffffffu, in ? d : 0xffffffffu);
            const unsigned below = peers & ((1u << lane) - 1);
            uint32_t old = 0;
            if (in) old = mine[d];
            __syncwarp();
            if (in && below == 0) mine[d] = old + __popc(peers);
            __syncwarp();
            rank[q] = old + __popc(below);
        }
        __syncthreads();
        // the warps' starts within the digit; the tile's items move its base on
        for (int d = threadIdx.x; d < D; d += THREADS) {
            uint32_t s = base[d];
            for (int w = 0; w < WARPS; ++w) {
                const uint32_t c = wc[w * D + d];
                wc[w * D + d] = s;
                s += c;
            }
            base[d] = s;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < ITEMS; ++q) {
            const long long i = t0 + warp * (32 * ITEMS) + q * 32 + lane;
            if (i >= hi) continue;
            const uint32_t pos = mine[key[q] >> shift & (D - 1)] + rank[q];
            if (order) {
                const bool empty = key[q] == (uint32_t)E;
                order[pos] = empty ? -1 : (int32_t)pair[q];
                place[pair[q]] = empty ? -1 : (int32_t)pos;
            } else {
                keys_out[pos] = key[q];
                pairs_out[pos] = pair[q];
            }
        }
        __syncthreads();
    }
}

// several passes: offsets[e] by bisection of the sorted pairs (-1 ends them)
__global__ void __launch_bounds__(THREADS) offsets_kernel(const int32_t *__restrict__ ids,
                                                          const int32_t *__restrict__ order, long long n, int E,
                                                          int32_t *__restrict__ offsets) {
    const int e = blockIdx.x * THREADS + threadIdx.x;
    if (e > E) return;
    long long lo = 0, hi = n;
    while (lo < hi) {
        const long long mid = (lo + hi) >> 1;
        const int32_t j = order[mid];
        if (j >= 0 && ids[j] < e) lo = mid + 1;
        else hi = mid;
    }
    offsets[e] = (int32_t)lo;
}

}  // namespace

size_t route_workspace_bytes(long long n_rows, int K, int E) {
    const long long n = n_rows * K;
    const Plan p = make_plan(n, E);
    const size_t table = up(sizeof(uint32_t) << p.bits) + up((sizeof(uint32_t) << p.bits) * p.blocks);
    // keys and pairs between passes, twice when there are two gaps or more
    const size_t lists = p.passes > 1 ? 2 * up(sizeof(uint32_t) * (size_t)n) * (p.passes > 2 ? 2 : 1) : 0;
    return table + lists;
}

cudaError_t launch_route(const int32_t *ids, long long n_rows, int K, int E, int32_t *offsets, int32_t *order,
                         int32_t *place, void *ws, cudaStream_t st) {
    const long long n = n_rows * K;
    if (n == 0) return cudaMemsetAsync(offsets, 0, sizeof(int32_t) * ((size_t)E + 1), st);
    const Plan p = make_plan(n, E);
    const int D = 1 << p.bits;
    char *w = static_cast<char *>(ws);
    uint32_t *totals = reinterpret_cast<uint32_t *>(w);
    w += up(sizeof(uint32_t) << p.bits);
    uint32_t *counts = reinterpret_cast<uint32_t *>(w);
    w += up((sizeof(uint32_t) << p.bits) * p.blocks);
    const size_t list = up(sizeof(uint32_t) * (size_t)n);
    uint32_t *buf[2][2];
    for (int g = 0; g < 2; ++g)
        for (int h = 0; h < 2; ++h) buf[g][h] = reinterpret_cast<uint32_t *>(w + (size_t)(2 * g + h) * list);
    const uint32_t *keys = nullptr, *pairs = nullptr;
    for (int q = 0; q < p.passes; ++q) {
        const bool last = q == p.passes - 1;
        const int shift = q * p.bits;
        count_kernel<<<p.blocks, THREADS, D * sizeof(uint32_t), st>>>(ids, keys, n, E, p.per_block, shift, p.bits,
                                                                      counts);
        scan_kernel<<<D, THREADS, 0, st>>>(counts, p.blocks, totals);
        uint32_t *ko = last ? nullptr : buf[q & 1][0], *po = last ? nullptr : buf[q & 1][1];
        move_kernel<<<p.blocks, THREADS, (size_t)D * (1 + WARPS) * sizeof(uint32_t), st>>>(
            ids, keys, pairs, n, E, p.per_block, shift, p.bits, counts, totals, ko, po, last ? order : nullptr,
            last ? place : nullptr, last && p.passes == 1 ? offsets : nullptr);
        keys = ko;
        pairs = po;
    }
    if (p.passes > 1) offsets_kernel<<<E / THREADS + 1, THREADS, 0, st>>>(ids, order, n, E, offsets);
    return cudaGetLastError();
}

}  // namespace sad
