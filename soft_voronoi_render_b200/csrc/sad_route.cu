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
//
// Several passes over many pairs are bound by their scattered writes: in the
// last one the pairs come in the order of their low digit, and each writes 4
// bytes of place to a sector of its own (2048 x 2048 x 8 pairs, 131,072 sites:
// 490 us for 1.6 GB).  Candidate lists are coherent, though: 4096 pairs of
// neighbouring rows hold a few hundred sites.  So there the pairs are sorted
// within tiles of 4096 first, in shared memory; only the tiles' runs of one
// expert (about 15 pairs each) are sorted by the passes above; and every tile
// then writes its part of order and place, in the pairs' own order.
//
// Measured: those lists 454 us (0.14 of the copy rate by the floor's bytes; 196
// us of it the tiles' sort, bound by instructions and shared memory, 110 us
// their writing, 74 us the runs' sort, 51 us the runs' lists, places and
// offsets); 768 x 512 x 8 pairs of 50,000 sites 89 us, 65,536 x 8 of 512
// experts 27 us, up to 1024 pairs 3 us in one launch.
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
    bool by_runs;
};

// Tiles that are sorted in shared memory, and the pairs from which on they are:
// a dozen launches against the scattered writes of seven.  Lists of images:
// 393,216 x 8 122 us by runs, 95 without; 1,048,576 x 8 206 and 233; 4,194,304
// x 8 462 and 1,040.  (Random lists of 4,194,304 x 8 over 131,072 sites have no
// runs: 3.6 ms against 2.4.)
constexpr int RUN_ITEMS = 16;
constexpr int RUN_TILE = THREADS * RUN_ITEMS;
constexpr long long RUN_PAIRS = 3 << 21;
constexpr int TILE_BITS = 12;      // a place in a tile, or a run's length less 1 ...
constexpr int RUN_KEY_BITS = 20;   // ... in one word with the key
static_assert(RUN_TILE == 1 << TILE_BITS && TILE_BITS + RUN_KEY_BITS == 32, "one word a pair");
constexpr int RUN_BLOCKS = 148 * 8;

Plan make_plan(long long n, int E) {
    int key_bits = 1;
    while ((1ll << key_bits) < (long long)E + 1) ++key_bits;
    Plan p;
    p.passes = (key_bits + MAX_BITS - 1) / MAX_BITS;
    p.bits = (key_bits + p.passes - 1) / p.passes;
    p.by_runs = p.passes > 1 && key_bits <= RUN_KEY_BITS && n >= RUN_PAIRS;
    const long long tiles = (n + TILE - 1) / TILE;
    p.blocks = (int)(tiles < MAX_BLOCKS ? (tiles ? tiles : 1) : MAX_BLOCKS);
    const long long tpb = (tiles + p.blocks - 1) / p.blocks;
    p.per_block = (tpb ? tpb : 1) * TILE;
    p.blocks = (int)((n + p.per_block - 1) / p.per_block);
    if (p.blocks < 1) p.blocks = 1;
    return p;
}

size_t move_shared(int D) { return (size_t)D * (sizeof(uint32_t) + WARPS * sizeof(uint16_t)); }
size_t up(size_t v) { return (v + 255) & ~size_t(255); }

__device__ __forceinline__ uint32_t key_of(int32_t id, int E) {
    return (uint32_t)id < (uint32_t)E ? (uint32_t)id : (uint32_t)E;
}

// items and items a block of a list whose length only the device knows
__device__ __forceinline__ void list_length(const uint32_t *__restrict__ length, long long &n, long long &per_block) {
    if (!length) return;
    n = min((long long)__ldg(length), n);
    const long long tiles = (n + TILE - 1) / TILE;
    per_block = (tiles + gridDim.x - 1) / gridDim.x * TILE;
}

// counts[digit][block]
__global__ void __launch_bounds__(THREADS) count_kernel(const int32_t *__restrict__ ids,
                                                        const uint2 *__restrict__ items, long long n, int E,
                                                        long long per_block, int shift, int bits,
                                                        uint32_t *__restrict__ counts,
                                                        const uint32_t *__restrict__ length) {
    extern __shared__ uint32_t hist[];
    list_length(length, n, per_block);
    const int D = 1 << bits;
    for (int d = threadIdx.x; d < D; d += THREADS) hist[d] = 0;
    __syncthreads();
    const long long lo = blockIdx.x * per_block, hi = min(n, lo + per_block);
    for (long long i = lo + threadIdx.x; i < hi; i += THREADS) {
        const uint32_t k = items ? items[i].x : key_of(ids[i], E);
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

// moves every item, a key and its pair, to its digit's place.  The first pass
// reads ids (the pair is the index); the last writes order and place.
__global__ void __launch_bounds__(THREADS, 4) move_kernel(const int32_t *__restrict__ ids,
                                                       const uint2 *__restrict__ items, long long n, int E,
                                                       long long per_block, int shift, int bits,
                                                       const uint32_t *__restrict__ counts,
                                                       const uint32_t *__restrict__ totals,
                                                       uint2 *__restrict__ items_out,
                                                       int32_t *__restrict__ order, int32_t *__restrict__ place,
                                                       int32_t *__restrict__ offsets,
                                                       const uint32_t *__restrict__ length) {
    extern __shared__ uint32_t smem[];
    list_length(length, n, per_block);
    __shared__ uint32_t warp_sum[WARPS];
    const int D = 1 << bits;
    uint32_t *base = smem;            // [D] next global position of each digit
    uint16_t *wc = reinterpret_cast<uint16_t *>(smem + D);  // [WARPS][D] counts, then starts in the tile
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    digit_bases(totals, D, base, warp_sum);
    // one pass sorts on the whole key: the digits' bases are the offsets
    if (offsets && blockIdx.x == 0)
        for (int d = threadIdx.x; d <= E; d += THREADS) offsets[d] = (int32_t)base[d];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += THREADS) base[d] += counts[(size_t)d * gridDim.x + blockIdx.x];
    const long long lo = blockIdx.x * per_block, hi = min(n, lo + per_block);
    for (long long t0 = lo; t0 < hi; t0 += TILE) {
        uint16_t *mine = wc + warp * D;
        for (int d = lane; d < D / 2; d += 32) reinterpret_cast<uint32_t *>(mine)[d] = 0;
        __syncwarp();
        uint32_t key[ITEMS], pair[ITEMS], rank[ITEMS];
#pragma unroll
        for (int q = 0; q < ITEMS; ++q) {
            const long long i = t0 + warp * (32 * ITEMS) + q * 32 + lane;
            const bool in = i < hi;
            uint2 v = make_uint2(0xffffffffu, 0);
            if (in) v = items ? items[i] : make_uint2(key_of(ids[i], E), (uint32_t)i);
            key[q] = v.x;
            pair[q] = v.y;
        }
#pragma unroll
        for (int q = 0; q < ITEMS; ++q) {
            const long long i = t0 + warp * (32 * ITEMS) + q * 32 + lane;
            const bool in = i < hi;
            const uint32_t d = key[q] >> shift & (D - 1);
            const unsigned peers = __match_any_sync(0xffffffffu, in ? d : 0xffffffffu);
            const unsigned below = peers & ((1u << lane) - 1);
            uint32_t old = 0;
            if (in) old = mine[d];
            __syncwarp();
            if (in && below == 0) mine[d] = (uint16_t)(old + __popc(peers));
            __syncwarp();
            rank[q] = old + __popc(below);
        }
        __syncthreads();
        // the warps' starts among the tile's items of a digit, two digits at a time
        uint32_t total[(1 << MAX_BITS) / (2 * THREADS)];
#pragma unroll
        for (int u = 0; u < (1 << MAX_BITS) / (2 * THREADS); ++u) {
            const int d = 2 * threadIdx.x + u * 2 * THREADS;
            if (d >= D) break;
            uint32_t at = 0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                uint32_t *c = reinterpret_cast<uint32_t *>(wc + w * D + d);
                const uint32_t add = *c;
                *c = at;
                at += add;
            }
            total[u] = at;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < ITEMS; ++q) {
            const long long i = t0 + warp * (32 * ITEMS) + q * 32 + lane;
            if (i >= hi) continue;
            const uint32_t d = key[q] >> shift & (D - 1), pos = base[d] + mine[d] + rank[q];
            if (order) {
                const bool empty = key[q] == (uint32_t)E;
                order[pos] = empty ? -1 : (int32_t)pair[q];
                place[pair[q]] = empty ? -1 : (int32_t)pos;
            } else {
                items_out[pos] = make_uint2(key[q], pair[q]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < (1 << MAX_BITS) / (2 * THREADS); ++u) {
            const int d = 2 * threadIdx.x + u * 2 * THREADS;
            if (d >= D) break;
            base[d] += total[u] & 0xffffu;
            base[d + 1] += total[u] >> 16;
        }
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

// ---------------------------------------------------------------------------
// by runs
// ---------------------------------------------------------------------------
// Sorts a tile of pairs by key in shared memory, stable; a pair is one word,
// key and place in the tile.  Writes the pairs' places in sorted order
// (local), a bit for every place where another key starts (heads) with the
// number of such places before each 32 (before), and for every run its first
// place and its word, key and length less 1; runs of tile t are entries
// t RUN_TILE + 0, 1, ...
constexpr int WORDS = RUN_TILE / 32;
__global__ void __launch_bounds__(THREADS, 4) tile_sort_kernel(const int32_t *__restrict__ ids, long long n, int E,
                                                               int passes, int bits, uint16_t *__restrict__ local,
                                                               uint32_t *__restrict__ heads,
                                                               uint16_t *__restrict__ heads_before,
                                                               uint32_t *__restrict__ run_word,
                                                               uint16_t *__restrict__ run_start,
                                                               uint32_t *__restrict__ run_count) {
    extern __shared__ uint32_t smem[];
    __shared__ uint32_t warp_sum[WARPS];
    __shared__ uint32_t word[WORDS], before[WORDS];
    const int D = 1 << bits;
    uint32_t *items = smem;                                           // [RUN_TILE]
    uint16_t *wc = reinterpret_cast<uint16_t *>(smem + RUN_TILE);     // [WARPS][D], then [RUN_TILE]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t0 = (long long)blockIdx.x * RUN_TILE;
    const int count = (int)min((long long)RUN_TILE, n - t0);
    const int p0 = warp * (32 * RUN_ITEMS) + lane;  // this thread's places: p0 + 32 q
    uint32_t item[RUN_ITEMS];
#pragma unroll
    for (int q = 0; q < RUN_ITEMS; ++q) {
        const int p = p0 + 32 * q;
        // places beyond the last pair have the largest digits and come last, so stay last
        item[q] = p < count ? key_of(__ldg(ids + t0 + p), E) << TILE_BITS | (uint32_t)p : 0xffffffffu;
    }
    uint16_t *mine = wc + warp * D;
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = TILE_BITS + pass * bits;
        for (int d = lane; d < D / 2; d += 32) reinterpret_cast<uint32_t *>(mine)[d] = 0;
        __syncwarp();
        uint32_t rank[RUN_ITEMS];
        // a match takes a round for each distinct digit of the warp, few here:
        // with a ballot a bit in its place the 2048 x 2048 lists took 428 us, not 225
#pragma unroll
        for (int q = 0; q < RUN_ITEMS; ++q) {
            const uint32_t d = item[q] >> shift & (D - 1);
            const unsigned peers = __match_any_sync(0xffffffffu, d);
            const unsigned below = peers & ((1u << lane) - 1);
            const uint32_t old = mine[d];
            __syncwarp();
            if (below == 0) mine[d] = (uint16_t)(old + __popc(peers));
            __syncwarp();
            rank[q] = old + __popc(below);
        }
        __syncthreads();
        // starts of the warps' items: digits in order, warps in order; a
        // thread takes 2 digits a step
        uint32_t carry = 0;
        for (int d0 = 0; d0 < D; d0 += 2 * THREADS) {
            const int d = d0 + 2 * threadIdx.x;
            uint32_t total = 0;  // two counts of 16 bits
            if (d < D) {
#pragma unroll
                for (int w = 0; w < WARPS; ++w) total += *reinterpret_cast<uint32_t *>(wc + w * D + d);
            }
            const uint32_t both_d = (total & 0xffffu) + (total >> 16);
            uint32_t s = both_d;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            if (lane == 31) warp_sum[warp] = s;
            __syncthreads();
            uint32_t start = carry + s - both_d;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                if (w < warp) start += warp_sum[w];
                carry += warp_sum[w];
            }
            if (d < D) {
                // both starts are at most 4096
                uint32_t at = start | (start + (total & 0xffffu)) << 16;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    uint32_t *c = reinterpret_cast<uint32_t *>(wc + w * D + d);
                    const uint32_t add = *c;
                    *c = at;
                    at += add;
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int q = 0; q < RUN_ITEMS; ++q) items[mine[item[q] >> shift & (D - 1)] + rank[q]] = item[q];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < RUN_ITEMS; ++q) item[q] = items[p0 + 32 * q];
    }
#pragma unroll
    for (int q = 0; q < RUN_ITEMS; ++q) {
        const int p = p0 + 32 * q;
        const bool head = p < count && (p == 0 || (items[p - 1] ^ item[q]) >> TILE_BITS);
        const uint32_t b = __ballot_sync(0xffffffffu, head);
        if (lane == 0) word[p >> 5] = b;
        if (p < count) local[t0 + p] = (uint16_t)(item[q] & (RUN_TILE - 1));
    }
    __syncthreads();
    static_assert(WORDS == 4 * 32, "one warp scans four words a lane");
    if (warp == 0) {
        uint32_t c[4], s = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) c[u] = __popc(word[lane * 4 + u]), s += c[u];
        const uint32_t sum = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        uint32_t b = s - sum;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            before[lane * 4 + u] = b;
            b += c[u];
        }
        if (lane == 31) run_count[blockIdx.x] = s;
    }
    __syncthreads();
    if (threadIdx.x < WORDS) {
        heads[(size_t)blockIdx.x * WORDS + threadIdx.x] = word[threadIdx.x];
        heads_before[(size_t)blockIdx.x * WORDS + threadIdx.x] = (uint16_t)before[threadIdx.x];
    }
    uint16_t *starts = wc;  // [runs]: the counters are done with
#pragma unroll
    for (int q = 0; q < RUN_ITEMS; ++q) {
        const int w = warp * RUN_ITEMS + q;
        const uint32_t b = word[w];
        if (b >> lane & 1u) starts[before[w] + __popc(b & ((1u << lane) - 1))] = (uint16_t)(32 * w + lane);
    }
    __syncthreads();
    const int runs = (int)(before[WORDS - 1] + __popc(word[WORDS - 1]));
    for (int r = threadIdx.x; r < runs; r += THREADS) {
        const int p = starts[r], end = r + 1 < runs ? starts[r + 1] : count;
        run_word[t0 + r] = (items[p] & ~(uint32_t)(RUN_TILE - 1)) | (uint32_t)(end - p - 1);
        run_start[t0 + r] = (uint16_t)p;
    }
}

// base[t] = runs of the tiles before t; base[tiles] = all
__global__ void __launch_bounds__(1024) run_base_kernel(const uint32_t *__restrict__ run_count, int tiles,
                                                        uint32_t *__restrict__ base) {
    constexpr int EACH = 8;
    __shared__ uint32_t warp_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (int t0 = 0; t0 < tiles; t0 += 1024 * EACH) {
        const int t = t0 + threadIdx.x * EACH;
        uint32_t v[EACH], sum = 0;
#pragma unroll
        for (int u = 0; u < EACH; ++u) v[u] = t + u < tiles ? run_count[t + u] : 0;
#pragma unroll
        for (int u = 0; u < EACH; ++u) sum += v[u];
        uint32_t s = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        uint32_t ws = warp_sum[lane];
        const uint32_t own = ws;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, ws, o);
            if (lane >= o) ws += u;
        }
        uint32_t start = carry + s - sum + __shfl_sync(0xffffffffu, ws - own, warp);
        carry += __shfl_sync(0xffffffffu, ws, 31);
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            if (t + u < tiles) base[t + u] = start;
            start += v[u];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) base[tiles] = carry;
}

// the runs of all tiles behind one another: word, and the run's entry
__global__ void __launch_bounds__(THREADS) run_list_kernel(const uint32_t *__restrict__ run_word,
                                                           const uint32_t *__restrict__ base,
                                                           uint2 *__restrict__ items) {
    const uint32_t from = base[blockIdx.x], count = base[blockIdx.x + 1] - from;
    const uint32_t t0 = blockIdx.x * (uint32_t)RUN_TILE;
    for (uint32_t r = threadIdx.x; r < count; r += THREADS) items[from + r] = make_uint2(run_word[t0 + r], t0 + r);
}

// pairs of a run, from its word
__device__ __forceinline__ uint32_t run_length(uint32_t word) { return (word & (RUN_TILE - 1)) + 1; }

// The sorted runs' first positions: a run of runs a block, its sum first,
// then its scan behind the sums of the blocks before it.  where[entry] is the
// position for the tiles, sorted[i] the same by rank for the offsets.
__global__ void __launch_bounds__(THREADS) run_sum_kernel(const uint2 *__restrict__ items,
                                                          const uint32_t *__restrict__ length,
                                                          uint32_t *__restrict__ sums) {
    __shared__ uint32_t warp_sum[WARPS];
    const uint32_t total = *length, each = (total + gridDim.x - 1) / gridDim.x;
    const uint32_t lo = min(blockIdx.x * each, total), hi = min(lo + each, total);
    uint32_t s = 0;
    for (uint32_t i = lo + threadIdx.x; i < hi; i += THREADS) s += run_length(items[i].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0;
        for (int w = 0; w < WARPS; ++w) s += warp_sum[w];
        sums[blockIdx.x] = s;
    }
}
__global__ void __launch_bounds__(THREADS) run_place_kernel(const uint2 *__restrict__ items,
                                                            const uint32_t *__restrict__ length,
                                                            const uint32_t *__restrict__ sums,
                                                            uint32_t *__restrict__ where,
                                                            uint32_t *__restrict__ sorted) {
    __shared__ uint32_t warp_sum[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t total = *length, each = (total + gridDim.x - 1) / gridDim.x;
    const uint32_t lo = min(blockIdx.x * each, total), hi = min(lo + each, total);
    uint32_t carry = 0;
    for (int b = threadIdx.x; b < blockIdx.x; b += THREADS) carry += sums[b];
#pragma unroll
    for (int o = 16; o; o >>= 1) carry += __shfl_xor_sync(0xffffffffu, carry, o);
    if (lane == 0) warp_sum[warp] = carry;
    __syncthreads();
    carry = 0;
    for (int w = 0; w < WARPS; ++w) carry += warp_sum[w];
    __syncthreads();
    for (uint32_t i0 = lo; i0 < hi; i0 += THREADS) {
        const uint32_t i = i0 + threadIdx.x;
        const uint2 run = i < hi ? items[i] : make_uint2(0, 0);
        const uint32_t e = run.y, v = i < hi ? run_length(run.x) : 0;
        uint32_t s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        uint32_t start = carry + s - v;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) start += warp_sum[w];
            carry += warp_sum[w];
        }
        if (i < hi) {
            where[e] = start;
            sorted[i] = start;
        }
        __syncthreads();
    }
}

// offsets[e]: the first position of the first run with a key of e or more
__global__ void __launch_bounds__(THREADS) run_offsets_kernel(const uint2 *__restrict__ items,
                                                              const uint32_t *__restrict__ sorted,
                                                              const uint32_t *__restrict__ length, long long n, int E,
                                                              int32_t *__restrict__ offsets) {
    const int e = blockIdx.x * THREADS + threadIdx.x;
    if (e > E) return;
    const uint32_t total = *length;
    uint32_t lo = 0, hi = total;
    while (lo < hi) {
        const uint32_t mid = (lo + hi) >> 1;
        if (__ldg(&items[mid].x) >> TILE_BITS < (uint32_t)e) lo = mid + 1;
        else hi = mid;
    }
    offsets[e] = (int32_t)(lo < total ? sorted[lo] : (uint32_t)n);
}

// a tile's part of order and place; FULL: a tile of RUN_TILE pairs
template <bool FULL>
__device__ __forceinline__ void tile_write(int count, uint32_t t0, const uint16_t (&idx)[RUN_ITEMS], uint32_t words,
                                           uint32_t befores, uint32_t live, const uint32_t *shift, int32_t *out,
                                           int32_t *__restrict__ order, int32_t *__restrict__ place) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int q = 0; q < RUN_ITEMS; ++q) {
        const uint32_t word = __shfl_sync(0xffffffffu, words, q), before = __shfl_sync(0xffffffffu, befores, q);
        const int p = warp * (32 * RUN_ITEMS) + 32 * q + lane;
        if (!FULL && p >= count) continue;
        const uint32_t pos = shift[before + __popc(word & (0xffffffffu >> (31 - lane))) - 1] + p;
        const bool empty = pos >= live;
        order[pos] = empty ? -1 : (int32_t)(t0 + idx[q]);
        out[idx[q]] = empty ? -1 : (int32_t)pos;
    }
    __syncthreads();
    place += t0;
    if (FULL && (reinterpret_cast<uintptr_t>(place) & 15) == 0) {
#pragma unroll
        for (int q = 0; q < RUN_ITEMS / 4; ++q)
            reinterpret_cast<int4 *>(place)[q * THREADS + threadIdx.x] = reinterpret_cast<const int4 *>(out)[q * THREADS + threadIdx.x];
    } else {
        for (int p = threadIdx.x; p < count; p += THREADS) place[p] = out[p];
    }
}
__global__ void __launch_bounds__(THREADS, 6) tile_write_kernel(long long n, const uint16_t *__restrict__ local,
                                                                const uint32_t *__restrict__ heads,
                                                                const uint16_t *__restrict__ heads_before,
                                                                const uint32_t *__restrict__ where,
                                                                const uint16_t *__restrict__ run_start,
                                                                const uint32_t *__restrict__ run_count,
                                                                const int32_t *__restrict__ offsets, int E,
                                                                int32_t *__restrict__ order,
                                                                int32_t *__restrict__ place) {
    __shared__ uint32_t shift[RUN_TILE];   // position less place in the tile, of each run
    __shared__ __align__(16) int32_t out[RUN_TILE];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t0 = (long long)blockIdx.x * RUN_TILE;
    const int count = (int)min((long long)RUN_TILE, n - t0);
    const uint32_t runs = run_count[blockIdx.x];
    // everything is loaded before the first wait; lane q has the q-th word of heads
    uint16_t idx[RUN_ITEMS];
#pragma unroll
    for (int q = 0; q < RUN_ITEMS; ++q) {
        const int p = warp * (32 * RUN_ITEMS) + 32 * q + lane;
        idx[q] = p < count ? local[t0 + p] : 0;
    }
    const size_t w = (size_t)blockIdx.x * WORDS + warp * RUN_ITEMS + (lane & (RUN_ITEMS - 1));
    const uint32_t words = __ldg(heads + w), befores = __ldg(heads_before + w);
    const uint32_t live = (uint32_t)__ldg(offsets + E);  // positions from here on are empty slots
    for (uint32_t r = threadIdx.x; r < runs; r += THREADS) shift[r] = where[t0 + r] - run_start[t0 + r];
    __syncthreads();
    if (count == RUN_TILE) tile_write<true>(count, (uint32_t)t0, idx, words, befores, live, shift, out, order, place);
    else tile_write<false>(count, (uint32_t)t0, idx, words, befores, live, shift, out, order, place);
}

// workspace of the sort by runs
struct RunSpace {
    uint32_t *totals, *counts, *base, *run_count, *heads, *sums, *run_word;
    uint2 *list[2];  // runs: key and length, entry
    uint16_t *local, *run_start, *heads_before;
    int tiles;
    size_t bytes;
    RunSpace(void *ws, long long n, const Plan &p) {
        tiles = (int)((n + RUN_TILE - 1) / RUN_TILE);
        const size_t slots = (size_t)tiles * RUN_TILE;
        char *base_p = static_cast<char *>(ws);
        size_t at = 0;
        auto take = [&](size_t b) {
            char *q = base_p + at;
            at += up(b);
            return q;
        };
        totals = reinterpret_cast<uint32_t *>(take(sizeof(uint32_t) << p.bits));
        counts = reinterpret_cast<uint32_t *>(take((sizeof(uint32_t) << p.bits) * RUN_BLOCKS));
        base = reinterpret_cast<uint32_t *>(take(sizeof(uint32_t) * ((size_t)tiles + 1)));
        run_count = reinterpret_cast<uint32_t *>(take(sizeof(uint32_t) * (size_t)tiles));
        heads = reinterpret_cast<uint32_t *>(take(slots / 8));
        sums = reinterpret_cast<uint32_t *>(take(sizeof(uint32_t) * RUN_BLOCKS));
        heads_before = reinterpret_cast<uint16_t *>(take(slots / 16));
        run_word = reinterpret_cast<uint32_t *>(take(sizeof(uint32_t) * slots));
        for (int g = 0; g < 2; ++g) list[g] = reinterpret_cast<uint2 *>(take(sizeof(uint2) * slots));
        local = reinterpret_cast<uint16_t *>(take(sizeof(uint16_t) * slots));
        run_start = reinterpret_cast<uint16_t *>(take(sizeof(uint16_t) * slots));
        bytes = at;
    }
};

cudaError_t route_by_runs(const int32_t *ids, long long n, int E, const Plan &p, int32_t *offsets, int32_t *order,
                          int32_t *place, void *ws, cudaStream_t st) {
    const RunSpace s(ws, n, p);
    const int D = 1 << p.bits;
    const uint32_t *length = s.base + s.tiles;
    const size_t sort_shared = RUN_TILE * sizeof(uint32_t) + (size_t)(WARPS * D > RUN_TILE ? WARPS * D : RUN_TILE) * sizeof(uint16_t);
    tile_sort_kernel<<<s.tiles, THREADS, sort_shared, st>>>(ids, n, E, p.passes, p.bits, s.local, s.heads,
                                                            s.heads_before, s.run_word, s.run_start, s.run_count);
    run_base_kernel<<<1, 1024, 0, st>>>(s.run_count, s.tiles, s.base);
    run_list_kernel<<<s.tiles, THREADS, 0, st>>>(s.run_word, s.base, s.list[0]);
    for (int q = 0; q < p.passes; ++q) {
        const uint2 *from = s.list[q & 1];
        const long long slots = (long long)s.tiles * RUN_TILE;
        const int shift = TILE_BITS + q * p.bits;
        count_kernel<<<RUN_BLOCKS, THREADS, D * sizeof(uint32_t), st>>>(nullptr, from, slots, E, 0, shift, p.bits,
                                                                        s.counts, length);
        scan_kernel<<<D, THREADS, 0, st>>>(s.counts, RUN_BLOCKS, s.totals);
        move_kernel<<<RUN_BLOCKS, THREADS, move_shared(D), st>>>(nullptr, from, slots, E, 0, shift, p.bits, s.counts,
                                                                 s.totals, s.list[~q & 1], nullptr, nullptr, nullptr,
                                                                 length);
    }
    const uint2 *runs = s.list[p.passes & 1];
    uint32_t *sorted = reinterpret_cast<uint32_t *>(s.list[~p.passes & 1]);
    // the words of the tiles' runs are in the list: their place takes the positions
    run_sum_kernel<<<RUN_BLOCKS, THREADS, 0, st>>>(runs, length, s.sums);
    run_place_kernel<<<RUN_BLOCKS, THREADS, 0, st>>>(runs, length, s.sums, s.run_word, sorted);
    run_offsets_kernel<<<E / THREADS + 1, THREADS, 0, st>>>(runs, sorted, length, n, E, offsets);
    tile_write_kernel<<<s.tiles, THREADS, 0, st>>>(n, s.local, s.heads, s.heads_before, s.run_word, s.run_start,
                                                   s.run_count, offsets, E, order, place);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// few pairs: one launch
// ---------------------------------------------------------------------------
// A pair's place is the number of words (key, pair) below its own: every
// thread of a block compares its pair with all of them, four to a load.  Each
// block does the same for its share of the offsets, found by bisection.
constexpr int FEW = 1024;
constexpr int FEW_OFFSETS = 8192;  // a block
__global__ void __launch_bounds__(FEW) few_kernel(const int32_t *__restrict__ ids, int n, int E,
                                                  int32_t *__restrict__ offsets, int32_t *__restrict__ order,
                                                  int32_t *__restrict__ place) {
    __shared__ __align__(16) uint32_t word[FEW];
    __shared__ uint32_t sorted[FEW];
    const int j = threadIdx.x;
    const uint32_t key = j < n ? key_of(__ldg(ids + j), E) : 0, mine = j < n ? key << 10 | (uint32_t)j : 0xffffffffu;
    word[j] = mine;
    __syncthreads();
    int rank = 0;
    const uint4 *four = reinterpret_cast<const uint4 *>(word);
    for (int i = 0; i < (n + 3) / 4; ++i) {
        const uint4 v = four[i];
        rank += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
    }
    if (j < n) {
        sorted[rank] = key;
        if (blockIdx.x == 0) {
            const bool empty = key == (uint32_t)E;
            order[rank] = empty ? -1 : j;
            place[j] = empty ? -1 : rank;
        }
    }
    __syncthreads();
    const int last = min(E, (blockIdx.x + 1) * FEW_OFFSETS - 1);
    for (int e = blockIdx.x * FEW_OFFSETS + j; e <= last; e += blockDim.x) {
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sorted[mid] < (uint32_t)e) lo = mid + 1;
            else hi = mid;
        }
        offsets[e] = lo;
    }
}
// the word has 22 bits for the key
bool is_few(long long n, int E) { return n <= FEW && E < 1 << 22; }

}  // namespace

size_t route_workspace_bytes(long long n_rows, int K, int E) {
    const long long n = n_rows * K;
    if (is_few(n, E)) return up(1);  // none needed: every size has some
    const Plan p = make_plan(n, E);
    if (p.by_runs) return RunSpace(nullptr, n, p).bytes;
    const size_t table = up(sizeof(uint32_t) << p.bits) + up((sizeof(uint32_t) << p.bits) * p.blocks);
    // a list between passes, two when there are two gaps or more
    const size_t lists = p.passes > 1 ? up(sizeof(uint2) * (size_t)n) * (p.passes > 2 ? 2 : 1) : 0;
    return table + lists;
}

cudaError_t launch_route(const int32_t *ids, long long n_rows, int K, int E, int32_t *offsets, int32_t *order,
                         int32_t *place, void *ws, cudaStream_t st) {
    const long long n = n_rows * K;
    if (n == 0) return cudaMemsetAsync(offsets, 0, sizeof(int32_t) * ((size_t)E + 1), st);
    if (is_few(n, E)) {
        const int threads = n <= 32 ? 128 : ((int)n + 31) / 32 * 32;
        few_kernel<<<E / FEW_OFFSETS + 1, threads, 0, st>>>(ids, (int)n, E, offsets, order, place);
        return cudaGetLastError();
    }
    const Plan p = make_plan(n, E);
    if (p.by_runs) return route_by_runs(ids, n, E, p, offsets, order, place, ws, st);
    const int D = 1 << p.bits;
    char *w = static_cast<char *>(ws);
    uint32_t *totals = reinterpret_cast<uint32_t *>(w);
    w += up(sizeof(uint32_t) << p.bits);
    uint32_t *counts = reinterpret_cast<uint32_t *>(w);
    w += up((sizeof(uint32_t) << p.bits) * p.blocks);
    const size_t list = up(sizeof(uint2) * (size_t)n);
    const uint2 *items = nullptr;
    for (int q = 0; q < p.passes; ++q) {
        const bool last = q == p.passes - 1;
        const int shift = q * p.bits;
        count_kernel<<<p.blocks, THREADS, D * sizeof(uint32_t), st>>>(ids, items, n, E, p.per_block, shift, p.bits,
                                                                      counts, nullptr);
        scan_kernel<<<D, THREADS, 0, st>>>(counts, p.blocks, totals);
        uint2 *to = last ? nullptr : reinterpret_cast<uint2 *>(w + (size_t)(q & 1) * list);
        move_kernel<<<p.blocks, THREADS, move_shared(D), st>>>(ids, items, n, E, p.per_block, shift, p.bits, counts,
                                                               totals, to, last ? order : nullptr,
                                                               last ? place : nullptr,
                                                               last && p.passes == 1 ? offsets : nullptr, nullptr);
        items = to;
    }
    if (p.passes > 1) offsets_kernel<<<E / THREADS + 1, THREADS, 0, st>>>(ids, order, n, E, offsets);
    return cudaGetLastError();
}

}  // namespace sad
