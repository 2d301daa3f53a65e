// k_embedding.cu - K8: embedding lookup with scaling, and its gradient by
// sorted ids.
//
//   out_t = scale * table[id_t]            (zeros where id_t is not in [0, rows))
//   grad_r = scale * sum over t with id_t = r of g_t, t ascending
//
// The lookup is HBM-bound: each row is read and written once. A group of L
// lanes copies K8_TOKENS rows at a time, so that their loads, whose addresses
// come from the ids, are in flight together.
//
// The gradient sorts the tokens by id (least significant digit first, stable,
// so that equal ids keep the order of their tokens) and adds runs of equal
// ids:
//   k8_sort_one    up to K8_ONE tokens: all digits in one block's shared memory
//   k8_count,      more tokens, per digit of up to 8 bits: how many of each
//   k8_scan,       value lie in each tile of K8_TILE tokens, the prefix over the
//   k8_scatter     tiles, and every token to its place
//   k8_heads,      (row form) which place of the output each run has
//   k8_scan
//   k8_runs        a warp adds 32 consecutive sorted tokens in fp32. A run that
//                  lies inside is written; the part of one that crosses into
//                  the next 32 goes to a partial row
//   k8_join        the partial rows of each crossing run, in order
// The order of every sum is fixed by the ids, so the bits repeat. Bound by the
// reading of g (once, in rows) and, for few tokens, by the launches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tt_internal.h"
#include "tt_rows.cuh"

namespace tt {
namespace {

constexpr int K8_THREADS = 256;
constexpr int K8_TOKENS = 4;

template <typename T, typename TO, typename ID, int E, int L>
__global__ void __launch_bounds__(K8_THREADS)
    k8_lookup(const T* __restrict__ table, int64_t rows, int d, const ID* __restrict__ ids, int64_t m, float scale,
              TO* __restrict__ out) {
    const int lane = threadIdx.x & (L - 1);
    const int64_t group = ((int64_t)blockIdx.x * K8_THREADS + threadIdx.x) / L;
    const int64_t groups = (int64_t)gridDim.x * K8_THREADS / L;
    for (int64_t t0 = group * K8_TOKENS; t0 < m; t0 += groups * K8_TOKENS) {
        int64_t id[K8_TOKENS];
#pragma unroll
        for (int q = 0; q < K8_TOKENS; ++q) id[q] = t0 + q < m ? (int64_t)__ldg(ids + t0 + q) : -1;
        for (int e = lane * E; e < d; e += L * E) {
            Raw<T, E> r[K8_TOKENS];
#pragma unroll
            for (int q = 0; q < K8_TOKENS; ++q) {
                if (id[q] >= 0 && id[q] < rows) r[q].load(table + id[q] * d + e); else r[q].zero();
            }
#pragma unroll
            for (int q = 0; q < K8_TOKENS; ++q) {
                if (t0 + q >= m) break;
                float x[E];
                r[q].get(x);
                // a padding row is zero whatever the scale
#pragma unroll
                for (int k = 0; k < E; ++k) x[k] = id[q] >= 0 && id[q] < rows ? x[k] * scale : 0.f;
                store_row<E>(out + (t0 + q) * d + e, x);
            }
        }
    }
}

template <typename T, typename TO, typename ID>
void lookup_shape(const void* table, int64_t rows, int d, const void* ids, int64_t m, float scale, void* out,
                  cudaStream_t s, int sm_count) {
    const T* t = static_cast<const T*>(table);
    const ID* i = static_cast<const ID*>(ids);
    TO* o = static_cast<TO*>(out);
    const int E = d % 8 == 0 ? 8 : 1;
    const int chunks = d / E;
    const int L = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
    const int64_t blocks = (m * L + (int64_t)K8_THREADS * K8_TOKENS - 1) / ((int64_t)K8_THREADS * K8_TOKENS);
    const int grid = (int)(blocks < 16 * sm_count ? blocks : 16 * sm_count);
    if (E == 8) {
        if (L == 8) k8_lookup<T, TO, ID, 8, 8><<<grid, K8_THREADS, 0, s>>>(t, rows, d, i, m, scale, o);
        else if (L == 16) k8_lookup<T, TO, ID, 8, 16><<<grid, K8_THREADS, 0, s>>>(t, rows, d, i, m, scale, o);
        else k8_lookup<T, TO, ID, 8, 32><<<grid, K8_THREADS, 0, s>>>(t, rows, d, i, m, scale, o);
    } else {
        if (L == 8) k8_lookup<T, TO, ID, 1, 8><<<grid, K8_THREADS, 0, s>>>(t, rows, d, i, m, scale, o);
        else if (L == 16) k8_lookup<T, TO, ID, 1, 16><<<grid, K8_THREADS, 0, s>>>(t, rows, d, i, m, scale, o);
        else k8_lookup<T, TO, ID, 1, 32><<<grid, K8_THREADS, 0, s>>>(t, rows, d, i, m, scale, o);
    }
}

template <typename T, typename TO>
void lookup_ids(const void* table, int64_t rows, int d, const void* ids, int id_bytes, int64_t m, float scale,
                void* out, cudaStream_t s, int sm_count) {
    if (id_bytes == 4) lookup_shape<T, TO, int32_t>(table, rows, d, ids, m, scale, out, s, sm_count);
    else lookup_shape<T, TO, int64_t>(table, rows, d, ids, m, scale, out, s, sm_count);
}

// ---------------------------------------------------------------------------
// the sort
// ---------------------------------------------------------------------------
constexpr int K8_SORT_THREADS = 256;
constexpr int K8_SORT_WARPS = K8_SORT_THREADS / 32;
constexpr int K8_KEYS = 16;                            // keys per thread
constexpr int K8_TILE = K8_SORT_THREADS * K8_KEYS;     // 4096
constexpr int K8_ONE_THREADS = 1024;
constexpr int K8_ONE = K8_ONE_THREADS * K8_KEYS;       // 16384
constexpr int K8_BINS = 256;
constexpr int K8_RUN = 32;                             // sorted tokens of a warp
constexpr int K8_RUN_WARPS = 8;
constexpr int K8_HEADS = 4096;                         // sorted tokens of a block of k8_heads

// Ids outside [0, rows) share the key `rows`, which sorts last.
template <typename ID>
__device__ __forceinline__ uint32_t key_of(ID id, uint32_t rows) {
    return id >= 0 && (uint64_t)id < rows ? (uint32_t)id : rows;
}

// One digit of a tile held in registers (key k of warp w and round r is the
// tile's element (w * K8_KEYS + r) * 32 + lane): cnt[w][v] becomes the number
// of keys with digit v in warp w, rank[r] the number of equal digits before
// the key in its warp. Keys past the end have digit >= bins.
__device__ __forceinline__ void warp_ranks(const uint32_t* digit, uint32_t (*cnt)[K8_BINS], int* rank) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int v = lane; v < K8_BINS; v += 32) cnt[warp][v] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < K8_KEYS; ++r) {
        const bool in = digit[r] < K8_BINS;
        const unsigned peers = __match_any_sync(0xffffffffu, digit[r]);
        const int before = __popc(peers & ((1u << lane) - 1u));
        const uint32_t old = in ? cnt[warp][digit[r]] : 0;
        __syncwarp();
        if (in && before == 0) cnt[warp][digit[r]] = old + __popc(peers);
        __syncwarp();
        rank[r] = (int)old + before;
    }
}

struct SortArgs {
    const void* ids;       // first pass; null afterwards
    const uint32_t* key_in;
    const uint32_t* pos_in;
    uint32_t* key_out;
    uint32_t* pos_out;
    int32_t* hist;         // [K8_BINS][tiles]
    int32_t* total;        // [K8_BINS]
    int64_t m;
    uint32_t rows;
    int tiles;
    int shift, bits;
};

template <typename ID>
__device__ __forceinline__ uint32_t load_key(const SortArgs& a, int64_t i) {
    return a.ids != nullptr ? key_of(__ldg(static_cast<const ID*>(a.ids) + i), a.rows) : __ldg(a.key_in + i);
}

template <typename ID>
__global__ void __launch_bounds__(K8_SORT_THREADS) k8_count(const SortArgs a) {
    __shared__ int h[K8_BINS];
    h[threadIdx.x] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * K8_TILE;
#pragma unroll
    for (int r = 0; r < K8_KEYS; ++r) {
        const int64_t i = base + r * K8_SORT_THREADS + threadIdx.x;
        if (i < a.m) atomicAdd(&h[(load_key<ID>(a, i) >> a.shift) & ((1u << a.bits) - 1u)], 1);
    }
    __syncthreads();
    a.hist[(int64_t)threadIdx.x * a.tiles + blockIdx.x] = h[threadIdx.x];
}

// Block b: exclusive prefix of row b of x ([rows][len]), in place, and its sum.
__global__ void __launch_bounds__(256) k8_scan(int32_t* __restrict__ x, int len, int32_t* __restrict__ total) {
    __shared__ int warp_tot[8];
    int32_t* row = x + (int64_t)blockIdx.x * len;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int run = 0;
    for (int base = 0; base < len; base += 256) {
        const int i = base + threadIdx.x;
        const int v = i < len ? row[i] : 0;
        int inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) warp_tot[warp] = inc;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            before += w < warp ? warp_tot[w] : 0;
            all += warp_tot[w];
        }
        if (i < len) row[i] = run + before + inc - v;
        run += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) total[blockIdx.x] = run;
}

// Exclusive prefix over the 256 threads of a block.
__device__ __forceinline__ int block_prefix256(int v, int* warp_tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) before += w < warp ? warp_tot[w] : 0;
    return before + inc - v;
}

template <typename ID>
__global__ void __launch_bounds__(K8_SORT_THREADS) k8_scatter(const SortArgs a) {
    __shared__ uint32_t cnt[K8_SORT_WARPS][K8_BINS];
    __shared__ int warp_tot[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t base = (int64_t)blockIdx.x * K8_TILE + (int64_t)warp * K8_KEYS * 32;
    uint32_t key[K8_KEYS], digit[K8_KEYS];
    int rank[K8_KEYS];
#pragma unroll
    for (int r = 0; r < K8_KEYS; ++r) {
        const int64_t i = base + r * 32 + lane;
        key[r] = i < a.m ? load_key<ID>(a, i) : 0u;
        digit[r] = i < a.m ? (key[r] >> a.shift) & ((1u << a.bits) - 1u) : (uint32_t)K8_BINS;
    }
    warp_ranks(digit, cnt, rank);
    const int first = block_prefix256(__ldg(a.total + threadIdx.x), warp_tot);  // has a barrier
    int at = first + __ldg(a.hist + (int64_t)threadIdx.x * a.tiles + blockIdx.x);
#pragma unroll
    for (int w = 0; w < K8_SORT_WARPS; ++w) {
        const int c = (int)cnt[w][threadIdx.x];
        cnt[w][threadIdx.x] = (uint32_t)at;
        at += c;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < K8_KEYS; ++r) {
        const int64_t i = base + r * 32 + lane;
        if (i >= a.m) continue;
        const uint32_t to = cnt[warp][digit[r]] + (uint32_t)rank[r];
        a.key_out[to] = key[r];
        a.pos_out[to] = a.ids != nullptr ? (uint32_t)i : __ldg(a.pos_in + i);
    }
}

// All digits in one block: keys and places go from registers through shared
// memory and back once per digit.
struct OneSmem {
    uint32_t key[K8_ONE];
    uint16_t pos[K8_ONE];
    uint32_t cnt[K8_ONE_THREADS / 32][K8_BINS];
    int warp_tot[8];
    int first[K8_BINS];
};

template <typename ID>
__global__ void __launch_bounds__(K8_ONE_THREADS)
    k8_sort_one(const ID* __restrict__ ids, int m, uint32_t rows, int passes, int bits, uint32_t* __restrict__ key_out,
                uint32_t* __restrict__ pos_out) {
    extern __shared__ __align__(16) uint8_t raw[];
    OneSmem& sm = *reinterpret_cast<OneSmem*>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the warps share the m tokens evenly: a warp's tokens are consecutive
    const int rounds = (m + K8_ONE_THREADS - 1) / K8_ONE_THREADS;
    const int base = warp * rounds * 32 + lane;
    uint32_t key[K8_KEYS], digit[K8_KEYS];
    uint16_t pos[K8_KEYS];
    int rank[K8_KEYS];
#pragma unroll
    for (int r = 0; r < K8_KEYS; ++r) {
        const int i = base + r * 32;
        const bool in = r < rounds && i < m;
        key[r] = in ? key_of(__ldg(ids + i), rows) : 0u;
        pos[r] = (uint16_t)i;
    }
    for (int p = 0; p < passes; ++p) {
        for (int v = lane; v < K8_BINS; v += 32) sm.cnt[warp][v] = 0;
        __syncwarp();
#pragma unroll
        for (int r = 0; r < K8_KEYS; ++r) {
            if (r >= rounds) break;
            const bool in = base + r * 32 < m;
            digit[r] = in ? (key[r] >> (p * bits)) & ((1u << bits) - 1u) : (uint32_t)K8_BINS;
            const unsigned peers = __match_any_sync(0xffffffffu, digit[r]);
            const int before = __popc(peers & ((1u << lane) - 1u));
            const uint32_t old = in ? sm.cnt[warp][digit[r]] : 0;
            __syncwarp();
            if (in && before == 0) sm.cnt[warp][digit[r]] = old + __popc(peers);
            __syncwarp();
            rank[r] = (int)old + before;
        }
        __syncthreads();
        int sum = 0;
        if (threadIdx.x < K8_BINS) {
#pragma unroll 8
            for (int w = 0; w < K8_ONE_THREADS / 32; ++w) {
                const int c = (int)sm.cnt[w][threadIdx.x];
                sm.cnt[w][threadIdx.x] = (uint32_t)sum;
                sum += c;
            }
            int inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) sm.warp_tot[warp] = inc;
            sm.first[threadIdx.x] = inc - sum;
        }
        __syncthreads();
        if (threadIdx.x < K8_BINS) {
            int before = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) before += w < warp ? sm.warp_tot[w] : 0;
            sm.first[threadIdx.x] += before;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < K8_KEYS; ++r) {
            if (r < rounds && digit[r] < K8_BINS) {
                const int to = sm.first[digit[r]] + (int)sm.cnt[warp][digit[r]] + rank[r];
                sm.key[to] = key[r];
                sm.pos[to] = pos[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < K8_KEYS; ++r) {
            const int i = base + r * 32;
            if (r < rounds && i < m) {
                key[r] = sm.key[i];
                pos[r] = sm.pos[i];
            }
        }
        // the next pass's writes to sm.key come after two more barriers
    }
#pragma unroll
    for (int r = 0; r < K8_KEYS; ++r) {
        const int i = base + r * 32;
        if (r < rounds && i < m) {
            key_out[i] = key[r];
            pos_out[i] = pos[r];
        }
    }
}

// ---------------------------------------------------------------------------
// the runs
// ---------------------------------------------------------------------------
struct RunArgs {
    const uint32_t* key;   // [m] sorted
    const uint32_t* pos;
    int64_t m;
    uint32_t rows;
    int d;
    float scale;
    int by_row;            // 1: output row = place of the run; 0: output row = id
    const int32_t* block_first;  // (by_row) runs before each block of k8_heads
    int32_t* place;        // (by_row) [chunks] runs before the warp's 32 tokens, within that block
    float* part;           // [chunks][2][d]
    int2* cross;           // crossing runs: (chunk they begin in, output row)
    int* cross_count;
    int64_t chunks;
};

__device__ __forceinline__ bool is_head(const RunArgs& a, int64_t i) {
    if (i >= a.m) return false;
    const uint32_t k = __ldg(a.key + i);
    return k < a.rows && (i == 0 || __ldg(a.key + i - 1) != k);
}

// Runs that begin in each 32 tokens: the prefix within the block's K8_HEADS
// tokens, and the block's sum.
__global__ void __launch_bounds__(128) k8_heads(const RunArgs a, int32_t* __restrict__ block_total) {
    __shared__ int warp_tot[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    static_assert(K8_HEADS == 128 * K8_RUN, "one thread per warp-chunk");
    const int64_t base = (int64_t)blockIdx.x * K8_HEADS;
    int mine = 0;  // thread t keeps the count of chunk t
    for (int c = 0; c < 32; ++c) {
        const int n = __popc(__ballot_sync(0xffffffffu, is_head(a, base + (warp * 32 + c) * K8_RUN + lane)));
        if (lane == c) mine = n;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warp_tot[w];
    const int64_t chunk = base / K8_RUN + threadIdx.x;
    if (chunk < a.chunks) a.place[chunk] = before + inc - mine;
    if (threadIdx.x == 127) block_total[blockIdx.x] = before + inc;
}

template <typename T, typename TO, typename ID, int E>
__global__ void __launch_bounds__(K8_RUN_WARPS * 32)
    k8_runs(const RunArgs a, const T* __restrict__ grad, TO* __restrict__ out, ID* __restrict__ out_ids) {
    constexpr int BATCH = 8;
    const int lane = threadIdx.x & 31;
    const int64_t chunk = (int64_t)blockIdx.x * K8_RUN_WARPS + (threadIdx.x >> 5);
    if (chunk >= a.chunks) return;
    const int64_t i0 = chunk * K8_RUN;
    const int64_t i = i0 + lane;
    const uint32_t key = i < a.m ? __ldg(a.key + i) : a.rows;
    const uint32_t pos = i < a.m ? __ldg(a.pos + i) : 0u;
    uint32_t prev = __shfl_up_sync(0xffffffffu, key, 1);
    if (lane == 0) prev = i0 > 0 ? __ldg(a.key + i0 - 1) : a.rows;
    const unsigned live = __ballot_sync(0xffffffffu, key < a.rows);
    if (live == 0) return;
    // bit q: token q begins a run (of those that count)
    const unsigned heads = __ballot_sync(0xffffffffu, key < a.rows && (prev != key || i == 0));
    const int count = __popc(live);  // live tokens come first
    const uint32_t last_key = __shfl_sync(0xffffffffu, key, 31);
    const bool goes_on = count == 32 && i0 + 32 < a.m && __ldg(a.key + i0 + 32) == last_key;
    int64_t first = 0;  // place of the first run that begins here
    if (a.by_row) first = (int64_t)__ldg(a.block_first + chunk / (K8_HEADS / K8_RUN)) + __ldg(a.place + chunk);
    const int e = (blockIdx.y * 32 + lane) * E;
    const bool in = e < a.d;
    if (out_ids != nullptr && blockIdx.y == 0 && (heads >> lane & 1u))
        out_ids[first + __popc(heads & ((1u << lane) - 1u))] = (ID)key;
    float acc[E];
#pragma unroll
    for (int k = 0; k < E; ++k) acc[k] = 0.f;
    int begun = 0;  // runs begun so far
    // write out the run that ends before token q
    auto flush = [&](int q) {
        const bool open = q == 32 && goes_on;
        if (begun == 0) {  // began in an earlier chunk
            if (in) store_row<E>(a.part + (chunk * 2) * a.d + e, acc);
        } else {
            const int64_t place = first + begun - 1;
            const int64_t row = a.by_row ? place : (int64_t)__shfl_sync(0xffffffffu, key, q - 1);
            if (open) {
                if (in) store_row<E>(a.part + (chunk * 2 + 1) * a.d + e, acc);
                if (lane == 0 && blockIdx.y == 0) a.cross[atomicAdd(a.cross_count, 1)] = make_int2((int)chunk, (int)row);
            } else if (in) {
                float y[E];
#pragma unroll
                for (int k = 0; k < E; ++k) y[k] = acc[k] * a.scale;
                store_row<E>(out + row * a.d + e, y);
            }
        }
    };
    for (int b = 0; b < count; b += BATCH) {
        Raw<T, E> r[BATCH];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const uint32_t p = __shfl_sync(0xffffffffu, pos, b + q);
            if (in && b + q < count) r[q].load(grad + (int64_t)p * a.d + e); else r[q].zero();
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            if (b + q >= count) break;
            if (heads >> (b + q) & 1u) {
                if (b + q > 0) flush(b + q);
                ++begun;
#pragma unroll
                for (int k = 0; k < E; ++k) acc[k] = 0.f;
            }
            float x[E];
            r[q].get(x);
#pragma unroll
            for (int k = 0; k < E; ++k) acc[k] += x[k];
        }
    }
    flush(count);
}

// A run that begins in chunk c and goes on: its own part row (slot 1 of c),
// then slot 0 of the chunks after c that it reaches. A warp adds up to
// K8_JOIN_WARP chunks; longer runs take the whole block, warp w the chunks
// c + 1 + w, c + 1 + w + 8, ..., and the warps' sums in order.
constexpr int K8_JOIN_WARPS = 8;
constexpr int K8_JOIN_WARP = 64;

template <int E>
__device__ __forceinline__ void add_parts(const RunArgs& a, int64_t c, int64_t from, int64_t to, int step, int e,
                                          float* acc) {
    constexpr int BATCH = 8;
    for (int64_t k0 = from; k0 < to; k0 += (int64_t)step * BATCH) {
        Raw<float, E> r[BATCH];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const int64_t k = k0 + (int64_t)q * step;
            if (k < to) r[q].load(a.part + (c + k) * 2 * a.d + e); else r[q].zero();
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            float x[E];
            r[q].get(x);
#pragma unroll
            for (int j = 0; j < E; ++j) acc[j] += x[j];
        }
    }
}

template <typename TO, int E>
__global__ void __launch_bounds__(K8_JOIN_WARPS * 32) k8_join(const RunArgs a, TO* __restrict__ out) {
    __shared__ int64_t reach[K8_JOIN_WARPS];
    __shared__ float sums[K8_JOIN_WARPS][32 * E];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = *a.cross_count;
    const int e = (blockIdx.y * 32 + lane) * E;
    const bool in = e < a.d;
    for (int b = blockIdx.x * K8_JOIN_WARPS; b < n; b += gridDim.x * K8_JOIN_WARPS) {
        int64_t k = 0;  // chunks after the first that the run reaches
        if (b + warp < n) {
            const int64_t c = a.cross[b + warp].x;
            const uint32_t key = __ldg(a.key + c * K8_RUN + K8_RUN - 1);
            while (true) {
                const int64_t i = (c + 1 + k + lane) * K8_RUN;
                const unsigned same = __ballot_sync(0xffffffffu, i < a.m && __ldg(a.key + i) == key);
                const int more = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
                k += more;
                if (more < 32) break;
            }
        }
        if (lane == 0) reach[warp] = k;
        __syncthreads();
        if (k > 0 && k <= K8_JOIN_WARP && in) {
            const int2 run = a.cross[b + warp];
            float acc[E];
            Raw<float, E> r;
            r.load(a.part + ((int64_t)run.x * 2 + 1) * a.d + e);
            r.get(acc);
            add_parts<E>(a, run.x, 1, k + 1, 1, e, acc);
#pragma unroll
            for (int j = 0; j < E; ++j) acc[j] *= a.scale;
            store_row<E>(out + (int64_t)run.y * a.d + e, acc);
        }
        for (int w = 0; w < K8_JOIN_WARPS; ++w) {
            const int64_t kw = reach[w];
            if (kw <= K8_JOIN_WARP) continue;  // the same for the whole block
            const int2 run = a.cross[b + w];
            float acc[E];
#pragma unroll
            for (int j = 0; j < E; ++j) acc[j] = 0.f;
            if (in) {
                if (warp == 0) {
                    Raw<float, E> r;
                    r.load(a.part + ((int64_t)run.x * 2 + 1) * a.d + e);
                    r.get(acc);
                }
                add_parts<E>(a, run.x, 1 + warp, kw + 1, K8_JOIN_WARPS, e, acc);
            }
#pragma unroll
            for (int j = 0; j < E; ++j) sums[warp][lane * E + j] = acc[j];
            __syncthreads();
            if (warp == 0 && in) {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    float t = sums[0][lane * E + j];
                    for (int q = 1; q < K8_JOIN_WARPS; ++q) t += sums[q][lane * E + j];
                    acc[j] = t * a.scale;
                }
                store_row<E>(out + (int64_t)run.y * a.d + e, acc);
            }
            __syncthreads();
        }
        __syncthreads();  // reach is written again
    }
}

int bit_length(uint32_t x) {
    int b = 0;
    while (x >> b) ++b;
    return b;
}

// Elements per lane: the fewest whose 32 lanes cover the row, among those
// that divide it; else the most that do.
int run_elems(int d) {
    int best = 1;
    for (int E = 1; E <= 8; E *= 2) {
        if (d % E != 0) break;
        best = E;
        if (32 * E >= d) break;
    }
    return best;
}

template <typename T, typename TO, typename ID, int E>
cudaError_t runs_launch(const RunArgs& a, const void* grad, void* out, void* out_ids, cudaStream_t s, int sm_count) {
    const int cols = (a.d + 32 * E - 1) / (32 * E);
    const dim3 grid((unsigned)((a.chunks + K8_RUN_WARPS - 1) / K8_RUN_WARPS), cols);
    note_launch_begin(TT_KIND_EMBEDDING, s);
    k8_runs<T, TO, ID, E><<<grid, K8_RUN_WARPS * 32, 0, s>>>(a, static_cast<const T*>(grad), static_cast<TO*>(out),
                                                            static_cast<ID*>(out_ids));
    note_launch_end(TT_KIND_EMBEDDING, s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.chunks < 2) return e;  // nothing crosses
    const int64_t most = (a.chunks + K8_JOIN_WARPS - 1) / K8_JOIN_WARPS;
    note_launch_begin(TT_KIND_EMBEDDING, s);
    k8_join<TO, E><<<dim3((unsigned)(most < 4 * sm_count ? most : 4 * sm_count), cols), K8_JOIN_WARPS * 32, 0, s>>>(
        a, static_cast<TO*>(out));
    note_launch_end(TT_KIND_EMBEDDING, s);
    return cudaGetLastError();
}

template <typename T, typename TO, typename ID>
cudaError_t runs_elems(const RunArgs& a, const void* grad, void* out, void* out_ids, cudaStream_t s, int sm_count) {
    switch (run_elems(a.d)) {
        case 8: return runs_launch<T, TO, ID, 8>(a, grad, out, out_ids, s, sm_count);
        case 4: return runs_launch<T, TO, ID, 4>(a, grad, out, out_ids, s, sm_count);
        case 2: return runs_launch<T, TO, ID, 2>(a, grad, out, out_ids, s, sm_count);
        default: return runs_launch<T, TO, ID, 1>(a, grad, out, out_ids, s, sm_count);
    }
}

struct GradPlan {
    int64_t tiles, chunks, heads;
    int passes, bits;
    size_t off_key[2], off_pos[2], off_hist, off_total, off_cross_count, off_cross, off_place, off_first, off_part, bytes;
};

GradPlan grad_plan(int64_t m, int64_t rows, int d) {
    GradPlan p;
    p.tiles = (m + K8_TILE - 1) / K8_TILE;
    p.chunks = (m + K8_RUN - 1) / K8_RUN;
    p.heads = (m + K8_HEADS - 1) / K8_HEADS;
    const int total = bit_length((uint32_t)rows);  // the key `rows` included
    p.passes = total > 0 ? (total + 7) / 8 : 1;
    p.bits = (total + p.passes - 1) / p.passes;
    if (p.bits < 1) p.bits = 1;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    p.off_cross_count = take(sizeof(int));
    for (int k = 0; k < 2; ++k) {
        p.off_key[k] = take((size_t)m * 4);
        p.off_pos[k] = take((size_t)m * 4);
    }
    p.off_hist = take((size_t)K8_BINS * p.tiles * 4);
    p.off_total = take(K8_BINS * 4);
    p.off_cross = take((size_t)p.chunks * sizeof(int2));
    p.off_place = take((size_t)p.chunks * 4);
    p.off_first = take((size_t)p.heads * 4);
    p.off_part = take((size_t)p.chunks * 2 * d * sizeof(float));
    p.bytes = off;
    return p;
}

template <typename ID>
cudaError_t sort_tokens(const GradPlan& p, const void* ids, int64_t m, uint32_t rows, uint8_t* ws, cudaStream_t s,
                        int* which) {
    uint32_t* key[2] = {reinterpret_cast<uint32_t*>(ws + p.off_key[0]), reinterpret_cast<uint32_t*>(ws + p.off_key[1])};
    uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(ws + p.off_pos[0]), reinterpret_cast<uint32_t*>(ws + p.off_pos[1])};
    cudaError_t e;
    if (m <= K8_ONE) {
        *which = 0;
        e = cudaFuncSetAttribute(k8_sort_one<ID>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(OneSmem));
        if (e != cudaSuccess) return e;
        note_launch_begin(TT_KIND_EMBEDDING, s);
        k8_sort_one<ID><<<1, K8_ONE_THREADS, sizeof(OneSmem), s>>>(static_cast<const ID*>(ids), (int)m, rows, p.passes,
                                                                  p.bits, key[0], pos[0]);
        note_launch_end(TT_KIND_EMBEDDING, s);
        return cudaGetLastError();
    }
    SortArgs a;
    a.hist = reinterpret_cast<int32_t*>(ws + p.off_hist);
    a.total = reinterpret_cast<int32_t*>(ws + p.off_total);
    a.m = m;
    a.rows = rows;
    a.tiles = (int)p.tiles;
    a.bits = p.bits;
    for (int q = 0; q < p.passes; ++q) {
        const int to = q & 1;
        a.ids = q == 0 ? ids : nullptr;
        a.key_in = key[to ^ 1];
        a.pos_in = pos[to ^ 1];
        a.key_out = key[to];
        a.pos_out = pos[to];
        a.shift = q * p.bits;
        note_launch_begin(TT_KIND_EMBEDDING, s);
        k8_count<ID><<<a.tiles, K8_SORT_THREADS, 0, s>>>(a);
        note_launch_end(TT_KIND_EMBEDDING, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        note_launch_begin(TT_KIND_EMBEDDING, s);
        k8_scan<<<K8_BINS, 256, 0, s>>>(a.hist, a.tiles, a.total);
        note_launch_end(TT_KIND_EMBEDDING, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        note_launch_begin(TT_KIND_EMBEDDING, s);
        k8_scatter<ID><<<a.tiles, K8_SORT_THREADS, 0, s>>>(a);
        note_launch_end(TT_KIND_EMBEDDING, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        *which = to;
    }
    return cudaSuccess;
}

template <typename ID>
cudaError_t embedding_grad_ids(const EmbeddingGrad& g, bool by_row, cudaStream_t s, int sm_count) {
    uint8_t* ws = static_cast<uint8_t*>(g.workspace);
    const GradPlan p = grad_plan(g.m, g.rows, g.d);
    cudaError_t e;
    if (!by_row) {
        const size_t bytes = (size_t)g.rows * g.d * (g.out_dtype == TT_F32 ? 4 : 2);
        if (bytes > 0 && (e = cudaMemsetAsync(g.out, 0, bytes, s)) != cudaSuccess) return e;
    }
    if (g.m == 0) return by_row ? cudaMemsetAsync(g.count, 0, sizeof(int32_t), s) : cudaSuccess;
    int* cross_count = reinterpret_cast<int*>(ws + p.off_cross_count);
    if ((e = cudaMemsetAsync(cross_count, 0, sizeof(int), s)) != cudaSuccess) return e;
    int which = 0;
    if ((e = sort_tokens<ID>(p, g.ids, g.m, (uint32_t)g.rows, ws, s, &which)) != cudaSuccess) return e;
    RunArgs a;
    a.key = reinterpret_cast<uint32_t*>(ws + p.off_key[which]);
    a.pos = reinterpret_cast<uint32_t*>(ws + p.off_pos[which]);
    a.m = g.m;
    a.rows = (uint32_t)g.rows;
    a.d = g.d;
    a.scale = g.scale;
    a.by_row = by_row ? 1 : 0;
    int32_t* first = reinterpret_cast<int32_t*>(ws + p.off_first);
    a.block_first = first;
    a.place = reinterpret_cast<int32_t*>(ws + p.off_place);
    a.part = reinterpret_cast<float*>(ws + p.off_part);
    a.cross = reinterpret_cast<int2*>(ws + p.off_cross);
    a.cross_count = cross_count;
    a.chunks = p.chunks;
    if (by_row) {
        note_launch_begin(TT_KIND_EMBEDDING, s);
        k8_heads<<<(unsigned)p.heads, 128, 0, s>>>(a, first);
        note_launch_end(TT_KIND_EMBEDDING, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        note_launch_begin(TT_KIND_EMBEDDING, s);
        k8_scan<<<1, 256, 0, s>>>(first, (int)p.heads, g.count);
        note_launch_end(TT_KIND_EMBEDDING, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (g.grad_dtype == TT_F32)
        return g.out_dtype == TT_F32
                   ? runs_elems<float, float, ID>(a, g.grad, g.out, g.out_ids, s, sm_count)
                   : runs_elems<float, __nv_bfloat16, ID>(a, g.grad, g.out, g.out_ids, s, sm_count);
    return g.out_dtype == TT_F32
               ? runs_elems<__nv_bfloat16, float, ID>(a, g.grad, g.out, g.out_ids, s, sm_count)
               : runs_elems<__nv_bfloat16, __nv_bfloat16, ID>(a, g.grad, g.out, g.out_ids, s, sm_count);
}

}  // namespace

size_t embedding_grad_bytes(int64_t m, int64_t rows, int d) { return grad_plan(m, rows, d).bytes; }

cudaError_t launch_embedding_grad(const EmbeddingGrad& g, bool by_row, cudaStream_t s, int sm_count) {
    return g.id_bytes == 4 ? embedding_grad_ids<int32_t>(g, by_row, s, sm_count)
                           : embedding_grad_ids<int64_t>(g, by_row, s, sm_count);
}

cudaError_t launch_embedding(const void* table, int table_dtype, int64_t rows, int d, const void* ids, int id_bytes,
                             int64_t m, float scale, void* out, int out_dtype, cudaStream_t s, int sm_count) {
    note_launch_begin(TT_KIND_EMBEDDING, s);
    if (table_dtype == TT_F32)
        out_dtype == TT_F32 ? lookup_ids<float, float>(table, rows, d, ids, id_bytes, m, scale, out, s, sm_count)
                            : lookup_ids<float, __nv_bfloat16>(table, rows, d, ids, id_bytes, m, scale, out, s, sm_count);
    else
        out_dtype == TT_F32
            ? lookup_ids<__nv_bfloat16, float>(table, rows, d, ids, id_bytes, m, scale, out, s, sm_count)
            : lookup_ids<__nv_bfloat16, __nv_bfloat16>(table, rows, d, ids, id_bytes, m, scale, out, s, sm_count);
    note_launch_end(TT_KIND_EMBEDDING, s);
    return cudaGetLastError();
}

}  // namespace tt
