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
//   k8_scatter     tiles (more than K8_FEW_TILES), and every token to its place
//   k8_heads,      (row form, not after k8_sort_one, which does it) which place
//   k8_scan        of the output each run has
//   k8_runs        a warp adds 32 consecutive sorted tokens in fp32, the block
//                  joins what its eight warps hold of one run, and writes it; the
//                  part of a run that reaches past the block goes to a partial row
//   k8_join        the partial rows of each such run, in order
// The kernels' launches overlap, so a block may be there before the data that it
// reads: what an earlier kernel of the call writes is read past L1 (__ldcg), whose
// lines another kernel of the call may have filled before that write.
// The order of every sum is fixed by the ids, so the bits repeat. Bound by the
// reading of g (once, in rows) and, for few tokens, by the launches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tt_device.cuh"
#include "tt_internal.h"
#include "tt_rows.cuh"

namespace tt {
namespace {

constexpr int K8_THREADS = 256;

// A lane's part of a row: K pieces of E elements, `step` columns apart, from
// column e on.
template <typename T, int E, int K>
struct Strip {
    Raw<T, E> r[K];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < K; ++j) r[j].zero();
    }
    __device__ __forceinline__ void load(const T* row, int e, int step, int d) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (e + j * step < d) r[j].load(row + e + j * step); else r[j].zero();
        }
    }
    __device__ __forceinline__ void get(float* x) const {
#pragma unroll
        for (int j = 0; j < K; ++j) r[j].get(x + j * E);
    }
};
template <int E, int K, typename TO>
__device__ __forceinline__ void store_strip(TO* row, int e, int step, int d, const float* x) {
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (e + j * step < d) store_row<E>(row + e + j * step, x + j * E);
}

// Loads of a row per lane, of two tokens at once: the narrower the loads, the more
// of them must be in flight (one load of four tokens against this, 32 * 10^6 elements
// in bf16 rows of 77: 68 against 49 us, of 300: 32 against 25, of 128: 24 against 22;
// 1024000 popular rows of 128: 71 against 66).
template <int E>
constexpr int lookup_pieces() { return E == 8 ? 2 : 4; }
constexpr int K8_TOKENS = 2;

// E elements per load, the most that divide the width.
template <typename T, typename TO, typename ID, int E, int L>
__global__ void __launch_bounds__(K8_THREADS)
    k8_lookup(const T* __restrict__ table, int64_t rows, int d, const ID* __restrict__ ids, int64_t m, float scale,
              TO* __restrict__ out) {
    constexpr int K = lookup_pieces<E>();
    const int lane = threadIdx.x & (L - 1);
    const int64_t group = ((int64_t)blockIdx.x * K8_THREADS + threadIdx.x) / L;
    const int64_t groups = (int64_t)gridDim.x * K8_THREADS / L;
    for (int64_t t0 = group * K8_TOKENS; t0 < m; t0 += groups * K8_TOKENS) {
        int64_t id[K8_TOKENS];
#pragma unroll
        for (int q = 0; q < K8_TOKENS; ++q) {
            id[q] = t0 + q < m ? (int64_t)__ldg(ids + t0 + q) : -1;
            if (id[q] >= rows) id[q] = -1;
        }
        for (int e = lane * E; e < d; e += L * E * K) {
            Strip<T, E, K> r[K8_TOKENS];
#pragma unroll
            for (int q = 0; q < K8_TOKENS; ++q) {
                if (id[q] >= 0) r[q].load(table + id[q] * d, e, L * E, d); else r[q].zero();
            }
#pragma unroll
            for (int q = 0; q < K8_TOKENS; ++q) {
                if (t0 + q >= m) break;
                float x[E * K];
                r[q].get(x);
                // a padding row is zero whatever the scale
#pragma unroll
                for (int k = 0; k < E * K; ++k) x[k] = id[q] >= 0 ? x[k] * scale : 0.f;
                store_strip<E, K>(out + (t0 + q) * d, e, L * E, d, x);
            }
        }
    }
}

template <typename T, typename TO, typename ID, int E>
void lookup_elems(const T* table, int64_t rows, int d, const ID* ids, int64_t m, float scale, TO* out, cudaStream_t s,
                  int sm_count) {
    auto launch = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        const int64_t per = (int64_t)K8_THREADS * K8_TOKENS;
        const int64_t blocks = (m * L + per - 1) / per;
        const int grid = (int)(blocks < 16 * sm_count ? blocks : 16 * sm_count);
        k8_lookup<T, TO, ID, E, L><<<grid, K8_THREADS, 0, s>>>(table, rows, d, ids, m, scale, out);
    };
    const int lanes = (d / E + lookup_pieces<E>() - 1) / lookup_pieces<E>();  // that cover a row
    if (lanes <= 2) launch(std::integral_constant<int, 2>());
    else if (lanes <= 4) launch(std::integral_constant<int, 4>());
    else if (lanes <= 8) launch(std::integral_constant<int, 8>());
    else if (lanes <= 16) launch(std::integral_constant<int, 16>());
    else launch(std::integral_constant<int, 32>());
}

template <typename T, typename TO, typename ID>
void lookup_shape(const void* table, int64_t rows, int d, const void* ids, int64_t m, float scale, void* out,
                  cudaStream_t s, int sm_count) {
    const T* t = static_cast<const T*>(table);
    const ID* i = static_cast<const ID*>(ids);
    TO* o = static_cast<TO*>(out);
    if (d % 8 == 0) lookup_elems<T, TO, ID, 8>(t, rows, d, i, m, scale, o, s, sm_count);
    else if (d % 4 == 0) lookup_elems<T, TO, ID, 4>(t, rows, d, i, m, scale, o, s, sm_count);
    else if (d % 2 == 0) lookup_elems<T, TO, ID, 2>(t, rows, d, i, m, scale, o, s, sm_count);
    else lookup_elems<T, TO, ID, 1>(t, rows, d, i, m, scale, o, s, sm_count);
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
constexpr int K8_KEYS = 16;                            // keys per thread of one block's sort
// Keys per thread of the sort by tiles (the gradient by rows of 10^6 tokens of 128
// bf16 takes 154 us with 8 of them and with 4, 162 with 16).
constexpr int K8_TILE_KEYS = 8;
constexpr int K8_TILE = K8_SORT_THREADS * K8_TILE_KEYS;  // 2048
constexpr int K8_ONE = 512 * K8_KEYS;                  // most tokens of one block's sort
constexpr int K8_ONE_SMALL = 256 * K8_KEYS;            // and of the smaller block's
constexpr int K8_BINS = 256;
// Up to this many tiles each block of k8_scatter adds the tiles' counts itself,
// a launch less per digit (the dense gradient of 8193 tokens 47 against 33 us,
// 65536 51 against 38, 130000 53 against 48; 300000, 147 tiles, 64 against 83).
constexpr int K8_FEW_TILES = 64;
constexpr int K8_RUN = 32;                             // sorted tokens of a warp
constexpr int K8_RUN_WARPS = 8;
constexpr int K8_HEADS = 4096;                         // sorted tokens of a block of k8_heads

// Ids outside [0, rows) share the key `rows`, which sorts last.
template <typename ID>
__device__ __forceinline__ uint32_t key_of(ID id, uint32_t rows) {
    return id >= 0 && (uint64_t)id < rows ? (uint32_t)id : rows;
}

// The place of a key: cnt (the warp's) holds where the next key of each digit
// goes; lanes with the same digit follow in their order.
__device__ __forceinline__ int warp_place(uint32_t digit, bool in, unsigned peers, uint32_t* cnt) {
    const int before = __popc(peers & lanemask_lt());
    const uint32_t at = in ? cnt[digit] : 0;
    __syncwarp();
    if (in && before == 0) cnt[digit] = at + __popc(peers);
    __syncwarp();
    return (int)at + before;
}

// A token in the sort: its key and its place in the call's ids.
struct SortArgs {
    const void* ids;       // first pass; null afterwards
    const uint2* in;       // (key, token)
    uint2* out;
    int32_t* hist;         // [tiles][K8_BINS] of few tiles, else [K8_BINS][tiles]
    int32_t* total;        // [K8_BINS]
    int* cross_count;      // zeroed by the first pass
    int64_t m;
    uint32_t rows;
    int tiles;
    int shift, bits;
    __device__ __forceinline__ uint32_t digit(uint32_t key) const { return (key >> shift) & ((1u << bits) - 1u); }
};

template <typename ID>
__device__ __forceinline__ uint2 load_token(const SortArgs& a, int64_t i) {
    if (a.ids != nullptr) return make_uint2(key_of(__ldg(static_cast<const ID*>(a.ids) + i), a.rows), (uint32_t)i);
    return __ldcg(a.in + i);
}

template <typename ID>
__global__ void __launch_bounds__(K8_SORT_THREADS) k8_count(const SortArgs a) {
    __shared__ int h[K8_BINS];
    pdl_trigger();
    h[threadIdx.x] = 0;
    __syncthreads();
    pdl_wait();
    if (a.ids != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.cross_count = 0;
    const int64_t base = (int64_t)blockIdx.x * K8_TILE;
    uint32_t key[K8_TILE_KEYS];
#pragma unroll
    for (int r = 0; r < K8_TILE_KEYS; ++r) {
        const int64_t i = base + r * K8_SORT_THREADS + threadIdx.x;
        key[r] = i < a.m ? load_token<ID>(a, i).x : 0u;
    }
#pragma unroll
    for (int r = 0; r < K8_TILE_KEYS; ++r)
        if (base + r * K8_SORT_THREADS + threadIdx.x < a.m) atomicAdd(&h[a.digit(key[r])], 1);
    __syncthreads();
    a.hist[a.tiles <= K8_FEW_TILES ? (int64_t)blockIdx.x * K8_BINS + threadIdx.x
                                   : (int64_t)threadIdx.x * a.tiles + blockIdx.x] = h[threadIdx.x];
}

// Block b: exclusive prefix of row b of x ([rows][len]), in place, and its sum.
__global__ void __launch_bounds__(256) k8_scan(int32_t* __restrict__ x, int len, int32_t* __restrict__ total) {
    __shared__ int warp_tot[8];
    pdl_trigger();
    pdl_wait();
    int32_t* row = x + (int64_t)blockIdx.x * len;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int run = 0;
    for (int base = 0; base < len; base += 256) {
        const int i = base + threadIdx.x;
        const int v = i < len ? __ldcg(row + i) : 0;
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

// The tile in the order of its digits in shared memory first, so that the
// stores to the digits' places are of runs of consecutive tokens.
template <typename ID>
__global__ void __launch_bounds__(K8_SORT_THREADS) k8_scatter(const SortArgs a) {
    __shared__ uint2 tile[K8_TILE];
    __shared__ uint32_t cnt[K8_SORT_WARPS][K8_BINS];
    __shared__ int to_out[K8_BINS];  // place in the output minus place in the tile, per digit
    __shared__ int warp_tot[2][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = (int64_t)blockIdx.x * K8_TILE;
    const int64_t base = first + (int64_t)warp * K8_TILE_KEYS * 32;
    pdl_trigger();
    for (int v = lane; v < K8_BINS; v += 32) cnt[warp][v] = 0;
    __syncwarp();
    pdl_wait();
    uint2 tok[K8_TILE_KEYS];
#pragma unroll
    for (int r = 0; r < K8_TILE_KEYS; ++r) {
        const int64_t i = base + r * 32 + lane;
        tok[r] = i < a.m ? load_token<ID>(a, i) : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int r = 0; r < K8_TILE_KEYS; ++r)
        if (base + r * 32 + lane < a.m) atomicAdd(&cnt[warp][a.digit(tok[r].x)], 1u);
    // tokens with this thread's digit: in all tiles, and in those before this one
    int all = 0, earlier = 0;
    if (a.tiles <= K8_FEW_TILES) {
#pragma unroll 16
        for (int t = 0; t < a.tiles; ++t) {
            const int c = __ldcg(a.hist + t * K8_BINS + threadIdx.x);
            all += c;
            if (t < blockIdx.x) earlier += c;
        }
    } else {
        all = __ldcg(a.total + threadIdx.x);
        earlier = __ldcg(a.hist + (int64_t)threadIdx.x * a.tiles + blockIdx.x);
    }
    const int before = block_prefix256(all, warp_tot[0]);  // has a barrier
    int sum = 0;
#pragma unroll
    for (int w = 0; w < K8_SORT_WARPS; ++w) {
        const int c = (int)cnt[w][threadIdx.x];
        cnt[w][threadIdx.x] = (uint32_t)sum;
        sum += c;
    }
    const int local = block_prefix256(sum, warp_tot[1]);
    to_out[threadIdx.x] = before + earlier - local;
#pragma unroll
    for (int w = 0; w < K8_SORT_WARPS; ++w) cnt[w][threadIdx.x] += (uint32_t)local;
    __syncthreads();
    unsigned peers[K8_TILE_KEYS];
#pragma unroll
    for (int r = 0; r < K8_TILE_KEYS; ++r)
        peers[r] = __match_any_sync(0xffffffffu, base + r * 32 + lane < a.m ? a.digit(tok[r].x) : (uint32_t)K8_BINS);
#pragma unroll
    for (int r = 0; r < K8_TILE_KEYS; ++r) {
        const bool in = base + r * 32 + lane < a.m;
        const int to = warp_place(a.digit(tok[r].x), in, peers[r], cnt[warp]);
        if (in) tile[to] = tok[r];
    }
    __syncthreads();
    const int here = a.m - first < K8_TILE ? (int)(a.m - first) : K8_TILE;
    for (int i = threadIdx.x; i < here; i += K8_SORT_THREADS) {
        const uint2 t = tile[i];
        a.out[to_out[a.digit(t.x)] + i] = t;
    }
}

// All digits in one block: keys and places go from registers through shared
// memory and back once per digit.
template <int THREADS>
struct OneSmem {
    uint32_t key[2][THREADS * K8_KEYS];
    uint16_t pos[2][THREADS * K8_KEYS];
    uint32_t cnt[THREADS / 32][K8_BINS];
    int warp_tot[32];
};

// Block 0 sorts; the others set the `zeros` 16-byte pieces at `zero` (and the
// last `tail` bytes), for the dense gradient's rows without a token. For the form
// by rows block 0 also counts the runs (`count`), and
// those before each K8_RUN tokens (`place`; `first` is zero, see k8_heads): two
// launches less.
template <typename ID, int THREADS, bool BY_ROW>
__global__ void __launch_bounds__(THREADS)
    k8_sort_one(const ID* __restrict__ ids, int m, uint32_t rows, int passes, int bits, uint2* __restrict__ out,
                int* __restrict__ cross_count, uint4* __restrict__ zero, int64_t zeros, int tail,
                int32_t* __restrict__ place, int32_t* __restrict__ first, int32_t* __restrict__ count) {
    constexpr int PARTS = THREADS / K8_BINS;           // threads per digit
    constexpr int PER = THREADS / 32 / PARTS;          // warps whose counts a thread adds
    extern __shared__ __align__(16) uint8_t raw[];
    OneSmem<THREADS>& sm = *reinterpret_cast<OneSmem<THREADS>*>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    if (blockIdx.x > 0) {
        const int64_t step = (int64_t)(gridDim.x - 1) * THREADS;
        for (int64_t v = (int64_t)(blockIdx.x - 1) * THREADS + threadIdx.x; v < zeros; v += step)
            zero[v] = make_uint4(0, 0, 0, 0);
        if (blockIdx.x == 1 && threadIdx.x < tail) reinterpret_cast<uint8_t*>(zero + zeros)[threadIdx.x] = 0;
        return;
    }
    if (threadIdx.x == 0) *cross_count = 0;
    // the warps share the m tokens evenly: a warp's tokens are consecutive
    const int rounds = (m + THREADS - 1) / THREADS;
    const int base = warp * rounds * 32 + lane;
    for (int i = threadIdx.x; i < m; i += THREADS) {
        sm.key[0][i] = key_of(__ldg(ids + i), rows);
        sm.pos[0][i] = (uint16_t)i;
    }
    const uint32_t mask = (1u << bits) - 1u;
    uint32_t* cnt = sm.cnt[warp];
    for (int p = 0; p < passes; ++p) {
        const uint32_t* key = sm.key[p & 1];
        const uint16_t* pos = sm.pos[p & 1];
        const int shift = p * bits;
        for (int v = lane; v < K8_BINS; v += 32) cnt[v] = 0;
        __syncthreads();  // the keys are there
#pragma unroll 4
        for (int r = 0; r < rounds; ++r)
            if (base + r * 32 < m) atomicAdd(cnt + (key[base + r * 32] >> shift & mask), 1u);
        __syncthreads();
        // the prefix over (digit, warp): PARTS threads per digit, PER warps each
        const int v = threadIdx.x / PARTS, part = threadIdx.x % PARTS;
        int c[PER], sum = 0;
#pragma unroll
        for (int w = 0; w < PER; ++w) {
            c[w] = (int)sm.cnt[part * PER + w][v];
            sum += c[w];
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) sm.warp_tot[warp] = inc;
        __syncthreads();
        const int tot = lane < THREADS / 32 ? sm.warp_tot[lane] : 0;
        int at = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? tot : 0);
#pragma unroll
        for (int w = 0; w < PER; ++w) {
            sm.cnt[part * PER + w][v] = (uint32_t)at;
            at += c[w];
        }
        __syncthreads();
        uint32_t* key_to = sm.key[(p & 1) ^ 1];
        uint16_t* pos_to = sm.pos[(p & 1) ^ 1];
        // lanes with the same digit: a vote per bit, of four rounds at once (on the
        // many values of a digit __match_any_sync takes half as long again)
        for (int r0 = 0; r0 < rounds; r0 += 4) {
            uint32_t k[4];
            unsigned peers[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = base + (r0 + q) * 32;
                const bool in = r0 + q < rounds && i < m;
                k[q] = in ? key[i] >> shift : 0u;
                peers[q] = __ballot_sync(0xffffffffu, in);
            }
            for (int b = 0; b < bits; ++b) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bool one = (k[q] >> b & 1u) != 0;
                    const unsigned v = __ballot_sync(0xffffffffu, one);
                    peers[q] &= one ? v : ~v;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = base + (r0 + q) * 32;
                const bool in = r0 + q < rounds && i < m;
                const int to = warp_place(k[q] & mask, in, peers[q], cnt);
                if (in) {
                    key_to[to] = key[i];
                    pos_to[to] = pos[i];
                }
            }
        }
        __syncthreads();
    }
    const uint32_t* key = sm.key[passes & 1];
    for (int i = threadIdx.x; i < m; i += THREADS) out[i] = make_uint2(key[i], sm.pos[passes & 1][i]);
    if constexpr (!BY_ROW) return;
    constexpr int PER_LANE = THREADS * K8_KEYS / K8_RUN / 32;
    const int chunks = (m + K8_RUN - 1) / K8_RUN;
    int* runs = reinterpret_cast<int*>(sm.cnt);
    for (int c = warp; c < chunks; c += THREADS / 32) {
        const int i = c * K8_RUN + lane;
        const bool head = i < m && key[i] < rows && (i == 0 || key[i - 1] != key[i]);
        const unsigned heads = __ballot_sync(0xffffffffu, head);
        if (lane == 0) runs[c] = __popc(heads);
    }
    __syncthreads();
    if (warp > 0) return;
    int own[PER_LANE], sum = 0;
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) {
        own[q] = lane * PER_LANE + q < chunks ? runs[lane * PER_LANE + q] : 0;
        sum += own[q];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    int before = inc - sum;
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) {
        if (lane * PER_LANE + q < chunks) place[lane * PER_LANE + q] = before;
        before += own[q];
    }
    if (lane < (m + K8_HEADS - 1) / K8_HEADS) first[lane] = 0;
    if (lane == 31) *count = inc;
}

// ---------------------------------------------------------------------------
// the runs
// ---------------------------------------------------------------------------
struct RunArgs {
    const uint2* tok;      // [m] sorted (key, token)
    int64_t m;
    uint32_t rows;
    int d;
    float scale;
    int by_row;            // 1: output row = place of the run; 0: output row = id
    const int32_t* block_first;  // (by_row) runs before each block of k8_heads
    int32_t* place;        // (by_row) [chunks] runs before a warp's 32 tokens, within that block
    float* part;           // [blocks][2][d]
    int2* cross;           // runs that go on past their block: (block, output row)
    int* cross_count;
    int64_t chunks;        // of 32 tokens
    __device__ __forceinline__ uint32_t key(int64_t i) const { return __ldcg(&tok[i].x); }
};

__device__ __forceinline__ bool is_head(const RunArgs& a, int64_t i) {
    if (i >= a.m) return false;
    const uint32_t k = a.key(i);
    return k < a.rows && (i == 0 || a.key(i - 1) != k);
}

// Runs that begin in each 32 tokens: the prefix within the block's K8_HEADS
// tokens, and the block's sum.
constexpr int K8_HEADS_THREADS = 512;
constexpr int K8_HEADS_CHUNKS = K8_HEADS / K8_RUN;

__global__ void __launch_bounds__(K8_HEADS_THREADS) k8_heads(const RunArgs a, int32_t* __restrict__ block_total) {
    constexpr int PER = K8_HEADS_CHUNKS / (K8_HEADS_THREADS / 32);
    static_assert(K8_HEADS_CHUNKS == 128, "four warps scan the counts");
    __shared__ int count[K8_HEADS_CHUNKS];
    __shared__ int warp_tot[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t base = (int64_t)blockIdx.x * K8_HEADS;
    pdl_trigger();
    pdl_wait();
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        const int n = __popc(__ballot_sync(0xffffffffu, is_head(a, base + (warp * PER + c) * K8_RUN + lane)));
        if (lane == 0) count[warp * PER + c] = n;
    }
    __syncthreads();
    int mine = 0, inc = 0;
    if (warp < 4) {
        inc = mine = count[threadIdx.x];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) warp_tot[warp] = inc;
    }
    __syncthreads();
    if (warp >= 4) return;
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warp_tot[w];
    const int64_t chunk = base / K8_RUN + threadIdx.x;
    if (chunk < a.chunks) a.place[chunk] = before + inc - mine;
    if (threadIdx.x == K8_HEADS_CHUNKS - 1) block_total[blockIdx.x] = before + inc;
}

// What a warp's 32 tokens leave open, for the block to join.
struct Open {
    int head;      // its first run began before it
    int through;   // and reaches past its end
    int tail;      // a run that began here reaches past its end
    int64_t row;   // that run's output row
};

template <typename T, typename TO, typename ID, int E, int K>
__global__ void __launch_bounds__(K8_RUN_WARPS * 32)
    k8_runs(const RunArgs a, const T* __restrict__ grad, TO* __restrict__ out, ID* __restrict__ out_ids) {
    constexpr int BATCH = K > 1 ? 4 : 8;
    constexpr int N = E * K;
    __shared__ float sums[K8_RUN_WARPS][2][N][32];  // of the open runs: head, tail
    __shared__ Open open[K8_RUN_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t chunk = (int64_t)blockIdx.x * K8_RUN_WARPS + warp;
    if (gridDim.x > 1) pdl_trigger();  // k8_join follows; a call's last kernel must not (tt_device.cuh)
    pdl_wait();
    const int64_t i0 = chunk * K8_RUN;
    const int64_t i = i0 + lane;
    const uint2 tok = i < a.m ? __ldcg(a.tok + i) : make_uint2(a.rows, 0u);
    const uint32_t key = tok.x;
    uint32_t prev = __shfl_up_sync(0xffffffffu, key, 1);
    if (lane == 0) prev = i0 > 0 && i0 < a.m ? a.key(i0 - 1) : a.rows;
    const int count = __popc(__ballot_sync(0xffffffffu, key < a.rows));  // those that count come first
    // bit q: token q begins a run (of those that count)
    const unsigned heads = __ballot_sync(0xffffffffu, key < a.rows && (prev != key || i == 0));
    const uint32_t last_key = __shfl_sync(0xffffffffu, key, 31);
    const bool goes_on = count == 32 && i0 + 32 < a.m && a.key(i0 + 32) == last_key;
    int64_t first = 0;  // place of the first run that begins here
    if (a.by_row && count > 0)
        first = (int64_t)__ldcg(a.block_first + chunk / K8_HEADS_CHUNKS) + __ldcg(a.place + chunk);
    const int e = (blockIdx.y * 32 * K + lane) * E;
    if (out_ids != nullptr && blockIdx.y == 0 && (heads >> lane & 1u))
        out_ids[first + __popc(heads & ((1u << lane) - 1u))] = (ID)key;
    if (lane == 0) open[warp] = {0, 0, 0, 0};
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    int begun = 0;  // runs begun so far
    auto write_row = [&](int64_t row, const float* v) {
        float y[N];
#pragma unroll
        for (int k = 0; k < N; ++k) y[k] = v[k] * a.scale;
        store_strip<E, K>(out + row * a.d, e, 32 * E, a.d, y);
    };
    // the run that ends before token q
    auto flush = [&](int q) {
        const bool on = q == 32 && goes_on;
        const int64_t row = a.by_row ? first + begun - 1 : (int64_t)__shfl_sync(0xffffffffu, key, q - 1);
        if (begun == 0 || on) {
#pragma unroll
            for (int k = 0; k < N; ++k) sums[warp][begun == 0 ? 0 : 1][k][lane] = acc[k];
            if (lane == 0) {
                if (begun == 0) {
                    open[warp].head = 1;
                    open[warp].through = on;
                } else {
                    open[warp].tail = 1;
                    open[warp].row = row;
                }
            }
        } else {
            write_row(row, acc);
        }
    };
    for (int b = 0; b < count; b += BATCH) {
        Strip<T, E, K> r[BATCH];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const uint32_t p = __shfl_sync(0xffffffffu, tok.y, b + q);
            if (b + q < count) r[q].load(grad + (int64_t)p * a.d, e, 32 * E, a.d); else r[q].zero();
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            if (b + q >= count) break;
            if (heads >> (b + q) & 1u) {
                if (b + q > 0) flush(b + q);
                ++begun;
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] = 0.f;
            }
            float x[N];
            r[q].get(x);
#pragma unroll
            for (int k = 0; k < N; ++k) acc[k] += x[k];
        }
    }
    if (count > 0) flush(count);
    __syncthreads();
    // Open runs within the block: the warp where one begins adds what the warps
    // after it hold of it; warp 0 also does so for the one that reaches into the
    // block. What reaches past the block becomes a partial row.
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const bool mine = which == 0 ? warp == 0 && open[0].head : open[warp].tail;
        if (!mine) continue;
        float s[N];
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = sums[warp][which][k][lane];
        bool on = which == 0 ? open[0].through != 0 : true;
        for (int w = warp + 1; on && w < K8_RUN_WARPS; ++w) {
#pragma unroll
            for (int k = 0; k < N; ++k) s[k] += sums[w][0][k][lane];
            on = open[w].through != 0;
        }
        if (which == 0 || on) {
            store_strip<E, K>(a.part + ((int64_t)blockIdx.x * 2 + which) * a.d, e, 32 * E, a.d, s);
            if (which == 1 && lane == 0 && blockIdx.y == 0)
                a.cross[atomicAdd(a.cross_count, 1)] = make_int2(blockIdx.x, (int)open[warp].row);
        } else {
            write_row(open[warp].row, s);
        }
    }
}

// A lane's part of a partial row, past L1.
__device__ __forceinline__ void load_part(Raw<float, 1>& r, const float* p) { r.a = __ldcg(p); }
__device__ __forceinline__ void load_part(Raw<float, 2>& r, const float* p) {
    r.a = __ldcg(reinterpret_cast<const float2*>(p));
}
__device__ __forceinline__ void load_part(Raw<float, 4>& r, const float* p) {
    r.a = __ldcg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ void load_part(Raw<float, 8>& r, const float* p) {
    r.a = __ldcg(reinterpret_cast<const float4*>(p));
    r.b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
}
template <int E, int K>
__device__ __forceinline__ void load_part(Strip<float, E, K>& s, const float* row, int e, int d) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (e + j * 32 * E < d) load_part(s.r[j], row + e + j * 32 * E); else s.r[j].zero();
    }
}

// A run that begins in block c and goes on: its own partial row (slot 1 of c),
// then slot 0 of the blocks after c that it reaches. A warp adds up to
// K8_JOIN_WARP of them; longer runs take the whole block, warp w the blocks
// c + 1 + w, c + 1 + w + 8, ..., and the warps' sums in order.
constexpr int K8_JOIN_WARPS = 8;
constexpr int K8_JOIN_WARP = 24;
constexpr int K8_BLOCK = K8_RUN * K8_RUN_WARPS;  // tokens of a block of k8_runs

template <int E, int K>
__device__ __forceinline__ void add_parts(const RunArgs& a, int64_t c, int64_t from, int64_t to, int step, int e,
                                          float* acc) {
    constexpr int BATCH = K > 1 ? 4 : 8;
    for (int64_t k0 = from; k0 < to; k0 += (int64_t)step * BATCH) {
        Strip<float, E, K> r[BATCH];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const int64_t k = k0 + (int64_t)q * step;
            if (k < to) load_part(r[q], a.part + (c + k) * 2 * a.d, e, a.d); else r[q].zero();
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            float x[E * K];
            r[q].get(x);
#pragma unroll
            for (int j = 0; j < E * K; ++j) acc[j] += x[j];
        }
    }
}

template <typename TO, int E, int K>
__global__ void __launch_bounds__(K8_JOIN_WARPS * 32) k8_join(const RunArgs a, TO* __restrict__ out) {
    __shared__ int64_t reach[K8_JOIN_WARPS];
    constexpr int N = E * K;
    __shared__ float sums[K8_JOIN_WARPS][N][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int n = __ldcg(a.cross_count);
    const int e = (blockIdx.y * 32 * K + lane) * E;
    // Neighbours in the list go to different blocks: the longest runs, of the
    // lowest ids where those are the popular ones, stand side by side.
    const int grid = gridDim.x;
    for (int b = blockIdx.x; b < n; b += grid * K8_JOIN_WARPS) {
        int64_t k = 0;  // blocks after the first that the run reaches
        if (b + warp * grid < n) {
            const int64_t c = __ldcg(&a.cross[b + warp * grid].x);
            const uint32_t key = a.key(c * K8_BLOCK + K8_BLOCK - 1);
            while (true) {
                const int64_t i = (c + 1 + k + lane) * K8_BLOCK;
                const unsigned same = __ballot_sync(0xffffffffu, i < a.m && a.key(i) == key);
                const int more = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
                k += more;
                if (more < 32) break;
            }
        }
        if (lane == 0) reach[warp] = k;
        __syncthreads();
        if (k > 0 && k <= K8_JOIN_WARP) {
            const int2 run = __ldcg(a.cross + b + warp * grid);
            float acc[N];
            Strip<float, E, K> r;
            load_part(r, a.part + ((int64_t)run.x * 2 + 1) * a.d, e, a.d);
            r.get(acc);
            add_parts<E, K>(a, run.x, 1, k + 1, 1, e, acc);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] *= a.scale;
            store_strip<E, K>(out + (int64_t)run.y * a.d, e, 32 * E, a.d, acc);
        }
        for (int w = 0; w < K8_JOIN_WARPS; ++w) {
            const int64_t kw = reach[w];
            if (kw <= K8_JOIN_WARP) continue;  // the same for the whole block
            const int2 run = __ldcg(a.cross + b + w * grid);
            float acc[N];
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.f;
            if (warp == 0) {
                Strip<float, E, K> r;
                load_part(r, a.part + ((int64_t)run.x * 2 + 1) * a.d, e, a.d);
                r.get(acc);
            }
            add_parts<E, K>(a, run.x, 1 + warp, kw + 1, K8_JOIN_WARPS, e, acc);
#pragma unroll
            for (int j = 0; j < N; ++j) sums[warp][j][lane] = acc[j];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    float t = sums[0][j][lane];
                    for (int q = 1; q < K8_JOIN_WARPS; ++q) t += sums[q][j][lane];
                    acc[j] = t * a.scale;
                }
                store_strip<E, K>(out + (int64_t)run.y * a.d, e, 32 * E, a.d, acc);
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

// Elements of a lane's load: the fewest whose 32 lanes cover the row, among
// those that divide it; else the most that do.
int run_elems(int d) {
    int best = 1;
    for (int E = 1; E <= 8; E *= 2) {
        if (d % E != 0) break;
        best = E;
        if (32 * E >= d) break;
    }
    return best;
}

template <typename T, typename TO, typename ID, int E, int K>
cudaError_t runs_launch(const RunArgs& a, const void* grad, void* out, void* out_ids, cudaStream_t s, int sm_count) {
    const int cols = (a.d + 32 * E * K - 1) / (32 * E * K);
    const int64_t blocks = (a.chunks + K8_RUN_WARPS - 1) / K8_RUN_WARPS;
    note_launch_begin(TT_KIND_EMBEDDING, s);
    cudaError_t e = launch_pdl(k8_runs<T, TO, ID, E, K>, dim3((unsigned)blocks, cols), dim3(K8_RUN_WARPS * 32), 0, s, a,
                               static_cast<const T*>(grad), static_cast<TO*>(out), static_cast<ID*>(out_ids));
    note_launch_end(TT_KIND_EMBEDDING, s);
    if (e != cudaSuccess || blocks < 2) return e;  // nothing crosses
    const int64_t most = (blocks + K8_JOIN_WARPS - 1) / K8_JOIN_WARPS;
    note_launch_begin(TT_KIND_EMBEDDING, s);
    e = launch_pdl(k8_join<TO, E, K>, dim3((unsigned)(most < 4 * sm_count ? most : 4 * sm_count), cols),
                   dim3(K8_JOIN_WARPS * 32), 0, s, a, static_cast<TO*>(out));
    note_launch_end(TT_KIND_EMBEDDING, s);
    return e;
}

template <typename T, typename TO, typename ID>
cudaError_t runs_elems(const RunArgs& a, const void* grad, void* out, void* out_ids, cudaStream_t s, int sm_count) {
    // Several loads of a row where one per lane does not cover it, up to eight
    // elements (one, and more blocks per row: 32 * 10^6 elements in rows of 77 fp32
    // 119 against 56 us, 65 bf16 105 against 50, 301 bf16 70 against 46).
    const int E = run_elems(a.d);
    const bool more = 32 * E < a.d;
    if (E == 8) return runs_launch<T, TO, ID, 8, 1>(a, grad, out, out_ids, s, sm_count);
    if (E == 4)
        return more ? runs_launch<T, TO, ID, 4, 2>(a, grad, out, out_ids, s, sm_count)
                    : runs_launch<T, TO, ID, 4, 1>(a, grad, out, out_ids, s, sm_count);
    if (E == 2)
        return more ? runs_launch<T, TO, ID, 2, 4>(a, grad, out, out_ids, s, sm_count)
                    : runs_launch<T, TO, ID, 2, 1>(a, grad, out, out_ids, s, sm_count);
    if (!more) return runs_launch<T, TO, ID, 1, 1>(a, grad, out, out_ids, s, sm_count);
    return a.d <= 128 ? runs_launch<T, TO, ID, 1, 4>(a, grad, out, out_ids, s, sm_count)
                      : runs_launch<T, TO, ID, 1, 8>(a, grad, out, out_ids, s, sm_count);
}

struct GradPlan {
    int64_t tiles, chunks, blocks, heads;
    int passes, bits;
    size_t off_tok[2], off_hist, off_total, off_cross_count, off_cross, off_place, off_first, off_part, bytes;
};

GradPlan grad_plan(int64_t m, int64_t rows, int d) {
    GradPlan p;
    p.tiles = (m + K8_TILE - 1) / K8_TILE;
    p.chunks = (m + K8_RUN - 1) / K8_RUN;
    p.blocks = (m + K8_BLOCK - 1) / K8_BLOCK;
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
    for (int k = 0; k < 2; ++k) p.off_tok[k] = take((size_t)m * sizeof(uint2));
    p.off_hist = take((size_t)K8_BINS * p.tiles * 4);
    p.off_total = take(K8_BINS * 4);
    p.off_cross = take((size_t)p.blocks * sizeof(int2));
    p.off_place = take((size_t)p.chunks * 4);
    p.off_first = take((size_t)p.heads * 4);
    p.off_part = take((size_t)p.blocks * 2 * d * sizeof(float));
    p.bytes = off;
    return p;
}

// Sorts the tokens into *sorted. The sort of one block also sets `bytes` of
// zeros at `zero` and counts the runs where `count` is given; the other one
// leaves both to the caller.
template <typename ID>
cudaError_t sort_tokens(const GradPlan& p, const void* ids, int64_t m, uint32_t rows, uint8_t* ws, void* zero,
                        size_t bytes, int32_t* count, cudaStream_t s, int sm_count, const uint2** sorted) {
    uint2* tok[2] = {reinterpret_cast<uint2*>(ws + p.off_tok[0]), reinterpret_cast<uint2*>(ws + p.off_tok[1])};
    int* cross_count = reinterpret_cast<int*>(ws + p.off_cross_count);
    cudaError_t e;
    if (m <= K8_ONE) {
        *sorted = tok[0];
        const int threads = m <= K8_ONE_SMALL ? 256 : 512;
        const int64_t fill = ((int64_t)(bytes / 16) + threads - 1) / threads;
        const int grid = bytes == 0 ? 1 : 1 + (int)(fill < 1 ? 1 : fill < sm_count - 1 ? fill : sm_count - 1);
        auto launch = [&](auto kernel, size_t smem) {
            if (smem > 48 * 1024 &&
                (e = allow_smem(kernel, smem)) != cudaSuccess)  // the same for every call
                return e;
            note_launch_begin(TT_KIND_EMBEDDING, s);
            kernel<<<grid, threads, smem, s>>>(static_cast<const ID*>(ids), (int)m, rows, p.passes, p.bits, tok[0],
                                               cross_count, static_cast<uint4*>(zero), (int64_t)(bytes / 16),
                                               (int)(bytes % 16), reinterpret_cast<int32_t*>(ws + p.off_place),
                                               reinterpret_cast<int32_t*>(ws + p.off_first), count);
            note_launch_end(TT_KIND_EMBEDDING, s);
            return cudaGetLastError();
        };
        if (threads == 256)
            return count != nullptr ? launch(k8_sort_one<ID, 256, true>, sizeof(OneSmem<256>))
                                    : launch(k8_sort_one<ID, 256, false>, sizeof(OneSmem<256>));
        return count != nullptr ? launch(k8_sort_one<ID, 512, true>, sizeof(OneSmem<512>))
                                : launch(k8_sort_one<ID, 512, false>, sizeof(OneSmem<512>));
    }
    SortArgs a;
    a.hist = reinterpret_cast<int32_t*>(ws + p.off_hist);
    a.total = reinterpret_cast<int32_t*>(ws + p.off_total);
    a.cross_count = cross_count;
    a.m = m;
    a.rows = rows;
    a.tiles = (int)p.tiles;
    a.bits = p.bits;
    for (int q = 0; q < p.passes; ++q) {
        a.ids = q == 0 ? ids : nullptr;
        a.in = tok[(q & 1) ^ 1];
        a.out = tok[q & 1];
        a.shift = q * p.bits;
        note_launch_begin(TT_KIND_EMBEDDING, s);
        if (q == 0) {
            k8_count<ID><<<a.tiles, K8_SORT_THREADS, 0, s>>>(a);
            e = cudaGetLastError();
        } else {
            e = launch_pdl(k8_count<ID>, dim3(a.tiles), dim3(K8_SORT_THREADS), 0, s, a);
        }
        note_launch_end(TT_KIND_EMBEDDING, s);
        if (e != cudaSuccess) return e;
        if (a.tiles > K8_FEW_TILES) {
            note_launch_begin(TT_KIND_EMBEDDING, s);
            e = launch_pdl(k8_scan, dim3(1 << p.bits), dim3(256), 0, s, a.hist, a.tiles, a.total);
            note_launch_end(TT_KIND_EMBEDDING, s);
            if (e != cudaSuccess) return e;
        }
        note_launch_begin(TT_KIND_EMBEDDING, s);
        e = launch_pdl(k8_scatter<ID>, dim3(a.tiles), dim3(K8_SORT_THREADS), 0, s, a);
        note_launch_end(TT_KIND_EMBEDDING, s);
        if (e != cudaSuccess) return e;
        *sorted = a.out;
    }
    return cudaSuccess;
}

template <typename ID>
cudaError_t embedding_grad_ids(const EmbeddingGrad& g, bool by_row, cudaStream_t s, int sm_count) {
    uint8_t* ws = static_cast<uint8_t*>(g.workspace);
    const GradPlan p = grad_plan(g.m, g.rows, g.d);
    cudaError_t e;
    const size_t zeros = by_row ? 0 : (size_t)g.rows * g.d * (g.out_dtype == TT_F32 ? 4 : 2);
    if (zeros > 0 && (g.m > K8_ONE || g.m == 0) && (e = cudaMemsetAsync(g.out, 0, zeros, s)) != cudaSuccess) return e;
    if (g.m == 0) return by_row ? cudaMemsetAsync(g.count, 0, sizeof(int32_t), s) : cudaSuccess;
    RunArgs a;
    if ((e = sort_tokens<ID>(p, g.ids, g.m, (uint32_t)g.rows, ws, g.out, zeros, by_row ? g.count : nullptr, s, sm_count,
                             &a.tok)) != cudaSuccess)
        return e;
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
    a.cross_count = reinterpret_cast<int*>(ws + p.off_cross_count);
    a.chunks = p.chunks;
    if (by_row && g.m > K8_ONE) {
        note_launch_begin(TT_KIND_EMBEDDING, s);
        e = launch_pdl(k8_heads, dim3((unsigned)p.heads), dim3(K8_HEADS_THREADS), 0, s, a, first);
        note_launch_end(TT_KIND_EMBEDDING, s);
        if (e != cudaSuccess) return e;
        note_launch_begin(TT_KIND_EMBEDDING, s);
        e = launch_pdl(k8_scan, dim3(1), dim3(256), 0, s, first, (int)p.heads, g.count);
        note_launch_end(TT_KIND_EMBEDDING, s);
        if (e != cudaSuccess) return e;
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
