// k_clip.cu - K9: the global norm of many tensors, and their scaling by it.
//
//   norm = sqrt(sum over all elements of all tensors of x^2)
//   c    = min(1, max_norm / (norm + 1e-6))
//   out  = x c, rounded to the tensor's type
//
// Bound by HBM, and by the launches for a few small tensors: two passes over
// the data (the scale needs every element), of which the second reads from L2
// what the first left there. Measured: 160 tensors of 1.1 GB scaled out of
// place in 192 + 351 us, 6.1 TB/s of the 3.3 GB moved (8 blocks per SM with
// longer ranges: 234 + 423 us). The tensors'
// addresses and sizes travel as kernel parameters, so a call copies nothing
// to the device and can be captured. The tensors are cut into chunks of
// K9_CHUNK bytes; every block owns a contiguous range of chunks, walks it
// upwards in the first pass and downwards in the second, whose first reads
// are then the first pass's last ones.
//
// The squares of 8 elements are added in fp32 and the groups in fp64. A
// group whose fp32 sum leaves [2^-80, 2^126], where squares overflow or
// underflow, is added in fp64 from the start; sums of one group are off by at
// most 8 roundings. Every block writes one partial sum, and each block of the
// second pass adds all of them in the same order: no atomics, no counter to
// reset, and the same bits on every run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tt_internal.h"
#include "tt_rows.cuh"

namespace tt {
namespace {

constexpr int K9_THREADS = 256;
constexpr int K9_VECS = 4;  // 16-byte loads in flight per thread
constexpr int K9_CHUNK = K9_THREADS * K9_VECS * 16;

struct ClipEntry {
    const void* in;
    void* out;
    int64_t n;
    int first;   // chunks before this tensor in the launch
    int dtype;
};

// Kernel parameters hold up to 32 KB; a launch with few tensors passes less.
template <int N>
struct ClipTable {
    int count, chunks;
    ClipEntry e[N];
};
constexpr int K9_SMALL = 32;
static_assert(sizeof(ClipTable<CLIP_MAX_TENSORS>) + 64 <= 32764, "kernel parameters");

__device__ __forceinline__ double square_sum8(const float* x) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(x[k], x[k], s);
    if (s <= 0x1p126f && s >= 0x1p-80f) return (double)s;
    double t = 0.0;  // overflow, underflow, NaN, or nothing but zeros
#pragma unroll
    for (int k = 0; k < 8; ++k) t = fma((double)x[k], (double)x[k], t);
    return t;
}

// Block sum of a double in a fixed order; the result is valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double* sm) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int q = 1; q < K9_THREADS / 32; ++q) v += sm[q];
    return v;
}

// Elements [lo, hi) of chunk c of a tensor, and where the 16-byte aligned
// part of them begins and ends.
struct Span {
    int64_t lo, hi, va, vb;
};
template <typename T>
__device__ __forceinline__ Span chunk_span(const T* p, int64_t n, int c) {
    constexpr int64_t PER = K9_CHUNK / sizeof(T);
    constexpr int E = 16 / sizeof(T);
    Span s;
    s.lo = c * PER;
    s.hi = s.lo + PER < n ? s.lo + PER : n;
    const int off = (int)((reinterpret_cast<uintptr_t>(p + s.lo) & 15) / sizeof(T));
    s.va = s.lo + (off ? E - off : 0);
    if (s.va > s.hi) s.va = s.hi;
    s.vb = s.va + (s.hi - s.va) / E * E;
    return s;
}

template <typename T>
__device__ double chunk_squares(const T* __restrict__ p, int64_t n, int c) {
    constexpr int E = 16 / sizeof(T);
    const Span s = chunk_span(p, n, c);
    const int vecs = (int)((s.vb - s.va) / E);
    const T* base = p + s.va;
    Raw<T, E> r[K9_VECS];
#pragma unroll
    for (int q = 0; q < K9_VECS; ++q) {
        const int v = q * K9_THREADS + threadIdx.x;
        if (v < vecs) r[q].load(base + (int64_t)v * E); else r[q].zero();
    }
    double sum = 0.0;
    if constexpr (E == 8) {
#pragma unroll
        for (int q = 0; q < K9_VECS; ++q) {
            float x[8];
            r[q].get(x);
            sum += square_sum8(x);
        }
    } else {
#pragma unroll
        for (int q = 0; q < K9_VECS; q += 2) {
            float x[8];
            r[q].get(x);
            r[q + 1].get(x + 4);
            sum += square_sum8(x);
        }
    }
    // at most E - 1 elements on either side
    const int64_t head = s.lo + threadIdx.x, tail = s.vb + threadIdx.x;
    if (head < s.va || tail < s.hi) {
        Raw<T, 1> one;
        float x;
        if (head < s.va) {
            one.load(p + head);
            one.get(&x);
            sum = fma((double)x, (double)x, sum);
        }
        if (tail < s.hi) {
            one.load(p + tail);
            one.get(&x);
            sum = fma((double)x, (double)x, sum);
        }
    }
    return sum;
}

template <typename T>
__device__ void chunk_scale(const T* p, T* out, int64_t n, int c, float scale) {
    constexpr int E = 16 / sizeof(T);
    const Span s = chunk_span(p, n, c);
    const int vecs = (int)((s.vb - s.va) / E);
    const T* base = p + s.va;
    T* obase = out + s.va;
    const bool aligned_out = (reinterpret_cast<uintptr_t>(obase) & 15) == 0;
    uint4 raw[K9_VECS];  // plain loads: out may be the same tensor
#pragma unroll
    for (int q = 0; q < K9_VECS; ++q) {
        const int v = q * K9_THREADS + threadIdx.x;
        if (v < vecs) raw[q] = *reinterpret_cast<const uint4*>(base + (int64_t)v * E);
    }
#pragma unroll
    for (int q = 0; q < K9_VECS; ++q) {
        const int v = q * K9_THREADS + threadIdx.x;
        if (v >= vecs) continue;
        float x[E];
        if constexpr (E == 8) {
            unpack_bf16x2(raw[q].x, x), unpack_bf16x2(raw[q].y, x + 2);
            unpack_bf16x2(raw[q].z, x + 4), unpack_bf16x2(raw[q].w, x + 6);
        } else {
            x[0] = __uint_as_float(raw[q].x), x[1] = __uint_as_float(raw[q].y);
            x[2] = __uint_as_float(raw[q].z), x[3] = __uint_as_float(raw[q].w);
        }
#pragma unroll
        for (int k = 0; k < E; ++k) x[k] *= scale;
        T* o = obase + (int64_t)v * E;
        if (aligned_out) {
            store_row<E>(o, x);
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k) store_row<1>(o + k, x + k);
        }
    }
    const int64_t head = s.lo + threadIdx.x, tail = s.vb + threadIdx.x;
    if (head < s.va) {
        const float x = (float)p[head] * scale;
        store_row<1>(out + head, &x);
    }
    if (tail < s.hi) {
        const float x = (float)p[tail] * scale;
        store_row<1>(out + tail, &x);
    }
}

// The tensor that owns chunk c of the launch.
template <int N>
__device__ __forceinline__ int find_tensor(const ClipTable<N>& t, int c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].first <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ void block_range(int chunks, int* lo, int* hi) {
    *lo = (int)((int64_t)chunks * blockIdx.x / gridDim.x);
    *hi = (int)((int64_t)chunks * (blockIdx.x + 1) / gridDim.x);
}

template <int N>
__global__ void __launch_bounds__(K9_THREADS)
    k9_squares(const __grid_constant__ ClipTable<N> t, double* __restrict__ part) {
    __shared__ double sm[K9_THREADS / 32];
    int lo, hi;
    block_range(t.chunks, &lo, &hi);
    double sum = 0.0;
    if (lo < hi) {
        int i = find_tensor(t, lo);
        for (int c = lo; c < hi; ++c) {
            while (i + 1 < t.count && t.e[i + 1].first <= c) ++i;
            const ClipEntry& e = t.e[i];
            sum += e.dtype == TT_F32
                       ? chunk_squares(static_cast<const float*>(e.in), e.n, c - e.first)
                       : chunk_squares(static_cast<const __nv_bfloat16*>(e.in), e.n, c - e.first);
        }
    }
    sum = block_sum(sum, sm);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The norm from the partial sums, in every thread.
__device__ __forceinline__ float total_norm(const double* __restrict__ part, int parts, double* sm) {
    double s = 0.0;
    for (int q = threadIdx.x; q < parts; q += K9_THREADS) s += __ldg(part + q);
    s = block_sum(s, sm);
    __shared__ float norm;
    if (threadIdx.x == 0) norm = (float)sqrt(s);
    __syncthreads();
    return norm;
}

__global__ void __launch_bounds__(K9_THREADS)
    k9_norm(const double* __restrict__ part, int parts, float* __restrict__ norm_out) {
    __shared__ double sm[K9_THREADS / 32];
    const float norm = total_norm(part, parts, sm);
    if (threadIdx.x == 0) *norm_out = norm;
}

template <int N>
__global__ void __launch_bounds__(K9_THREADS)
    k9_scale(const __grid_constant__ ClipTable<N> t, const double* __restrict__ part, int parts, float max_norm,
             float* __restrict__ norm_out) {
    __shared__ double sm[K9_THREADS / 32];
    const float norm = total_norm(part, parts, sm);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    const float ratio = max_norm / (norm + 1e-6f);
    // NaN stays, but no limit is not exceeded by an infinite norm
    const float scale = ratio >= 1.0f || (isinf(max_norm) && isinf(norm)) ? 1.0f : ratio;
    int lo, hi;
    block_range(t.chunks, &lo, &hi);
    if (lo >= hi) return;
    int i = find_tensor(t, hi - 1);
    for (int c = hi - 1; c >= lo; --c) {
        while (t.e[i].first > c) --i;
        const ClipEntry& e = t.e[i];
        if (scale == 1.0f && e.in == e.out) continue;  // nothing to change
        if (e.dtype == TT_F32)
            chunk_scale(static_cast<const float*>(e.in), static_cast<float*>(e.out), e.n, c - e.first, scale);
        else
            chunk_scale(static_cast<const __nv_bfloat16*>(e.in), static_cast<__nv_bfloat16*>(e.out), e.n, c - e.first,
                        scale);
    }
}

int clip_grid(int sm_count) { return 48 * sm_count; }

int64_t tensor_chunks(const ClipList& l, int i) {
    const int64_t per = K9_CHUNK / (l.dtype[i] == TT_F32 ? 4 : 2);
    return (l.n[i] + per - 1) / per;
}

template <int N>
cudaError_t launch_part(const ClipList& l, int first, int count, bool scale, double* part, int parts, float max_norm,
                        float* norm, cudaStream_t s, int grid) {
    ClipTable<N> t;
    t.count = 0;
    int64_t chunks = 0;
    for (int i = first; i < first + count; ++i) {
        if (l.n[i] == 0) continue;
        t.e[t.count++] = {l.in[i], scale ? l.out[i] : nullptr, l.n[i], (int)chunks, l.dtype[i]};
        chunks += tensor_chunks(l, i);
    }
    t.chunks = (int)chunks;
    note_launch_begin(TT_KIND_CLIP, s);
    if (scale)
        k9_scale<N><<<grid, K9_THREADS, 0, s>>>(t, part, parts, max_norm, norm);
    else
        k9_squares<N><<<grid, K9_THREADS, 0, s>>>(t, part);
    note_launch_end(TT_KIND_CLIP, s);
    return cudaGetLastError();
}

// The tensors of the launch that starts at `first`: as many as the table
// holds while their chunks stay below 2^31 (one tensor's always do).
int launch_count(const ClipList& l, int first, int64_t* chunks) {
    int k = 0;
    *chunks = 0;
    while (first + k < l.count && k < CLIP_MAX_TENSORS) {
        const int64_t c = tensor_chunks(l, first + k);
        if (k > 0 && *chunks + c >= INT32_MAX) break;
        *chunks += c;
        ++k;
    }
    return k;
}

}  // namespace

size_t clip_workspace_bytes(const ClipList& l, int sm_count) {
    int launches = 0;
    int64_t chunks;
    for (int i = 0; i < l.count; i += launch_count(l, i, &chunks)) ++launches;
    return (size_t)(launches > 0 ? launches : 1) * clip_grid(sm_count) * sizeof(double);
}

cudaError_t launch_clip(const ClipList& l, bool scale, float max_norm, float* norm, double* part, cudaStream_t s,
                        int sm_count) {
    cudaError_t e;
    int parts = 0;
    for (int pass = 0; pass < (scale ? 2 : 1); ++pass) {
        int i = 0;
        do {  // at least one launch, so that no tensors give norm 0
            int64_t chunks;
            const int k = launch_count(l, i, &chunks);
            int grid = clip_grid(sm_count);
            if (chunks < grid) grid = chunks > 0 ? (int)chunks : 1;
            double* p = pass == 0 ? part + parts : part;
            e = k <= K9_SMALL ? launch_part<K9_SMALL>(l, i, k, pass == 1, p, parts, max_norm, norm, s, grid)
                              : launch_part<CLIP_MAX_TENSORS>(l, i, k, pass == 1, p, parts, max_norm, norm, s, grid);
            if (e != cudaSuccess) return e;
            if (pass == 0) parts += grid;
            i += k;
        } while (i < l.count);
    }
    if (scale) return cudaSuccess;
    note_launch_begin(TT_KIND_CLIP, s);
    k9_norm<<<1, K9_THREADS, 0, s>>>(part, parts, norm);
    note_launch_end(TT_KIND_CLIP, s);
    return cudaGetLastError();
}

}  // namespace tt
