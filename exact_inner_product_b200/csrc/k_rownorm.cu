// k_rownorm.cu - K7: layer norm, its gradient, and the gradient of the L2
// normalisation (K1), all row-wise.
//
// Layer norm of a row x of d numbers, with xhat = (x - mean) rstd:
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps)
//   y = xhat w + bias
// Its gradient for the row's dy, with g = dy w:
//   dx = rstd (g - sum(g) / d - xhat sum(g xhat) / d)
//   dw = sum over rows of dy xhat,  dbias = sum over rows of dy
// L2 normalisation y = x / norm, norm = sqrt(max(sum x^2, 1e-12)):
//   dx = (dy - y sum(y dy)) / norm; where the maximum is the constant, norm
//   does not depend on x and dx = dy / norm.
//
// All are HBM-bound: each row is read once into registers and every sum is
// taken from there (the variance from the centred values, not from the sum
// of squares, which cancels when the mean is large). A row belongs to a
// group of L lanes of one warp, or to a block when it is too wide for a
// warp's registers. Chunks of 8 elements per lane where d is a multiple of 8
// (rows are then 16-byte aligned), single elements otherwise.
//
// The column sums dw and dbias: each thread keeps its columns' sums in
// registers over all the rows it handles, the block adds its warps' sums in
// shared memory and writes one partial row; a second kernel adds the partial
// rows. Every order is fixed by the sizes, so the result repeats bit for bit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tt_internal.h"
#include "tt_rows.cuh"

namespace tt {
namespace {

constexpr int K7_THREADS = 256;
constexpr int K7_WARPS = K7_THREADS / 32;

// ---------------------------------------------------------------------------
// a row per group of L lanes
// ---------------------------------------------------------------------------
template <typename T, typename TW, int E, int L, int CH>
__global__ void __launch_bounds__(K7_THREADS)
    k7_layernorm(const T* __restrict__ x, const TW* __restrict__ w, const TW* __restrict__ bias, T* __restrict__ y,
                 float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t n, int d, float eps) {
    constexpr int RPW = 32 / L;
    const int lane = threadIdx.x & (L - 1);
    const int64_t first = ((int64_t)blockIdx.x * K7_WARPS + (threadIdx.x >> 5)) * RPW;
    const int64_t step = (int64_t)gridDim.x * K7_WARPS * RPW;
    for (int64_t base = first; base < n; base += step) {  // the same for all lanes of a warp
        const int64_t row = base + (threadIdx.x & 31) / L;
        const bool live = row < n;
        const T* xr = x + row * d;
        Raw<T, E> raw[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + lane) * E;
            if (live && e < d) raw[c].load(xr + e); else raw[c].zero();
        }
        float v[CH * E];
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            raw[c].get(v + c * E);
#pragma unroll
            for (int k = 0; k < E; ++k) sum += v[c * E + k];
        }
        const float mean = group_sum<L>(sum) / (float)d;
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const bool in = (c * L + lane) * E < d;
#pragma unroll
            for (int k = 0; k < E; ++k) {
                v[c * E + k] = v[c * E + k] - mean;
                if (in) sq = fmaf(v[c * E + k], v[c * E + k], sq);
            }
        }
        const float rstd = 1.0f / sqrtf(group_sum<L>(sq) / (float)d + eps);
        if (!live) continue;
        T* yr = y + row * d;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + lane) * E;
            if (e >= d) continue;
            float ww[E], bb[E], out[E];
            Raw<TW, E> r;
            if (w) r.load(w + e), r.get(ww);
            if (bias) r.load(bias + e), r.get(bb);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                out[k] = v[c * E + k] * rstd;
                if (w) out[k] *= ww[k];
                if (bias) out[k] += bb[k];
            }
            store_row<E>(yr + e, out);
        }
        if (lane == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
    }
}

template <typename T, typename TW, int E, int L, int CH>
__global__ void __launch_bounds__(K7_THREADS)
    k7_layernorm_grad(const T* __restrict__ dy, const T* __restrict__ x, const TW* __restrict__ w,
                      const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* __restrict__ dx,
                      float* __restrict__ part, int64_t n, int d) {
    constexpr int RPW = 32 / L;
    extern __shared__ float red[];  // [K7_WARPS][L * CH * E]: one column sum of each warp
    const int lane = threadIdx.x & (L - 1);
    const int warp = threadIdx.x >> 5;
    const int64_t first = ((int64_t)blockIdx.x * K7_WARPS + warp) * RPW;
    const int64_t step = (int64_t)gridDim.x * K7_WARPS * RPW;
    float dw[CH * E], db[CH * E];
#pragma unroll
    for (int i = 0; i < CH * E; ++i) dw[i] = db[i] = 0.f;
    const float inv_d = 1.0f / (float)d;
    for (int64_t base = first; base < n; base += step) {
        const int64_t row = base + (threadIdx.x & 31) / L;
        const bool live = row < n;
        Raw<T, E> rx[CH], rg[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + lane) * E;
            if (live && e < d) {
                rx[c].load(x + row * d + e);
                rg[c].load(dy + row * d + e);
            } else {
                rx[c].zero();
                rg[c].zero();
            }
        }
        const float mean = live ? __ldg(mean_in + row) : 0.f;
        const float rstd = live ? __ldg(rstd_in + row) : 0.f;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + lane) * E;
            float xv[E], gv[E], ww[E];
            rx[c].get(xv);
            rg[c].get(gv);
            if (w && e < d) {
                Raw<TW, E> r;
                r.load(w + e);
                r.get(ww);
            }
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float xh = (xv[k] - mean) * rstd;
                if (e < d) {
                    dw[c * E + k] = fmaf(gv[k], xh, dw[c * E + k]);
                    db[c * E + k] += gv[k];
                }
                const float g = w && e < d ? __fmul_rn(gv[k], ww[k]) : gv[k];
                s1 += g;
                s2 = fmaf(g, e < d ? xh : 0.f, s2);
            }
        }
        s1 = group_sum<L>(s1) * inv_d;
        s2 = group_sum<L>(s2) * inv_d;
        if (!live || dx == nullptr) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + lane) * E;
            if (e >= d) continue;
            float xv[E], gv[E], ww[E], out[E];
            rx[c].get(xv);
            rg[c].get(gv);
            if (w) {
                Raw<TW, E> r;
                r.load(w + e);
                r.get(ww);
            }
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float xh = (xv[k] - mean) * rstd;
                const float g = w ? __fmul_rn(gv[k], ww[k]) : gv[k];
                out[k] = rstd * fmaf(-xh, s2, g - s1);
            }
            store_row<E>(dx + row * d + e, out);
        }
    }
    if (part == nullptr) return;
    // the block's column sums: the lane groups of a warp, then the warps
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CH * E; ++i) {
            float s = which == 0 ? dw[i] : db[i];
#pragma unroll
            for (int o = L; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if ((threadIdx.x & 31) < L) red[warp * (L * CH * E) + (i / E * L + lane) * E + i % E] = s;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < d; e += K7_THREADS) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < K7_WARPS; ++q) s += red[q * (L * CH * E) + e];
            part[((int64_t)blockIdx.x * 2 + which) * d + e] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// a row per block
// ---------------------------------------------------------------------------
// Sums of a and b over the block, given to every thread. `sm` holds two
// buffers that alternate between calls, so one barrier per call suffices.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 (*sm)[32], int& turn) {
    a = group_sum<32>(a);
    b = group_sum<32>(b);
    float2* buf = sm[turn];
    turn ^= 1;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
    for (int q = 0; q < warps; ++q) {
        s.x += buf[q].x;
        s.y += buf[q].y;
    }
    return s;
}

template <typename T, typename TW, int E, int CH>
__global__ void __launch_bounds__(512)
    k7_layernorm_wide(const T* __restrict__ x, const TW* __restrict__ w, const TW* __restrict__ bias,
                      T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t n, int d,
                      float eps) {
    __shared__ float2 sm[2][32];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const T* xr = x + row * d;
        Raw<T, E> raw[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * (int)blockDim.x + (int)threadIdx.x) * E;
            if (e < d) raw[c].load(xr + e); else raw[c].zero();
        }
        float v[CH * E];
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            raw[c].get(v + c * E);
#pragma unroll
            for (int k = 0; k < E; ++k) sum += v[c * E + k];
        }
        const float mean = block_sum2(sum, 0.f, sm, turn).x / (float)d;
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const bool in = (c * (int)blockDim.x + (int)threadIdx.x) * E < d;
#pragma unroll
            for (int k = 0; k < E; ++k) {
                v[c * E + k] = v[c * E + k] - mean;
                if (in) sq = fmaf(v[c * E + k], v[c * E + k], sq);
            }
        }
        const float rstd = 1.0f / sqrtf(block_sum2(sq, 0.f, sm, turn).x / (float)d + eps);
        T* yr = y + row * d;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * (int)blockDim.x + (int)threadIdx.x) * E;
            if (e >= d) continue;
            float ww[E], bb[E], out[E];
            Raw<TW, E> r;
            if (w) r.load(w + e), r.get(ww);
            if (bias) r.load(bias + e), r.get(bb);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                out[k] = v[c * E + k] * rstd;
                if (w) out[k] *= ww[k];
                if (bias) out[k] += bb[k];
            }
            store_row<E>(yr + e, out);
        }
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
    }
}

template <typename T, typename TW, int E, int CH>
__global__ void __launch_bounds__(512)
    k7_layernorm_grad_wide(const T* __restrict__ dy, const T* __restrict__ x, const TW* __restrict__ w,
                           const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                           T* __restrict__ dx, float* __restrict__ part, int64_t n, int d) {
    __shared__ float2 sm[2][32];
    int turn = 0;
    float dw[CH * E], db[CH * E];
#pragma unroll
    for (int i = 0; i < CH * E; ++i) dw[i] = db[i] = 0.f;
    const float inv_d = 1.0f / (float)d;
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        Raw<T, E> rx[CH], rg[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * (int)blockDim.x + (int)threadIdx.x) * E;
            if (e < d) {
                rx[c].load(x + row * d + e);
                rg[c].load(dy + row * d + e);
            } else {
                rx[c].zero();
                rg[c].zero();
            }
        }
        const float mean = __ldg(mean_in + row), rstd = __ldg(rstd_in + row);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * (int)blockDim.x + (int)threadIdx.x) * E;
            if (e >= d) continue;
            float xv[E], gv[E], ww[E];
            rx[c].get(xv);
            rg[c].get(gv);
            if (w) {
                Raw<TW, E> r;
                r.load(w + e);
                r.get(ww);
            }
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float xh = (xv[k] - mean) * rstd;
                dw[c * E + k] = fmaf(gv[k], xh, dw[c * E + k]);
                db[c * E + k] += gv[k];
                const float g = w ? __fmul_rn(gv[k], ww[k]) : gv[k];
                s1 += g;
                s2 = fmaf(g, xh, s2);
            }
        }
        const float2 s = block_sum2(s1, s2, sm, turn);
        if (dx == nullptr) continue;
        s1 = s.x * inv_d;
        s2 = s.y * inv_d;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * (int)blockDim.x + (int)threadIdx.x) * E;
            if (e >= d) continue;
            float xv[E], gv[E], ww[E], out[E];
            rx[c].get(xv);
            rg[c].get(gv);
            if (w) {
                Raw<TW, E> r;
                r.load(w + e);
                r.get(ww);
            }
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float xh = (xv[k] - mean) * rstd;
                const float g = w ? __fmul_rn(gv[k], ww[k]) : gv[k];
                out[k] = rstd * fmaf(-xh, s2, g - s1);
            }
            store_row<E>(dx + row * d + e, out);
        }
    }
    if (part == nullptr) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e = (c * (int)blockDim.x + (int)threadIdx.x) * E;
        if (e >= d) continue;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            part[((int64_t)blockIdx.x * 2) * d + e + k] = dw[c * E + k];
            part[((int64_t)blockIdx.x * 2 + 1) * d + e + k] = db[c * E + k];
        }
    }
}

// Column sums of the blocks' partial rows: 32 columns per block, 8 threads
// per column over the rows, then those in order. part is [rows][2 d]: dw, db.
__global__ void __launch_bounds__(256)
    k7_columns(const float* __restrict__ part, int rows, int d, float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float sm[8][32];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + cx;
    float s = 0.f;
    if (col < 2 * d)
#pragma unroll 4
        for (int r = ry; r < rows; r += 8) s += __ldg(part + (int64_t)r * 2 * d + col);
    sm[ry][cx] = s;
    __syncthreads();
    if (ry == 0 && col < 2 * d) {
        float t = sm[0][cx];
#pragma unroll
        for (int q = 1; q < 8; ++q) t += sm[q][cx];
        float* out = col < d ? dw : db;
        if (out) out[col < d ? col : col - d] = t;
    }
}

// ---------------------------------------------------------------------------
// the gradient of the L2 normalisation: d a multiple of 16, at most 512
// ---------------------------------------------------------------------------
template <typename T, typename TG, int L, int CH>
__global__ void __launch_bounds__(K7_THREADS)
    k7_normalize_grad(const TG* __restrict__ dy, const T* __restrict__ x, T* __restrict__ dx, int64_t n, int d) {
    constexpr int RPW = 32 / L;
    const int lane = threadIdx.x & (L - 1);
    const int64_t first = ((int64_t)blockIdx.x * K7_WARPS + (threadIdx.x >> 5)) * RPW;
    const int64_t step = (int64_t)gridDim.x * K7_WARPS * RPW;
    for (int64_t base = first; base < n; base += step) {
        const int64_t row = base + (threadIdx.x & 31) / L;
        const bool live = row < n;
        Raw<T, 8> rx[CH];
        Raw<TG, 8> rg[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + lane) * 8;
            if (live && e < d) {
                rx[c].load(x + row * d + e);
                rg[c].load(dy + row * d + e);
            } else {
                rx[c].zero();
                rg[c].zero();
            }
        }
        float xv[CH * 8], gv[CH * 8];
        float sq = 0.f, in = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            rx[c].get(xv + 8 * c);
            rg[c].get(gv + 8 * c);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sq = fmaf(xv[8 * c + k], xv[8 * c + k], sq);
                in = fmaf(xv[8 * c + k], gv[8 * c + k], in);
            }
        }
        sq = group_sum<L>(sq);
        in = group_sum<L>(in);
        const bool clamped = sq < 1e-12f;
        const float norm = sqrtf(fmaxf(sq, 1e-12f));
        const float inv = 1.0f / norm;
        // y sum(y dy) = x sum(x dy) / norm^2
        const float coef = clamped ? 0.f : in / fmaxf(sq, 1e-12f);
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + lane) * 8;
            if (e >= d) continue;
            float out[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k] = fmaf(-xv[8 * c + k], coef, gv[8 * c + k]) * inv;
            store_row<8>(dx + row * d + e, out);
        }
    }
}

int grid_for(int64_t units, int per_block, int cap) {
    const int64_t blocks = (units + per_block - 1) / per_block;
    return (int)(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}

// How a layer-norm row is laid on threads: E elements per chunk, L lanes of a
// warp per row (0: a block of `threads`), CH chunks per thread.
struct RowShape {
    int E, L, CH, threads;
};

RowShape layernorm_shape(int d) {
    RowShape r;
    r.E = d % 8 == 0 ? 8 : 1;
    const int chunks = d / r.E;
    r.threads = K7_THREADS;
    if (r.E == 8) {
        if (chunks <= 8) return r.L = 8, r.CH = 1, r;
        if (chunks <= 16) return r.L = 16, r.CH = 1, r;
        if (chunks <= 32) return r.L = 32, r.CH = 1, r;
        if (chunks <= 64) return r.L = 32, r.CH = 2, r;
        if (chunks <= 128) return r.L = 32, r.CH = 4, r;
        r.L = 0;
        r.CH = chunks <= 256 ? 1 : chunks <= 512 ? 2 : 4;
        if (chunks > 1024) r.threads = 512;
        return r;
    }
    if (chunks <= 32) return r.L = 32, r.CH = 1, r;
    if (chunks <= 128) return r.L = 32, r.CH = 4, r;
    if (chunks <= 512) return r.L = 32, r.CH = 16, r;
    r.L = 0;
    r.CH = chunks <= 2048 ? 8 : 32;
    if (chunks > 8192) r.threads = 512;
    return r;
}

int grad_blocks(int64_t n, const RowShape& r, int sm_count) {
    if (r.L == 0) return grid_for(n, 1, 3 * sm_count);
    return grid_for(n, K7_WARPS * (32 / r.L), 2 * sm_count);
}

struct LnArgs {
    const void *dy, *x, *w, *bias;
    void* y;
    float *mean, *rstd, *part;
    int64_t n;
    int d;
    float eps;
    int grid;
    cudaStream_t s;
};

template <typename T, typename TW, int E, int L, int CH>
void ln_launch(const LnArgs& a, bool grad, const RowShape& r) {
    const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.dy);
    const TW *w = static_cast<const TW*>(a.w), *bias = static_cast<const TW*>(a.bias);
    T* y = static_cast<T*>(a.y);
    if constexpr (L > 0) {
        if (grad)
            k7_layernorm_grad<T, TW, E, L, CH><<<a.grid, K7_THREADS, K7_WARPS * L * CH * E * sizeof(float), a.s>>>(
                dy, x, w, a.mean, a.rstd, y, a.part, a.n, a.d);
        else
            k7_layernorm<T, TW, E, L, CH><<<a.grid, K7_THREADS, 0, a.s>>>(x, w, bias, y, a.mean, a.rstd, a.n, a.d,
                                                                          a.eps);
    } else {
        if (grad)
            k7_layernorm_grad_wide<T, TW, E, CH><<<a.grid, r.threads, 0, a.s>>>(dy, x, w, a.mean, a.rstd, y, a.part,
                                                                                a.n, a.d);
        else
            k7_layernorm_wide<T, TW, E, CH><<<a.grid, r.threads, 0, a.s>>>(x, w, bias, y, a.mean, a.rstd, a.n, a.d,
                                                                           a.eps);
    }
}

template <typename T, typename TW>
void ln_shape(const LnArgs& a, bool grad, const RowShape& r) {
    if (r.E == 8) {
        if (r.L == 8) return ln_launch<T, TW, 8, 8, 1>(a, grad, r);
        if (r.L == 16) return ln_launch<T, TW, 8, 16, 1>(a, grad, r);
        if (r.L == 32 && r.CH == 1) return ln_launch<T, TW, 8, 32, 1>(a, grad, r);
        if (r.L == 32 && r.CH == 2) return ln_launch<T, TW, 8, 32, 2>(a, grad, r);
        if (r.L == 32) return ln_launch<T, TW, 8, 32, 4>(a, grad, r);
        if (r.CH == 1) return ln_launch<T, TW, 8, 0, 1>(a, grad, r);
        if (r.CH == 2) return ln_launch<T, TW, 8, 0, 2>(a, grad, r);
        return ln_launch<T, TW, 8, 0, 4>(a, grad, r);
    }
    if (r.L == 32 && r.CH == 1) return ln_launch<T, TW, 1, 32, 1>(a, grad, r);
    if (r.L == 32 && r.CH == 4) return ln_launch<T, TW, 1, 32, 4>(a, grad, r);
    if (r.L == 32) return ln_launch<T, TW, 1, 32, 16>(a, grad, r);
    if (r.CH == 8) return ln_launch<T, TW, 1, 0, 8>(a, grad, r);
    return ln_launch<T, TW, 1, 0, 32>(a, grad, r);
}

cudaError_t ln_dispatch(const LnArgs& a, int x_dtype, int w_dtype, bool grad, const RowShape& r) {
    note_launch_begin(TT_KIND_ROWNORM, a.s);
    if (x_dtype == TT_F32)
        w_dtype == TT_F32 ? ln_shape<float, float>(a, grad, r) : ln_shape<float, __nv_bfloat16>(a, grad, r);
    else
        w_dtype == TT_F32 ? ln_shape<__nv_bfloat16, float>(a, grad, r)
                          : ln_shape<__nv_bfloat16, __nv_bfloat16>(a, grad, r);
    note_launch_end(TT_KIND_ROWNORM, a.s);
    return cudaGetLastError();
}

template <typename T, typename TG>
void normalize_grad_shape(const void* dy, const void* x, void* dx, int64_t n, int d, cudaStream_t s, int sm_count) {
    const TG* g = static_cast<const TG*>(dy);
    const T* xx = static_cast<const T*>(x);
    T* o = static_cast<T*>(dx);
    const int L = d <= 64 ? 8 : d <= 128 ? 16 : 32;
    const int grid = grid_for(n, K7_WARPS * (32 / L), 16 * sm_count);
    if (L == 8) k7_normalize_grad<T, TG, 8, 1><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
    else if (L == 16) k7_normalize_grad<T, TG, 16, 1><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
    else if (d <= 256) k7_normalize_grad<T, TG, 32, 1><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
    else k7_normalize_grad<T, TG, 32, 2><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
}

}  // namespace

size_t layernorm_grad_bytes(int64_t n, int d, int sm_count) {
    return (size_t)grad_blocks(n, layernorm_shape(d), sm_count) * 2 * d * sizeof(float);
}

cudaError_t launch_layernorm(const void* x, int x_dtype, int64_t n, int d, const void* w, const void* bias,
                             int w_dtype, float eps, void* y, float* mean, float* rstd, cudaStream_t s, int sm_count) {
    const RowShape r = layernorm_shape(d);
    const int grid = r.L ? grid_for(n, K7_WARPS * (32 / r.L), 16 * sm_count) : grid_for(n, 1, 16 * sm_count);
    const LnArgs a = {nullptr, x, w, bias, y, mean, rstd, nullptr, n, d, eps, grid, s};
    return ln_dispatch(a, x_dtype, w_dtype, false, r);
}

cudaError_t launch_layernorm_grad(const void* dy, const void* x, int x_dtype, int64_t n, int d, const void* w,
                                  int w_dtype, const float* mean, const float* rstd, void* dx, float* dw, float* db,
                                  float* part, cudaStream_t s, int sm_count) {
    const RowShape r = layernorm_shape(d);
    const bool columns = dw != nullptr || db != nullptr;
    const int grid = grad_blocks(n, r, sm_count);
    const LnArgs a = {dy, x, w, nullptr, dx, const_cast<float*>(mean), const_cast<float*>(rstd),
                      columns ? part : nullptr, n, d, 0.f, grid, s};
    cudaError_t e = ln_dispatch(a, x_dtype, w_dtype, true, r);
    if (e != cudaSuccess || !columns) return e;
    note_launch_begin(TT_KIND_ROWNORM, s);
    k7_columns<<<(2 * d + 31) / 32, 256, 0, s>>>(part, grid, d, dw, db);
    note_launch_end(TT_KIND_ROWNORM, s);
    return cudaGetLastError();
}

cudaError_t launch_normalize_grad(const void* dy, int dy_dtype, const void* x, int x_dtype, int64_t n, int d, void* dx,
                                  cudaStream_t s, int sm_count) {
    note_launch_begin(TT_KIND_ROWNORM, s);
    if (x_dtype == TT_F32)
        dy_dtype == TT_F32 ? normalize_grad_shape<float, float>(dy, x, dx, n, d, s, sm_count)
                           : normalize_grad_shape<float, __nv_bfloat16>(dy, x, dx, n, d, s, sm_count);
    else
        dy_dtype == TT_F32 ? normalize_grad_shape<__nv_bfloat16, float>(dy, x, dx, n, d, s, sm_count)
                           : normalize_grad_shape<__nv_bfloat16, __nv_bfloat16>(dy, x, dx, n, d, s, sm_count);
    note_launch_end(TT_KIND_ROWNORM, s);
    return cudaGetLastError();
}

}  // namespace tt
