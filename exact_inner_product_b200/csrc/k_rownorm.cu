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
// All are HBM-bound: each row is read once into registers, where every sum is
// taken (the variance from the centred values, not from the sum of squares,
// which cancels when the mean is large). A row belongs to a group of L lanes
// of one warp, or to a block or a team of warps when it is too wide for a warp's
// registers; a group walks over its rows, and several rows, or the next one, are
// in flight while it works on one. The arithmetic is on fp32 pairs (f32x2), which halves the
// instructions that otherwise bound the gradient.
//
// Rows travel as 16-byte pieces between memory and registers, 8 elements per
// chunk. Rows whose width is a multiple of 8 begin on a 16-byte boundary; other
// rows begin `off` elements after one, and their chunks are those of memory, so
// that chunk i holds columns 8 i - off and on, and the first and last ones
// elements of the neighbours, which count as zeros and are not written. A group
// sees only rows whose numbers agree modulo 8, so its off, and with it each
// thread's columns, stay the same from row to row: the column sums stay in
// registers, and the thread's weights, loaded once, in its own shared memory
// (element by element, 100000 x 777 bf16 took 432 us forward and 602 us back; so
// 128 and 161, beside 86 and 115 for 776).
//
// The column sums dw and dbias: each thread keeps its columns' sums in
// registers over all the rows it handles, the block adds its warps' sums in
// shared memory and writes one partial row; a second kernel adds the partial
// rows. Every order is fixed by the sizes, so the result repeats bit for bit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tt_device.cuh"
#include "tt_internal.h"
#include "tt_rows.cuh"

namespace tt {
namespace {

constexpr int K7_THREADS = 256;
constexpr int K7_WARPS = K7_THREADS / 32;

// The gradient's blocks: its threads hold two sums per column, and with the row
// at hand and the next one on its way that is 128 registers and more for CH = 4
// chunks, so those blocks have 12 warps and one fits an SM (65536 x 1000 bf16:
// 16 warps that wait for their loads 105 us, 12 that have them ahead 82 us).
template <int CH>
constexpr int grad_warps() { return CH >= 4 ? 12 : K7_WARPS; }
template <int CH>
constexpr int grad_resident() { return CH >= 4 ? 1 : 2; }

__device__ __forceinline__ float sum2(f32x2 a) {
    const float2 v = unpair(a);
    return v.x + v.y;
}

// 8 elements as four pairs.
template <typename T>
__device__ __forceinline__ void pairs8(const Raw<T, 8>& r, f32x2* v) {
    float x[8];
    r.get(x);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = pair(x[2 * k], x[2 * k + 1]);
}
template <typename T>
__device__ __forceinline__ void load_pairs8(const T* p, f32x2* v) {
    Raw<T, 8> r;
    r.load(p);
    pairs8(r, v);
}
template <typename T>
__device__ __forceinline__ void store_pairs8(T* p, const f32x2* v) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 u = unpair(v[k]);
        x[2 * k] = u.x;
        x[2 * k + 1] = u.y;
    }
    store_row<8>(p, x);
}

// Which of the 8 elements of the chunk at column col belong to the row, as bits.
constexpr uint32_t WHOLE = 0xFFu;
__device__ __forceinline__ uint32_t kept(int col, int d) {
    const int lo = col < 0 ? -col : 0, hi = d - col < 8 ? d - col : 8;
    return lo < hi ? (WHOLE >> (8 - hi)) & (WHOLE << lo) : 0u;
}
// x where bit k is set, else 0.
__device__ __forceinline__ float keep_f32(float x, uint32_t keep, int k) { return keep >> k & 1u ? x : 0.f; }
// The chunk with zeros where it is not kept.
__device__ __forceinline__ void clear_others(Raw<__nv_bfloat16, 8>& r, uint32_t keep) {
    if (keep == WHOLE) return;
    auto mask = [&](int j) {
        return (keep >> (2 * j) & 1u ? 0xFFFFu : 0u) | (keep >> (2 * j + 1) & 1u ? 0xFFFF0000u : 0u);
    };
    r.a.x &= mask(0), r.a.y &= mask(1), r.a.z &= mask(2), r.a.w &= mask(3);
}
__device__ __forceinline__ void clear_others(Raw<float, 8>& r, uint32_t keep) {
    if (keep == WHOLE) return;
    r.a = make_float4(keep_f32(r.a.x, keep, 0), keep_f32(r.a.y, keep, 1), keep_f32(r.a.z, keep, 2),
                      keep_f32(r.a.w, keep, 3));
    r.b = make_float4(keep_f32(r.b.x, keep, 4), keep_f32(r.b.y, keep, 5), keep_f32(r.b.z, keep, 6),
                      keep_f32(r.b.w, keep, 7));
}

// The chunk of memory at p (16-byte aligned); `end` is the tensor's, past which
// nothing is read (zeros). What is not the row's is cleared where the chunk is
// used: done here it would wait for the load.
__device__ __forceinline__ void load_chunk(Raw<__nv_bfloat16, 8>& r, const __nv_bfloat16* p, const __nv_bfloat16* end) {
    if (p + 8 <= end) {
        r.load(p);
    } else {
        const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
        auto word = [&](int j) {
            return (p + 2 * j < end ? (uint32_t)u[2 * j] : 0u) | (p + 2 * j + 1 < end ? (uint32_t)u[2 * j + 1] << 16 : 0u);
        };
        r.a = make_uint4(word(0), word(1), word(2), word(3));
    }
}
__device__ __forceinline__ void load_chunk(Raw<float, 8>& r, const float* p, const float* end) {
    if (p + 8 <= end) {
        r.load(p);
    } else {
        auto one = [&](int k) { return p + k < end ? __ldg(p + k) : 0.f; };
        r.a = make_float4(one(0), one(1), one(2), one(3));
        r.b = make_float4(one(4), one(5), one(6), one(7));
    }
}
template <typename T>
__device__ __forceinline__ void store_kept(T* p, const f32x2* v, uint32_t keep) {
    if (keep == WHOLE) {
        store_pairs8(p, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 u = unpair(v[k]);
        if (keep >> (2 * k) & 1u) store_row<1>(p + 2 * k, &u.x);
        if (keep >> (2 * k + 1) & 1u) store_row<1>(p + 2 * k + 1, &u.y);
    }
}

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

// Who shares a row: L lanes of a warp (L > 0), or the block (L = 0).
template <int L, int WARPS = K7_WARPS>
struct Group {
    int lane, size, turn;
    int64_t row, step;  // the group's first row, and the distance to its next
    __device__ __forceinline__ Group() : turn(0) {
        if constexpr (L > 0) {
            lane = threadIdx.x & (L - 1);
            size = L;
            row = ((int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5)) * (32 / L) + (threadIdx.x & 31) / L;
            step = (int64_t)gridDim.x * WARPS * (32 / L);
        } else {
            lane = threadIdx.x;
            size = blockDim.x;
            row = blockIdx.x;
            step = gridDim.x;
        }
    }
    // Whether any group of the warp (block) still has a row: the loops of all
    // its threads turn the same number of times.
    __device__ __forceinline__ bool any(int64_t n) const {
        if constexpr (L > 0) return row - (threadIdx.x & 31) / L < n;
        return row < n;
    }
    __device__ __forceinline__ float2 sums(float a, float b, float2 (*sm)[32]) {
        if constexpr (L > 0) return make_float2(group_sum<L>(a), group_sum<L>(b));
        return block_sum2(a, b, sm, turn);
    }
};

// A thread's weights (and biases) of its CH chunks: read from memory where the
// chunks are aligned with the columns, else kept in shared memory, pieces of 16
// bytes side by side over the block.
template <typename TW, int CH, bool ALIGNED>
struct Weights {
    const TW* w;
    float4* own;
    // `place`: 2 CH x blockDim.x pieces
    __device__ __forceinline__ Weights(const TW* weights, float4* place, int lane, int size, int off, int d)
        : w(weights), own(place + threadIdx.x) {
        if constexpr (!ALIGNED) {
            if (w == nullptr) return;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int col = (c * size + lane) * 8 - off + k;
                    x[k] = 0.f;
                    if (col >= 0 && col < d) {
                        Raw<TW, 1> r;
                        r.load(w + col);
                        r.get(x + k);
                    }
                }
                own[(2 * c) * blockDim.x] = make_float4(x[0], x[1], x[2], x[3]);
                own[(2 * c + 1) * blockDim.x] = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
    __device__ __forceinline__ void get(int c, int col, f32x2* v) const {
        if constexpr (ALIGNED) {
            load_pairs8(w + col, v);
        } else {
            const float4 a = own[(2 * c) * blockDim.x], b = own[(2 * c + 1) * blockDim.x];
            v[0] = pair(a.x, a.y), v[1] = pair(a.z, a.w), v[2] = pair(b.x, b.y), v[3] = pair(b.z, b.w);
        }
    }
};

// Elements between a 16-byte boundary and the group's rows.
template <typename T, bool ALIGNED>
__device__ __forceinline__ int row_offset(int64_t row, int d) {
    if constexpr (ALIGNED) return 0;
    return (int)(row * d % (16 / (int)sizeof(T)));
}

// Rows a group has at hand at once: narrow rows are short loads, and several of
// them share the weights and hide each other's sums (400000 x 200 bf16: 120 to
// 114 us forward, 142 to 126 back; 10^6 x 40 fp32 113 to 93 back).
template <int L, int CH, bool ALIGNED>
constexpr int forward_rows() { return ALIGNED && L > 0 && CH == 1 ? 2 : 1; }
template <int CH>
constexpr int grad_rows() { return CH == 1 ? 4 : 2; }

template <typename T, typename TW, int L, int CH, bool ALIGNED>
__global__ void __launch_bounds__(L > 0 ? K7_THREADS : CH == 8 ? 320 : 512)
    k7_layernorm(const T* __restrict__ x, const TW* __restrict__ w, const TW* __restrict__ bias, T* __restrict__ y,
                 float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t n, int d, float eps) {
    constexpr int R = forward_rows<L, CH, ALIGNED>();
    // The next row's loads ahead pay where a block has a row (30000 x 2400 bf16: 98 us
    // ahead, 113 not), and for rows whose first and last chunks need work before the
    // sums (400000 x 201 bf16: 121 against 157); with a warp per whole row the other
    // warps' loads do as well in most cases (200003 x 512 fp32: 140 us ahead, 136 not;
    // 65536 x 1000 bf16: 70 against 63; but 200003 x 512 bf16: 89 against 99), and so
    // they do with four chunks.
    constexpr bool AHEAD = L == 0 ? ALIGNED : !ALIGNED && CH <= 2;
    __shared__ float2 sm[2][32];
    extern __shared__ float4 places[];
    Group<L> g;
    const int off = row_offset<T, ALIGNED>(g.row, d);
    const T* end = x + n * d;
    const Weights<TW, CH, ALIGNED> ww(w, places, g.lane, g.size, off, d);
    const Weights<TW, CH, ALIGNED> bb(bias, places + 2 * CH * blockDim.x, g.lane, g.size, off, d);
    auto column = [&](int c) { return (c * g.size + g.lane) * 8 - off; };
    uint32_t keep[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) keep[c] = kept(column(c), d);
    // One chunk: its weights stay in registers (400000 x 200 fp32 138 against 130 us).
    constexpr bool HELD = CH == 1;
    f32x2 wv[4], bv[4];
    if (HELD && w && keep[0] != 0) ww.get(0, column(0), wv);
    if (HELD && bias && keep[0] != 0) bb.get(0, column(0), bv);
    Raw<T, 8> next[R][CH];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = row + r * g.step;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                next[r][c].zero();
                if (at < n && keep[c] != 0) {
                    if constexpr (ALIGNED) next[r][c].load(x + at * d + column(c));
                    else load_chunk(next[r][c], x + at * d + column(c), end);
                }
            }
        }
    };
    // A product with 1/d and rsqrtf instead of divisions and a square root, which
    // are a tenth of a narrow row's instructions, at 2 units in the last place more
    // (400000 x 200 bf16 114 against 100 us, fp32 130 against 122). Not with four
    // chunks, where the compiler's order of the loads then costs more (100000 x 776
    // bf16 85 against 104 us).
    constexpr bool DIVIDE = L > 0 && CH == 4;
    const float inv_d = 1.0f / (float)d;
    auto over_d = [&](float sum) { return DIVIDE ? sum / (float)d : sum * inv_d; };
    // The mean takes the product's remainder too, which a division would not have:
    // a row of one number whose sum is exact has that number as its mean, and not one
    // beside it, which rstd would blow up (12289 at 500 columns: y = -0.3 for 0).
    auto mean_of = [&](float sum) {
        const float m = over_d(sum);
        if (DIVIDE) return m;
        const float rest = fmaf(-m, (float)d, sum);
        return rest == rest ? fmaf(rest, inv_d, m) : m;  // an infinite mean stays
    };
    if (AHEAD) load(g.row);
    for (; g.any(n); g.row += R * g.step) {
        if (!AHEAD) load(g.row);
        f32x2 v[R][CH * 4];
        float mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f32x2 s = pair(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (!ALIGNED) clear_others(next[r][c], keep[c]);
                pairs8(next[r][c], v[r] + 4 * c);
#pragma unroll
                for (int k = 0; k < 4; ++k) s = add2(s, v[r][4 * c + k]);
            }
            mean[r] = sum2(s);
        }
        if (AHEAD) load(g.row + R * g.step);
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = mean_of(g.sums(mean[r], 0.f, sm).x);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const f32x2 minus = pair(-mean[r], -mean[r]);
            f32x2 s = pair(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[r][4 * c + k] = add2(v[r][4 * c + k], minus);
                if (ALIGNED || keep[c] == WHOLE) {
                    if (keep[c] != 0) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) s = fma2(v[r][4 * c + k], v[r][4 * c + k], s);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 u = unpair(v[r][4 * c + k]);
                        const f32x2 in = pair(keep_f32(u.x, keep[c], 2 * k), keep_f32(u.y, keep[c], 2 * k + 1));
                        s = fma2(in, in, s);
                    }
                }
            }
            rstd[r] = sum2(s);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float var = over_d(g.sums(rstd[r], 0.f, sm).x) + eps;
            rstd[r] = DIVIDE ? 1.0f / sqrtf(var) : rsqrtf(var);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (keep[c] == 0) continue;
            if (!HELD && w) ww.get(c, column(c), wv);
            if (!HELD && bias) bb.get(c, column(c), bv);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t at = g.row + r * g.step;
                if (at >= n) continue;
                const f32x2 r2 = pair(rstd[r], rstd[r]);
                f32x2 out[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    out[k] = mul2(v[r][4 * c + k], r2);
                    if (w) out[k] = mul2(out[k], wv[k]);
                    if (bias) out[k] = add2(out[k], bv[k]);
                }
                if constexpr (ALIGNED) store_pairs8(y + at * d + column(c), out);
                else store_kept(y + at * d + column(c), out, keep[c]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = g.row + r * g.step;
            if (g.lane == 0 && at < n) {
                if (mean_out) mean_out[at] = mean[r];
                if (rstd_out) rstd_out[at] = rstd[r];
            }
        }
    }
}

// The block's column sums to its partial row: lane groups that have the same
// columns, then the rest in order.
template <typename T, int L, int CH, int WARPS, bool ALIGNED>
__device__ __forceinline__ void write_columns(const f32x2* dw, const f32x2* db, const Group<L, WARPS>& g, float* red,
                                              float* row, int d) {
    constexpr int RPW = 32 / L;
    constexpr int ROWS = ALIGNED ? WARPS : WARPS * RPW;  // rows of `red`
    constexpr int WIDTH = L * CH * 8;                    // [ROWS][WIDTH], by chunk
    const int warp = threadIdx.x >> 5, sub = (threadIdx.x & 31) / L;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CH * 4; ++i) {
            float2 s = unpair(which == 0 ? dw[i] : db[i]);
            if constexpr (ALIGNED) {
#pragma unroll
                for (int o = L; o < 32; o <<= 1) {
                    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
                    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
                }
            }
            if (!ALIGNED || sub == 0)
                *reinterpret_cast<float2*>(red + (ALIGNED ? warp : warp * RPW + sub) * WIDTH +
                                           (i / 4 * L + g.lane) * 8 + i % 4 * 2) = s;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < d; e += 32 * WARPS) {
            float s = 0.f;
            // row q of `red` is of rows congruent to the block's first + q modulo 8
            const int64_t at = (int64_t)blockIdx.x * WARPS * RPW;
#pragma unroll 8
            for (int q = 0; q < ROWS; ++q) s += red[q * WIDTH + e + row_offset<T, ALIGNED>(at + q, d)];
            row[which * d + e] = s;
        }
    }
}

template <typename T, typename TW, int L, int CH, bool ALIGNED>
__global__ void __launch_bounds__(32 * grad_warps<CH>(), grad_resident<CH>())
    k7_layernorm_grad(const T* __restrict__ dy, const T* __restrict__ x, const TW* __restrict__ w,
                      const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* __restrict__ dx,
                      float* __restrict__ part, int64_t n, int d) {
    // The next row's loads ahead, where the registers hold them: fp32 rows of four
    // chunks do not fit beside the sums (100000 x 776 fp32 314 against 182 us), nor
    // do unaligned bf16 ones (100000 x 777: 184 against 161 us).
    constexpr bool AHEAD = CH <= 2 || (ALIGNED && sizeof(T) == 2);
    constexpr int WARPS = grad_warps<CH>();
    extern __shared__ float4 places[];  // the threads' weights; at the end the warps' column sums
    Group<L, WARPS> g;
    const int off = row_offset<T, ALIGNED>(g.row, d);
    const T *x_end = x + n * d, *dy_end = dy + n * d;
    const Weights<TW, CH, ALIGNED> ww(w, places, g.lane, L, off, d);
    f32x2 dw[CH * 4], db[CH * 4];
#pragma unroll
    for (int i = 0; i < CH * 4; ++i) dw[i] = db[i] = pair(0.f, 0.f);
    const float inv_d = 1.0f / (float)d;
    Raw<T, 8> nx[CH], ng[CH];
    float n_mean, n_rstd;
    auto load = [&](int64_t row) {
        const bool live = row < n;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * L + g.lane) * 8 - off;
            nx[c].zero();
            ng[c].zero();
            if (live && col < d) {
                if constexpr (ALIGNED) {
                    nx[c].load(x + row * d + col);
                    ng[c].load(dy + row * d + col);
                } else {
                    load_chunk(nx[c], x + row * d + col, x_end);
                    load_chunk(ng[c], dy + row * d + col, dy_end);
                }
            }
        }
        n_mean = live ? __ldg(mean_in + row) : 0.f;
        n_rstd = live ? __ldg(rstd_in + row) : 0.f;
    };
    if (AHEAD) load(g.row);
    for (; g.any(n); g.row += g.step) {
        if (!AHEAD) load(g.row);
        Raw<T, 8> rx[CH], rg[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            rx[c] = nx[c];
            rg[c] = ng[c];
            if (!ALIGNED) {
                const uint32_t keep = kept((c * L + g.lane) * 8 - off, d);
                clear_others(rx[c], keep);
                clear_others(rg[c], keep);
            }
        }
        const f32x2 minus = pair(-n_mean, -n_mean), r2 = pair(n_rstd, n_rstd);
        const bool live = g.row < n;
        if (AHEAD) load(g.row + g.step);
        f32x2 s1 = pair(0.f, 0.f), s2 = s1;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * L + g.lane) * 8 - off;
            if (col >= d) continue;
            f32x2 xv[4], gv[4], wv[4];
            pairs8(rx[c], xv);
            pairs8(rg[c], gv);  // zeros outside the row, so what xhat is there does not matter
            if (w) ww.get(c, col, wv);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x2 xh = mul2(add2(xv[k], minus), r2);
                dw[4 * c + k] = fma2(gv[k], xh, dw[4 * c + k]);
                db[4 * c + k] = add2(db[4 * c + k], gv[k]);
                if (w) gv[k] = mul2(gv[k], wv[k]);
                s1 = add2(s1, gv[k]);
                s2 = fma2(gv[k], xh, s2);
            }
        }
        const float2 s = make_float2(group_sum<L>(sum2(s1)), group_sum<L>(sum2(s2)));
        if (!live || dx == nullptr) continue;
        const f32x2 m1 = pair(-s.x * inv_d, -s.x * inv_d), m2 = pair(-s.y * inv_d, -s.y * inv_d);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * L + g.lane) * 8 - off;
            if (col >= d) continue;
            f32x2 xv[4], gv[4], wv[4], out[4];
            pairs8(rx[c], xv);
            pairs8(rg[c], gv);
            if (w) ww.get(c, col, wv);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x2 xh = mul2(add2(xv[k], minus), r2);
                if (w) gv[k] = mul2(gv[k], wv[k]);
                out[k] = mul2(fma2(xh, m2, add2(gv[k], m1)), r2);
            }
            if constexpr (ALIGNED) store_pairs8(dx + g.row * d + col, out);
            else store_kept(dx + g.row * d + col, out, kept(col, d));
        }
    }
    if (part != nullptr)
        write_columns<T, L, CH, WARPS, ALIGNED>(dw, db, g, reinterpret_cast<float*>(places),
                                                part + (int64_t)blockIdx.x * 2 * d, d);
}

// The same for narrow rows (a multiple of 8, up to 512 columns), several at once.
template <typename T, typename TW, int L, int CH>
__global__ void __launch_bounds__(K7_THREADS, 2)
    k7_layernorm_grad_rows(const T* __restrict__ dy, const T* __restrict__ x, const TW* __restrict__ w,
                           const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* __restrict__ dx,
                           float* __restrict__ part, int64_t n, int d) {
    constexpr int R = grad_rows<CH>();
    extern __shared__ float red[];
    Group<L> g;
    auto column = [&](int c) { return (c * L + g.lane) * 8; };
    f32x2 dw[CH * 4], db[CH * 4];
#pragma unroll
    for (int i = 0; i < CH * 4; ++i) dw[i] = db[i] = pair(0.f, 0.f);
    const float inv_d = 1.0f / (float)d;
    for (; g.any(n); g.row += R * g.step) {
        Raw<T, 8> rx[R][CH], rg[R][CH];
        f32x2 minus[R], r2[R];
        float2 s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = g.row + r * g.step;
            const bool live = at < n;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                rx[r][c].zero();
                rg[r][c].zero();
                if (live && column(c) < d) {
                    rx[r][c].load(x + at * d + column(c));
                    rg[r][c].load(dy + at * d + column(c));
                }
            }
            const float mean = live ? __ldg(mean_in + at) : 0.f, rstd = live ? __ldg(rstd_in + at) : 0.f;
            minus[r] = pair(-mean, -mean);
            r2[r] = pair(rstd, rstd);
        }
        f32x2 s1[R], s2[R];
#pragma unroll
        for (int r = 0; r < R; ++r) s1[r] = s2[r] = pair(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (column(c) >= d) continue;
            f32x2 wv[4];
            if (w) load_pairs8(w + column(c), wv);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f32x2 xv[4], gv[4];
                pairs8(rx[r][c], xv);
                pairs8(rg[r][c], gv);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 xh = mul2(add2(xv[k], minus[r]), r2[r]);
                    dw[4 * c + k] = fma2(gv[k], xh, dw[4 * c + k]);
                    db[4 * c + k] = add2(db[4 * c + k], gv[k]);
                    if (w) gv[k] = mul2(gv[k], wv[k]);
                    s1[r] = add2(s1[r], gv[k]);
                    s2[r] = fma2(gv[k], xh, s2[r]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = make_float2(group_sum<L>(sum2(s1[r])), group_sum<L>(sum2(s2[r])));
        if (dx == nullptr) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (column(c) >= d) continue;
            f32x2 wv[4];
            if (w) load_pairs8(w + column(c), wv);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t at = g.row + r * g.step;
                if (at >= n) continue;
                const f32x2 m1 = pair(-s[r].x * inv_d, -s[r].x * inv_d), m2 = pair(-s[r].y * inv_d, -s[r].y * inv_d);
                f32x2 xv[4], gv[4], out[4];
                pairs8(rx[r][c], xv);
                pairs8(rg[r][c], gv);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 xh = mul2(add2(xv[k], minus[r]), r2[r]);
                    if (w) gv[k] = mul2(gv[k], wv[k]);
                    out[k] = mul2(fma2(xh, m2, add2(gv[k], m1)), r2[r]);
                }
                store_pairs8(dx + at * d + column(c), out);
            }
        }
    }
    if (part != nullptr)
        write_columns<T, L, CH, K7_WARPS, true>(dw, db, g, red, part + (int64_t)blockIdx.x * 2 * d, d);
}

// ---------------------------------------------------------------------------
// the gradient of wide rows (above 1024 columns): a team of warps per row
// ---------------------------------------------------------------------------
// Each thread has CH chunks of a row and keeps their weights and column sums in
// registers; a team works on R rows at once, whose loads are in flight together
// and whose sums share a barrier. A block holds as many teams as fit. (A block
// per row, one row ahead: 30000 x 2400 bf16 145 against 112 us, fp32 250 against
// 172; 2401 columns 245 against 135 and 282 against 190.)
template <int CH>
constexpr int team_threads() { return CH == 8 ? 320 : 512; }
template <typename T, int CH>
constexpr int team_rows() { return CH >= 4 ? 1 : (sizeof(T) == 2 ? 4 : 2) / CH; }

struct Team {
    int lane, size, id, turn;
    int64_t row, step;
    float* buf;  // [2][warps][8]
    __device__ __forceinline__ Team(int threads, float* sm) : size(threads), turn(0) {
        id = (int)threadIdx.x / size;
        lane = (int)threadIdx.x - id * size;
        const int teams = (int)blockDim.x / size;
        row = (int64_t)blockIdx.x * teams + id;
        step = (int64_t)gridDim.x * teams;
        buf = sm + id * (size >> 5) * 16;
    }
    // f of the sums of K values over the team, given to every thread. A warp halves
    // the number of values per lane with each exchange; each lane then adds the
    // warps' sums of one value, in order, and passes it on. The two buffers
    // alternate, so one barrier per call suffices.
    template <int K, typename F>
    __device__ __forceinline__ void sums(float* v, F f) {
        const int l = threadIdx.x & 31;
        int o = 16;
#pragma unroll
        for (int half = K / 2; half >= 1; half >>= 1, o >>= 1) {
            const bool up = l & o;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float give = up ? v[i] : v[i + half];
                v[i] = (up ? v[i + half] : v[i]) + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
#pragma unroll
        for (int q = 16 / K; q >= 1; q >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], q);
        float* b = buf + turn * (size >> 5) * 8;
        turn ^= 1;
        if ((l & (32 / K - 1)) == 0) b[(lane >> 5) * 8 + l / (32 / K)] = v[0];
        named_bar_sync(1 + id, size);
        float s = 0.f;
        for (int q = 0; q < size >> 5; ++q) s += b[q * 8 + l % K];
        s = f(s);
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = __shfl_sync(0xffffffffu, s, i);
    }
};

// The eight weights at column col, where the row has them.
template <bool ALIGNED, typename TW>
__device__ __forceinline__ void load_weights(const TW* w, int col, uint32_t keep, f32x2* v) {
    if (ALIGNED && keep != 0) {
        load_pairs8(w + col, v);
        return;
    }
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        x[k] = 0.f;
        if (keep >> k & 1u) {
            Raw<TW, 1> r;
            r.load(w + col + k);
            r.get(x + k);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = pair(x[2 * k], x[2 * k + 1]);
}

template <typename T, typename TW, int CH, bool ALIGNED>
__global__ void __launch_bounds__(team_threads<CH>(), 1)
    k7_layernorm_grad_team(const T* __restrict__ dy, const T* __restrict__ x, const TW* __restrict__ w,
                           const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* __restrict__ dx,
                           float* __restrict__ part, int64_t n, int d, int size) {
    constexpr int R = team_rows<T, CH>();
    constexpr bool HELD = CH <= 2;
    __shared__ float4 sm[team_threads<CH>() / 32 * 4];
    extern __shared__ float red[];  // the teams' column sums
    Team t(size, reinterpret_cast<float*>(sm));
    const int off = row_offset<T, ALIGNED>(t.row, d);
    const T *x_end = x + n * d, *dy_end = dy + n * d;
    auto column = [&](int c) { return (c * size + t.lane) * 8 - off; };
    auto keep = [&](int c) { return ALIGNED ? (column(c) < d ? WHOLE : 0u) : kept(column(c), d); };
    f32x2 wv[HELD ? CH * 4 : 4], dw[CH * 4], db[CH * 4];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (HELD && w) load_weights<ALIGNED>(w, column(c), keep(c), wv + 4 * c);
    }
#pragma unroll
    for (int i = 0; i < CH * 4; ++i) dw[i] = db[i] = pair(0.f, 0.f);
    const float inv_d = 1.0f / (float)d;
    for (; t.row < n; t.row += R * t.step) {
        Raw<T, 8> rx[R][CH], rg[R][CH];
        float mean[R], rstd[R], s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = t.row + r * t.step;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                rx[r][c].zero();
                rg[r][c].zero();
                if (at < n && keep(c) != 0) {
                    if constexpr (ALIGNED) {
                        rx[r][c].load(x + at * d + column(c));
                        rg[r][c].load(dy + at * d + column(c));
                    } else {
                        load_chunk(rx[r][c], x + at * d + column(c), x_end);
                        load_chunk(rg[r][c], dy + at * d + column(c), dy_end);
                    }
                }
            }
            mean[r] = at < n ? __ldg(mean_in + at) : 0.f;
            rstd[r] = at < n ? __ldg(rstd_in + at) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const f32x2 minus = pair(-mean[r], -mean[r]), r2 = pair(rstd[r], rstd[r]);
            f32x2 s1 = pair(0.f, 0.f), s2 = s1;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (keep(c) == 0) continue;
                if (!ALIGNED) {
                    clear_others(rx[r][c], keep(c));
                    clear_others(rg[r][c], keep(c));
                }
                if (!HELD && w) load_weights<ALIGNED>(w, column(c), keep(c), wv);
                const f32x2* wc = wv + (HELD ? 4 * c : 0);
                f32x2 xv[4], gv[4];
                pairs8(rx[r][c], xv);
                pairs8(rg[r][c], gv);  // zeros outside the row, so what xhat is there does not matter
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 xh = mul2(add2(xv[k], minus), r2);
                    dw[4 * c + k] = fma2(gv[k], xh, dw[4 * c + k]);
                    db[4 * c + k] = add2(db[4 * c + k], gv[k]);
                    if (w) gv[k] = mul2(gv[k], wc[k]);
                    s1 = add2(s1, gv[k]);
                    s2 = fma2(gv[k], xh, s2);
                }
            }
            s[2 * r] = sum2(s1);
            s[2 * r + 1] = sum2(s2);
        }
        if (dx == nullptr) continue;
        t.template sums<2 * R>(s, [&](float v) { return -v * inv_d; });
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (keep(c) == 0) continue;
            if (!HELD && w) load_weights<ALIGNED>(w, column(c), keep(c), wv);
            const f32x2* wc = wv + (HELD ? 4 * c : 0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t at = t.row + r * t.step;
                if (at >= n) continue;
                const f32x2 minus = pair(-mean[r], -mean[r]), r2 = pair(rstd[r], rstd[r]);
                const f32x2 m1 = pair(s[2 * r], s[2 * r]), m2 = pair(s[2 * r + 1], s[2 * r + 1]);
                f32x2 xv[4], gv[4], out[4];
                pairs8(rx[r][c], xv);
                pairs8(rg[r][c], gv);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 xh = mul2(add2(xv[k], minus), r2);
                    if (w) gv[k] = mul2(gv[k], wc[k]);
                    out[k] = mul2(fma2(xh, m2, add2(gv[k], m1)), r2);
                }
                if constexpr (ALIGNED) store_pairs8(dx + at * d + column(c), out);
                else store_kept(dx + at * d + column(c), out, keep(c));
            }
        }
    }
    if (part == nullptr) return;
    float* row = part + (int64_t)blockIdx.x * 2 * d;
    const int teams = (int)blockDim.x / size;
    if (teams == 1) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 a = unpair(dw[4 * c + k]), b = unpair(db[4 * c + k]);
                float* at = row + column(c) + 2 * k;
                if (keep(c) >> (2 * k) & 1u) at[0] = a.x, at[d] = b.x;
                if (keep(c) >> (2 * k + 1) & 1u) at[1] = a.y, at[d + 1] = b.y;
            }
        }
        return;
    }
    // the teams' sums in order
    const int width = size * CH * 8;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CH * 4; ++i)
            *reinterpret_cast<float2*>(red + t.id * width + (i / 4 * size + t.lane) * 8 + i % 4 * 2) =
                unpair(which == 0 ? dw[i] : db[i]);
        __syncthreads();
        for (int e = threadIdx.x; e < d; e += blockDim.x) {
            float sum = 0.f;
            for (int q = 0; q < teams; ++q)
                sum += red[q * width + e + row_offset<T, ALIGNED>((int64_t)blockIdx.x * teams + q, d)];
            row[which * d + e] = sum;
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
    pdl_wait();  // the partial rows
    float s = 0.f;
    if (col < 2 * d)
#pragma unroll 8
        for (int r = ry; r < rows; r += 8) s += __ldcg(part + (int64_t)r * 2 * d + col);
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
    Group<L> g;
    for (; g.any(n); g.row += g.step) {
        const bool live = g.row < n;
        Raw<T, 8> rx[CH];
        Raw<TG, 8> rg[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + g.lane) * 8;
            if (live && e < d) {
                rx[c].load(x + g.row * d + e);
                rg[c].load(dy + g.row * d + e);
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
        const float square = fmaxf(sq, 1e-12f);
        const float inv = 1.0f / sqrtf(square);
        // y sum(y dy) = x sum(x dy) / norm^2
        const float coef = sq < 1e-12f ? 0.f : in / square;
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * L + g.lane) * 8;
            if (e >= d) continue;
            float out[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k] = fmaf(-xv[8 * c + k], coef, gv[8 * c + k]) * inv;
            store_row<8>(dx + g.row * d + e, out);
        }
    }
}

int grid_for(int64_t units, int per_block, int cap) {
    const int64_t blocks = (units + per_block - 1) / per_block;
    return (int)(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}

// How a layer-norm row is laid on threads: L lanes of a warp (0: a block of
// `threads`; the gradient's team of `threads`), CH chunks of 8 elements per
// thread. Up to 1024 columns a warp per row is faster than a block (1000 bf16
// columns: 65 against 91 us forward) or a team (65536 x 1000 bf16 85 against 104 us
// back). Forward the team is not faster (16384 x 4096 bf16 84, a block 75).
struct RowShape {
    bool aligned;
    int L, CH, threads;
    // the wide rows' gradient: teams of `threads` per block
    int teams() const { return threads < 512 ? 512 / threads : 1; }
};

RowShape layernorm_shape(int d, bool grad) {
    RowShape r;
    r.aligned = d % 8 == 0;
    r.threads = K7_THREADS;
    const int chunks = r.aligned ? d / 8 : (d + 14) / 8;  // that a row can touch
    r.CH = 1;
    r.L = chunks <= 2 ? 2 : chunks <= 4 ? 4 : chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
    if (chunks <= 32) return r;
    r.CH = chunks <= 64 ? 2 : 4;
    if (chunks <= 128) return r;
    r.L = 0;
    if (grad || chunks > 2048) {  // 8 chunks: 16384 columns that are no multiple of 8
        r.CH = chunks <= 256 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8;
        r.threads = (chunks + 32 * r.CH - 1) / (32 * r.CH) * 32;
    } else {
        r.CH = chunks <= 256 ? 1 : chunks <= 512 ? 2 : 4;
        if (chunks > 1024) r.threads = 512;
    }
    return r;
}

// Blocks of `teams` rows each: rows of a team agree modulo 8, unless they are aligned.
int row_blocks(int64_t n, int teams, int cap, bool aligned) {
    const int g = grid_for(n, teams, cap);
    if (aligned || (int64_t)g * teams >= n) return g;
    int every = 8;  // a multiple of this many blocks
    for (int t = teams; every > 1 && t % 2 == 0; t /= 2) every /= 2;
    return g / every * every;
}

int grad_blocks(int64_t n, const RowShape& r, int sm_count) {
    if (r.L == 0) return row_blocks(n, r.teams(), sm_count, r.aligned);
    if (r.CH < 4) return grid_for(n, grad_warps<1>() * (32 / r.L), grad_resident<1>() * sm_count);
    // an even number, so that a warp's rows agree modulo 8
    return grid_for(n, grad_warps<4>(), grad_resident<4>() * (sm_count / 2 * 2));
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

template <typename T, typename TW, int L, int CH, bool ALIGNED>
cudaError_t ln_launch(const LnArgs& a, bool grad, const RowShape& r) {
    const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.dy);
    const TW *w = static_cast<const TW*>(a.w), *bias = static_cast<const TW*>(a.bias);
    T* y = static_cast<T*>(a.y);
    const int warps = grad ? grad_warps<CH>() : K7_WARPS;
    const int threads = L > 0 ? 32 * warps : r.threads;
    const int own = ALIGNED ? 0 : threads * CH * 32;  // a thread's weights
    const int red = L > 0 ? (ALIGNED ? warps : warps * 32 / (L > 0 ? L : 1)) * L * CH * 32 : 0;
    const int smem = grad ? (red > own ? red : own) : 2 * own;
    // a block per row has up to 512 threads (320 with eight chunks)
    constexpr int WIDEST = ALIGNED || L > 0 ? 0 : 2 * (CH == 8 ? 320 : 512) * CH * 32;
    auto raise = [&](auto* kernel) {
        const int most = smem > WIDEST ? smem : WIDEST;
        return most <= 48 * 1024 ? cudaSuccess : allow_smem(kernel, most);
    };
    auto run_grad = [&](auto* kernel) {
        if (const cudaError_t e = raise(kernel); e != cudaSuccess) return e;
        kernel<<<a.grid, threads, smem, a.s>>>(dy, x, w, a.mean, a.rstd, y, a.part, a.n, a.d);
        return cudaGetLastError();
    };
    if (grad) {
        if constexpr (L == 0) {
            const int block = r.teams() * r.threads;
            const int sums = r.teams() > 1 ? block * CH * 32 : 0;
            k7_layernorm_grad_team<T, TW, CH, ALIGNED><<<a.grid, block, sums, a.s>>>(dy, x, w, a.mean, a.rstd, y,
                                                                                     a.part, a.n, a.d, r.threads);
            return cudaGetLastError();
        } else if constexpr (ALIGNED && CH <= 2) {
            return run_grad(&k7_layernorm_grad_rows<T, TW, L, CH>);
        } else {
            return run_grad(&k7_layernorm_grad<T, TW, L, CH, ALIGNED>);
        }
    }
    const auto kernel = &k7_layernorm<T, TW, L, CH, ALIGNED>;
    if (const cudaError_t e = raise(kernel); e != cudaSuccess) return e;
    kernel<<<a.grid, threads, smem, a.s>>>(x, w, bias, y, a.mean, a.rstd, a.n, a.d, a.eps);
    return cudaGetLastError();
}

template <typename T, typename TW, bool ALIGNED>
cudaError_t ln_shape(const LnArgs& a, bool grad, const RowShape& r) {
    if (r.L == 2) return ln_launch<T, TW, 2, 1, ALIGNED>(a, grad, r);
    if (r.L == 4) return ln_launch<T, TW, 4, 1, ALIGNED>(a, grad, r);
    if (r.L == 8) return ln_launch<T, TW, 8, 1, ALIGNED>(a, grad, r);
    if (r.L == 16) return ln_launch<T, TW, 16, 1, ALIGNED>(a, grad, r);
    if (r.L == 32 && r.CH == 1) return ln_launch<T, TW, 32, 1, ALIGNED>(a, grad, r);
    if (r.L == 32 && r.CH == 2) return ln_launch<T, TW, 32, 2, ALIGNED>(a, grad, r);
    if (r.L == 32) return ln_launch<T, TW, 32, 4, ALIGNED>(a, grad, r);
    if (r.CH == 1) return ln_launch<T, TW, 0, 1, ALIGNED>(a, grad, r);
    if (r.CH == 2) return ln_launch<T, TW, 0, 2, ALIGNED>(a, grad, r);
    if (r.CH == 4) return ln_launch<T, TW, 0, 4, ALIGNED>(a, grad, r);
    return ln_launch<T, TW, 0, 8, false>(a, grad, r);
}

template <typename T, typename TW>
cudaError_t ln_width(const LnArgs& a, bool grad, const RowShape& r) {
    return r.aligned ? ln_shape<T, TW, true>(a, grad, r) : ln_shape<T, TW, false>(a, grad, r);
}

cudaError_t ln_dispatch(const LnArgs& a, int x_dtype, int w_dtype, bool grad, const RowShape& r) {
    note_launch_begin(TT_KIND_ROWNORM, a.s);
    cudaError_t e;
    if (x_dtype == TT_F32)
        e = w_dtype == TT_F32 ? ln_width<float, float>(a, grad, r) : ln_width<float, __nv_bfloat16>(a, grad, r);
    else
        e = w_dtype == TT_F32 ? ln_width<__nv_bfloat16, float>(a, grad, r)
                              : ln_width<__nv_bfloat16, __nv_bfloat16>(a, grad, r);
    note_launch_end(TT_KIND_ROWNORM, a.s);
    return e;
}

template <typename T, typename TG>
void normalize_grad_shape(const void* dy, const void* x, void* dx, int64_t n, int d, cudaStream_t s, int sm_count) {
    const TG* g = static_cast<const TG*>(dy);
    const T* xx = static_cast<const T*>(x);
    T* o = static_cast<T*>(dx);
    const int L = d <= 16 ? 2 : d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32;
    const int grid = grid_for(n, K7_WARPS * (32 / L), 16 * sm_count);
    if (L == 2) k7_normalize_grad<T, TG, 2, 1><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
    else if (L == 4) k7_normalize_grad<T, TG, 4, 1><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
    else if (L == 8) k7_normalize_grad<T, TG, 8, 1><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
    else if (L == 16) k7_normalize_grad<T, TG, 16, 1><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
    else if (d <= 256) k7_normalize_grad<T, TG, 32, 1><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
    else k7_normalize_grad<T, TG, 32, 2><<<grid, K7_THREADS, 0, s>>>(g, xx, o, n, d);
}

}  // namespace

size_t layernorm_grad_bytes(int64_t n, int d, int sm_count) {
    return (size_t)grad_blocks(n, layernorm_shape(d, true), sm_count) * 2 * d * sizeof(float);
}

cudaError_t launch_layernorm(const void* x, int x_dtype, int64_t n, int d, const void* w, const void* bias,
                             int w_dtype, float eps, void* y, float* mean, float* rstd, cudaStream_t s, int sm_count) {
    const RowShape r = layernorm_shape(d, false);
    // unaligned rows: blocks that stay, for their weights are loaded first
    const int grid = r.L == 0 ? row_blocks(n, 1, (r.aligned ? 2048 : 1024) / r.threads * sm_count, r.aligned)
                              : grid_for(n, K7_WARPS * (32 / r.L), (r.aligned ? 32 : 6) * sm_count);
    const LnArgs a = {nullptr, x, w, bias, y, mean, rstd, nullptr, n, d, eps, grid, s};
    return ln_dispatch(a, x_dtype, w_dtype, false, r);
}

cudaError_t launch_layernorm_grad(const void* dy, const void* x, int x_dtype, int64_t n, int d, const void* w,
                                  int w_dtype, const float* mean, const float* rstd, void* dx, float* dw, float* db,
                                  float* part, cudaStream_t s, int sm_count) {
    const RowShape r = layernorm_shape(d, true);
    const bool columns = dw != nullptr || db != nullptr;
    const int grid = grad_blocks(n, r, sm_count);
    const LnArgs a = {dy, x, w, nullptr, dx, const_cast<float*>(mean), const_cast<float*>(rstd),
                      columns ? part : nullptr, n, d, 0.f, grid, s};
    cudaError_t e = ln_dispatch(a, x_dtype, w_dtype, true, r);
    if (e != cudaSuccess || !columns) return e;
    note_launch_begin(TT_KIND_ROWNORM, s);
    e = launch_pdl(k7_columns, dim3((2 * d + 31) / 32), dim3(256), 0, s, static_cast<const float*>(part), grid, d, dw, db);
    note_launch_end(TT_KIND_ROWNORM, s);
    return e;
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
