// k_softmax_grad.cu - K6: the gradient of the in-batch sampled softmax (K5)
// with respect to the user and item rows, without writing the b x nc matrix.
//
// With l_ij = (u_i . v_j) / tau - log q_j, P_ij = exp(l_ij - lse_i) for the
// columns in row i's sum (0 for the others), and w_i the loss's weight of row
// i (the gradient of loss_i, plus that of the mean over the valid rows; 0 for
// padding):
//   grad_u_i = w_i / tau (sum_j P_ij v_j - v_i)
//   grad_v_j = 1 / tau (sum_i w_i P_ij u_i - [j < b] w_j u_j)
// The diagonal is kept out of the matrix products: its coefficient
// P_ii - 1 = expm1(-loss_i) (both terms of the sums above together) is applied
// in fp32 at the end, so that the one large entry of a row is not rounded and
// does not cancel.
//
// Kernels, in launch order (each may start while the one before it still runs
// and waits for its end before it touches memory; see pdl_wait):
//   table_clear  (with item ids) empty the table that numbers the ids
//   k6_prepare   per column: bias -log q_j log2(e), item group; per row:
//                w_i, -lse_i log2(e) (-inf where w_i = 0), expm1(-loss_i);
//                with padding, copies of users and items whose padded rows
//                are zero (what a padded row holds, NaN even, never matters)
//   k6_products  both gradients' products. One pass keeps 128 users and runs
//                over the items, the other keeps 128 items and runs over the
//                users; each forms the logits of a 128 x TN tile again on the
//                tensor cores, turns them into P in registers, writes P as
//                bf16 over the logits in tensor memory and multiplies it from
//                there with the tile of rows that is still in shared memory
//   k6_finish    adds the partial products of each row, scales them by its sums
//                of P, adds the diagonal, applies the loss's scale, and rounds to
//                bf16
//
// P is rounded to bf16 (at most a relative 2^-8 of each term, of either sign):
// its products with bf16 rows are then exact and add in fp32. The gradient of a
// user is a sum over differences v_j - v_i (and that of an item nearly one over
// differences of users), so what the vectors have in common cancels between the
// product and the diagonal, but only if the coefficients add up to what they did
// before the rounding: the P of a flat softmax are near one another and may all be
// rounded the same way, and 2^-8 of a large common component is more than the
// result. So the epilogue also adds each row's P before and after the rounding, in
// fp32, and k6_finish scales the row's product by the ratio of the two sums. What
// the rounding then leaves goes by the spread of the rows that are added, at most
// 2^-7 of sum P |v_j - mean|. The scale is held to 1 / (1 +- 2^-8), which it does
// not leave where the terms have one sign; weights of both signs can bring the
// sums near zero.
// Recomputing the logits in both passes costs 2 of the 8 b nc d operations and
// a second exponential per logit; one pass would need either atomic additions
// of b x d (or nc x d) sums per tile, whose order changes the result, or
// their partial sums in HBM (2.1 GB at 16384 x 32768 x 128).
//
// Bound by the tensor cores for d >= 128 and by the exponentials below; the
// epilogue (about 6 instructions per logit, 2 of them the sums of P, and 2 more
// with item ids) overlaps with both by two groups of warps and two to three logit
// tiles in flight. Measured on a B200, 8 b nc d operations in k6_products: 16384 x
// 32768 x 128 456 us (1.21 PFLOP/s) without masks, 498 us with all (without the
// sums of P 418 and 459); 16384^2 x 256 412 us (1.33); 32768^2 x 64 without masks
// 789 us (2.7 T exponentials/s; without the sums 682); 8192^2 x 512 668 us (one
// stage of rows fits beside the kept tile, and the logits are formed for each half
// of the columns).
//
// The tiles of both passes, row tile after row tile, form one line that is cut
// evenly among the SMs, so a few row tiles with long sums use the whole GPU
// too; the parts of a row tile are added in k6_finish in the order of the
// line. Every wait is bounded; on expiry the kernel records an error code,
// every output becomes NaN, and the host check reports a timeout.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "tt_device.cuh"
#include "tt_internal.h"
#include "tt_rows.cuh"
#include "tt_softmax.cuh"

namespace tt {
namespace {

constexpr int K6_M = 128;            // kept rows per tile (TMEM lanes)
// Groups of four epilogue warps, one tile each in turn. At most as many as there
// are logit buffers (2 at least): a group that waits for a tile has seen the
// logits of the tile K6_GROUPS before it, and with it every earlier round of the
// buffer, so the parity it waits for cannot be that of a round before.
constexpr int K6_GROUPS = 2;
static_assert(K6_GROUPS <= 2, "no more than the fewest logit buffers");
constexpr int K6_EPI_WARPS = 4 * K6_GROUPS;
constexpr int K6_THREADS = 32 * (4 + K6_EPI_WARPS);  // warps 0-3: copies, logits, products, none
// Registers: the four first warps give back what the epilogue takes.
// setmaxnreg.inc draws on the registers the block was launched with, and a
// split above them would wait forever: launch_products refuses it.
constexpr int K6_ROLE_REGS = 64;
constexpr int K6_EPI_REGS = 208;
constexpr int K6_SPLIT_REGS = 128 * K6_ROLE_REGS + 32 * K6_EPI_WARPS * K6_EPI_REGS;
static_assert(K6_THREADS % 128 == 0, "whole warpgroups: setmaxnreg is theirs");
static_assert(K6_SPLIT_REGS <= 16384 / (K6_THREADS / 32 / 4 * 32) / 8 * 8 * K6_THREADS, "register split");
constexpr int K6_TMEM_COLS = 512;
constexpr int K6_MAX_BUFS = 4;       // logit tiles in tensor memory
constexpr int K6_MAX_STAGES = 8;
constexpr int K6_SMEM_BUDGET = 227 * 1024;
constexpr int K6_HALF = 256;         // widest product of one unit; wider rows take two
constexpr float K6_LOG2E = 1.4426950408889634f;
constexpr int K6_PREP_THREADS = 256;

struct K6Ctl {
    uint64_t full[K6_MAX_STAGES], empty[K6_MAX_STAGES];
    uint64_t xfull, xempty;
    uint64_t sfull[K6_MAX_BUFS];  // logits of a tile are in tensor memory
    uint64_t pfull[K6_MAX_BUFS];  // P is there in their place
    uint64_t pdone[K6_MAX_BUFS];  // the product with P is done
    uint64_t accfull, accempty;
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(K6Ctl) <= 1024, "the control block's place in shared memory");

// What a row brings as one of a tile's columns or kept rows (arrays padded to
// whole tiles): bias, added to acc log2(e) / tau (items -log q log2(e), users
// -lse log2(e), -inf where w = 0), and the item group.
struct K6Side {
    float* bias;
    int* grp;
};

// The line of `work` tiles cut evenly among `grid` blocks: block c begins at
// floor(work c / grid).
struct K6Cut {
    int64_t each;
    int rest, grid;
    K6Cut() = default;
    K6Cut(int64_t work, int g) : each(work / g), rest((int)(work % g)), grid(g) {}
    __device__ __forceinline__ int64_t begin(int c) const { return each * c + rest * c / grid; }
    // the block that has tile w
    __device__ __forceinline__ int block_of(int64_t w) const {
        int c = (int)((double)w / ((double)each + (double)rest / grid));
        if (c >= grid) c = grid - 1;
        while (c > 0 && begin(c) > w) --c;
        while (begin(c + 1) <= w) ++c;
        return c;
    }
};

struct K6Params {
    K6Side item;          // [nc]
    K6Side user;          // [b]
    const float* weight;  // [b] w_i, padded
    float* part;          // [units + grid][128][width] partial products
    float* sums;          // [units + grid][K6_GROUPS][2][128] sums of P, before and after its rounding
    int* err;
    int b, nc, d;
    float a2;             // log2(e) / tau
    int kchunks;          // 64-element pieces of a row
    int halves, width;    // products of `width` columns, in `halves` units
    int stages, bufs;
    int weighted;         // the items' pass multiplies P by w_i (else the rows' common weight is applied at the end)
    K6Cut cut;
    uint32_t idesc_s;
};

// Unit u: half u / (row tiles of both passes), then the users' row tiles, then the items'.
struct K6Unit {
    int pass, half, tile, cols;  // cols: tiles of the other side
    int64_t begin;               // its first tile on the line
};

template <int TN>
struct K6Line {
    int ru, rv;  // row tiles of users, items
    int cu, cv;  // column tiles of users, items
    __host__ __device__ K6Line(int b, int nc)
        : ru((b + K6_M - 1) / K6_M), rv((nc + K6_M - 1) / K6_M), cu((b + TN - 1) / TN), cv((nc + TN - 1) / TN) {}
    __host__ __device__ int64_t per_half() const { return (int64_t)ru * cv + (int64_t)rv * cu; }
    __host__ __device__ K6Unit unit(int u) const {
        K6Unit r;
        r.half = u / (ru + rv);
        const int q = u - r.half * (ru + rv);
        r.pass = q < ru ? 0 : 1;
        r.tile = r.pass == 0 ? q : q - ru;
        r.cols = r.pass == 0 ? cv : cu;
        r.begin = (int64_t)r.half * per_half() + (r.pass == 0 ? (int64_t)r.tile * cv : (int64_t)ru * cv + (int64_t)r.tile * cu);
        return r;
    }
    // the unit that holds tile w of the line
    __host__ __device__ int unit_of(int64_t w) const {
        const int half = (int)(w / per_half());
        const int64_t q = w - (int64_t)half * per_half();
        const int64_t first = (int64_t)ru * cv;
        return half * (ru + rv) + (q < first ? (int)(q / cv) : ru + (int)((q - first) / cu));
    }
};

// ---------------------------------------------------------------------------
// preparation
// ---------------------------------------------------------------------------
struct K6Prep {
    const float* logq;
    const int64_t* item_ids;
    const uint8_t* valid;
    const float *lse, *loss, *grad_loss, *grad_mean;
    unsigned long long* keys;
    int log2_slots;
    K6Side item, user;
    float *weight, *diag, *common;
    const uint4 *users, *items;  // copied where valid is given
    uint4 *users_c, *items_c;
    int b, nc, vpr;              // vpr: 16-byte pieces of a row
    int* err;
};

__global__ void __launch_bounds__(K6_PREP_THREADS) k6_prepare(const K6Prep p) {
    __shared__ int valid_rows;
    const int tid = blockIdx.x * K6_PREP_THREADS + threadIdx.x;
    const int threads = gridDim.x * K6_PREP_THREADS;
    pdl_trigger();
    if (threadIdx.x == 0) valid_rows = 0;
    __syncthreads();
    pdl_wait();  // the empty table, the call's inputs, and whoever used the workspace before
    if (p.valid != nullptr && p.grad_mean != nullptr) {  // every block counts all rows
        int n = 0;
        const bool words = (reinterpret_cast<uintptr_t>(p.valid) & 15) == 0;
        const int whole = words ? p.b / 16 : 0;
        auto set = [](uint32_t w) { return __popc(__vminu4(w, 0x01010101u)); };  // bytes that are not zero
        for (int i = threadIdx.x; i < whole; i += K6_PREP_THREADS) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.valid) + i);
            n += set(v.x) + set(v.y) + set(v.z) + set(v.w);
        }
        for (int i = 16 * whole + threadIdx.x; i < p.b; i += K6_PREP_THREADS) n += p.valid[i] != 0;
        n = __reduce_add_sync(0xffffffffu, n);
        if ((threadIdx.x & 31) == 0) atomicAdd(&valid_rows, n);
        __syncthreads();
    }
    // the weight of every valid row, where there is no gradient per row
    const int count = p.valid != nullptr ? valid_rows : p.b;
    const float mean_w = p.grad_mean != nullptr && count > 0 ? *p.grad_mean / (float)count : 0.f;
    if (tid == 0) *p.err = 0;
    if (tid == 0) *p.common = p.grad_loss != nullptr ? 1.f : mean_w;
    // past the end, to whole tiles: columns without a share
    for (int j = p.nc + tid; j < (p.nc + K6_M - 1) / K6_M * K6_M; j += threads) {
        p.item.bias[j] = -INFINITY;
        p.item.grp[j] = -2;
    }
    for (int j = p.b + tid; j < (p.b + K6_M - 1) / K6_M * K6_M; j += threads) {
        p.user.bias[j] = -INFINITY;
        p.user.grp[j] = -2;
        p.weight[j] = 0.f;
    }
    for (int j = tid; j < p.nc; j += threads) {
        const bool ok = p.valid == nullptr || p.valid[j] != 0;
        p.item.bias[j] = ok ? (p.logq != nullptr ? -p.logq[j] * K6_LOG2E : 0.f) : -INFINITY;
        const int grp = p.item_ids != nullptr ? item_group((unsigned long long)p.item_ids[j], p.keys, p.log2_slots) : 0;
        p.item.grp[j] = grp;
        if (j < p.b) {
            const float w = ok ? (p.grad_loss != nullptr ? p.grad_loss[j] : 0.f) + mean_w : 0.f;
            p.weight[j] = w;
            p.diag[j] = ok ? expm1f(-p.loss[j]) : 0.f;
            p.user.bias[j] = w != 0.f ? -p.lse[j] * K6_LOG2E : -INFINITY;
            p.user.grp[j] = grp;
        }
    }
    if (p.valid == nullptr) return;
    const int64_t total = (int64_t)p.nc * p.vpr;
    for (int64_t v = tid; v < total; v += threads) {
        const int j = (int)(v / p.vpr);
        const bool ok = p.valid[j] != 0;
        p.items_c[v] = ok ? __ldg(p.items + v) : make_uint4(0, 0, 0, 0);
        if (j < p.b) p.users_c[v] = ok ? __ldg(p.users + v) : make_uint4(0, 0, 0, 0);
    }
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------
// A place in a ring of buffers and the parity of its current round.
struct Ring {
    int at, len;
    uint32_t phase;
    __device__ __forceinline__ explicit Ring(int n) : at(0), len(n), phase(0) {}
    __device__ __forceinline__ void next() {
        if (++at == len) {
            at = 0;
            phase ^= 1;
        }
    }
};

// A thread's sum of one row's P after the rounding, two at a time. Mixed additions
// (fp32 + bf16) where the test for hits keeps the integer pipe busy, else the bf16
// pair unpacked and a packed addition (16384 x 32768 x 128 with all masks 532
// against 551 us a call, without masks 490 against 481; 32768^2 x 64 836 against 811).
template <bool MIXED>
struct RoundedSum;
template <>
struct RoundedSum<false> {
    f32x2 s;
    __device__ __forceinline__ RoundedSum() : s(pair(0.f, 0.f)) {}
    __device__ __forceinline__ void add(uint32_t bits) {
        s = add2(s, pair(__uint_as_float(bits << 16), __uint_as_float(bits & 0xFFFF0000u)));
    }
    __device__ __forceinline__ float total() const {
        const float2 v = unpair(s);
        return v.x + v.y;
    }
};
template <>
struct RoundedSum<true> {
    float s;
    __device__ __forceinline__ RoundedSum() : s(0.f) {}
    __device__ __forceinline__ void add(uint32_t bits) {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
            "add.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %0, hi, %0;\n\t}"
            : "+f"(s)
            : "r"(bits));
    }
    __device__ __forceinline__ float total() const { return s; }
};

template <int K>
struct Kind {
    static constexpr int value = K;
};

template <int TN, bool HITS>
__global__ void __launch_bounds__(K6_THREADS, 1)
    k6_products(const __grid_constant__ CUtensorMap tm_ux, const __grid_constant__ CUtensorMap tm_uy,
                const __grid_constant__ CUtensorMap tm_vx, const __grid_constant__ CUtensorMap tm_vy,
                const K6Params p) {
    constexpr int XCHUNK = K6_M * 128;  // bytes of a 64-element piece of the kept tile
    constexpr int YCHUNK = TN * 128;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* xsm = smem;                                   // [kchunks][128 x 128 B]
    uint8_t* ring = smem + (size_t)p.kchunks * XCHUNK;     // [stages][kchunks][TN x 128 B]
    const int ystage = p.kchunks * YCHUNK;
    // [stages][3][TN]: bias, group, weight of the stage's rows
    float* cols_sm = reinterpret_cast<float*>(ring + (size_t)p.stages * ystage);
    K6Ctl* ctl = reinterpret_cast<K6Ctl*>(cols_sm + (size_t)p.stages * 3 * TN);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const K6Line<TN> line(p.b, p.nc);
    const int64_t w0 = p.cut.begin(blockIdx.x);
    const int64_t w1 = p.cut.begin(blockIdx.x + 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        mbar_init(&ctl->xfull, 1);
        mbar_init(&ctl->xempty, 1);
        for (int q = 0; q < p.bufs; ++q) {
            mbar_init(&ctl->sfull[q], 1);
            mbar_init(&ctl->pfull[q], 4);
            mbar_init(&ctl->pdone[q], 1);
        }
        mbar_init(&ctl->accfull, 1);
        mbar_init(&ctl->accempty, K6_EPI_WARPS);
        mbar_init(&ctl->drain[0], 1);
        mbar_init(&ctl->drain[1], 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, K6_TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    pdl_trigger();
    pdl_wait();  // k6_prepare
    const uint32_t acc_cols = (uint32_t)((p.width + 31) / 32 * 32);  // the product; the logit tiles follow
    volatile int* abort = &ctl->abort;

    if (warp < 4) {
    regs_dec<K6_ROLE_REGS>();
    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            uint32_t n = 0;  // tiles loaded
            int seg = 0;     // kept tiles loaded
            bool ok = true;
            for (int64_t w = w0; ok && w < w1; ++seg) {
                const K6Unit u = line.unit(line.unit_of(w));
                const int t0 = (int)(w - u.begin);
                const int t1 = (int)(u.begin + u.cols < w1 ? u.cols : w1 - u.begin);
                const CUtensorMap* tx = u.pass == 0 ? &tm_ux : &tm_vx;
                const CUtensorMap* ty = u.pass == 0 ? &tm_vy : &tm_uy;
                if (!mbar_wait(&ctl->xempty, (seg & 1) ^ 1, abort)) { ok = false; break; }
                mbar_arrive_expect_tx(&ctl->xfull, (uint32_t)(p.kchunks * XCHUNK));
                for (int kc = 0; kc < p.kchunks; ++kc)
                    tma_load_2d(xsm + (size_t)kc * XCHUNK, tx, &ctl->xfull, kc * 64, u.tile * K6_M);
                for (int t = t0; t < t1; ++t, ++n) {
                    const int s = n % p.stages;
                    if (!mbar_wait(&ctl->empty[s], ((n / p.stages) & 1) ^ 1, abort)) { ok = false; break; }
                    const bool weights = u.pass == 1 && p.weighted;
                    const K6Side& ys = u.pass == 0 ? p.item : p.user;
                    float* cs = cols_sm + s * 3 * TN;
                    mbar_arrive_expect_tx(&ctl->full[s], (uint32_t)(ystage + (1 + HITS + weights) * TN * 4));
                    bulk_load(cs, ys.bias + (int64_t)t * TN, &ctl->full[s], TN * 4);
                    if (HITS) bulk_load(cs + TN, ys.grp + (int64_t)t * TN, &ctl->full[s], TN * 4);
                    if (weights) bulk_load(cs + 2 * TN, p.weight + (int64_t)t * TN, &ctl->full[s], TN * 4);
                    for (int kc = 0; kc < p.kchunks; ++kc)
                        tma_load_2d(ring + (size_t)s * ystage + (size_t)kc * YCHUNK, ty, &ctl->full[s], kc * 64, t * TN);
                }
                w += t1 - t0;
            }
            if (!ok) {
                atomicExch(p.err, ERR_TIMEOUT_TMA);
                *abort = 1;
            }
            // Every issued load must land before the block may exit.
            const uint32_t first = n > (uint32_t)p.stages ? n - p.stages : 0;
            for (uint32_t j = first; j < n; ++j) mbar_wait(&ctl->full[j % p.stages], (j / p.stages) & 1, nullptr);
            if (seg > 0) mbar_wait(&ctl->xfull, (seg - 1) & 1, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------ logits ------------------------------
        // One thread issues the logits of every tile, as soon as its buffer (the
        // product of the tile that had it before) and its stage are there.
        if (lane == 0) {
            const uint32_t xdesc = umma_desc_lo(smem_u32(xsm)), ydesc = umma_desc_lo(smem_u32(ring));
            Ring st(p.stages), bf(p.bufs);
            bool ok = true;
            int seg = 0;
            for (int64_t w = w0; ok && w < w1; ++seg) {
                const K6Unit u = line.unit(line.unit_of(w));
                const int64_t end = u.begin + u.cols < w1 ? u.begin + u.cols : w1;
                if (!mbar_wait(&ctl->xfull, seg & 1, abort)) { ok = false; break; }
                for (; w < end; ++w) {
                    if (!mbar_wait(&ctl->pdone[bf.at], bf.phase ^ 1, abort)) { ok = false; break; }
                    if (!mbar_wait(&ctl->full[st.at], st.phase, abort)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + acc_cols + (uint32_t)(bf.at * TN);
                    uint32_t a = xdesc, b = ydesc + (uint32_t)(st.at * ystage >> 4);
                    for (int kc = 0; kc < p.kchunks; ++kc, a += XCHUNK >> 4, b += YCHUNK >> 4) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16(d_tmem, umma_desc_of(a + kk * 2, UMMA_KMAJOR_HI), umma_desc_of(b + kk * 2, UMMA_KMAJOR_HI),
                                      p.idesc_s, (kc | kk) != 0 ? 1u : 0u);
                    }
                    umma_commit(&ctl->sfull[bf.at]);
                    st.next();
                    bf.next();
                }
                if (ok) umma_commit(&ctl->xempty);  // the kept tile is free after this
            }
            if (!ok) {
                atomicExch(p.err, ERR_TIMEOUT_MMA);
                *abort = 1;
            }
            // Wait for every MMA issued by this thread before TMEM is freed.
            umma_commit(&ctl->drain[0]);
            mbar_wait(&ctl->drain[0], 0, nullptr);
        }
    } else if (warp == 2) {
        // ------------------------------ products ------------------------------
        // Another thread issues the product of every tile once P is there, and
        // with it frees the tile's stage and buffer.
        if (lane == 0) {
            const uint32_t ydesc = umma_desc_lo(smem_u32(ring)) | ((uint32_t)(YCHUNK >> 4) << 16);
            Ring st(p.stages), bf(p.bufs);
            bool ok = true;
            int seg = 0;
            for (int64_t w = w0; ok && w < w1; ++seg) {
                const K6Unit u = line.unit(line.unit_of(w));
                const int64_t end = u.begin + u.cols < w1 ? u.begin + u.cols : w1;
                const int cols = p.d - u.half * K6_HALF < K6_HALF ? p.d - u.half * K6_HALF : K6_HALF;
                const uint32_t idesc = umma_idesc_bf16_bmn(K6_M, cols);
                const uint32_t half = (uint32_t)(u.half * (K6_HALF / 64) * YCHUNK) >> 4;
                uint32_t accumulate = 0;
                if (!mbar_wait(&ctl->accempty, (seg & 1) ^ 1, abort)) { ok = false; break; }
                for (; w < end; ++w) {
                    if (!mbar_wait(&ctl->pfull[bf.at], bf.phase, abort)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a = tmem_base + acc_cols + (uint32_t)(bf.at * TN);
                    const uint32_t b = ydesc + (uint32_t)(st.at * ystage >> 4) + half;
#pragma unroll
                    for (int kk = 0; kk < TN / 16; ++kk) {
                        umma_bf16_ts(tmem_base, a + kk * 8, umma_desc_of(b + kk * (2048 >> 4), UMMA_MNMAJOR_HI), idesc,
                                     accumulate);
                        accumulate = 1;
                    }
                    umma_commit(&ctl->pdone[bf.at]);
                    umma_commit(&ctl->empty[st.at]);
                    st.next();
                    bf.next();
                }
                if (ok) umma_commit(&ctl->accfull);
            }
            if (!ok) {
                atomicExch(p.err, ERR_TIMEOUT_MMA);
                *abort = 1;
            }
            umma_commit(&ctl->drain[1]);
            mbar_wait(&ctl->drain[1], 0, nullptr);
        }
    }
    } else {
        regs_inc<K6_EPI_REGS>();
        // ------------------------------ epilogue ------------------------------
        // Group g takes tiles g, g + K6_GROUPS, ...; warp w of it TMEM lanes
        // 32 (w % 4) .., as two blocks of 16 in the fragment layout: a thread has
        // rows lane / 4 + {0, 8, 16, 24} and, of each 8 columns, the pair
        // 2 (lane % 4). Its columns' constants then fit in registers (a whole row
        // per thread would read them all from shared memory, at the cost of the
        // exponentials themselves).
        const int ew = warp - 4;
        const int group = ew / (4);
        const int quarter = warp & 3;
        const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
        const f32x2 a2v = pair(p.a2, p.a2);
        bool ok = true;
        Ring st(p.stages), bf(p.bufs);
        int turn = 0;  // the group of the tile that st and bf stand at
        auto step_on = [&](int& t) {
            ++t;
            st.next();
            bf.next();
            turn = turn + 1 == K6_GROUPS ? 0 : turn + 1;
        };
        int seg = 0;
        for (int64_t w = w0; ok && w < w1; ++seg) {
            const int uid = line.unit_of(w);
            const K6Unit u = line.unit(uid);
            const int t0 = (int)(w - u.begin);
            const int t1 = (int)(u.begin + u.cols < w1 ? u.cols : w1 - u.begin);
            const int rows = u.pass == 0 ? p.b : p.nc;
            const K6Side& xs = u.pass == 0 ? p.user : p.item;
            const int row0 = u.tile * K6_M + quarter * 32 + (lane >> 2);
            const int col0 = 2 * (lane & 3);
            f32x2 rbias[4];
            int rgrp[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = row0 + 8 * q;
                const bool in = row < rows;
                const float rb = in ? xs.bias[row] : -INFINITY;
                rbias[q] = pair(rb, rb);
                rgrp[q] = in ? xs.grp[row] : -1;
            }
            // the thread's share of its rows' sums of P, before and after the rounding
            f32x2 exact_sum[4];
            RoundedSum<HITS> round_sum[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) exact_sum[q] = pair(0.f, 0.f);
            // A tile to P, in steps of 64 columns of one 16-row block. P of a step
            // covers logits that the block's threads have read already. Loads and
            // stores of 8 columns each: larger ones tie 32 registers into one
            // operand, which the packed arithmetic then copies out of and into
            // (1.5 moves per logit; 16384 x 32768 x 128 470 against 450 us).
            // kind: bit 0 columns have weights; bit 1 (without item ids) a column
            // may be a row.
            auto tile = [&](uint32_t buf, const float* cs, int tt, auto kind) {
                constexpr bool WEIGHTS = (decltype(kind)::value & 1) != 0, DIAGONAL = (decltype(kind)::value & 2) != 0;
#pragma unroll 1
                for (int h = 0; h < TN / 64; ++h) {
                    f32x2 cb[8];
                    [[maybe_unused]] int2 cg[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        cb[e] = *reinterpret_cast<const f32x2*>(cs + h * 64 + 8 * e + col0);
                        if constexpr (HITS) cg[e] = *reinterpret_cast<const int2*>(cs + TN + h * 64 + 8 * e + col0);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t at = buf + ((uint32_t)(16 * k) << 16);
                        float v[32];
#pragma unroll
                        for (int e = 0; e < 8; ++e) tmem_ld_frag8(at + h * 64 + 8 * e, v + 4 * e);
                        tmem_ld_wait();
                        fence_regs(v);
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const f32x2 acc = pair(v[4 * e + 2 * q], v[4 * e + 2 * q + 1]);
                                float2 x = unpair(add2(fma2(acc, a2v, cb[e]), rbias[2 * k + q]));
                                if constexpr (HITS) {  // the diagonal among them
                                    x.x = cg[e].x == rgrp[2 * k + q] ? -INFINITY : x.x;
                                    x.y = cg[e].y == rgrp[2 * k + q] ? -INFINITY : x.y;
                                }
                                if constexpr (DIAGONAL) {
                                    const int i = row0 + 16 * k + 8 * q, j = tt * TN + h * 64 + 8 * e + col0;
                                    x.x = i == j ? -INFINITY : x.x;
                                    x.y = i == j + 1 ? -INFINITY : x.y;
                                }
                                float2 y = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                                if constexpr (WEIGHTS) {
                                    const float2 ww = *reinterpret_cast<const float2*>(cs + 2 * TN + h * 64 + 8 * e + col0);
                                    y.x *= ww.x;
                                    y.y *= ww.y;
                                }
                                const uint32_t bits = bf16x2_bits(y.x, y.y);
                                pk[2 * e + q] = bits;
                                exact_sum[2 * k + q] = add2(exact_sum[2 * k + q], pair(y.x, y.y));
                                round_sum[2 * k + q].add(bits);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) tmem_st_frag4(at + h * 32 + 4 * e, pk[2 * e], pk[2 * e + 1]);
                    }
                }
            };
            const bool weights = u.pass == 1 && p.weighted;
            // to the first tile of this segment that is this group's
            int t = t0;
            while (turn != group && t < t1) step_on(t);
            while (t < t1) {
                if (!mbar_wait(&ctl->sfull[bf.at], bf.phase, abort)) { ok = false; break; }
                // the stage's column constants (complete before its logits were issued)
                if (!mbar_wait(&ctl->full[st.at], st.phase, abort)) { ok = false; break; }
                tc_fence_after();
                const uint32_t buf = lane_base + acc_cols + (uint32_t)(bf.at * TN);
                const float* cs = cols_sm + st.at * 3 * TN;
                const bool diagonal = !HITS && t * TN < (u.tile + 1) * K6_M && u.tile * K6_M < (t + 1) * TN;
                if (!diagonal) {
                    if (weights) tile(buf, cs, t, Kind<1>{}); else tile(buf, cs, t, Kind<0>{});
                } else if constexpr (!HITS) {
                    if (weights) tile(buf, cs, t, Kind<3>{}); else tile(buf, cs, t, Kind<2>{});
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->pfull[bf.at]);
#pragma unroll
                for (int q = 0; q < K6_GROUPS; ++q)
                    if (t < t1) step_on(t);
            }
            if (!ok) break;
            {
                float* sums = p.sums + ((int64_t)(uid + blockIdx.x) * K6_GROUPS + group) * 2 * K6_M + quarter * 32 + (lane >> 2);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 a = unpair(exact_sum[q]);
                    float exact = a.x + a.y, rounded = round_sum[q].total();
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        exact += __shfl_xor_sync(0xffffffffu, exact, o);
                        rounded += __shfl_xor_sync(0xffffffffu, rounded, o);
                    }
                    if ((lane & 3) == 0) {
                        sums[8 * q] = exact;
                        sums[K6_M + 8 * q] = rounded;
                    }
                }
            }
            // the product of this segment
            if (!mbar_wait(&ctl->accfull, seg & 1, abort)) { ok = false; break; }
            tc_fence_after();
            const int width = p.d - u.half * K6_HALF < K6_HALF ? p.d - u.half * K6_HALF : K6_HALF;
            float* out = p.part + ((int64_t)(uid + blockIdx.x) * K6_M + quarter * 32 + lane) * p.width;
            for (int c = group * 32; c < width; c += K6_GROUPS * 32) {
                Cols32 v;
                tmem_ld_32cols(lane_base + c, v.x);
                tmem_ld_wait();
                fence_regs(v);
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    if (c + e < width)
                        *reinterpret_cast<float4*>(out + c + e) = make_float4(v.x[e], v.x[e + 1], v.x[e + 2], v.x[e + 3]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->accempty);
            w += t1 - t0;
        }
        if (!ok) {
            atomicExch(p.err, ERR_TIMEOUT_EPI);
            *abort = 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, K6_TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// the sums of the parts, the diagonal, the scale
// ---------------------------------------------------------------------------
struct K6Finish {
    const float* part;
    const float* sums;
    const float *weight, *diag;  // [b]
    const float* common;         // factor of the items' products
    const __nv_bfloat16 *users, *items;
    __nv_bfloat16 *grad_users, *grad_items;
    const int* err;
    int b, nc, d, width;
    K6Cut cut;
    float inv_tau;
};

// A block takes 32 consecutive rows of one row tile (of the users, then of the
// items) and one half of the columns; which parts of the line belong to the
// tile is found once per block.
constexpr int K6_FIN_ROWS = 32;
// The ratio of a row's sums of P before and after the rounding to bf16 lies between these.
constexpr float K6_SCALE_MIN = 256.f / 257.f, K6_SCALE_MAX = 256.f / 255.f;

template <int TN>
__global__ void __launch_bounds__(256) k6_finish(const K6Finish p) {
    __shared__ int first, parts;
    __shared__ float sums[8][2][K6_FIN_ROWS], scale[K6_FIN_ROWS];
    const K6Line<TN> line(p.b, p.nc);
    // no pdl_trigger: the last kernel, and its rows may be the next call's (tt_device.cuh)
    const int per_tile = K6_M / K6_FIN_ROWS;
    const int q = blockIdx.x / per_tile;  // row tile
    const int pass = q < line.ru ? 0 : 1;
    const int half = blockIdx.y;
    const int uid = half * (line.ru + line.rv) + q;
    if (threadIdx.x == 0) {
        const K6Unit u = line.unit(uid);
        int c = p.cut.block_of(u.begin);
        first = c;
        while (c < p.cut.grid && p.cut.begin(c) < u.begin + u.cols) ++c;
        parts = c - first;
    }
    __syncthreads();
    pdl_wait();  // k6_products
    const int row0 = (pass == 0 ? q : q - line.ru) * K6_M + (blockIdx.x % per_tile) * K6_FIN_ROWS;
    const int rows = pass == 0 ? p.b : p.nc;
    const int col0 = half * K6_HALF, cols = p.d - col0 < K6_HALF ? p.d - col0 : K6_HALF;
    const bool failed = *p.err != 0;
    const float common = pass == 1 ? *p.common : 1.f;
    // the rows' sums of P: a warp per eighth of the parts, then the eight in order
    {
        const int r = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const float* src = p.sums + (int64_t)(uid + first) * K6_GROUPS * 2 * K6_M + row0 % K6_M + r;
        float exact = 0.f, rounded = 0.f;
#pragma unroll 4
        for (int c = warp; c < parts * K6_GROUPS; c += 8) {
            exact += __ldcg(src + (int64_t)c * 2 * K6_M);
            rounded += __ldcg(src + (int64_t)c * 2 * K6_M + K6_M);
        }
        sums[warp][0][r] = exact;
        sums[warp][1][r] = rounded;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int q = 1; q < 8; ++q) {
                exact += sums[q][0][r];
                rounded += sums[q][1][r];
            }
            // no sum: nothing was added
            scale[r] = rounded != 0.f ? fminf(fmaxf(exact / rounded, K6_SCALE_MIN), K6_SCALE_MAX) : 1.f;
        }
        __syncthreads();
    }
    for (int v = threadIdx.x; v < K6_FIN_ROWS * (cols / 8); v += 256) {
        const int r = v / (cols / 8), c8 = (v - r * (cols / 8)) * 8;
        const int i = row0 + r;
        if (i >= rows) break;
        float acc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
        const float* src = p.part + ((int64_t)(uid + first) * K6_M + i % K6_M) * p.width + c8;
#pragma unroll 4
        for (int c = 0; c < parts; ++c, src += (int64_t)K6_M * p.width) {
            // past L1: written by the kernel before, beside which this one may have started
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
            const float4 y = __ldcg(reinterpret_cast<const float4*>(src) + 1);
            acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
            acc[4] += y.x, acc[5] += y.y, acc[6] += y.z, acc[7] += y.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= scale[r];
        const float w = i < p.b ? p.weight[i] : 0.f;
        float out[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) out[k] = pass == 0 ? 0.f : acc[k] * common * p.inv_tau;
        if (w != 0.f) {
            // past L1, and not as read-only data: with padding these are copies that
            // k6_prepare wrote, maybe when this block was there already
            Raw<__nv_bfloat16, 8> other;
            float x[8];
            other.a = __ldcg(reinterpret_cast<const uint4*>((pass == 0 ? p.items : p.users) + (int64_t)i * p.d + col0 + c8));
            other.get(x);
            const float c_ii = p.diag[i];
            if (pass == 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k) out[k] = fmaf(c_ii, x[k], acc[k]) * w * p.inv_tau;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) out[k] = fmaf(c_ii * w, x[k], acc[k] * common) * p.inv_tau;
            }
        }
        if (failed) {
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k] = NAN;
        }
        store_row<8>((pass == 0 ? p.grad_users : p.grad_items) + (int64_t)i * p.d + col0 + c8, out);
    }
}

int log2_ceil(int64_t x) {
    int l = 0;
    while (((int64_t)1 << l) < x) ++l;
    return l;
}

template <int TN>
int stages_for(int kchunks) {
    const int fixed = 1024 + kchunks * K6_M * 128 + (int)sizeof(K6Ctl);
    const int s = (K6_SMEM_BUDGET - fixed) / (kchunks * TN * 128 + TN * 12);
    return s < K6_MAX_STAGES ? s : K6_MAX_STAGES;
}

}  // namespace

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
SoftmaxGradPlan softmax_grad_plan(int b, int nc, int d, bool item_ids, bool copies, int sm_count) {
    SoftmaxGradPlan pl;
    const int kchunks = (d + 63) / 64;
    // 64 columns where shared memory holds no two tiles of 128 rows of 5 pieces and
    // more (the logits' products read the kept tile twice as often then: 16384^2 x
    // 256 436 against 429 us)
    pl.tile_cols = d <= 256 ? 128 : 64;
    pl.halves = (d + K6_HALF - 1) / K6_HALF;
    pl.width = d < K6_HALF ? d : K6_HALF;
    const int acc = (pl.width + 31) / 32 * 32;
    pl.bufs = (K6_TMEM_COLS - acc) / pl.tile_cols;  // 2 to 4
    if (pl.bufs > K6_MAX_BUFS) pl.bufs = K6_MAX_BUFS;
    pl.stages = pl.tile_cols == 128 ? stages_for<128>(kchunks) : stages_for<64>(kchunks);
    int64_t units;
    if (pl.tile_cols == 128) {
        const K6Line<128> line(b, nc);
        pl.work = line.per_half() * pl.halves;
        units = (int64_t)(line.ru + line.rv) * pl.halves;
    } else {
        const K6Line<64> line(b, nc);
        pl.work = line.per_half() * pl.halves;
        units = (int64_t)(line.ru + line.rv) * pl.halves;
    }
    pl.grid = pl.work < sm_count ? (int)pl.work : sm_count;
    pl.log2_slots = item_ids ? log2_ceil(2 * (int64_t)(nc > 32 ? nc : 32)) : 0;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    pl.off_err = take(sizeof(int));  // first: tt_inbatch_softmax_check reads it at offset 0
    const size_t b_pad = ((size_t)b + K6_M - 1) / K6_M * K6_M, nc_pad = ((size_t)nc + K6_M - 1) / K6_M * K6_M;
    pl.off_item = take(nc_pad * 8);  // biases, then groups
    pl.off_user = take(b_pad * 8);
    pl.off_weight = take(b_pad * sizeof(float));
    pl.off_diag = take((size_t)b * sizeof(float));
    pl.off_common = take(sizeof(float));
    pl.off_keys = take(item_ids ? ((size_t)1 << pl.log2_slots) * sizeof(unsigned long long) : 0);
    pl.off_users_c = take(copies ? (size_t)b * d * 2 : 0);
    pl.off_items_c = take(copies ? (size_t)nc * d * 2 : 0);
    pl.off_part = take((size_t)(units + pl.grid) * K6_M * pl.width * sizeof(float));
    pl.off_sums = take((size_t)(units + pl.grid) * K6_GROUPS * 2 * K6_M * sizeof(float));
    pl.bytes = off;
    return pl;
}

namespace {

template <int TN, bool HITS>
cudaError_t launch_products(const SoftmaxGradPlan& pl, const SoftmaxGrad& g, const K6Params& p, cudaStream_t s) {
    const int smem = 1024 + p.kchunks * K6_M * 128 + p.stages * (p.kchunks * TN * 128 + TN * 12) + (int)sizeof(K6Ctl);
    cudaError_t e = allow_smem(k6_products<TN, HITS>, K6_SMEM_BUDGET);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, k6_products<TN, HITS>)) != cudaSuccess) return e;
    if (attr.numRegs * K6_THREADS < K6_SPLIT_REGS) return cudaErrorInvalidConfiguration;  // the register split would not fit
    note_launch_begin(TT_KIND_SOFTMAX_GRAD, s);
    e = launch_pdl(k6_products<TN, HITS>, dim3(pl.grid), dim3(K6_THREADS), smem, s, g.tm_ux, g.tm_uy, g.tm_vx, g.tm_vy, p);
    note_launch_end(TT_KIND_SOFTMAX_GRAD, s);
    return e;
}

template <int TN>
cudaError_t launch_all(const SoftmaxGradPlan& pl, const SoftmaxGrad& g, cudaStream_t s, int sm_count) {
    uint8_t* ws = static_cast<uint8_t*>(g.workspace);
    const bool hits = g.item_ids != nullptr;
    cudaError_t e;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(ws + pl.off_keys);
    if (hits) {
        const int64_t slots = (int64_t)1 << pl.log2_slots;
        const int64_t blocks = (slots + 255) / 256;
        note_launch_begin(TT_KIND_SOFTMAX_GRAD, s);
        table_clear<<<(int)(blocks < 4 * sm_count ? blocks : 4 * sm_count), 256, 0, s>>>(keys, slots);
        note_launch_end(TT_KIND_SOFTMAX_GRAD, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    K6Prep q;
    q.logq = g.logq;
    q.item_ids = g.item_ids;
    q.valid = g.valid;
    q.lse = g.lse;
    q.loss = g.loss;
    q.grad_loss = g.grad_loss;
    q.grad_mean = g.grad_mean;
    q.keys = keys;
    q.log2_slots = pl.log2_slots;
    const size_t b_pad = ((size_t)g.b + K6_M - 1) / K6_M * K6_M, nc_pad = ((size_t)g.nc + K6_M - 1) / K6_M * K6_M;
    q.item.bias = reinterpret_cast<float*>(ws + pl.off_item);
    q.item.grp = reinterpret_cast<int*>(q.item.bias + nc_pad);
    q.user.bias = reinterpret_cast<float*>(ws + pl.off_user);
    q.user.grp = reinterpret_cast<int*>(q.user.bias + b_pad);
    q.weight = reinterpret_cast<float*>(ws + pl.off_weight);
    q.diag = reinterpret_cast<float*>(ws + pl.off_diag);
    q.common = reinterpret_cast<float*>(ws + pl.off_common);
    q.users = static_cast<const uint4*>(g.users);
    q.items = static_cast<const uint4*>(g.items);
    q.users_c = reinterpret_cast<uint4*>(ws + pl.off_users_c);
    q.items_c = reinterpret_cast<uint4*>(ws + pl.off_items_c);
    q.b = g.b;
    q.nc = g.nc;
    q.vpr = g.d / 8;
    q.err = reinterpret_cast<int*>(ws + pl.off_err);
    // a thread per column, or per 16-byte piece to copy
    const int64_t prep = ((int64_t)g.nc * (g.valid != nullptr ? q.vpr : 1) + K6_PREP_THREADS - 1) / K6_PREP_THREADS;
    const dim3 prep_grid((unsigned)(prep < 4 * sm_count ? prep : 4 * sm_count));
    note_launch_begin(TT_KIND_SOFTMAX_GRAD, s);
    if (hits) {
        e = launch_pdl(k6_prepare, prep_grid, dim3(K6_PREP_THREADS), 0, s, q);
    } else {
        k6_prepare<<<prep_grid, K6_PREP_THREADS, 0, s>>>(q);
        e = cudaGetLastError();
    }
    note_launch_end(TT_KIND_SOFTMAX_GRAD, s);
    if (e != cudaSuccess) return e;

    K6Params p;
    p.item = q.item;
    p.user = q.user;
    p.weight = q.weight;
    p.part = reinterpret_cast<float*>(ws + pl.off_part);
    p.sums = reinterpret_cast<float*>(ws + pl.off_sums);
    p.err = q.err;
    p.b = g.b;
    p.nc = g.nc;
    p.d = g.d;
    p.a2 = (float)(1.4426950408889634 / (double)g.tau);
    p.kchunks = (g.d + 63) / 64;
    p.halves = pl.halves;
    p.width = pl.width;
    p.stages = pl.stages;
    p.bufs = pl.bufs;
    p.weighted = g.grad_loss != nullptr ? 1 : 0;
    p.cut = K6Cut(pl.work, pl.grid);
    p.idesc_s = umma_idesc_bf16(K6_M, TN);
    e = hits ? launch_products<TN, true>(pl, g, p, s) : launch_products<TN, false>(pl, g, p, s);
    if (e != cudaSuccess) return e;

    K6Finish f;
    f.part = p.part;
    f.sums = p.sums;
    f.weight = q.weight;
    f.diag = q.diag;
    f.common = q.common;
    const bool copies = g.valid != nullptr;
    f.users = static_cast<const __nv_bfloat16*>(copies ? static_cast<const void*>(q.users_c) : g.users);
    f.items = static_cast<const __nv_bfloat16*>(copies ? static_cast<const void*>(q.items_c) : g.items);
    f.grad_users = static_cast<__nv_bfloat16*>(g.grad_users);
    f.grad_items = static_cast<__nv_bfloat16*>(g.grad_items);
    f.err = q.err;
    f.b = g.b;
    f.nc = g.nc;
    f.d = g.d;
    f.width = pl.width;
    f.cut = p.cut;
    f.inv_tau = (float)(1.0 / (double)g.tau);
    const K6Line<TN> line(g.b, g.nc);
    note_launch_begin(TT_KIND_SOFTMAX_GRAD, s);
    e = launch_pdl(k6_finish<TN>, dim3((unsigned)(line.ru + line.rv) * (K6_M / K6_FIN_ROWS), pl.halves), dim3(256), 0, s, f);
    note_launch_end(TT_KIND_SOFTMAX_GRAD, s);
    return e;
}

}  // namespace

cudaError_t launch_softmax_grad(const SoftmaxGradPlan& pl, const SoftmaxGrad& g, cudaStream_t s, int sm_count) {
    return pl.tile_cols == 128 ? launch_all<128>(pl, g, s, sm_count) : launch_all<64>(pl, g, s, sm_count);
}

}  // namespace tt
