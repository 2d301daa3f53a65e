// tt_softmax.cuh - what the in-batch softmax (k_softmax.cu) and its gradient
// (k_softmax_grad.cu) share: packed fp32 arithmetic, the base-2 exponential,
// and the table that numbers the item ids.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tt_device.cuh"

namespace tt {

// Packed fp32 pairs (sm_100 f32x2): two lanes of work per instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Keep the compiler from moving uses of TMEM-loaded registers above the
// tcgen05.wait::ld that makes them valid.
__device__ __forceinline__ void fence_regs(float (&x)[32]) {
    asm volatile(""
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]),
                   "+f"(x[6]), "+f"(x[7]), "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]),
                   "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]), "+f"(x[16]), "+f"(x[17]),
                   "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]),
                   "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]),
                   "+f"(x[30]), "+f"(x[31]));
}
__device__ __forceinline__ void fence_regs(Cols32& c) { fence_regs(c.x); }

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------------------
// Item groups: equal ids <=> equal group numbers. The group of an id is the
// slot it occupies in an open-addressing table of 2^log2_slots keys, at least
// twice as many as there are columns.
// ---------------------------------------------------------------------------
constexpr unsigned long long TABLE_EMPTY = 0x8000000000000000ull;  // free table slot

static __global__ void table_clear(unsigned long long* keys, int64_t slots) {
    for (int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; t < slots;
         t += (int64_t)gridDim.x * blockDim.x)
        keys[t] = TABLE_EMPTY;
}

// Fibonacci hashing (Knuth, TAOCP vol. 3, 6.4): multiply by 2^64 / golden
// ratio and keep the top bits.
__device__ __forceinline__ int64_t table_hash(unsigned long long id, int log2_slots) {
    return (int64_t)((id * 0x9E3779B97F4A7C15ull) >> (64 - log2_slots));
}

__device__ __forceinline__ int item_group(unsigned long long id, unsigned long long* keys, int log2_slots) {
    const int64_t slots = (int64_t)1 << log2_slots;
    if (id == TABLE_EMPTY) return (int)slots;  // the one id the table cannot hold has a group of its own
    // linear probing; the table has at least twice as many slots as columns,
    // so a free or matching slot is always found
    int64_t h = table_hash(id, log2_slots);
    for (int64_t probe = 0; probe < slots; ++probe) {
        // a popular id is found by a plain read, without the atomic's queue
        unsigned long long prev = *reinterpret_cast<volatile unsigned long long*>(keys + h);
        if (prev == TABLE_EMPTY) prev = atomicCAS(keys + h, TABLE_EMPTY, id);
        if (prev == TABLE_EMPTY || prev == id) return (int)h;
        h = (h + 1) & (slots - 1);
    }
    return 0;
}

}  // namespace tt
