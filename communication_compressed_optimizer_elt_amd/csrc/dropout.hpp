// dropout.hpp -- counter-based dropout (gfx950).
//
// Element e (counted from chunk 0 of the whole tensor) takes the 16-bit half
// (e & 1) of word (e % 8) / 2 of the Philox4x32-10 block e / 8, keyed by the
// shared seed; it is kept iff that draw is at least T = round(65536 p).  No
// mask is stored: the backward pass draws the same numbers again.
//
// Why 16 bits: one Philox block costs 20 32x32->64 products, which run at a
// quarter of the vector rate; at one block for eight elements drawing costs
// less than moving eight bf16 values, at one block for four it would not.
#pragma once

#include "device_common.hpp"
#include "number.hpp"

namespace demo {

constexpr uint32_t kTagDropout = 2u;

struct Drop {
    uint64_t first;      // Philox block of element 0
    uint32_t k0, k1;     // seed
    uint32_t step, c3;   // counter words 2 and 3
    uint32_t threshold;  // draws below it are dropped, 0..65536
    float scale;         // of the kept elements
    uint32_t on;
};

// the eight draws of Philox block `blk`, two in a word
__device__ __forceinline__ void draw_block(const Drop& d, uint64_t blk, uint32_t (&w)[4]) {
    philox4x32_10((uint32_t)blk, (uint32_t)(blk >> 32), d.step, d.c3, d.k0, d.k1, w);
}

// v[j] = v[j] * scale where the block's draw keeps it, else 0
__device__ __forceinline__ void drop_drawn(const Drop& d, const uint32_t (&w)[4], float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        v[2 * j] = (w[j] & 0xFFFFu) >= d.threshold ? v[2 * j] * d.scale : 0.f;
        v[2 * j + 1] = (w[j] >> 16) >= d.threshold ? v[2 * j + 1] * d.scale : 0.f;
    }
}

// v[j] = element j of Philox block `blk` is kept ? v[j] * scale : 0
__device__ __forceinline__ void drop_block(const Drop& d, uint64_t blk, float (&v)[8]) {
    uint32_t w[4];
    draw_block(d, blk, w);
    drop_drawn(d, w, v);
}

// bit j: element e + j is kept, e counted from the tensor's element 0 (they may
// reach into the next block)
__device__ __forceinline__ uint32_t kept8(const Drop& d, uint64_t e) {
    const uint64_t blk = d.first + (e >> 3);
    const uint32_t from = (uint32_t)e & 7u;
    uint32_t w[4], keep = 0;
    draw_block(d, blk, w);
#pragma unroll
    for (int j = 0; j < 8; j++) keep |= (uint32_t)((w[j >> 1] >> 16 * (j & 1) & 0xFFFFu) >= d.threshold) << j;
    if (from) {
        draw_block(d, blk + 1, w);
#pragma unroll
        for (int j = 0; j < 8; j++) keep |= (uint32_t)((w[j >> 1] >> 16 * (j & 1) & 0xFFFFu) >= d.threshold) << (8 + j);
    }
    return keep >> from;
}

// v[j] = element e + j is kept ? v[j] * scale : 0
__device__ __forceinline__ void drop8(const Drop& d, uint64_t e, float (&v)[8]) {
    const uint32_t keep = kept8(d, e);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = keep >> j & 1 ? v[j] * d.scale : 0.f;
}

struct DropoutArgs {
    const void* x;
    const void* residual;  // NULL: none
    void* y;
    uint64_t n;
    Drop drop;
};

// y = residual + (kept ? x * scale : 0), each in fp32 and rounded once.  A
// dropped element is not read into the result, so NaN or infinity there leaves
// no trace.  One work-item per Philox block, whose eight bf16 values are one
// 16-byte access.  Bound by memory: the gradient of 16384 x 8192 bf16 takes 88
// us (6.1 TB/s); 2561 x 768 fp32 with a residual 5.2 to 6.2 us, 16 x 2048 bf16 2.2
// to 2.6 us, which is the launch.
template <typename T, bool RES>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs p) {
    const T* x = (const T*)p.x;
    const T* res = (const T*)p.residual;
    T* y = (T*)p.y;
    const uint64_t blocks = (p.n + 7) >> 3, step = (uint64_t)gridDim.x * 256;
    for (uint64_t b = (uint64_t)blockIdx.x * 256 + threadIdx.x; b < blocks; b += step) {
        const uint64_t e = b * 8;
        if (e + 8 <= p.n) {
            float v[8], r[8];
            load8(x + e, v);
            if (RES) load8(res + e, r);
            drop_block(p.drop, p.drop.first + b, v);
            if (RES) {
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] += r[j];
            }
            store8(y + e, v);
        } else {
            float v[8];
            const int left = (int)(p.n - e);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = j < left ? to_float(x[e + j]) : 0.f;
            drop_block(p.drop, p.drop.first + b, v);
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j < left) y[e + j] = from_float<T>(RES ? v[j] + to_float(res[e + j]) : v[j]);
        }
    }
}

}  // namespace demo
