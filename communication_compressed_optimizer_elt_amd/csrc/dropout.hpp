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

// bit j: element j of the eight of Philox block `blk` is kept
__device__ __forceinline__ uint32_t keep_block(const Drop& d, uint64_t blk) {
    uint32_t w[4];
    philox4x32_10((uint32_t)blk, (uint32_t)(blk >> 32), d.step, d.c3, d.k0, d.k1, w);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        m |= (uint32_t)((w[j] & 0xFFFFu) >= d.threshold) << (2 * j);
        m |= (uint32_t)((w[j] >> 16) >= d.threshold) << (2 * j + 1);
    }
    return m;
}

// bit j: element e + j is kept, j < 8, e counted from the tensor's element 0
__device__ __forceinline__ uint32_t keep8(const Drop& d, uint64_t e) {
    const uint64_t blk = d.first + (e >> 3);
    const uint32_t sh = (uint32_t)e & 7u;
    uint32_t m = keep_block(d, blk);
    if (sh) m = (m | keep_block(d, blk + 1) << 8) >> sh;
    return m;
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
// no trace.  One work-item per Philox block.
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
            const uint32_t keep = keep_block(p.drop, p.drop.first + b);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                v[j] = keep >> j & 1 ? v[j] * p.drop.scale : 0.f;
                if (RES) v[j] += r[j];
            }
            store8(y + e, v);
        } else {
            const uint32_t keep = keep_block(p.drop, p.drop.first + b);
            for (int j = 0; e + j < p.n; j++) {
                float v = keep >> j & 1 ? to_float(x[e + j]) * p.drop.scale : 0.f;
                if (RES) v += to_float(res[e + j]);
                y[e + j] = from_float<T>(v);
            }
        }
    }
}

}  // namespace demo
