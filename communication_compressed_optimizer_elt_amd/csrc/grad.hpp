// grad.hpp -- the gradient between the backward pass and the step: its global
// norm over many tensors, and its scaled copy (gfx950).
//
//   S = sum over all tensors of x^2,   c = min(1, max_norm / (sqrt(S) + 1e-6)),   dst = c src
//
// S is summed in fp64 from the first square on, so no gradient of fp32 overflows
// or vanishes in it; that costs two fp64 instructions an element, far below
// what the loads take.  The tensors' table is part of a launch's arguments:
// nothing is copied to the device, and a captured call holds it.  A launch's
// elements are cut into chunks that never cross a tensor; a workgroup takes
// every grid-th chunk and finds its tensor by halving.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "number.hpp"

namespace demo {

constexpr int kTable = 120;  // tensors of a launch: 3840 of the 4096 bytes of arguments

struct TensorEntry {
    const void* src;
    void* dst;
    uint64_t n;
    uint32_t first;  // chunks of the launch before this tensor's
    uint32_t kind;   // type of src, 4 * type of dst, 16: both are 16-byte aligned
};

struct GradArgs {
    TensorEntry table[kTable];
    uint32_t count, chunks;
    uint32_t chunk;         // elements of a chunk, a multiple of 2048
    float max_norm;
    const double* sumsq;    // scaled copy: S
    float* norm;            // scaled copy: sqrt(S) goes here (NULL: not wanted)
    double* partial;        // norm: a sum for each workgroup
};
static_assert(sizeof(GradArgs) <= 4096, "arguments of a launch");

// the tensor of chunk c: the last one that begins at or before it
__device__ __forceinline__ uint32_t tensor_of(const GradArgs& p, uint32_t c) {
    uint32_t lo = 0, hi = p.count;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (p.table[mid].first <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

// f(type of src) for the entry's kind
template <typename F>
__device__ __forceinline__ void with_type(uint32_t type, F f) {
    if (type == 0) f((const float*)nullptr);
    else if (type == 1) f((const f16_t*)nullptr);
    else f((const bf16_t*)nullptr);
}

// sum over a workgroup of 64 NW lanes; once in a kernel
template <int NW>
__device__ __forceinline__ double sum_block(double v) {
    __shared__ double part[NW];
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0;
#pragma unroll
    for (int w = 0; w < NW; w++) s += part[w];
    return s;
}

// squares of n elements from x, this work-item's share of 64 NW
template <int NW, typename T>
__device__ __forceinline__ double squares(const T* x, uint32_t n, bool wide) {
    constexpr uint32_t kStep = NW * 64;
    double a[4] = {};
    if (wide) {
        uint32_t i = threadIdx.x * 8;
#pragma unroll 4
        for (; i + 8 <= n; i += kStep * 8) {
            float v[8];
            load8(x + i, v);
#pragma unroll
            for (int j = 0; j < 8; j++) a[j & 3] = fma((double)v[j], (double)v[j], a[j & 3]);
        }
        i = (n & ~7u) + threadIdx.x;
        if (threadIdx.x < 8 && i < n) a[0] = fma((double)to_float(x[i]), (double)to_float(x[i]), a[0]);
    } else {
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < n; i += kStep) a[0] = fma((double)to_float(x[i]), (double)to_float(x[i]), a[0]);
    }
    return (a[0] + a[1]) + (a[2] + a[3]);
}

// Sum of the squares of a launch's tensors, one for each workgroup.
template <int NW>
__global__ __launch_bounds__(64 * NW) void grad_norm_kernel(GradArgs p) {
    double sum = 0;
    for (uint32_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
        const TensorEntry& t = p.table[tensor_of(p, c)];
        const uint64_t at = (uint64_t)(c - t.first) * p.chunk;
        const uint32_t n = (uint32_t)min((uint64_t)p.chunk, t.n - at);
        with_type(t.kind & 3u, [&](auto* type) {
            sum += squares<NW>((decltype(type))t.src + at, n, t.kind & 16u);
        });
    }
    sum = sum_block<NW>(sum);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = sum;
}

// The partial sums, in an order that their number fixes.
__global__ __launch_bounds__(1024) void grad_join_kernel(const double* partial, uint32_t count, double* sumsq) {
    double sum = 0;
    for (uint32_t i = threadIdx.x; i < count; i += 1024) sum += partial[i];
    sum = sum_block<16>(sum);
    if (threadIdx.x == 0) *sumsq = sum;
}

// dst = c src, rounded once.  Where c is 1 and a tensor is its own destination
// nothing is read or written: a step that is not clipped costs the launch.
template <typename S, typename D>
__device__ __forceinline__ void scale_chunk(const S* x, D* y, uint32_t n, bool wide, float c) {
    if (wide) {
        uint32_t i = threadIdx.x * 8;
#pragma unroll 4
        for (; i + 8 <= n; i += 2048) {
            float v[8];
            load8(x + i, v);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] *= c;
            store8(y + i, v);
        }
        i = (n & ~7u) + threadIdx.x;
        if (threadIdx.x < 8 && i < n) y[i] = from_float<D>(to_float(x[i]) * c);
    } else {
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < n; i += 256) y[i] = from_float<D>(to_float(x[i]) * c);
    }
}

__global__ __launch_bounds__(256) void grad_scale_kernel(GradArgs p) {
    const double norm = sqrt(*p.sumsq), q = (double)p.max_norm / (norm + 1e-6);
    const float c = q >= 1.0 ? 1.f : (float)q;  // NaN stays NaN
    if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = (float)norm;
    for (uint32_t b = blockIdx.x; b < p.chunks; b += gridDim.x) {
        const TensorEntry& t = p.table[tensor_of(p, b)];
        if (c == 1.f && t.src == t.dst) continue;
        const uint64_t at = (uint64_t)(b - t.first) * p.chunk;
        const uint32_t n = (uint32_t)min((uint64_t)p.chunk, t.n - at);
        with_type(t.kind & 3u, [&](auto* type) {
            typedef std::remove_const_t<std::remove_pointer_t<decltype(type)>> T;
            const T* x = (const T*)t.src + at;
            if ((t.kind >> 2 & 3u) == 0) scale_chunk(x, (float*)t.dst + at, n, t.kind & 16u, c);
            else scale_chunk(x, (T*)t.dst + at, n, t.kind & 16u, c);
        });
    }
}

}  // namespace demo
