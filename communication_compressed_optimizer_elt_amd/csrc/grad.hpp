// grad.hpp -- the gradient between the backward pass and the step: its global
// norm over many tensors, and its scaled copy (gfx950).
//
//   S = sum over all tensors of x^2,   c = min(1, max_norm / (sqrt(S) + 1e-6)),   dst = c src
//
// S is summed in fp64 from the first square on, so no gradient of fp32 overflows
// or vanishes in it; that costs two fp64 instructions an element, far below
// what the loads take.  The tensors' table is part of a launch's arguments:
// nothing is copied to the device, and a captured call holds it.  A launch's
// elements are cut into chunks that never cross a tensor; a chunk is a
// wave's.
//
// Bound by bytes: the norm of 640 million fp32 takes 443 us (5.8 TB/s) and their
// clipped copy 832 (6.2 TB/s); of 44 bf16 tensors of 268 million elements 102 us
// (5.3 TB/s), the copy to fp32 248 (6.5 TB/s).  A tensor that is not 16-byte aligned on
// both sides is copied element by element, as pieces behind one of odd size are: 44 of
// 6.1 million elements to a flat gradient one element further on, bf16 318 us against
// 282, fp32 472 against 360.  Small lists are bound by their kernels' own latency: 64 vectors of
// 2048, 64 waves on 256 CUs, 15 us for the two calls, whose three kernels take 11.7.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "number.hpp"

namespace demo {

constexpr int kTable = 120;  // tensors of a launch: 3840 of the 4096 bytes of arguments

struct GradArgs {
    const void* src[kTable];
    void* dst[kTable];
    uint64_t n[kTable];
    uint32_t first[kTable];  // chunks of the launch before this tensor's
    uint32_t kind[kTable];   // type of src, 4 * type of dst, 16: both are 16-byte aligned
    uint32_t count, chunks;
    uint32_t chunk;          // elements of a chunk, a multiple of 2048
    double max_norm;
    const double* sumsq;     // scaled copy: S
    float* norm;             // scaled copy: sqrt(S) goes here (NULL: not wanted)
    double* partial;         // norm: a sum for each workgroup
};
static_assert(sizeof(GradArgs) <= 4096, "arguments of a launch");

// A chunk's tensor is the last one that begins at or before it: all lanes look at
// once (halving, seven loads one after the other, took half of a small call).
struct Piece {
    uint32_t tensor, n;
    uint64_t at;  // its first element
};
__device__ __forceinline__ Piece piece_of(const GradArgs& p, uint32_t c) {
    static_assert(kTable <= 128, "two looks a lane");
    const uint32_t lane = threadIdx.x & 63;
    const bool low = lane < p.count && p.first[lane] <= c;
    const bool high = lane + 64 < p.count && p.first[min(lane + 64, (uint32_t)kTable - 1)] <= c;
    const uint32_t t = __builtin_popcountll(__ballot(low)) + __builtin_popcountll(__ballot(high)) - 1;
    const uint64_t at = (uint64_t)(c - p.first[t]) * p.chunk;
    return {t, (uint32_t)min((uint64_t)p.chunk, p.n[t] - at), at};
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

// N neighbouring values in one access
template <typename T, int N>
struct Vec {
    typedef T type __attribute__((ext_vector_type(N)));
};

// squares of n elements from x, this lane's share of a wave
template <typename T>
__device__ __forceinline__ double squares(const T* x, uint32_t n, bool wide) {
    constexpr uint32_t V = 16 / sizeof(T);
    typedef typename Vec<T, V>::type vec;
    const uint32_t lane = threadIdx.x & 63;
    double a[4] = {};
    uint32_t i = lane;
    if (wide) {
#pragma unroll 8
        for (uint32_t k = lane * V; k + V <= n; k += 64 * V) {
            const vec v = *(const vec*)(x + k);
#pragma unroll
            for (int j = 0; j < (int)V; j++) a[j & 3] = fma((double)(float)v[j], (double)(float)v[j], a[j & 3]);
        }
        i += n & ~(V - 1);
    }
#pragma unroll 4
    for (; i < n; i += 64) {
        const double v = to_float(x[i]);
        a[0] = fma(v, v, a[0]);
    }
    return (a[0] + a[1]) + (a[2] + a[3]);
}

// Sum of the squares of a launch's tensors, one for each workgroup, whose NW waves
// take a chunk each (of a small list, which one workgroup does alone, several).
template <int NW>
__global__ __launch_bounds__(64 * NW) void grad_norm_kernel(GradArgs p) {
    double sum = 0;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint32_t c = blockIdx.x * NW + wave; c < p.chunks; c += gridDim.x * NW) {
        const Piece t = piece_of(p, c);
        const uint32_t kind = p.kind[t.tensor];
        with_type(kind & 3u, [&](auto* type) { sum += squares((decltype(type))p.src[t.tensor] + t.at, t.n, kind & 16u); });
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
template <typename S, typename D, bool PAST>
__device__ __forceinline__ void scale_chunk(const S* x, D* y, uint32_t n, bool wide, float c) {
    typedef typename Vec<S, 4>::type from;
    typedef typename Vec<D, 4>::type to;
    const uint32_t lane = threadIdx.x & 63;
    uint32_t i = lane;
    if (wide) {
#pragma unroll 8
        for (uint32_t k = lane * 4; k + 4 <= n; k += 256) {
            const from v = PAST ? __builtin_nontemporal_load((const from*)(x + k)) : *(const from*)(x + k);
            to w;
#pragma unroll
            for (int j = 0; j < 4; j++) w[j] = from_float<D>(to_float(v[j]) * c);
            if (PAST) __builtin_nontemporal_store(w, (to*)(y + k));
            else *(to*)(y + k) = w;
        }
        i += n & ~3u;
    }
#pragma unroll 4
    for (; i < n; i += 64) y[i] = from_float<D>(to_float(x[i]) * c);
}

template <bool PAST>
__global__ __launch_bounds__(256) void grad_scale_kernel(GradArgs p) {
    const double norm = sqrt(*p.sumsq), reach = norm + 1e-6;
    // compared before divided: an infinite limit holds an infinite norm too; NaN stays NaN
    const float c = p.max_norm >= reach ? 1.f : (float)(p.max_norm / reach);
    if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = (float)norm;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint32_t b = blockIdx.x * 4 + wave; b < p.chunks; b += gridDim.x * 4) {
        const Piece t = piece_of(p, b);
        const void* src = p.src[t.tensor];
        void* dst = p.dst[t.tensor];
        const uint32_t kind = p.kind[t.tensor];
        if (c == 1.f && src == dst) continue;
        with_type(kind & 3u, [&](auto* type) {
            typedef std::remove_const_t<std::remove_pointer_t<decltype(type)>> T;
            const T* x = (const T*)src + t.at;
            if ((kind >> 2 & 3u) == 0) scale_chunk<T, float, PAST>(x, (float*)dst + t.at, t.n, kind & 16u, c);
            else scale_chunk<T, T, PAST>(x, (T*)dst + t.at, t.n, kind & 16u, c);
        });
    }
}

}  // namespace demo
