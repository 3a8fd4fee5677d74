// number.hpp -- what the linear-layer operators share: the storage types (fp32,
// fp16, bf16, 8-bit e4m3 and e5m2) with their conversions, which round to
// nearest even by the hardware's instructions, and the order of tiles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace demo {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;
typedef float float4_v __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2_v __attribute__((ext_vector_type(2)));

template <typename T>
__device__ __forceinline__ float to_float(T x) { return (float)x; }
template <typename T>
__device__ __forceinline__ T from_float(float x) { return (T)x; }

// eight values from a 16-byte aligned address
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4_v a = *(const float4_v*)p, b = *(const float4_v*)(p + 4);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = a[j], v[4 + j] = b[j];
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    static_assert(sizeof(T) == 2, "two-byte type");
    typedef T vec __attribute__((ext_vector_type(8)));
    const vec a = *(const vec*)p;
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = (float)a[j];
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *(float4_v*)p = float4_v{v[0], v[1], v[2], v[3]};
    *(float4_v*)(p + 4) = float4_v{v[4], v[5], v[6], v[7]};
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    static_assert(sizeof(T) == 2, "two-byte type");
    typedef T vec __attribute__((ext_vector_type(8)));
    vec a;
#pragma unroll
    for (int j = 0; j < 8; j++) a[j] = (T)v[j];
    *(vec*)p = a;
}

// store8 past the caches
template <typename T>
__device__ __forceinline__ void stream8(T* p, const float (&v)[8]) {
    static_assert(sizeof(T) == 2, "two-byte type");
    typedef T vec __attribute__((ext_vector_type(8)));
    vec a;
#pragma unroll
    for (int j = 0; j < 8; j++) a[j] = (T)v[j];
    __builtin_nontemporal_store(a, (vec*)p);
}

// 16 bytes, four or eight values from, and eight to, any element's address: one access
// each (two for eight fp32 values), which the hardware splits where it has to
typedef uint4_v uint4_any __attribute__((aligned(2)));
template <typename T>
__device__ __forceinline__ uint4_v load16_any(const T* p) { return *(const uint4_any*)p; }
template <typename T>
__device__ __forceinline__ auto load4_any(const T* p) {
    typedef T vec __attribute__((ext_vector_type(4)));
    typedef uint2_v uint2_any __attribute__((aligned(2)));
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(vec, load16_any(p));
    else return __builtin_bit_cast(vec, (uint2_v)(*(const uint2_any*)p));
}
template <typename T>
__device__ __forceinline__ void load8_any(const T* p, float (&v)[8]) {
    constexpr int N = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(N)));
#pragma unroll
    for (int i = 0; i < 8; i += N) {
        const vec a = __builtin_bit_cast(vec, load16_any(p + i));
#pragma unroll
        for (int j = 0; j < N; j++) v[i + j] = to_float(a[j]);
    }
}
template <typename T>
__device__ __forceinline__ void store8_any(T* p, const float (&v)[8]) {
    constexpr int N = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(N)));
#pragma unroll
    for (int i = 0; i < 8; i += N) {
        vec a;
#pragma unroll
        for (int j = 0; j < N; j++) a[j] = from_float<T>(v[i + j]);
        *(uint4_any*)(p + i) = __builtin_bit_cast(uint4_v, a);
    }
}

constexpr int kE4M3 = 0, kE5M2 = 1;

// Tile of workgroup `id`: the 8 XCDs, which take ids in turn, get runs of
// neighbouring tiles each, and a run goes down kTileRun row tiles before it
// takes the next column tile, so that one XCD's workgroups share rows of both
// operands of a product in its L2, and the pieces of a transposed row that
// they write lie side by side.
constexpr uint32_t kTileRun = 8;

__device__ __forceinline__ void tile_of(uint32_t tiles_m, uint32_t tiles_n, uint32_t id, uint32_t& tm, uint32_t& tn) {
    const uint32_t tiles = tiles_m * tiles_n, q = tiles / kXcds, r = tiles % kXcds, x = id % kXcds;
    id = x * q + min(x, r) + id / kXcds;
    const uint32_t band = kTileRun * tiles_n, first = id / band * kTileRun, high = min(tiles_m - first, kTileRun);
    tm = first + id % band % high;
    tn = id % band / high;
}

}  // namespace demo
