// quantize.hpp -- block-scaled 8-bit operands of the matrix product (gfx950).
//
// Each block of 128 values (a run of 128 along a row, or a 128 x 128 square)
// gets the scale 2^e with the smallest e >= -127 for which the block's largest
// finite magnitude is at most fmax * 2^e (fmax = 448 for e4m3, 57344 for e5m2:
// 1.75 times a power of two, so e follows from the magnitude's bits).  Scaling
// by a power of two is exact, so a code is one rounding of its value, and the
// scale byte e + 127 is what the scaled matrix instruction takes.
//
// One workgroup reads a 128 x 128 square once and writes both orientations:
// work-item t holds rows 8 (t / 16) .. +7 of columns 8 (t % 16) .. +7, so eight
// codes in a row make one 8-byte store of the row operand and eight codes in
// a column one 8-byte LDS store of the transposed one.  The square's maxima go
// through 16-lane exchanges (rows) and a small LDS table (columns).
#pragma once

#include "dropout.hpp"

namespace demo {

constexpr int kBlk = 128;

struct QuantArgs {
    const void* src;
    uint64_t ld;          // elements between rows of src
    uint32_t rows, cols;
    uint8_t *q, *s;       // row operand: codes and scale bytes (NULL: not wanted)
    uint64_t pitch;
    uint32_t s_pitch;
    uint8_t *qt, *st;     // transposed operand
    uint64_t pitch_t;
    uint32_t s_pitch_t;
    uint32_t tiles_c;     // column tiles
    uint32_t wide;        // rows of src are 16-byte aligned and cols a multiple of 8
    Drop drop;
};

// magnitude bits of a finite value, 0 for infinity and NaN
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    return u < 0x7F800000u ? u : 0u;
}

// scale byte of a block whose largest finite magnitude has the bits u
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t u) {
    const int b = (int)(u >> 23) - (FMT == kE4M3 ? 8 : 15) + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(b, 0);
}

// 2^-e of a scale byte e + 127 <= 247
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t max16(uint32_t u) {  // over 16 neighbouring lanes
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) u = max(u, (uint32_t)__shfl_xor((int)u, s));
    return u;
}

template <typename T, int FMT, bool TILE>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs p) {
    __shared__ uint32_t colmax[4][kBlk];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kBlk * kBlk];
    const int t = threadIdx.x, g = t >> 4, h = t & 15, wave = t >> 6;
    const uint32_t tc = blockIdx.x % p.tiles_c, tr = blockIdx.x / p.tiles_c;
    const uint32_t r0 = tr * kBlk + g * 8, c0 = tc * kBlk + h * 8;

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t r = r0 + i;
#pragma unroll
        for (int j = 0; j < 8; j++) v[i][j] = 0.f;
        if (r < p.rows && c0 < p.cols) {
            const T* src = (const T*)p.src + (uint64_t)r * p.ld + c0;
            if (p.wide) {
                load8(src, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (c0 + j < p.cols) v[i][j] = to_float(src[j]);
            }
        }
    }
    if (p.drop.on) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t r = r0 + i;
            if (r < p.rows && c0 < p.cols) {
                const uint32_t keep = keep8(p.drop, (uint64_t)r * p.cols + c0);
#pragma unroll
                for (int j = 0; j < 8; j++) v[i][j] = keep >> j & 1 ? v[i][j] * p.drop.scale : 0.f;
            }
        }
    }
    // infinities become NaN here, so that both formats store NaN for them
    uint32_t rowmax[8], cmax[8];
#pragma unroll
    for (int j = 0; j < 8; j++) cmax[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        rowmax[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const uint32_t u = finite_bits(v[i][j]);
            if ((__float_as_uint(v[i][j]) & 0x7F800000u) == 0x7F800000u) v[i][j] = __uint_as_float(0x7FC00000u);
            rowmax[i] = max(rowmax[i], u);
            cmax[j] = max(cmax[j], u);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) rowmax[i] = max16(rowmax[i]);
#pragma unroll
    for (int j = 0; j < 8; j++) {
        cmax[j] = max(cmax[j], (uint32_t)__shfl_xor((int)cmax[j], 16));
        cmax[j] = max(cmax[j], (uint32_t)__shfl_xor((int)cmax[j], 32));
    }
    if ((t & 63) < 16) {
#pragma unroll
        for (int j = 0; j < 8; j++) colmax[wave][h * 8 + j] = cmax[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const int c = h * 8 + j;
        cmax[j] = max(max(colmax[0][c], colmax[1][c]), max(colmax[2][c], colmax[3][c]));
    }
    if (TILE) {
        uint32_t all = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) all = max(all, cmax[j]);
        all = max16(all);
#pragma unroll
        for (int j = 0; j < 8; j++) cmax[j] = rowmax[j] = all;
    }
    if (p.q) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t r = r0 + i, b = scale_byte<FMT>(rowmax[i]);
            const float k = inverse_scale(b);
            if (r < p.rows) {
                const uint32_t lo = codes4<FMT>(v[i][0] * k, v[i][1] * k, v[i][2] * k, v[i][3] * k);
                const uint32_t hi = codes4<FMT>(v[i][4] * k, v[i][5] * k, v[i][6] * k, v[i][7] * k);
                *(uint2_v*)(p.q + (uint64_t)r * p.pitch + c0) = uint2_v{lo, hi};
                if (h == 0) {
                    uint8_t* s = p.s + (uint64_t)r * p.s_pitch;
                    s[tc] = (uint8_t)b;
                    if (tc + 1 == p.tiles_c)
                        for (uint32_t c = tc + 1; c < p.s_pitch; c++) s[c] = 0;
                }
            }
        }
    }
    if (p.qt) {
        // 8-byte slot g of column c sits at g ^ (c / 8): the 16 lanes of one g
        // then cover all banks, and a pair of slots stays one 16-byte chunk
        const uint32_t tiles_r = (p.rows + kBlk - 1) / kBlk;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int c = h * 8 + j;
            const uint32_t b = scale_byte<FMT>(cmax[j]);
            const float k = inverse_scale(b);
            const uint32_t lo = codes4<FMT>(v[0][j] * k, v[1][j] * k, v[2][j] * k, v[3][j] * k);
            const uint32_t hi = codes4<FMT>(v[4][j] * k, v[5][j] * k, v[6][j] * k, v[7][j] * k);
            *(uint2_v*)(turned + c * kBlk + 8 * (g ^ h)) = uint2_v{lo, hi};
            if (g == 0 && c0 + j < p.cols) {
                uint8_t* s = p.st + (uint64_t)(c0 + j) * p.s_pitch_t;
                s[tr] = (uint8_t)b;
                if (tr + 1 == tiles_r)
                    for (uint32_t r = tr + 1; r < p.s_pitch_t; r++) s[r] = 0;
            }
        }
        __syncthreads();
#pragma unroll
        for (int it = 0; it < 4; it++) {
            const int idx = it * 256 + t, c = idx >> 3, chunk = idx & 7, x = c >> 3;
            uint4_v w = *(const uint4_v*)(turned + c * kBlk + 16 * (chunk ^ (x >> 1)));
            if (x & 1) w = uint4_v{w[2], w[3], w[0], w[1]};
            const uint32_t col = tc * kBlk + c;
            if (col < p.cols) *(uint4_v*)(p.qt + (uint64_t)col * p.pitch_t + tr * kBlk + 16 * chunk) = w;
        }
    }
}

}  // namespace demo
