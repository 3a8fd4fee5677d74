// mx_quantize.hpp -- 4-bit operands of the matrix product (gfx950): e2m1 codes
// with a power of two for each block of 32 values.
//
// A block's scale is 2^e with the smallest e >= -127 for which its largest
// magnitude is at most 6 * 2^e (6 is 1.5 times a power of two, so e follows from
// the magnitude's bits); a code is then one rounding of its value, by the
// hardware's scaled conversion.  The format has no NaN: a block with an infinity
// or a NaN gets the scale byte 255, which stands for NaN.
//
// A workgroup reads a square of 128 x 128 once and writes both orientations,
// work-item t holding rows 8 (t / 16) .. +7 of columns 8 (t % 16) .. +7 as in
// quantize_kernel.  A block of a row is then four neighbouring lanes, and the 32
// rows of a column's block are one wave's: no maximum leaves its wave.
//
// Bound by issue: 8192 x 2048 fp32 as squares, both orientations, takes 20.0 us (85
// MB, 4.2 TB/s; waves wait to issue 67% of their time), 8192 x 2048 fp16 14.4 us (51
// MB, 3.5 TB/s; 47%).  More rounds of workgroups reach no higher rate: 16384 x 8192
// bf16, 16 of them, 101 us (411 MB, 4.1 TB/s).  16384 x 2047 bf16 24 us where caches
// hold the source (41 with a load for each value), 32 where they do not.
#pragma once

#include "quantize.hpp"

namespace demo {

constexpr int kMx = 32;

struct MxArgs {
    const void* src;
    uint64_t ld;
    uint32_t rows, cols;
    uint8_t *q, *s;  // row operand: codes and scale bytes (NULL: not wanted)
    uint64_t pitch;  // bytes
    uint32_t s_pitch;
    uint8_t *qt, *st;  // transposed operand
    uint64_t pitch_t;
    uint32_t s_pitch_t;
    uint32_t tiles_r, tiles_c;  // squares
    Drop drop;
};

// scale byte of a block whose largest magnitude has the fp32 bits u
__device__ __forceinline__ uint32_t mx_byte(uint32_t u) {
    if (u >= 0x7F800000u) return 255u;
    return (uint32_t)max((int)(u >> 23) - 2 + ((u & 0x7FFFFFu) > 0x400000u ? 1 : 0), 0);
}

// maximum over four neighbouring lanes
__device__ __forceinline__ uint32_t max4(uint32_t u) { return max_dpp<0x4E>(max_dpp<0xB1>(u)); }

// eight codes of a row's, or of a column's, eight values over a scale
__device__ __forceinline__ uint32_t mx_row(const FloatSquare& q, int i, float k) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q.v[i][0], q.v[i][1], k, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q.v[i][2], q.v[i][3], k, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q.v[i][4], q.v[i][5], k, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q.v[i][6], q.v[i][7], k, 3);
}
__device__ __forceinline__ uint32_t mx_col(const FloatSquare& q, int j, float k) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q.v[0][j], q.v[1][j], k, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q.v[2][j], q.v[3][j], k, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q.v[4][j], q.v[5][j], k, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q.v[6][j], q.v[7][j], k, 3);
}
template <typename T>
__device__ __forceinline__ uint32_t mx_four(uint32_t a, uint32_t b, uint32_t c, uint32_t d, float k) {
    uint32_t w = 0;
    if constexpr (__is_same(T, bf16_t)) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(b2, a), k, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(b2, b), k, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(b2, c), k, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(b2, d), k, 3);
    } else {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2, a), k, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2, b), k, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2, c), k, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2, d), k, 3);
    }
}
template <typename T>
__device__ __forceinline__ uint32_t mx_row(const PairSquare<T>& q, int i, float k) {
    return mx_four<T>(q.v[i][0], q.v[i][1], q.v[i][2], q.v[i][3], k);
}
template <typename T>
__device__ __forceinline__ uint32_t mx_col(const PairSquare<T>& q, int j, float k) {
    return mx_four<T>(q.down(0, j), q.down(2, j), q.down(4, j), q.down(6, j), k);
}

// eight values from any element's address, `left` of them in the row; v is 0 before
template <typename T>
__device__ __forceinline__ void load_any(const T* src, uint32_t left, uint32_t (&v)[4]) {
    if (left < 8) return load_each(src, left, v);
    const uint4_v x = load16_any(src);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = x[j];
}
__device__ __forceinline__ void load_any(const float* src, uint32_t left, float (&v)[8]) {
    if (left < 8) return load_each(src, left, v);
    const uint4_v x = load16_any(src), y = load16_any(src + 4);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = __uint_as_float(x[j]), v[4 + j] = __uint_as_float(y[j]);
}

// WIDE: rows of src are 16-byte aligned and cols a multiple of 8.  DROP: the
// source through a dropout's gradient, as fp32 from there on.
template <typename T, bool TILE, bool DROP, bool WIDE>
__global__ __launch_bounds__(256, 4) void mx_quantize_kernel(MxArgs p) {
    typedef Square<T> SQ;
    constexpr int kWords = SQ::kPacked ? 4 : 8;  // of a row in memory
    constexpr int kTurned = 68;                  // bytes of a column in LDS: 17 words keep columns off each other's banks
    __shared__ uint32_t turned[kBlk * kTurned / 4];
    __shared__ uint32_t bytes[kBlk];
    const int t = threadIdx.x, g = t >> 4, h = t & 15, wave = t >> 6;
    uint32_t tr, tc;
    tile_of(p.tiles_r, p.tiles_c, blockIdx.x, tr, tc);
    const uint32_t r0 = tr * kBlk + g * 8, c0 = tc * kBlk + h * 8;

    SQ sq;
    {
        const T* src = (const T*)p.src;
        if (WIDE) {
            // what lies outside repeats the last row or columns, and becomes zero
            const uint32_t c = min(c0, p.cols - 8);
#pragma unroll
            for (int i = 0; i < 8; i++) load_wide(src + (uint64_t)min(r0 + i, p.rows - 1) * p.ld + c, sq.v[i]);
            if ((tr + 1) * kBlk > p.rows || (tc + 1) * kBlk > p.cols) {
#pragma unroll
                for (int i = 0; i < 8; i++)
#pragma unroll
                    for (int j = 0; j < kWords; j++)
                        if (r0 + i >= p.rows || c0 >= p.cols) sq.v[i][j] = 0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) {
#pragma unroll
                for (int j = 0; j < kWords; j++) sq.v[i][j] = 0;
                if (r0 + i < p.rows && c0 < p.cols) load_any(src + (uint64_t)(r0 + i) * p.ld + c0, p.cols - c0, sq.v[i]);
            }
        }
    }
    const auto out = [&] {
        if constexpr (!DROP) {
            return sq;
        } else {
            FloatSquare f;
            if constexpr (SQ::kPacked) f = sq.times(1.f);
            else f = sq;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint64_t e = (uint64_t)(r0 + i) * p.cols + c0;
                if (WIDE) drop_block(p.drop, p.drop.first + (e >> 3), f.v[i]);
                else drop8(p.drop, e, f.v[i]);
            }
            return f;
        }
    }();
    typedef std::remove_const_t<decltype(out)> OUT;
    constexpr int kCols = OUT::kPacked ? 4 : 8;  // words of a work-item's columns' maxima
    // fp32 bits of a magnitude as the square keeps it
    auto float_bits = [&](uint32_t u) {
        if constexpr (OUT::kPacked) return __float_as_uint(OUT::number(u));
        else return u;
    };
    uint32_t rowmax[8], cmax[kCols], colbits[8];
    out.template maxima<false>(rowmax, cmax, 0);
    if (TILE) {
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) all = max(all, rowmax[i]);
        all = max_rows<false>(max4(all));
#pragma unroll
        for (int i = 0; i < 8; i++) rowmax[i] = colbits[i] = all;
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) rowmax[i] = max4(rowmax[i]);
#pragma unroll
        for (int j = 0; j < kCols; j++) cmax[j] = max_rows<OUT::kPacked>(cmax[j]);
#pragma unroll
        for (int j = 0; j < 8; j++)
            colbits[j] = OUT::kPacked ? cmax[j / 2 % kCols] >> 16 * (j & 1) & 0xFFFFu : cmax[j % kCols];
    }
    if (p.q) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t r = r0 + i, b = mx_byte(float_bits(rowmax[i]));
            if (r < p.rows) {
                *(uint32_t*)(p.q + (uint64_t)r * p.pitch + tc * 64 + h * 4) = b == 255u ? 0u : mx_row(out, i, scale_of(b));
                uint8_t* s = p.s + (uint64_t)r * p.s_pitch;
                if ((h & 3) == 0) s[tc * 4 + (h >> 2)] = (uint8_t)b;
                if (h == 0 && tc + 1 == p.tiles_c)
                    for (uint32_t c = p.tiles_c * 4; c < p.s_pitch; c += 4) *(uint32_t*)(s + c) = 0;
            }
        }
    }
    if (p.qt) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int c = h * 8 + j;
            const uint32_t b = mx_byte(float_bits(colbits[j]));
            turned[c * (kTurned / 4) + g] = b == 255u ? 0u : mx_col(out, j, scale_of(b));
            if ((g & 3) == 0) ((uint8_t*)bytes)[c * 4 + wave] = (uint8_t)b;
        }
        __syncthreads();
#pragma unroll
        for (int it = 0; it < 2; it++) {
            const int idx = it * 256 + t, c = idx >> 2, chunk = idx & 3;
            const uint32_t* w = turned + c * (kTurned / 4) + 4 * chunk;
            const uint32_t col = tc * kBlk + c;
            if (col < p.cols)
                *(uint4_v*)(p.qt + (uint64_t)col * p.pitch_t + tr * 64 + 16 * chunk) = uint4_v{w[0], w[1], w[2], w[3]};
        }
        if (t < kBlk && tc * kBlk + t < p.cols) {
            uint8_t* s = p.st + (uint64_t)(tc * kBlk + t) * p.s_pitch_t;
            *(uint32_t*)(s + tr * 4) = bytes[t];
            if (tr + 1 == p.tiles_r)
                for (uint32_t r = p.tiles_r * 4; r < p.s_pitch_t; r += 4) *(uint32_t*)(s + r) = 0;
        }
    }
}

struct MxValuesArgs {
    const uint8_t *q, *s;
    uint64_t pitch, ld;
    uint32_t s_pitch, rows, cols;
    void* dst;
};

// Values of eight codes a work-item, by rows; WIDE: dst takes eight at a time.  Bound
// by bytes: 8192 x 2048 to bf16, 42 MB, takes 7.7 to 9 us (4.7 to 5.5 TB/s).
template <typename T, bool WIDE>
__global__ __launch_bounds__(256) void mx_values_kernel(MxValuesArgs p) {
    const uint32_t groups = (p.cols + 7) / 8;
    const uint64_t total = (uint64_t)p.rows * groups;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (uint64_t)gridDim.x * 256) {
        const uint32_t r = (uint32_t)(i / groups), c = (uint32_t)(i % groups) * 8;
        const uint32_t w = *(const uint32_t*)(p.q + r * p.pitch + c / 2);
        const uint32_t b = p.s[(uint64_t)r * p.s_pitch + c / kMx];
        const float k = b == 255u ? __uint_as_float(0x7FC00000u) : scale_of(b);
        typedef float v2f __attribute__((ext_vector_type(2)));
        const v2f x[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3)};
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = x[j >> 1][j & 1] * k;
        T* to = (T*)p.dst + r * p.ld + c;
        if (WIDE) {
            store8(to, v);
        } else if (c + 8 <= p.cols) {
            store8_any(to, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (c + j < p.cols) to[j] = from_float<T>(v[j]);
        }
    }
}

}  // namespace demo
