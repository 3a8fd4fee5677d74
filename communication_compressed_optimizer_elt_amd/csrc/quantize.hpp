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
// through 16-lane exchanges (rows) and a small LDS table (columns); 16-bit
// sources stay pairs of 16 bits, whose magnitudes compare as integers, until
// the hardware's scaled conversion makes codes of them.
//
// Bound by memory where it is large: 16384 x 8192 bf16 to e4m3, both operands
// (537 MB), takes 99 us in a layer (5.4 TB/s; 112 us before the pieces of a
// transposed row were written side by side and the source read past the
// caches), 112 to 121 us back to back.  8192 x 2048 fp32 in squares (101 MB) takes
// 24 us and 16384 x 2048 bf16 through a dropout to e5m2 (134 MB) 36 us, one or
// two rounds of workgroups whose loads, arithmetic and stores coincide: waves
// wait to issue for 62% and 45% of their time.  Workgroups that stay and load
// their next square early spilled for fp32 sources, 64 registers a square, and
// took twice as long (54 us for the weight); 16-bit squares are 32 registers of
// 83 (106 with a dropout) and have not been tried so.  2561 x 768 bf16 takes 7.1
// us: its 126 workgroups leave half of the CUs idle, and a wave's load, maxima,
// exchange and store follow one another.
//
// Sources of odd width or pitch are read value by value: 16384 x 8191 bf16 212
// us, 8192 x 2047 fp32 in squares 42 us, 16384 x 2047 bf16 through a dropout 71
// us.  The fp32 kernels spill 57 to 76 scalar registers to lanes of vector
// registers, most of them on the path for infinities and NaN; those with a
// dropout on such sources also 8 to 10 vector registers to scratch (16384 x 2047:
// 86 us against 54 us of 2048 columns, 21 MB written on top).
#pragma once

#include <type_traits>

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
    uint32_t odd_from;    // 16-bit sources: least magnitude whose product with the dropout's scale is no number
    Drop drop;
};

// scale byte of a block whose largest finite magnitude has the fp32 bits u
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t u) {
    const int b = (int)(u >> 23) - (FMT == kE4M3 ? 8 : 15) + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(b, 0);
}

// the scale of a byte
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

// maxima over 16 neighbouring lanes, and over the wave's four lanes of equal l % 16
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t u) {
    return max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t max16(uint32_t u) {
    u = max_dpp<0xB1>(u);   // lanes 1 0 3 2
    u = max_dpp<0x4E>(u);   // lanes 2 3 0 1
    u = max_dpp<0x141>(u);  // halves of a row mirrored
    return max_dpp<0x140>(u);  // rows mirrored
}
typedef uint32_t uint2_s __attribute__((ext_vector_type(2)));
typedef uint16_t us2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}
template <bool PACKED>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    return PACKED ? pk_max(a, b) : max(a, b);
}
template <bool PACKED>
__device__ __forceinline__ uint32_t max_rows(uint32_t u) {
    uint2_s r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    u = larger<PACKED>(r[0], r[1]);
    r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return larger<PACKED>(r[0], r[1]);
}

// Two codes, of values over a scale 2^e, into half HI of a word.  The
// hardware divides and rounds once, to nearest even; its scale is the
// exponent of the float.
typedef short s2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
template <int FMT, bool HI>
__device__ __forceinline__ s2 codes2(s2 old, float x, float y, float scale) {
    return FMT == kE4M3 ? __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(old, x, y, scale, HI)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(old, x, y, scale, HI);
}
template <int FMT, bool HI, typename T>
__device__ __forceinline__ s2 codes2(s2 old, uint32_t pair, float scale) {
    if constexpr (sizeof(T) == 2 && __is_same(T, bf16_t)) {
        const b2 v = __builtin_bit_cast(b2, pair);
        return FMT == kE4M3 ? __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(old, v, scale, HI)
                            : __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(old, v, scale, HI);
    } else {
        const h2 v = __builtin_bit_cast(h2, pair);
        return FMT == kE4M3 ? __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(old, v, scale, HI)
                            : __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(old, v, scale, HI);
    }
}

// A work-item's 8 x 8 values as floats: magnitudes are compared as fp32 bits.
// Those from `from` on are no numbers.
struct FloatSquare {
    static constexpr bool kPacked = false;
    static constexpr uint32_t kInf = 0x7F800000u;
    float v[8][8];

    static __device__ __forceinline__ bool odd(uint32_t u, uint32_t from) { return u >= from; }
    // magnitude; FINITE: 0 for infinity and NaN
    template <bool FINITE>
    __device__ __forceinline__ uint32_t size(int i, int j, uint32_t from) const {
        const uint32_t u = __float_as_uint(v[i][j]) & 0x7FFFFFFFu;
        return FINITE && u >= from ? 0u : u;
    }
    // maxima of the rows and of the columns, words of 32 bits
    template <bool FINITE>
    __device__ __forceinline__ void maxima(uint32_t (&r)[8], uint32_t (&c)[8], uint32_t from) const {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            r[i] = 0;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t u = size<FINITE>(i, j, from);
                r[i] = max(r[i], u);
                c[j] = i ? max(c[j], u) : u;
            }
        }
    }
    // the rare path computes from the values again instead of keeping what
    // the usual one had of them in registers
    __device__ __forceinline__ void renew() {
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 8; j++) asm volatile("" : "+v"(v[i][j]));
    }
    __device__ __forceinline__ void odd_to_nan(uint32_t from) {
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 8; j++)
                if ((__float_as_uint(v[i][j]) & 0x7FFFFFFFu) >= from) v[i][j] = __uint_as_float(0x7FC00000u);
    }
    template <int FMT>
    __device__ __forceinline__ uint2_v row_codes(int i, float k) const {
        s2 a = {}, b = {};
        a = codes2<FMT, false>(a, v[i][0], v[i][1], k), a = codes2<FMT, true>(a, v[i][2], v[i][3], k);
        b = codes2<FMT, false>(b, v[i][4], v[i][5], k), b = codes2<FMT, true>(b, v[i][6], v[i][7], k);
        return uint2_v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    }
    template <int FMT>
    __device__ __forceinline__ uint2_v col_codes(int j, float k) const {
        s2 a = {}, b = {};
        a = codes2<FMT, false>(a, v[0][j], v[1][j], k), a = codes2<FMT, true>(a, v[2][j], v[3][j], k);
        b = codes2<FMT, false>(b, v[4][j], v[5][j], k), b = codes2<FMT, true>(b, v[6][j], v[7][j], k);
        return uint2_v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    }
};

// The same as pairs of 16-bit values of a row: magnitudes are compared as
// their own bits, two at a time.
template <typename T>
struct PairSquare {
    static constexpr bool kPacked = true;
    static constexpr uint32_t kInf = __is_same(T, bf16_t) ? 0x7F80u : 0x7C00u;
    uint32_t v[8][4];

    static __device__ __forceinline__ bool odd(uint32_t u, uint32_t from) {
        return (u & 0x7FFFu) >= from || (u >> 16 & 0x7FFFu) >= from;
    }
    template <bool FINITE>
    __device__ __forceinline__ uint32_t size(int i, int j, uint32_t from) const {
        uint32_t u = v[i][j] & 0x7FFF7FFFu;
        if (FINITE && (u & 0xFFFFu) >= from) u &= 0xFFFF0000u;
        if (FINITE && (u >> 16) >= from) u &= 0xFFFFu;
        return u;
    }
    // maxima of the rows, and of the columns as pairs
    template <bool FINITE>
    __device__ __forceinline__ void maxima(uint32_t (&r)[8], uint32_t (&c)[4], uint32_t from) const {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            uint32_t row = 0;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t u = size<FINITE>(i, j, from);
                row = j ? pk_max(row, u) : u;
                c[j] = i ? pk_max(c[j], u) : u;
            }
            r[i] = max(row & 0xFFFFu, row >> 16);
        }
    }
    static __device__ __forceinline__ float number(uint32_t u) { return (float)__builtin_bit_cast(T, (uint16_t)u); }
    __device__ __forceinline__ void renew() {
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) asm volatile("" : "+v"(v[i][j]));
    }
    __device__ __forceinline__ void odd_to_nan(uint32_t from) {
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if ((v[i][j] & 0x7FFFu) >= from) v[i][j] |= 0x7FFFu;
                if ((v[i][j] >> 16 & 0x7FFFu) >= from) v[i][j] |= 0x7FFF0000u;
            }
    }
    // draws become masks of what a dropout leaves out (a threshold below 65536)
    static __device__ __forceinline__ void left_out(uint32_t (&w)[4], uint32_t threshold) {
        const us2 t = {(uint16_t)threshold, (uint16_t)threshold};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            us2 out = __builtin_elementwise_sub_sat(t, __builtin_bit_cast(us2, w[j]));  // 0: kept
            out = __builtin_elementwise_min(out, us2{1, 1}) * us2{0xFFFF, 0xFFFF};
            w[j] = __builtin_bit_cast(uint32_t, out);
        }
    }
    // row i without that, or with a bit for each value it keeps
    __device__ __forceinline__ void drop_out(int i, const uint32_t (&w)[4]) {
#pragma unroll
        for (int j = 0; j < 4; j++) v[i][j] &= ~w[j];
    }
    __device__ __forceinline__ void drop_kept(int i, uint32_t keep) {
#pragma unroll
        for (int j = 0; j < 4; j++)
            v[i][j] &= (keep >> 2 * j & 1 ? 0xFFFFu : 0u) | (keep >> (2 * j + 1) & 1 ? 0xFFFF0000u : 0u);
    }
    // the values times a scale
    __device__ __forceinline__ FloatSquare times(float scale) const {
        FloatSquare f;
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 8; j++) f.v[i][j] = number(v[i][j >> 1] >> 16 * (j & 1)) * scale;
        return f;
    }
    template <int FMT>
    __device__ __forceinline__ uint2_v row_codes(int i, float k) const {
        s2 a = {}, b = {};
        a = codes2<FMT, false, T>(a, v[i][0], k), a = codes2<FMT, true, T>(a, v[i][1], k);
        b = codes2<FMT, false, T>(b, v[i][2], k), b = codes2<FMT, true, T>(b, v[i][3], k);
        return uint2_v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    }
    // column j of rows i, i + 1 as a pair
    __device__ __forceinline__ uint32_t down(int i, int j) const {
        return __builtin_amdgcn_perm(v[i + 1][j >> 1], v[i][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
    }
    template <int FMT>
    __device__ __forceinline__ uint2_v col_codes(int j, float k) const {
        s2 a = {}, b = {};
        a = codes2<FMT, false, T>(a, down(0, j), k), a = codes2<FMT, true, T>(a, down(2, j), k);
        b = codes2<FMT, false, T>(b, down(4, j), k), b = codes2<FMT, true, T>(b, down(6, j), k);
        return uint2_v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    }
};

template <typename T>
struct Square : PairSquare<T> {};
template <>
struct Square<float> : FloatSquare {};

// Eight neighbours of a row, as pairs or floats: in 16-byte loads past the
// caches (the source is read once), or the first `left` one by one into zeros
template <typename T>
__device__ __forceinline__ void load_wide(const T* src, uint32_t (&v)[4]) {
    const uint4_v w = __builtin_nontemporal_load((const uint4_v*)src);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = w[j];
}
__device__ __forceinline__ void load_wide(const float* src, float (&v)[8]) {
    const float4_v a = __builtin_nontemporal_load((const float4_v*)src);
    const float4_v b = __builtin_nontemporal_load((const float4_v*)(src + 4));
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = a[j], v[4 + j] = b[j];
}
template <typename T>
__device__ __forceinline__ void load_each(const T* src, uint32_t left, uint32_t (&v)[4]) {
    const uint16_t* s = (const uint16_t*)src;
#pragma unroll
    for (int j = 0; j < 8; j++)
        if ((uint32_t)j < left) v[j >> 1] |= (uint32_t)s[j] << 16 * (j & 1);
}
__device__ __forceinline__ void load_each(const float* src, uint32_t left, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j++)
        if ((uint32_t)j < left) v[j] = src[j];
}

// DROP: the source through a dropout's gradient.  A product with the scale, in
// fp32, grows with the value: 16-bit sources find their maxima, and what
// overflows, as pairs without the scale (16384 x 2048 bf16 36 us, as products
// 37.5 us; 8192 x 2048 20 and 22 us).  WIDE: rows of src are 16-byte aligned
// and cols a multiple of 8.
template <typename T, int FMT, bool TILE, bool DROP, bool WIDE>
__global__ __launch_bounds__(256, 4) void quantize_kernel(QuantArgs p) {
    typedef Square<T> SQ;
    constexpr int kCols = SQ::kPacked ? 4 : 8;  // words of a work-item's columns' maxima, and of a row
    __shared__ __attribute__((aligned(16))) uint32_t colmax[4][16 * kCols];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kBlk * kBlk];
    const int t = threadIdx.x, g = t >> 4, h = t & 15, wave = t >> 6;
    // neighbouring squares go to one XCD, whose L2 gathers their single scale bytes
    const uint32_t tiles_r = (p.rows + kBlk - 1) / kBlk;
    uint32_t tr, tc;
    tile_of(tiles_r, p.tiles_c, blockIdx.x, tr, tc);
    const uint32_t r0 = tr * kBlk + g * 8, c0 = tc * kBlk + h * 8;

    SQ sq;
    {
        const T* src = (const T*)p.src;
        if (WIDE) {
            // what lies outside repeats the last row or columns, and becomes zero
            const uint32_t c = min(c0, p.cols - 8);
#pragma unroll
            for (int i = 0; i < 8; i++) load_wide(src + (uint64_t)min(r0 + i, p.rows - 1) * p.ld + c, sq.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) {
#pragma unroll
                for (int j = 0; j < kCols; j++) sq.v[i][j] = 0;
                if (r0 + i < p.rows && c0 < p.cols) load_each(src + (uint64_t)(r0 + i) * p.ld + c0, p.cols - c0, sq.v[i]);
            }
        }
        uint32_t drawn[8][4];
        if (WIDE && DROP) {  // drawn while the loads are under way
#pragma unroll
            for (int i = 0; i < 8; i++) {
                draw_block(p.drop, p.drop.first + (((uint64_t)(r0 + i) * p.cols + c0) >> 3), drawn[i]);
                if constexpr (SQ::kPacked) SQ::left_out(drawn[i], p.drop.threshold);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        const bool past = WIDE && ((tr + 1) * kBlk > p.rows || (tc + 1) * kBlk > p.cols);
        const bool none = DROP && SQ::kPacked && p.drop.threshold == 65536u;  // nothing is kept
        if (past || none) {
#pragma unroll
            for (int i = 0; i < 8; i++)
#pragma unroll
                for (int j = 0; j < kCols; j++)
                    if (none || r0 + i >= p.rows || c0 >= p.cols) sq.v[i][j] = 0;
        }
        if constexpr (DROP) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint64_t e = (uint64_t)(r0 + i) * p.cols + c0;
                if constexpr (SQ::kPacked) {
                    if (WIDE) sq.drop_out(i, drawn[i]);
                    else sq.drop_kept(i, kept8(p.drop, e));
                } else {
                    if (WIDE) drop_drawn(p.drop, drawn[i], sq.v[i]);
                    else drop8(p.drop, e, sq.v[i]);
                }
            }
        }
    }
    const uint32_t odd_from = DROP && SQ::kPacked ? p.odd_from : SQ::kInf;
    // fp32 bits of a maximum as the square keeps it
    auto float_bits = [&](uint32_t u) {
        if constexpr (SQ::kPacked) return __float_as_uint(DROP ? SQ::number(u) * p.drop.scale : SQ::number(u));
        else return u;
    };
    uint32_t rowmax[8], cmax[kCols], any = 0;
    sq.template maxima<false>(rowmax, cmax, odd_from);
#pragma unroll
    for (int j = 0; j < kCols; j++) any |= SQ::odd(cmax[j], odd_from);
    if (any) {  // infinities and NaN: no part of a maximum, and NaN in the end
        sq.renew();
        sq.template maxima<true>(rowmax, cmax, odd_from);
        sq.odd_to_nan(odd_from);
    }
    const auto out = [&] {
        if constexpr (DROP && SQ::kPacked) return sq.times(p.drop.scale);
        else return sq;
    }();
#pragma unroll
    for (int i = 0; i < 8; i++) rowmax[i] = max16(rowmax[i]);
    auto rows_out = [&] {
        if (p.q) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint32_t r = r0 + i, b = scale_byte<FMT>(float_bits(rowmax[i]));
                if (r < p.rows) {
                    *(uint2_v*)(p.q + (uint64_t)r * p.pitch + c0) = out.template row_codes<FMT>(i, scale_of(b));
                    if (h == 0) {
                        uint8_t* s = p.s + (uint64_t)r * p.s_pitch;
                        s[tc] = (uint8_t)b;
                        if (tc + 1 == p.tiles_c)
                            for (uint32_t c = tc + 1; c < p.s_pitch; c++) s[c] = 0;
                    }
                }
            }
        }
    };
    if (!TILE) rows_out();
#pragma unroll
    for (int j = 0; j < kCols; j++) cmax[j] = max_rows<SQ::kPacked>(cmax[j]);
    if ((t & 63) < 16) {
#pragma unroll
        for (int j = 0; j < kCols; j += 4)
            *(uint4_v*)&colmax[wave][h * kCols + j] = uint4_v{cmax[j], cmax[j + 1], cmax[j + 2], cmax[j + 3]};
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; w++)
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
            const uint4_v o = *(const uint4_v*)&colmax[w][h * kCols + j];
#pragma unroll
            for (int q = 0; q < 4; q++) cmax[j + q] = larger<SQ::kPacked>(cmax[j + q], o[q]);
        }
    uint32_t colbits[8];
#pragma unroll
    for (int j = 0; j < 8; j++) colbits[j] = SQ::kPacked ? cmax[j / 2 % kCols] >> 16 * (j & 1) & 0xFFFFu : cmax[j % kCols];
    if (TILE) {
        uint32_t all = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) all = max(all, colbits[j]);
        all = max16(all);
#pragma unroll
        for (int j = 0; j < 8; j++) colbits[j] = rowmax[j] = all;
    }
    if (TILE) rows_out();
    if (p.qt) {
        // 8-byte slot g of column c sits at g ^ (c / 8): the 16 lanes of one g
        // then cover all banks, and a pair of slots stays one 16-byte chunk
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int c = h * 8 + j;
            const uint32_t b = scale_byte<FMT>(float_bits(colbits[j]));
            *(uint2_v*)(turned + c * kBlk + 8 * (g ^ h)) = out.template col_codes<FMT>(j, scale_of(b));
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
