// norm.hpp -- root-mean-square norm in front of the linear layer (gfx950).
//
//   h = residual + x, rounded to the tensors' type;   r = 1 / sqrt(mean(h^2) + eps);   y = (h r) w
//
// and backwards, with n = h r and g = dy w:
//
//   dx = r (g - n mean(g n)) + dresidual;   dw = sum over rows of dy n
//
// A row stays in the registers of W waves (lane l of wave w holds the eight
// columns from 512 (v W + w) + 8 l on, v < NV), so it is read once; a block of
// 128 columns is 16 neighbouring lanes, whose largest magnitude and codes need
// no memory in between.  y is quantised from fp32, as the quantiser would
// quantise an fp32 y.
#pragma once

#include "quantize.hpp"

namespace demo {

struct NormArgs {
    const void *x, *res;  // res NULL: none
    const float* w;
    void *h, *y;          // NULL: not wanted
    float* rstd;          // NULL: not wanted
    uint8_t *q, *s;       // operand: codes and scale bytes (NULL: not wanted)
    uint64_t ld_x, ld_res, ld_h, ld_y, pitch;
    uint32_t s_pitch, fmt, rows, cols;
    float eps;
};

// eight values of a row from column c on; those at and behind `cols` are 0
template <bool WIDE, typename T>
__device__ __forceinline__ void load_row8(const T* row, uint32_t c, uint32_t cols, float (&v)[8]) {
    if (WIDE) {
        if (c < cols) {
            load8(row + c, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = c + j < cols ? to_float(row[c + j]) : 0.f;
    }
}
template <bool WIDE, typename T>
__device__ __forceinline__ void store_row8(T* row, uint32_t c, uint32_t cols, const float (&v)[8]) {
    if (WIDE) {
        if (c < cols) store8(row + c, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (c + j < cols) row[c + j] = from_float<T>(v[j]);
    }
}

__device__ __forceinline__ float sum_wave(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// sum over the W waves of a row; `part` is used in turn by two calls
template <int W>
__device__ __forceinline__ float sum_row(float v, float (&part)[W]) {
    v = sum_wave(v);
    if (W == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6 & (W - 1)] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; i++) s += part[i];
    return s;
}

// y = (h r) w: both kernels that quantise it compute it so, to the same bits
__device__ __forceinline__ float normed(float h, float r, float w) { return h * r * w; }

// the magnitude that counts for a block's scale: 0 for infinity and NaN
__device__ __forceinline__ uint32_t finite_bits(float v) {
    const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
    return u >= FloatSquare::kInf ? 0u : u;
}
__device__ __forceinline__ float odd_as_nan(float v) {
    return (__float_as_uint(v) & 0x7FFFFFFFu) >= FloatSquare::kInf ? __uint_as_float(0x7FC00000u) : v;
}

template <int FMT>
__device__ __forceinline__ uint2_v codes8(const float (&v)[8], float k) {
    s2 a = {}, b = {};
    a = codes2<FMT, false>(a, v[0], v[1], k), a = codes2<FMT, true>(a, v[2], v[3], k);
    b = codes2<FMT, false>(b, v[4], v[5], k), b = codes2<FMT, true>(b, v[6], v[7], k);
    return uint2_v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}

template <typename T, int W, int NV, bool WIDE>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void norm_kernel(NormArgs p) {
    constexpr int kRows = W < 4 ? 4 / W : 1;  // of a workgroup
    __shared__ float part[2][W];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = wave & (W - 1);
    const uint32_t c0 = w * 512 + lane * 8;
    float weight[NV][8];
#pragma unroll
    for (int v = 0; v < NV; v++) load_row8<WIDE>(p.w, c0 + v * W * 512, p.cols, weight[v]);
    int turn = 0;
    for (uint32_t row = blockIdx.x * kRows + (kRows > 1 ? wave / W : 0); row < p.rows; row += gridDim.x * kRows) {
        float h[NV][8], sum = 0.f;
        const T* x = (const T*)p.x + row * p.ld_x;
#pragma unroll
        for (int v = 0; v < NV; v++) load_row8<WIDE>(x, c0 + v * W * 512, p.cols, h[v]);
        if (p.res) {
            const T* res = (const T*)p.res + row * p.ld_res;
            float a[NV][8];
#pragma unroll
            for (int v = 0; v < NV; v++) load_row8<WIDE>(res, c0 + v * W * 512, p.cols, a[v]);
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int j = 0; j < 8; j++) h[v][j] = to_float(from_float<T>(h[v][j] + a[v][j]));
        }
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int j = 0; j < 8; j++) sum = fmaf(h[v][j], h[v][j], sum);
        const float r = 1.f / sqrtf(sum_row<W>(sum, part[turn]) / (float)p.cols + p.eps);
        turn ^= 1;
        if (p.h) {
#pragma unroll
            for (int v = 0; v < NV; v++) store_row8<WIDE>((T*)p.h + row * p.ld_h, c0 + v * W * 512, p.cols, h[v]);
        }
        if (p.rstd && w == 0 && lane == 0) p.rstd[row] = r;
        if (!p.y && !p.q) continue;
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int j = 0; j < 8; j++) h[v][j] = normed(h[v][j], r, weight[v][j]);
        if (p.y) {
#pragma unroll
            for (int v = 0; v < NV; v++) store_row8<WIDE>((T*)p.y + row * p.ld_y, c0 + v * W * 512, p.cols, h[v]);
        }
        if (p.q) {
#pragma unroll
            for (int v = 0; v < NV; v++) {
                const uint32_t c = c0 + v * W * 512;
                uint32_t most = 0;
                if (c + 8 > p.cols) {  // codes behind the last column are 0 whatever r is
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (c + j >= p.cols) h[v][j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    most = max(most, finite_bits(h[v][j]));
                    h[v][j] = odd_as_nan(h[v][j]);
                }
                most = max16(most);
                const uint32_t b = p.fmt == kE4M3 ? scale_byte<kE4M3>(most) : scale_byte<kE5M2>(most);
                if (c < p.pitch)
                    *(uint2_v*)(p.q + row * p.pitch + c) =
                        p.fmt == kE4M3 ? codes8<kE4M3>(h[v], scale_of(b)) : codes8<kE5M2>(h[v], scale_of(b));
                // bytes behind the last block belong to no column and come out as 0
                if ((lane & 15) == 0 && c / kBlk < p.s_pitch) p.s[(uint64_t)row * p.s_pitch + c / kBlk] = (uint8_t)b;
            }
        }
    }
}

struct NormTurnArgs {
    const void* h;
    const float *w, *rstd;
    uint8_t *qt, *st;
    uint64_t ld_h, pitch_t;
    uint32_t s_pitch_t, rows, cols, tiles_c;
};

// The transposed operand, blocks along the rows, from h and r: squares of 128 x
// 128 as in quantize_kernel, with y in place of a source.
template <typename T, int FMT, bool WIDE>
__global__ __launch_bounds__(256, 4) void norm_turn_kernel(NormTurnArgs p) {
    __shared__ __attribute__((aligned(16))) uint32_t colmax[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kBlk * kBlk];
    const int t = threadIdx.x, g = t >> 4, h = t & 15, wave = t >> 6;
    const uint32_t tiles_r = (p.rows + kBlk - 1) / kBlk;
    uint32_t tr, tc;
    tile_of(tiles_r, p.tiles_c, blockIdx.x, tr, tc);
    const uint32_t r0 = tr * kBlk + g * 8, c0 = tc * kBlk + h * 8;
    FloatSquare sq;
    float weight[8], r[8];
    load_row8<WIDE>(p.w, c0, p.cols, weight);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const bool in = r0 + i < p.rows;
        r[i] = in ? p.rstd[r0 + i] : 0.f;
        load_row8<WIDE>((const T*)p.h + (uint64_t)(r0 + i) * p.ld_h, c0, in ? p.cols : 0, sq.v[i]);
    }
    uint32_t cmax[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        cmax[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float y = r0 + i < p.rows ? normed(sq.v[i][j], r[i], weight[j]) : 0.f;
            cmax[j] = max(cmax[j], finite_bits(y));
            sq.v[i][j] = odd_as_nan(y);
        }
        cmax[j] = max_rows<false>(cmax[j]);
    }
    if ((t & 63) < 16) {
        *(uint4_v*)&colmax[wave][h * 8] = uint4_v{cmax[0], cmax[1], cmax[2], cmax[3]};
        *(uint4_v*)&colmax[wave][h * 8 + 4] = uint4_v{cmax[4], cmax[5], cmax[6], cmax[7]};
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; w++)
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const uint4_v o = *(const uint4_v*)&colmax[w][h * 8 + j];
#pragma unroll
            for (int q = 0; q < 4; q++) cmax[j + q] = max(cmax[j + q], o[q]);
        }
    // 8-byte slot g of column c at g ^ (c / 8), as in quantize_kernel
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const int c = h * 8 + j;
        const uint32_t b = scale_byte<FMT>(cmax[j]);
        *(uint2_v*)(turned + c * kBlk + 8 * (g ^ h)) = sq.col_codes<FMT>(j, scale_of(b));
        if (g == 0 && c0 + j < p.cols) {
            uint8_t* s = p.st + (uint64_t)(c0 + j) * p.s_pitch_t;
            s[tr] = (uint8_t)b;
            if (tr + 1 == tiles_r)
                for (uint32_t i = tr + 1; i < p.s_pitch_t; i++) s[i] = 0;
        }
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 4; it++) {
        const int idx = it * 256 + t, c = idx >> 3, chunk = idx & 7, x = c >> 3;
        uint4_v o = *(const uint4_v*)(turned + c * kBlk + 16 * (chunk ^ (x >> 1)));
        if (x & 1) o = uint4_v{o[2], o[3], o[0], o[1]};
        const uint32_t col = tc * kBlk + c;
        if (col < p.cols) *(uint4_v*)(p.qt + (uint64_t)col * p.pitch_t + tr * kBlk + 16 * chunk) = o;
    }
}

struct NormBackArgs {
    const void *dy, *h, *dres;  // dres NULL: none
    const float *w, *rstd;
    void* dx;
    float* partial;  // [workgroup][cols] sums of dw (NULL: not wanted)
    uint64_t ld_dy, ld_h, ld_dres, ld_dx;
    uint32_t rows, cols;
};

// A workgroup takes every grid-th row and keeps its part of dw in registers.
template <typename T, int W, int NV, bool WIDE>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void norm_back_kernel(NormBackArgs p) {
    constexpr int kRows = W < 4 ? 4 / W : 1;
    __shared__ float part[2][W];
    __shared__ float sums[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? W * NV * 512 : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = wave & (W - 1);
    const uint32_t c0 = w * 512 + lane * 8;
    float weight[NV][8], dw[NV][8] = {};
#pragma unroll
    for (int v = 0; v < NV; v++) load_row8<WIDE>(p.w, c0 + v * W * 512, p.cols, weight[v]);
    int turn = 0;
    for (uint32_t row = blockIdx.x * kRows + (kRows > 1 ? wave / W : 0); row < p.rows; row += gridDim.x * kRows) {
        float n[NV][8], g[NV][8], sum = 0.f;
        const float r = p.rstd[row];
#pragma unroll
        for (int v = 0; v < NV; v++) {
            load_row8<WIDE>((const T*)p.h + row * p.ld_h, c0 + v * W * 512, p.cols, n[v]);
            load_row8<WIDE>((const T*)p.dy + row * p.ld_dy, c0 + v * W * 512, p.cols, g[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int j = 0; j < 8; j++) {
                n[v][j] *= r;
                dw[v][j] = fmaf(g[v][j], n[v][j], dw[v][j]);
                g[v][j] *= weight[v][j];
                sum = fmaf(g[v][j], n[v][j], sum);
            }
        const float mean = sum_row<W>(sum, part[turn]) / (float)p.cols;
        turn ^= 1;
        float a[NV][8] = {};
        if (p.dres) {
#pragma unroll
            for (int v = 0; v < NV; v++)
                load_row8<WIDE>((const T*)p.dres + row * p.ld_dres, c0 + v * W * 512, p.cols, a[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; v++) {
#pragma unroll
            for (int j = 0; j < 8; j++) a[v][j] += r * (g[v][j] - n[v][j] * mean);
            store_row8<WIDE>((T*)p.dx + row * p.ld_dx, c0 + v * W * 512, p.cols, a[v]);
        }
    }
    if (!p.partial) return;
    if (kRows > 1) {  // the workgroup's waves, in their order
        if (wave > 0) {
#pragma unroll
            for (int v = 0; v < NV; v++) store8(&sums[wave - 1][v * 512 + lane * 8], dw[v]);
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int i = 0; i < kRows - 1; i++)
#pragma unroll
            for (int v = 0; v < NV; v++) {
                float o[8];
                load8(&sums[i][v * 512 + lane * 8], o);
#pragma unroll
                for (int j = 0; j < 8; j++) dw[v][j] += o[j];
            }
    }
#pragma unroll
    for (int v = 0; v < NV; v++)
        store_row8<WIDE>(p.partial + (uint64_t)blockIdx.x * p.cols, c0 + v * W * 512, p.cols, dw[v]);
}

// dw = addend + the workgroups' sums: 32 columns by 32 groups of them, each in
// the order of the workgroups, then the groups in theirs.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* partial, uint32_t count, uint32_t cols,
                                                         const float* addend, float* dw) {
    __shared__ float sums[32][33];
    const uint32_t lane = threadIdx.x & 31, group = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (uint32_t i = group; i < count; i += 32) sum += partial[(uint64_t)i * cols + c];
    }
    sums[group][lane] = sum;
    __syncthreads();
    if (group == 0 && c < cols) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i++) s += sums[i][lane];
        dw[c] = addend ? addend[c] + s : s;
    }
}

}  // namespace demo
