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

// eight values of a row as they lie in memory: 16-bit types two in a word
template <typename T>
struct Raw8 {
    uint32_t w[sizeof(T) * 2];
};

// from column c on; those at and behind `cols` are 0
template <bool WIDE, typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* row, uint32_t c, uint32_t cols) {
    Raw8<T> r;
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) * 2; j++) r.w[j] = 0;
    if (WIDE ? c < cols : c + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++) {
            const T* from = row + c + i * (16 / sizeof(T));
            const uint4_v x = WIDE ? *(const uint4_v*)from : load16_any(from);
#pragma unroll
            for (int j = 0; j < 4; j++) r.w[i * 4 + j] = x[j];
        }
    } else if (WIDE) {
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (c + j < cols) r.w[j] = __float_as_uint(row[c + j]);
    } else {
        const uint16_t* from = (const uint16_t*)row;
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (c + j < cols) r.w[j >> 1] |= (uint32_t)from[c + j] << 16 * (j & 1);
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void values8(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
        if constexpr (sizeof(T) == 4) v[j] = __uint_as_float(r.w[j]);
        else v[j] = (float)__builtin_bit_cast(T, (uint16_t)(r.w[j >> 1] >> 16 * (j & 1)));
    }
}
template <bool WIDE, typename T>
__device__ __forceinline__ void load_row8(const T* row, uint32_t c, uint32_t cols, float (&v)[8]) {
    values8(load_raw8<WIDE>(row, c, cols), v);
}
template <bool WIDE, typename T>
__device__ __forceinline__ void store_row8(T* row, uint32_t c, uint32_t cols, const float (&v)[8]) {
    if (WIDE) {
        if (c < cols) store8(row + c, v);
    } else if (c + 8 <= cols) {
        store8_any(row + c, v);
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

// sum over the W waves of a row, this one being number w; `part` is used in turn by two calls
template <int W>
__device__ __forceinline__ float sum_row(float v, float (&part)[W], int w) {
    v = sum_wave(v);
    if (W == 1) return v;
    if ((threadIdx.x & 63) == 0) part[w] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; i++) s += part[i];
    return s;
}

// y = (h r) w: both kernels that quantise it compute it so, to the same bits
__device__ __forceinline__ float normed(float h, float r, float w) { return h * r * w; }

// Largest finite magnitudes of M rows of N values, as fp32 bits; infinities among
// them become NaN.  A maximum leaves NaN out by itself, and NaN becomes a NaN code.
template <int M, int N>
__device__ __forceinline__ void finite_maxima(float (&v)[M][N], uint32_t (&most)[M]) {
    float m[M], all = 0.f;
#pragma unroll
    for (int i = 0; i < M; i++) {
        m[i] = 0.f;
#pragma unroll
        for (int j = 0; j < N; j++) m[i] = fmaxf(m[i], fabsf(v[i][j]));
        all = fmaxf(all, m[i]);
    }
    if (__float_as_uint(all) == FloatSquare::kInf) {
#pragma unroll
        for (int i = 0; i < M; i++) {
            m[i] = 0.f;
#pragma unroll
            for (int j = 0; j < N; j++) {
                v[i][j] = fabsf(v[i][j]) < __uint_as_float(FloatSquare::kInf) ? v[i][j] : __uint_as_float(0x7FC00000u);
                m[i] = fmaxf(m[i], fabsf(v[i][j]));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < M; i++) most[i] = __float_as_uint(m[i]);
}

template <int FMT>
__device__ __forceinline__ uint2_v codes8(const float (&v)[8], float k) {
    s2 a = {}, b = {};
    a = codes2<FMT, false>(a, v[0], v[1], k), a = codes2<FMT, true>(a, v[2], v[3], k);
    b = codes2<FMT, false>(b, v[4], v[5], k), b = codes2<FMT, true>(b, v[6], v[7], k);
    return uint2_v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}

// Waves of a workgroup: rows of one wave share a workgroup, four at a time
template <int W>
constexpr int kNormWaves = W == 1 ? 4 : W;

// Each row is read and written once.  Where a workgroup has several rows, which is
// beyond six waves a row or a million workgroups, a wave loads its part of the next one
// before it works on this one (not of rows of two eighths a work-item).  Bound by
// bytes: 16384 x 2048 bf16 with residual, h, statistics and an operand, 237 MB, takes 43
// us (5.5 TB/s), 4096 x 8192 with y 48 us.  Eight columns a lane are 16 bytes of a
// 16-bit type, and 16 lanes a block of the operand.  Rows that are not WIDE (16-byte
// aligned, columns a multiple of 8) take the same accesses at any alignment, but the
// last columns: 16384 x 2047 with y 81 to 87 us, 177 with an access for each value.
template <typename T, int W, int NV, bool WIDE>
__global__ __launch_bounds__(64 * kNormWaves<W>) void norm_kernel(NormArgs p) {
    constexpr uint32_t kRows = kNormWaves<W> / W;  // of a workgroup
    __shared__ float part[2][W];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = wave % W;
    const uint32_t c0 = w * 512 + lane * 8, step = gridDim.x * kRows;
    uint32_t row = blockIdx.x * kRows + wave / W;
    if (row >= p.rows) return;  // rows of several waves are a workgroup's own: all of them go
    float weight[NV][8];
    Raw8<T> next[NV], next_res[NV];
    auto fetch = [&] {
#pragma unroll
        for (int v = 0; v < NV; v++) {
            next[v] = load_raw8<WIDE>((const T*)p.x + row * p.ld_x, c0 + v * W * 512, p.cols);
            if (p.res) next_res[v] = load_raw8<WIDE>((const T*)p.res + row * p.ld_res, c0 + v * W * 512, p.cols);
        }
    };
    if (NV == 1) fetch();  // rows of more are not loaded ahead: their registers are not there
#pragma unroll
    for (int v = 0; v < NV; v++) load_row8<WIDE>(p.w, c0 + v * W * 512, p.cols, weight[v]);
    for (int turn = 0;; turn ^= 1) {
        const uint32_t here = row;
        float h[NV][8], sum = 0.f;
        if (NV > 1) fetch();
#pragma unroll
        for (int v = 0; v < NV; v++) {
            values8(next[v], h[v]);
            if (p.res) {
                float a[8];
                values8(next_res[v], a);
#pragma unroll
                for (int j = 0; j < 8; j++) h[v][j] = to_float(from_float<T>(h[v][j] + a[j]));
            }
        }
        row += step;
        const bool more = row < p.rows;
        if (NV == 1 && more) fetch();  // while this row is worked on
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int j = 0; j < 8; j++) sum = fmaf(h[v][j], h[v][j], sum);
        const float r = rsqrtf(sum_row<W>(sum, part[turn], w) / (float)p.cols + p.eps);
        if (p.h) {
#pragma unroll
            for (int v = 0; v < NV; v++) store_row8<WIDE>((T*)p.h + here * p.ld_h, c0 + v * W * 512, p.cols, h[v]);
        }
        if (p.rstd && w == 0 && lane == 0) p.rstd[here] = r;
        if (p.y || p.q) {
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int j = 0; j < 8; j++) h[v][j] = normed(h[v][j], r, weight[v][j]);
        }
        if (p.y) {
#pragma unroll
            for (int v = 0; v < NV; v++) store_row8<WIDE>((T*)p.y + here * p.ld_y, c0 + v * W * 512, p.cols, h[v]);
        }
        if (p.q) {
            uint32_t most[NV];
            if (c0 + (NV - 1) * W * 512 + 8 > p.cols) {  // codes behind the last column are 0 whatever r is
#pragma unroll
                for (int v = 0; v < NV; v++)
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (c0 + v * W * 512 + j >= p.cols) h[v][j] = 0.f;
            }
            finite_maxima(h, most);
#pragma unroll
            for (int v = 0; v < NV; v++) {
                const uint32_t c = c0 + v * W * 512;
                most[v] = max16(most[v]);
                const uint32_t b = p.fmt == kE4M3 ? scale_byte<kE4M3>(most[v]) : scale_byte<kE5M2>(most[v]);
                if (c < p.pitch)
                    *(uint2_v*)(p.q + here * p.pitch + c) =
                        p.fmt == kE4M3 ? codes8<kE4M3>(h[v], scale_of(b)) : codes8<kE5M2>(h[v], scale_of(b));
                // bytes behind the last block belong to no column and come out as 0
                if ((lane & 15) == 0 && c / kBlk < p.s_pitch) p.s[(uint64_t)here * p.s_pitch + c / kBlk] = (uint8_t)b;
            }
        }
        if (!more) return;
    }
}

struct NormTurnArgs {
    const void* h;
    const float *w, *rstd;
    uint8_t *qt, *st;
    uint64_t ld_h, pitch_t;
    uint32_t s_pitch_t, rows, cols, tiles_c;
};

// The transposed operand, blocks along the rows, from h and r: 128 rows x 64
// columns a workgroup, work-item t holding rows 8 (t / 16) .. +7 of columns 4 (t %
// 16) .. +3.  The quantiser's squares of 128 x 128 need twice the registers here and
// spilled (33 us), and 512 work-items for such a square waited for one another (16384
// x 2048 bf16 20 us with h in the caches, 16.5 so).  Bound by bytes: 100 MB in 23.7
// us behind the norm, which leaves h in the last cache only.
template <typename T, int FMT, bool WIDE>
__global__ __launch_bounds__(256) void norm_turn_kernel(NormTurnArgs p) {
    constexpr int kCols = 64;
    __shared__ __attribute__((aligned(16))) uint32_t colmax[4][kCols];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kCols * kBlk];
    const int t = threadIdx.x, g = t >> 4, h = t & 15, wave = t >> 6;
    const uint32_t tiles_r = (p.rows + kBlk - 1) / kBlk;
    uint32_t tr, tc;
    tile_of(tiles_r, p.tiles_c, blockIdx.x, tr, tc);
    const uint32_t r0 = tr * kBlk + g * 8, c0 = tc * kCols + h * 4;
    float x[8][4], y[4][8], weight[4] = {}, r[8];
    const bool full = (tr + 1) * kBlk <= p.rows;
    const T* from = (const T*)p.h + r0 * p.ld_h + c0;
    typedef T vec __attribute__((ext_vector_type(4)));
    if (WIDE && full) {
        vec w[8] = {};
        if (c0 < p.cols) {
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = *(const vec*)(from + i * p.ld_h);
            const float4_v k = *(const float4_v*)(p.w + c0);
#pragma unroll
            for (int j = 0; j < 4; j++) weight[j] = k[j];
        }
        load8(p.rstd + r0, r);
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) x[i][j] = (float)w[i][j];
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const bool in = r0 + i < p.rows;
            r[i] = in ? p.rstd[r0 + i] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) x[i][j] = 0.f;
            if (in && c0 + 4 <= p.cols) {
                const vec v = load4_any(from + i * p.ld_h);
#pragma unroll
                for (int j = 0; j < 4; j++) x[i][j] = (float)v[j];
            } else if (in) {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (c0 + j < p.cols) x[i][j] = to_float(from[i * p.ld_h + j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; j++) weight[j] = c0 + j < p.cols ? p.w[c0 + j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int i = 0; i < 8; i++) y[j][i] = normed(x[i][j], r[i], weight[j]);
    if (!full) {  // codes behind the last row are 0, not -0
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (r0 + i >= p.rows) y[0][i] = y[1][i] = y[2][i] = y[3][i] = 0.f;
    }
    uint32_t cmax[4];
    finite_maxima(y, cmax);
#pragma unroll
    for (int j = 0; j < 4; j++) cmax[j] = max_rows<false>(cmax[j]);
    if ((t & 63) < 16) *(uint4_v*)&colmax[wave][h * 4] = uint4_v{cmax[0], cmax[1], cmax[2], cmax[3]};
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; w++) {
        const uint4_v o = *(const uint4_v*)&colmax[w][h * 4];
#pragma unroll
        for (int j = 0; j < 4; j++) cmax[j] = max(cmax[j], o[j]);
    }
    // 8-byte slot g of column c at g ^ (c / 4), as in quantize_kernel
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int c = h * 4 + j;
        const uint32_t b = scale_byte<FMT>(cmax[j]);
        *(uint2_v*)(turned + c * kBlk + 8 * (g ^ h)) = codes8<FMT>(y[j], scale_of(b));
        if (g == 0 && c0 + j < p.cols) {
            uint8_t* s = p.st + (uint64_t)(c0 + j) * p.s_pitch_t;
            s[tr] = (uint8_t)b;
            if (tr + 1 == tiles_r)
                for (uint32_t i = tr + 1; i < p.s_pitch_t; i++) s[i] = 0;
        }
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 2; it++) {
        const int idx = it * 256 + t, c = idx >> 3, chunk = idx & 7, x = c >> 2;
        uint4_v o = *(const uint4_v*)(turned + c * kBlk + 16 * (chunk ^ (x >> 1)));
        if (x & 1) o = uint4_v{o[2], o[3], o[0], o[1]};
        const uint32_t col = tc * kCols + c;
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

// Rows that a workgroup of the backward pass works on at a time: up to eight waves
template <int W>
constexpr int kBackRows = W <= 4 ? 8 / W : 1;

// Bound by bytes: 16384 x 2048 bf16 with a residual's gradient, 268 MB, takes 48.5 us
// (5.5 TB/s) and the join 4.7; 2561 x 768 fp32 8.4 and 3.7 us, where the launches'
// ends show.  dw's sums stay in registers over a workgroup's rows, so that 512 rows
// of them are all that the join reads, at any number of rows.
//
// A workgroup takes every grid-th kBackRows rows and keeps its part of dw in
// registers until the end; its waves meet as often, with rows or without.
template <typename T, int W, int NV, bool WIDE>
__global__ __launch_bounds__(64 * W * kBackRows<W>) void norm_back_kernel(NormBackArgs p) {
    constexpr uint32_t kRows = kBackRows<W>;
    __shared__ float part[2][kRows][W];
    __shared__ __attribute__((aligned(16))) float sums[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? W * NV * 512 : 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = wave % W, group = wave / W;
    const uint32_t c0 = w * 512 + lane * 8, step = gridDim.x * kRows;
    uint32_t row = blockIdx.x * kRows + group;
    float weight[NV][8], dw[NV][8] = {};
    Raw8<T> next_h[NV], next_dy[NV], next_res[NV];
    auto fetch = [&] {  // of the next row, or nothing
        const uint32_t cols = row < p.rows ? p.cols : 0;
#pragma unroll
        for (int v = 0; v < NV; v++) {
            next_h[v] = load_raw8<WIDE>((const T*)p.h + row * p.ld_h, c0 + v * W * 512, cols);
            next_dy[v] = load_raw8<WIDE>((const T*)p.dy + row * p.ld_dy, c0 + v * W * 512, cols);
            if (p.dres) next_res[v] = load_raw8<WIDE>((const T*)p.dres + row * p.ld_dres, c0 + v * W * 512, cols);
        }
    };
    auto fetch_weight = [&] {
#pragma unroll
        for (int v = 0; v < NV; v++) load_row8<WIDE>(p.w, c0 + v * W * 512, p.cols, weight[v]);
    };
    // Rows of two eighths a work-item have no registers to load the next one ahead in, and
    // read w again (4096 x 16384 bf16 104 to 116 us, 125 with w kept).  They spill all the
    // same, 2 to 5 registers of 128, at any alignment 10 to 12; w kept spills more.
    if (NV == 1) fetch(), fetch_weight();
    int turn = 0;
    for (uint32_t first = blockIdx.x * kRows; first < p.rows; first += step, turn ^= 1) {
        const uint32_t here = row;
        const bool on = here < p.rows;
        float n[NV][8], g[NV][8], a[NV][8] = {}, sum = 0.f;
        const float r = on ? p.rstd[here] : 0.f;
        if (NV > 1) fetch(), fetch_weight();
#pragma unroll
        for (int v = 0; v < NV; v++) {
            values8(next_h[v], n[v]);
            values8(next_dy[v], g[v]);
            if (p.dres) values8(next_res[v], a[v]);
        }
        row += step;
        if (NV == 1 && first + step < p.rows) fetch();  // while this row is worked on
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int j = 0; j < 8; j++) {
                n[v][j] *= r;
                dw[v][j] = fmaf(g[v][j], n[v][j], dw[v][j]);
                g[v][j] *= weight[v][j];
                sum = fmaf(g[v][j], n[v][j], sum);
            }
        const float mean = sum_row<W>(sum, part[turn][group], w) / (float)p.cols;
#pragma unroll
        for (int v = 0; v < NV; v++) {
#pragma unroll
            for (int j = 0; j < 8; j++) a[v][j] += r * (g[v][j] - n[v][j] * mean);
            if (on) store_row8<WIDE>((T*)p.dx + here * p.ld_dx, c0 + v * W * 512, p.cols, a[v]);
        }
    }
    if (!p.partial) return;
    if (kRows > 1) {  // the workgroup's rows, in their order
        if (group > 0) {
#pragma unroll
            for (int v = 0; v < NV; v++) store8(&sums[group - 1][c0 + v * W * 512], dw[v]);
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (uint32_t i = 0; i < kRows - 1; i++)
#pragma unroll
            for (int v = 0; v < NV; v++) {
                float o[8];
                load8(&sums[i][c0 + v * W * 512], o);
#pragma unroll
                for (int j = 0; j < 8; j++) dw[v][j] += o[j];
            }
    }
#pragma unroll
    for (int v = 0; v < NV; v++)
        store_row8<WIDE>(p.partial + (uint64_t)blockIdx.x * p.cols, c0 + v * W * 512, p.cols, dw[v]);
}

// dw = addend + the workgroups' sums: 16 columns by 64 groups of them, each in
// the order of the workgroups, then the groups in theirs.  Added in 64 bits: 72
// roundings in a row would be most of dw's error (1.7e-7 of its norm; so 6e-8),
// and what bounds the kernel is its launch and one pass over the sums.
constexpr int kJoinCols = 16;
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* partial, uint32_t count, uint32_t cols,
                                                         const float* addend, float* dw) {
    constexpr int kGroups = 1024 / kJoinCols;
    __shared__ double sums[kGroups][kJoinCols + 1];
    const uint32_t lane = threadIdx.x % kJoinCols, group = threadIdx.x / kJoinCols, c = blockIdx.x * kJoinCols + lane;
    double sum = 0;
    if (c < cols) {
#pragma unroll 8
        for (uint32_t i = group; i < count; i += kGroups) sum += partial[(uint64_t)i * cols + c];
    }
    sums[group][lane] = sum;
    __syncthreads();
    if (group == 0 && c < cols) {
        double s = addend ? addend[c] : 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; i++) s += sums[i][lane];
        dw[c] = (float)s;
    }
}

}  // namespace demo
