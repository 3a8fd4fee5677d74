// mx_product.hpp -- matrix product of 4-bit operands (gfx950).
//
//   C[i, j] = addend[i, j] + drop( sum_b 2^(ea[i,b] + eb[j,b]) sum_{k in block b} A[i,k] B[j,k] )
//
// with blocks of 32 along the sum.  The scaled matrix instructions take 128 of
// the sum at a time: lane l holds 32 codes (16 bytes) of row l % 16 and their
// scale byte, which is just one block.  Products of two codes are multiples of
// 1/4 up to 36, so nothing of them is lost; the sums are fp32's.
//
// Memory is cut as for the 8-bit product: 128 bytes of a row at a time, here
// 256 codes and 8 scale bytes ("a step").  Lane l takes chunks 2 (l / 16) and + 1
// of a step's eight chunks of 16 bytes, one for each of two instructions, and so
// the scale bytes 2 (l / 16) and + 1.
#pragma once

#include "product_big.hpp"

namespace demo {

constexpr int kFP4 = 4;  // the instruction's code of the format
constexpr int kStepK = 128;  // bytes of a step
constexpr int kStepScales = 8;

// acc += 16 x 16 pieces of A's SM and B's SN fragments over half a step, with
// byte Q of the scale words.  Columns of C run along the instruction's rows: a
// lane's four sums are neighbours in memory.
template <int Q, int SM, int SN>
__device__ __forceinline__ void mx_multiply(v4f (&acc)[SM][SN], const v4i (&fa)[SM], const v4i (&fb)[SN],
                                            const uint32_t (&ea)[SM], const uint32_t (&eb)[SN]) {
    const auto wide = [](const v4i& x) { return __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1); };
#pragma unroll
    for (int i = 0; i < SM; i++)
#pragma unroll
        for (int j = 0; j < SN; j++)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(fb[j]), wide(fa[i]), acc[i][j], kFP4, kFP4,
                                                                         Q, (int)eb[j], Q, (int)ea[i]);
}

// BM x BN of C by WM x WN waves, one of the splits of the sum (grid y), loads
// and stages as in product_kernel.  Scale bytes come 16 of a row at a time, for
// two steps.
template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void mx_kernel(ProductArgs p) {
    constexpr int NW = WM * WN, SM = BM / WM / 16, SN = BN / WN / 16;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;
    constexpr int kStage = (BM + BN) * kStepK, kScales = (BM + BN) * 2 * kStepScales;
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0 && (BM + BN) / 64 <= NW, "loads per wave");
    static_assert(NW * finish_bytes<SM, SN>() <= 2 * kStage, "the way out fits the stages");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint8_t* scales = lds + 2 * kStage;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t tm, tn;
    tile_of(p.tiles_m, p.tiles_n, blockIdx.x, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * BN;
    const uint32_t kb0 = blockIdx.y * p.kb_split, kb1 = min(kb0 + p.kb_split, p.kb);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);

    // this lane's place in the loads: row 8 (wave + i NW) + lane / 8
    const uint8_t* ga = p.a + (uint64_t)m0 * p.pitch;
    const uint8_t* gb = p.b + (uint64_t)n0 * p.pitch;
    uint32_t oa[LA], ob[LB];
#pragma unroll
    for (int i = 0; i < LA; i++) {
        const uint32_t r = 8 * (wave + i * NW) + (lane >> 3);
        oa[i] = min(r, p.m - 1 - m0) * p.pitch + ((lane & 7) ^ (r >> 1 & 7)) * 16;
    }
#pragma unroll
    for (int i = 0; i < LB; i++) {
        const uint32_t r = 8 * (wave + i * NW) + (lane >> 3);
        ob[i] = min(r, p.n - 1 - n0) * p.pitch + ((lane & 7) ^ (r >> 1 & 7)) * 16;
    }
    const bool scale_of_a = wave * 64 < BM;
    const uint32_t srow = scale_of_a ? min((uint32_t)(wave * 64 + lane), p.m - 1 - m0)
                                     : min((uint32_t)(wave * 64 - BM + lane), p.n - 1 - n0);
    const uint8_t* gs = scale_of_a ? p.sa + (uint64_t)m0 * p.s_pitch : p.sb + (uint64_t)n0 * p.s_pitch;
    const uint32_t os = srow * p.s_pitch;

    auto fetch = [&](uint32_t kb) {
        const uint32_t at = lds0 + (kb & 1) * kStage;
#pragma unroll
        for (int i = 0; i < LA; i++) load_lds16(ga + (uint64_t)kb * kStepK, oa[i], at + (wave + i * NW) * 1024);
#pragma unroll
        for (int i = 0; i < LB; i++) load_lds16(gb + (uint64_t)kb * kStepK, ob[i], at + BM * kStepK + (wave + i * NW) * 1024);
        if ((kb & 1) == 0 && wave < (BM + BN) / 64)  // two steps' scale bytes
            load_lds16(gs + kb * kStepScales, os, lds0 + 2 * kStage + (kb >> 1 & 1) * kScales + wave * 1024);
    };

    const int wm = wave % WM, wn = wave / WM, row = lane & 15, g = lane >> 4;
    const int c0 = ((2 * g) ^ (row >> 1)) * 16, c1 = ((2 * g + 1) ^ (row >> 1)) * 16;
    v4f acc[SM][SN] = {};
    uint32_t ea[SM], eb[SN];
    fetch(kb0);
    for (uint32_t kb = kb0; kb < kb1; kb++) {
        // step kb has landed, and everyone has read the stage that is filled next
        sync_loads<0>();
        if (kb + 1 < kb1) fetch(kb + 1);
        const uint8_t* stage = lds + (kb & 1) * kStage;
        const uint8_t* sc = scales + (kb >> 1 & 1) * kScales + (kb & 1) * kStepScales + 2 * g;
#pragma unroll
        for (int i = 0; i < SM; i++) ea[i] = *(const uint16_t*)(sc + ((wm * SM + i) * 16 + row) * 16);
#pragma unroll
        for (int i = 0; i < SN; i++) eb[i] = *(const uint16_t*)(sc + (BM + (wn * SN + i) * 16 + row) * 16);
        const uint8_t* sa = stage + (wm * SM * 16 + row) * kStepK;
        const uint8_t* sb = stage + (BM + wn * SN * 16 + row) * kStepK;
        v4i fa[SM], fb[SN];
#pragma unroll
        for (int i = 0; i < SN; i++) fb[i] = *(const v4i*)(sb + i * 16 * kStepK + c0);
#pragma unroll
        for (int i = 0; i < SM; i++) fa[i] = *(const v4i*)(sa + i * 16 * kStepK + c0);
        mx_multiply<0>(acc, fa, fb, ea, eb);
#pragma unroll
        for (int i = 0; i < SN; i++) fb[i] = *(const v4i*)(sb + i * 16 * kStepK + c1);
#pragma unroll
        for (int i = 0; i < SM; i++) fa[i] = *(const v4i*)(sa + i * 16 * kStepK + c1);
        mx_multiply<1>(acc, fa, fb, ea, eb);
    }
    __syncthreads();
    finish<SM, SN>(target(p, blockIdx.y), acc, (float*)(lds + wave * finish_bytes<SM, SN>()), m0 + wm * SM * 16,
                   n0 + wn * SN * 16, 0, 0, lane);
}

// Few rows: 16 columns of C for up to 16 rows by NW waves that share the sum
// among them, each taking every NW-th step straight from memory.
template <int NW>
__global__ __launch_bounds__(64 * NW) void mx_few_kernel(ProductArgs p) {
    __shared__ __attribute__((aligned(16))) float sums[NW][16 * 20];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, g = lane >> 4;
    const uint32_t n0 = blockIdx.x * 16;
    const uint32_t ra = min((uint32_t)row, p.m - 1), rb = min(n0 + row, p.n - 1);
    const uint8_t *qa = p.a + (uint64_t)ra * p.pitch + g * 32, *xa = p.sa + (uint64_t)ra * p.s_pitch + g * 2;
    const uint8_t *qb = p.b + (uint64_t)rb * p.pitch + g * 32, *xb = p.sb + (uint64_t)rb * p.s_pitch + g * 2;
    v4f acc[1][1] = {};
    for (uint32_t kb = wave; kb < p.kb; kb += NW) {
        const uint32_t ea[1] = {*(const uint16_t*)(xa + kb * kStepScales)}, eb[1] = {*(const uint16_t*)(xb + kb * kStepScales)};
        const v4i a0[1] = {*(const v4i*)(qa + kb * kStepK)}, a1[1] = {*(const v4i*)(qa + kb * kStepK + 16)};
        const v4i b0[1] = {*(const v4i*)(qb + kb * kStepK)}, b1[1] = {*(const v4i*)(qb + kb * kStepK + 16)};
        mx_multiply<0>(acc, a0, b0, ea, eb);
        mx_multiply<1>(acc, a1, b1, ea, eb);
    }
    *(v4f*)&sums[wave][row * 20 + 4 * g] = acc[0][0];
    __syncthreads();
    if (threadIdx.x < 32) {  // two lanes a row, eight columns each
        const uint32_t r = threadIdx.x >> 1, c = (threadIdx.x & 1) * 8;
        float v[8] = {};
        for (int w = 0; w < NW; w++) {
            const float* s = &sums[w][r * 20 + c];
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] += s[q];
        }
        finish8(p, r, n0 + c, 0, v);
    }
}

}  // namespace demo
