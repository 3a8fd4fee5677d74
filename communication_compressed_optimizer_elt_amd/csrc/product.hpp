// product.hpp -- matrix product of block-scaled 8-bit operands (gfx950).
//
//   C[i, j] = addend[i, j] + drop( sum_b 2^(ea[i,b] + eb[j,b]) sum_{k in block b} A[i,k] B[j,k] )
//
// Both operands are stored along the summed axis with the pitch padded to 128
// by zeros, so no tail of the sum needs care.  There are two ways to multiply:
//
//  * scaled 8-bit matrix instructions (4.75 PFLOP/s from registers): they
//    apply both scales by themselves and accumulate in fp32, but line up the
//    eight products of each 8 neighbouring values of the sum at the largest of
//    them and keep 13 binary places below it.  Measured on sums of 2048 and
//    8192 (root mean square, relative to the result's): 1.5e-5 on normal
//    values, 4.0e-5 to 4.7e-5 (4.4e-4 at most) where 0.4% of the channels are 20
//    times larger.  Rounding to bf16 is off by 1.7e-3, 35 to 110 times that;
//    rounding to fp16 by 2.07e-4, 4 to 14 times that, and both together by up
//    to 2.11e-4.  16-bit results take it for twice the rate; a caller for whom
//    that is too much asks for an fp32 result;
//  * bf16 matrix instructions (2.38 PFLOP/s from registers) on codes widened
//    to bf16 with their scale, which is exact, and whose products and sums are
//    those of fp32: fp32 results take it (WIDE).  A code times its scale has to
//    stay within bf16's range, between 2^-126 and 2^128 (one and two rows are
//    multiplied in fp32, with the scales last).
#pragma once

#include <type_traits>

#include "dropout.hpp"

namespace demo {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kBlkK = 128;  // codes per scale
constexpr uint32_t kF32 = 0, kF16 = 1, kBF16 = 2;

struct ProductArgs {
    const uint8_t *a, *b;    // codes
    const uint8_t *sa, *sb;  // scale bytes
    uint32_t m, n;
    uint32_t kb;             // blocks of 128 along the sum
    uint32_t pitch;          // of both operands' codes
    uint32_t s_pitch;        // of both operands' scale bytes
    void* c;
    const void* addend;      // NULL: none
    uint64_t ldc, ld_addend;
    uint32_t dtype;
    uint32_t wide;  // n is a multiple of 8, and eight neighbours of c and addend are aligned accesses of 16 bytes
    uint32_t tiles_m, tiles_n;
    uint32_t kb_split;  // blocks of 128 along the sum of one split, a multiple of 4
    float* partial;     // [split][m][n] sums of more than one split, else NULL
    Drop drop;
};

// 64 lanes' 16 bytes at base + offset into LDS at `lds` + 16 lane, in flight
// until the next vmcnt wait.  The register that holds the LDS address is an
// input, written by the compiler, which knows what is in it; one instruction
// has to stand between that and the load.
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(lds), "v"(offset), "s"(base) : "memory");
}
// the same with 4 bytes a lane
__device__ __forceinline__ void load_lds4(const uint8_t* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, %2" ::"{m0}"(lds), "v"(offset), "s"(base) : "memory");
}

// C[i, j+from..j+7] from eight sums: drop, add, round once, store, element by
// element or (wide, from 0, eight left) in aligned accesses
template <typename T>
__device__ __forceinline__ void put_row(const ProductArgs& p, uint32_t i, uint32_t j, int from, int count, float (&v)[8],
                                        bool wide) {
    T* c = (T*)p.c + (uint64_t)i * p.ldc + j;
    const T* add = (const T*)p.addend + (p.addend ? (uint64_t)i * p.ld_addend + j : 0);
    if (wide) {
        if (p.addend) {
            float w[8];
            load8(add, w);
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] += w[q];
        }
        store8(c, v);
        return;
    }
#pragma unroll
    for (int q = 0; q < 8; q++)
        if (q >= from && q < count) c[q] = from_float<T>((p.addend ? to_float(add[q]) : 0.f) + v[q]);
}

__device__ __forceinline__ void finish8(const ProductArgs& p, uint32_t i, uint32_t j, int from, float (&v)[8]) {
    if (i >= p.m || j >= p.n) return;
    const int count = (int)min(p.n - j, 8u);
    if (p.drop.on) {
        drop8(p.drop, (uint64_t)i * p.n + j, v);
    }
    if (p.dtype == kF32) put_row<float>(p, i, j, from, count, v, p.wide);
    else if (p.dtype == kF16) put_row<f16_t>(p, i, j, from, count, v, p.wide);
    else put_row<bf16_t>(p, i, j, from, count, v, p.wide);
}

// eight raw neighbours of a row
template <typename T>
struct Row8 {
    typedef T vec __attribute__((ext_vector_type(8)));
};

// The same for P rows at once, in aligned accesses: every load of the addend
// is in flight before the first sum, every store behind the last.  16-bit rows
// go past the caches (logits of 2048 tokens: 368 us, 421 us through them);
// fp32 rows, 16 bytes of every 32 at a time, do not (2048 x 8192 x 8192: 254
// us, 266 us past them).  on[r]: the row and its eight columns are this tile's
// to write.
template <typename T, int P>
__device__ __forceinline__ void finish_rows(const ProductArgs& p, const uint64_t (&i)[P], uint32_t j, const bool (&on)[P],
                                            float (&v)[P][8]) {
    typedef typename Row8<T>::vec vec;
    if (p.addend) {
        vec w[P];
#pragma unroll
        for (int r = 0; r < P; r++)
            if (on[r]) w[r] = *(const vec*)((const T*)p.addend + i[r] * p.ld_addend + j);
#pragma unroll
        for (int r = 0; r < P; r++)
            if (on[r]) {
#pragma unroll
                for (int q = 0; q < 8; q++) v[r][q] += (float)w[r][q];
            }
    }
#pragma unroll
    for (int r = 0; r < P; r++)
        if (on[r]) {
            if constexpr (sizeof(T) == 2) stream8((T*)p.c + i[r] * p.ldc + j, v[r]);
            else store8((T*)p.c + i[r] * p.ldc + j, v[r]);
        }
}

// A wave's SM x SN accumulators of 16 x 16 (lane l holds row l % 16, columns 4
// (l / 16) .. +3 of each) go to C through a piece of LDS of the wave's own, 32
// rows at a time: a lane then holds eight neighbours, which makes one 16-byte
// access of a 16-bit row and one Philox block.  Four floats of padding a row
// keep the accesses off each other's banks.  Rows below lo_i and columns below
// lo_j are another tile's.
template <int SM, int SN>
constexpr int finish_bytes() { return 16 * (SM < 2 ? 1 : 2) * (SN * 16 + 4) * 4; }

template <int N>
using Int = std::integral_constant<int, N>;

// f(Int<s>()) of a run-time s < N: registers have no index.  The branches are
// told apart at their ends, or the compiler would make one of them that finds
// the accumulators in memory.
template <int N, int T = 0, typename F>
__device__ __forceinline__ void pick(int s, F f) {
    if constexpr (T < N) {
        if (s == T) {
            f(Int<T>());
            asm volatile("; %0" ::"n"(T));
        } else {
            pick<N, T + 1>(s, f);
        }
    }
}

// S pieces of 16 H rows x 16 SN columns; write(Int<t>()) puts piece t into the
// slab.
template <int S, int H, int SN, typename F>
__device__ __forceinline__ void finish_pieces(const ProductArgs& p, float* slab, uint32_t i0, uint32_t j0, uint32_t lo_i,
                                              uint32_t lo_j, int lane, F write) {
    constexpr int kRow = SN * 16 + 4, kLanes = SN * 2, kRows = 64 / kLanes, P = 16 * H / kRows;
    static_assert(P >= 1, "a pass fits a piece");
    const uint32_t j = j0 + lane % kLanes * 8;
    const bool col = j + 8 > lo_j && j < p.n;
#pragma unroll 1
    for (int s = 0; s < S; s++) {
        pick<S>(s, write);
        wave_lds_sync();
        const uint32_t top = i0 + s * 16 * H;
        if (p.wide) {
            float v[P][8];
            uint64_t i[P];
            bool on[P];
#pragma unroll
            for (int r = 0; r < P; r++) {
                i[r] = top + r * kRows + lane / kLanes;
                on[r] = col && i[r] >= lo_i && i[r] < p.m;
                load8(slab + (r * kRows + lane / kLanes) * kRow + lane % kLanes * 8, v[r]);
            }
            if (p.drop.on) {
#pragma unroll
                for (int r = 0; r < P; r++)
                    drop_block(p.drop, p.drop.first + ((i[r] * p.n + j) >> 3), v[r]);
            }
            if (p.dtype == kF32) finish_rows<float, P>(p, i, j, on, v);
            else if (p.dtype == kF16) finish_rows<f16_t, P>(p, i, j, on, v);
            else finish_rows<bf16_t, P>(p, i, j, on, v);
        } else {
#pragma unroll 1
            for (int r = lane / kLanes; r < 16 * H; r += kRows) {
                float v[8];
                load8(slab + r * kRow + lane % kLanes * 8, v);
                if (top + r >= lo_i) finish8(p, top + r, j, max(lo_j, j) - j, v);
            }
        }
        wave_lds_sync();
    }
}

template <int SM, int SN>
__device__ __forceinline__ void finish(const ProductArgs& p, const v4f (&acc)[SM][SN], float* slab, uint32_t i0,
                                       uint32_t j0, uint32_t lo_i, uint32_t lo_j, int lane) {
    constexpr int H = SM < 2 ? 1 : 2, kRow = SN * 16 + 4;
    static_assert(SM % H == 0, "whole pieces");
    finish_pieces<SM / H, H, SN>(p, slab, i0, j0, lo_i, lo_j, lane, [&](auto T) {
        constexpr int t = decltype(T)::value;
#pragma unroll
        for (int i = 0; i < H; i++)
#pragma unroll
            for (int c = 0; c < SN; c++)
                *(v4f*)(slab + (i * 16 + (lane & 15)) * kRow + c * 16 + 4 * (lane >> 4)) = acc[t * H + i][c];
    });
}

typedef __bf16 v8b __attribute__((ext_vector_type(8)));

// 2^(byte - 127)
__device__ __forceinline__ float scale_float(uint32_t byte) {
    return __uint_as_float(max(byte << 23, 0x00400000u));
}

// eight codes (two words) as bf16 times their scale: exact
template <int FMT>
__device__ __forceinline__ v8b widen(int lo, int hi, float scale) {
    typedef __bf16 v2b __attribute__((ext_vector_type(2)));
    v2b w[4];
    if (FMT == kE4M3) {
        w[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, scale, false);
        w[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, scale, true);
        w[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, scale, false);
        w[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, scale, true);
    } else {
        w[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)lo, scale, false);
        w[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)lo, scale, true);
        w[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)hi, scale, false);
        w[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)hi, scale, true);
    }
    return v8b{w[0][0], w[0][1], w[1][0], w[1][1], w[2][0], w[2][1], w[3][0], w[3][1]};
}

// acc += 16 x 16 pieces of A's SM and B's SN fragments over 128 of the sum.  A
// fragment's lane l holds 32 codes of row l % 16, those of chunks 2 (l / 16)
// and + 1; both operands use the same order, so any order is right.  ea and eb
// hold the rows' scale bytes in their lowest bytes.  Columns of C run along
// the instruction's rows: a lane's four sums are neighbours in memory.
template <int FA, int FB, bool WIDE, int SM, int SN>
__device__ __forceinline__ void multiply(v4f (&acc)[SM][SN], const v8i (&fa)[SM], const v8i (&fb)[SN],
                                         const uint32_t (&ea)[SM], const uint32_t (&eb)[SN]) {
    if constexpr (WIDE) {
        float ka[SM], kb[SN];
#pragma unroll
        for (int i = 0; i < SM; i++) ka[i] = scale_float(ea[i] & 255u);
#pragma unroll
        for (int j = 0; j < SN; j++) kb[j] = scale_float(eb[j] & 255u);
#pragma unroll
        for (int q = 0; q < 4; q++) {
            v8b wb[SN];
#pragma unroll
            for (int j = 0; j < SN; j++) wb[j] = widen<FB>(fb[j][2 * q], fb[j][2 * q + 1], kb[j]);
#pragma unroll
            for (int i = 0; i < SM; i++) {
                const v8b wa = widen<FA>(fa[i][2 * q], fa[i][2 * q + 1], ka[i]);
#pragma unroll
                for (int j = 0; j < SN; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa, acc[i][j], 0, 0, 0);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < SM; i++)
#pragma unroll
            for (int j = 0; j < SN; j++)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i], acc[i][j], FB, FA, 0,
                                                                             (int)eb[j], 0, (int)ea[i]);
    }
}

// Where this workgroup's sums go: the result, or its split's plane of the partial sums.
__device__ __forceinline__ ProductArgs target(const ProductArgs& p, uint32_t split) {
    ProductArgs t = p;
    if (p.partial) {
        t.c = p.partial + (uint64_t)split * p.m * p.n;
        t.ldc = p.n;
        t.dtype = kF32;
        t.addend = nullptr;
        t.wide = p.n % 8 == 0;
        t.drop.on = 0;
    }
    return t;
}

// All but the N newest of this wave's loads have landed and its LDS reads are
// done; then the same holds for every wave.
template <int N>
__device__ __forceinline__ void sync_loads() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// BM x BN of C by WM x WN waves, one of the splits of the sum (grid y).  LDS
// holds two blocks of 128 along the sum, filled by loads that go from memory to
// LDS one block ahead; one barrier a block.  What hides the waits is a second
// workgroup on the CU (four of 64 x 64): three or four stages, and with them
// fewer workgroups, measured slower (2048 x 2048 x 2048 in tiles of 64: 15.8
// us, 19.2 and 18.2 with three and four; 11.8 against 12.0 us at 2304 x 768 x
// 2560, where no CU has more than two; 4096 x 8192 x 2048 in tiles of 128: 71
// us, 112 with four), and so did 8 waves of half the size (17.6 us).  Row r's
// 16-byte chunk c sits at c ^ (r / 2 & 7), which spreads 16 rows' reads of one
// chunk over all 64 banks; loads into LDS write lanes in order, so the exchange
// is made on their source addresses.  Fp32 results in tiles of 64 have a kernel
// of their own below.  Rows past the matrix repeat its last row; what they give is not stored.
template <int FA, int FB, bool WIDE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void product_kernel(ProductArgs p) {
    constexpr int NW = WM * WN, SM = BM / WM / 16, SN = BN / WN / 16;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;
    constexpr int kStage = (BM + BN) * kBlkK, kScales = (BM + BN) * 4;
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
        for (int i = 0; i < LA; i++) load_lds16(ga + kb * kBlkK, oa[i], at + (wave + i * NW) * 1024);
#pragma unroll
        for (int i = 0; i < LB; i++) load_lds16(gb + kb * kBlkK, ob[i], at + BM * kBlkK + (wave + i * NW) * 1024);
        if ((kb & 3) == 0 && wave < (BM + BN) / 64)  // four blocks' scale bytes
            load_lds4(gs + kb, os, lds0 + 2 * kStage + (kb >> 2 & 1) * kScales + wave * 256);
    };

    const int wm = wave % WM, wn = wave / WM, row = lane & 15, g = lane >> 4;
    const int c0 = ((2 * g) ^ (row >> 1)) * 16, c1 = ((2 * g + 1) ^ (row >> 1)) * 16;
    v4f acc[SM][SN] = {};
    uint32_t ea[SM], eb[SN];
    fetch(kb0);
    for (uint32_t kb = kb0; kb < kb1; kb++) {
        // block kb has landed, and everyone has read the stage that is filled next
        sync_loads<0>();
        if (kb + 1 < kb1) fetch(kb + 1);
        const uint8_t* stage = lds + (kb & 1) * kStage;
        if ((kb & 3) == 0) {
            const uint32_t* sc = (const uint32_t*)(scales + (kb >> 2 & 1) * kScales);
#pragma unroll
            for (int i = 0; i < SM; i++) ea[i] = sc[(wm * SM + i) * 16 + row];
#pragma unroll
            for (int i = 0; i < SN; i++) eb[i] = sc[BM + (wn * SN + i) * 16 + row];
        }
        const uint8_t* sa = stage + (wm * SM * 16 + row) * kBlkK;
        const uint8_t* sb = stage + (BM + wn * SN * 16 + row) * kBlkK;
        v8i fa[SM], fb[SN];
#pragma unroll
        for (int i = 0; i < SN; i++)
            fb[i] = __builtin_shufflevector(*(const v4i*)(sb + i * 16 * kBlkK + c0),
                                            *(const v4i*)(sb + i * 16 * kBlkK + c1), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int i = 0; i < SM; i++)
            fa[i] = __builtin_shufflevector(*(const v4i*)(sa + i * 16 * kBlkK + c0),
                                            *(const v4i*)(sa + i * 16 * kBlkK + c1), 0, 1, 2, 3, 4, 5, 6, 7);
        multiply<FA, FB, WIDE>(acc, fa, fb, ea, eb);
#pragma unroll
        for (int i = 0; i < SM; i++) ea[i] >>= 8;
#pragma unroll
        for (int i = 0; i < SN; i++) eb[i] >>= 8;
    }
    __syncthreads();
    finish<SM, SN>(target(p, blockIdx.y), acc, (float*)(lds + wave * finish_bytes<SM, SN>()), m0 + wm * SM * 16,
                   n0 + wn * SN * 16, 0, 0, lane);
}

// 64 x 64 of C with an fp32 result: four waves that share the sum, a quarter of
// each block of 128 each.  A wave then widens 32 codes of 64 rows of both
// operands for its 16 matrix instructions, half of what it would widen for 32 x
// 32 of C and the whole block: 2304 x 768 x 2560 takes 17.2 us (18.8 so), 2048 x
// 2048 x 8192 75 us (85 so).  Bound by issue: widening and matrix instructions
// of a SIMD's waves take turns (six VALU instructions for each matrix one, whose
// units are busy for 28% of the time), on 432 tiles that the CUs share unevenly;
// two blocks a barrier gave nothing (19.4 against
// 18.4 us with an addend).  Loads, stages and chunks as in product_kernel.  In
// the end wave w takes rows 16 w .. +15 and adds the others' sums in the order
// w, w+3, w+2, w+1 (mod 4): three exchanges through two halves of LDS.
template <int FA, int FB>
__global__ __launch_bounds__(256, 4) void product_shared_kernel(ProductArgs p) {
    constexpr int T = 64, kStage = 2 * T * kBlkK, kScales = 2 * T * 4, kPiece = 64 * 4 * 16;
    static_assert(8 * kPiece <= 2 * kStage && 4 * finish_bytes<1, 4>() <= 2 * kStage, "the way out fits the stages");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint8_t* scales = lds + 2 * kStage;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t tm, tn;
    tile_of(p.tiles_m, p.tiles_n, blockIdx.x, tm, tn);
    const uint32_t m0 = tm * T, n0 = tn * T;
    const uint32_t kb0 = blockIdx.y * p.kb_split, kb1 = min(kb0 + p.kb_split, p.kb);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);

    // this lane's place in the loads: row 8 (wave + 4 i) + lane / 8
    const uint8_t* ga = p.a + (uint64_t)m0 * p.pitch;
    const uint8_t* gb = p.b + (uint64_t)n0 * p.pitch;
    uint32_t oa[2], ob[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t r = 8 * (wave + i * 4) + (lane >> 3), c = ((lane & 7) ^ (r >> 1 & 7)) * 16;
        oa[i] = min(r, p.m - 1 - m0) * p.pitch + c;
        ob[i] = min(r, p.n - 1 - n0) * p.pitch + c;
    }
    const uint32_t srow = min((uint32_t)lane, wave ? p.n - 1 - n0 : p.m - 1 - m0);
    const uint8_t* gs = wave ? p.sb + (uint64_t)n0 * p.s_pitch : p.sa + (uint64_t)m0 * p.s_pitch;
    const uint32_t os = srow * p.s_pitch;
    auto fetch = [&](uint32_t kb) {
        const uint32_t at = lds0 + (kb & 1) * kStage;
#pragma unroll
        for (int i = 0; i < 2; i++) load_lds16(ga + kb * kBlkK, oa[i], at + (wave + i * 4) * 1024);
#pragma unroll
        for (int i = 0; i < 2; i++) load_lds16(gb + kb * kBlkK, ob[i], at + T * kBlkK + (wave + i * 4) * 1024);
        if ((kb & 3) == 0 && wave < 2)  // four blocks' scale bytes
            load_lds4(gs + kb, os, lds0 + 2 * kStage + (kb >> 2 & 1) * kScales + wave * 256);
    };

    // eight codes of row `row` of a fragment: half g % 2 of chunk 2 wave + g / 2
    const int row = lane & 15, g = lane >> 4;
    const uint32_t at = row * kBlkK + ((2 * wave + (g >> 1)) ^ (row >> 1)) * 16 + (g & 1) * 8;
    v4f acc[4][4] = {};
    uint32_t ea[4], eb[4];
    fetch(kb0);
    for (uint32_t kb = kb0; kb < kb1; kb++) {
        // block kb has landed, and everyone has read the stage that is filled next
        sync_loads<0>();
        if (kb + 1 < kb1) fetch(kb + 1);
        const uint8_t* stage = lds + (kb & 1) * kStage + at;
        if ((kb & 3) == 0) {
            const uint32_t* sc = (const uint32_t*)(scales + (kb >> 2 & 1) * kScales) + row;
#pragma unroll
            for (int i = 0; i < 4; i++) ea[i] = sc[i * 16], eb[i] = sc[T + i * 16];
        }
        uint2_v fa[4], fb[4];
#pragma unroll
        for (int i = 0; i < 4; i++) fb[i] = *(const uint2_v*)(stage + (T + i * 16) * kBlkK);
#pragma unroll
        for (int i = 0; i < 4; i++) fa[i] = *(const uint2_v*)(stage + i * 16 * kBlkK);
        v8b wb[4];
#pragma unroll
        for (int j = 0; j < 4; j++) wb[j] = widen<FB>((int)fb[j][0], (int)fb[j][1], scale_float(eb[j] & 255u));
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const v8b wa = widen<FA>((int)fa[i][0], (int)fa[i][1], scale_float(ea[i] & 255u));
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa, acc[i][j], 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) ea[i] >>= 8, eb[i] >>= 8;
    }
    __syncthreads();

    v4f* half = (v4f*)lds;  // place [exchange % 2][taker][column][lane]
    auto give = [&](int x) {  // to wave w + x
        const int to = (wave + x) & 3;
        pick<4>(to, [&](auto I) {
#pragma unroll
            for (int j = 0; j < 4; j++) half[((x & 1) * 4 + to) * 256 + j * 64 + lane] = acc[decltype(I)::value][j];
        });
    };
    v4f own[1][4];
    pick<4>(wave, [&](auto I) {
#pragma unroll
        for (int j = 0; j < 4; j++) own[0][j] = acc[decltype(I)::value][j];
    });
    auto take = [&](int x) {
#pragma unroll
        for (int j = 0; j < 4; j++) own[0][j] += half[((x & 1) * 4 + wave) * 256 + j * 64 + lane];
    };
    give(1);
    __syncthreads();
    give(2), take(1);
    __syncthreads();
    give(3), take(2);
    __syncthreads();
    take(3);
    __syncthreads();
    finish<1, 4>(target(p, blockIdx.y), own, (float*)(lds + wave * finish_bytes<1, 4>()), m0 + wave * 16, n0, 0, 0, lane);
}

// 32 codes from a 16-byte aligned address
__device__ __forceinline__ v8i load_codes(const uint8_t* p) {
    return __builtin_shufflevector(*(const v4i*)p, *(const v4i*)(p + 16), 0, 1, 2, 3, 4, 5, 6, 7);
}

// Few rows: 16 columns of C for up to 16 rows by NW waves that share the sum
// among them, each taking every NW-th block of 128 straight from memory
// (nothing is used twice), and add up in LDS in the order of the waves.  Bound
// by latency: a wave has the loads of one block in flight (the compiler does
// not unroll a loop of matrix instructions whose length it does not know), and
// 2048 columns make 128 workgroups: waves wait for 95% of their time.  16 x 2048
// x 8192 takes 12.2 to 13.2 us (13.1 with 16 waves where it took 12.8), 16 x 8192
// x 2048 6.9 to 7.6 us.
template <int FA, int FB, bool WIDE, int NW>
__global__ __launch_bounds__(64 * NW) void product_few_kernel(ProductArgs p) {
    __shared__ __attribute__((aligned(16))) float sums[NW][16 * 20];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, g = lane >> 4;
    const uint32_t n0 = blockIdx.x * 16;
    const uint32_t ra = min((uint32_t)row, p.m - 1), rb = min(n0 + row, p.n - 1);
    const uint8_t *qa = p.a + (uint64_t)ra * p.pitch + g * 32, *xa = p.sa + (uint64_t)ra * p.s_pitch;
    const uint8_t *qb = p.b + (uint64_t)rb * p.pitch + g * 32, *xb = p.sb + (uint64_t)rb * p.s_pitch;
    v4f acc[1][1] = {};
    for (uint32_t kb = wave; kb < p.kb; kb += NW) {
        const uint32_t ea[1] = {xa[kb]}, eb[1] = {xb[kb]};
        const v8i fa[1] = {load_codes(qa + kb * kBlkK)}, fb[1] = {load_codes(qb + kb * kBlkK)};
        multiply<FA, FB, WIDE>(acc, fa, fb, ea, eb);
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

// two floats of two codes
template <int FMT, bool HI>
__device__ __forceinline__ void floats2(uint32_t w, float& x, float& y) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    const v2f r = FMT == kE4M3 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w, HI) : __builtin_amdgcn_cvt_pk_f32_bf8((int)w, HI);
    x = r[0], y = r[1];
}

// One or two rows, as a token at a time makes them: a wave for each column of
// C, its lanes along the sum, 16 codes each, in fp32; the eight lanes of a
// block of 128 scale what they have of it.  No matrix instruction, whose other
// 15 rows would be empty: one row x 2048 x 8192 takes 5.8 us against 8.5 us of
// product_few_kernel beside it (6.0 to 6.4 us with inputs that no cache holds),
// 16384 x 8192 24.7 against 29.7 us (5.4 TB/s of codes);
// two rows 6.1 against 9.0 us; at four rows the gain is gone (8.2, 9.7 us, and
// 7.3 against 5.4 us with 8192 columns of 2048).
template <int FA, int FB, int M>
__global__ __launch_bounds__(256) void product_rows_kernel(ProductArgs p) {
    const int lane = threadIdx.x & 63;
    const uint32_t j = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (j >= p.n) return;
    const uint8_t *qb = p.b + (uint64_t)j * p.pitch, *xb = p.sb + (uint64_t)j * p.s_pitch;
    float sum[M] = {};
#pragma unroll M == 1 ? 8 : 4
    for (uint32_t k = lane * 16; k < p.pitch; k += 1024) {
        const v4i b = *(const v4i*)(qb + k);
        const int eb = xb[k >> 7];
        v4i a[M];
        int ea[M];
#pragma unroll
        for (int i = 0; i < M; i++) {
            a[i] = *(const v4i*)(p.a + (uint64_t)i * p.pitch + k);
            ea[i] = p.sa[(uint64_t)i * p.s_pitch + (k >> 7)];
        }
#pragma unroll
        for (int i = 0; i < M; i++) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 4; w++) {
                float x[4], y[4];
                floats2<FA, false>(a[i][w], x[0], x[1]), floats2<FA, true>(a[i][w], x[2], x[3]);
                floats2<FB, false>(b[w], y[0], y[1]), floats2<FB, true>(b[w], y[2], y[3]);
#pragma unroll
                for (int q = 0; q < 4; q++) s = fmaf(x[q], y[q], s);
            }
            sum[i] += ldexpf(s, ea[i] + eb - 254);
        }
    }
#pragma unroll
    for (int i = 0; i < M; i++)
#pragma unroll
        for (int d = 32; d; d >>= 1) sum[i] += __shfl_xor(sum[i], d);
    if (lane < M) {
        float v[8] = {M > 1 && lane ? sum[M - 1] : sum[0]};
        if (p.drop.on) drop8(p.drop, (uint64_t)lane * p.n + j, v);
        if (p.dtype == kF32) put_row<float>(p, lane, j, 0, 1, v, false);
        else if (p.dtype == kF16) put_row<f16_t>(p, lane, j, 0, 1, v, false);
        else put_row<bf16_t>(p, lane, j, 0, 1, v, false);
    }
}

// The splits' partial sums, added in their order, to the result.  They were
// written just before and come from the caches; what this costs is in the
// figures by which sums are split.
__global__ __launch_bounds__(256) void product_join_kernel(ProductArgs p, uint32_t splits) {
    const uint32_t groups = (p.n + 7) / 8;
    const uint64_t total = (uint64_t)p.m * groups, plane = (uint64_t)p.m * p.n;
    for (uint64_t t = (uint64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (uint64_t)gridDim.x * 256) {
        const uint32_t i = (uint32_t)(t / groups), j = (uint32_t)(t % groups) * 8;
        const float* s = p.partial + (uint64_t)i * p.n + j;
        const int count = (int)min(p.n - j, 8u);
        float v[8] = {};
        for (uint32_t z = 0; z < splits; z++) {
            if (p.n % 8 == 0) {
                float w[8];
                load8(s + z * plane, w);
#pragma unroll
                for (int q = 0; q < 8; q++) v[q] += w[q];
            } else {
#pragma unroll
                for (int q = 0; q < 8; q++)
                    if (q < count) v[q] += s[z * plane + q];
            }
        }
        finish8(p, i, j, 0, v);
    }
}

}  // namespace demo
