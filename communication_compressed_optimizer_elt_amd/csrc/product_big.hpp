// product_big.hpp -- the matrix product's kernels for large results (gfx950):
// 256 x 256 of C a workgroup, one workgroup a CU.  LDS holds two stages of 128
// along the sum, as in product_kernel; tiles that would pass the matrix' end
// are moved back inside, and write only what is theirs.
//
// Matrix instructions stand in assembly because the compiler, given a choice,
// moves the sums between both register files (it spilled 270 registers).  They
// are volatile and in order; what reads or writes their registers otherwise is
// at least eight of them away, and the way out begins behind a wait.
#pragma once

#include "product.hpp"

namespace demo {

constexpr int kBig = 256;
constexpr int kBigStage = 2 * kBig * kBlkK, kBigScales = 2 * kBig * 4;
constexpr size_t kBigLds = 2 * (kBigStage + kBigScales);

__device__ __forceinline__ void fence_order() { __builtin_amdgcn_sched_barrier(0); }

// d += a b, 128 along the sum, at byte Q of the scale words
template <int FMT_A, int FMT_B, int Q>
__device__ __forceinline__ void mma8(v4f& d, const v8i& a, const v8i& b, uint32_t ea, uint32_t eb) {
    asm volatile(
        "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%5,0] op_sel_hi:[%6,%6,0] cbsz:%7 blgp:%8"
        : "+a"(d)
        : "v"(a), "v"(b), "v"(ea), "v"(eb), "n"(Q & 1), "n"(Q >> 1), "n"(FMT_A), "n"(FMT_B));
}
// The tile and its loads.  Load x of an operand
// takes rows 8 (wave + 4 x) + lane / 8; all of them share one chunk offset
// because 4 x rows of 8 leave (row / 2) % 8 as it is.
struct BigTile {
    uint32_t m0, n0, lo_i, lo_j;
    const uint8_t *ga, *gb, *gsa, *gsb;
    uint32_t offset, p32, s_offset, lds, lds_scales;
    int lane, wave, wm, wn, row;
    uint32_t c0, c1;  // this lane's two chunks of a fragment
};

__device__ __forceinline__ BigTile big_tile(const ProductArgs& p, uint8_t* lds) {
    BigTile t;
    t.lane = threadIdx.x & 63;
    t.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t tm, tn;
    tile_of(p.tiles_m, p.tiles_n, blockIdx.x, tm, tn);
    t.lo_i = tm * kBig;
    t.lo_j = tn * kBig;
    t.m0 = min(t.lo_i, p.m - kBig);
    t.n0 = min(t.lo_j, p.n - kBig);
    t.ga = p.a + (uint64_t)(t.m0 + 8 * t.wave) * p.pitch;
    t.gb = p.b + (uint64_t)(t.n0 + 8 * t.wave) * p.pitch;
    t.gsa = p.sa + (uint64_t)(t.m0 + 64 * t.wave) * p.s_pitch;
    t.gsb = p.sb + (uint64_t)(t.n0 + 64 * t.wave) * p.s_pitch;
    t.offset = (t.lane >> 3) * p.pitch + (((t.lane & 7) ^ (t.lane >> 4) ^ (t.wave & 1) * 4) * 16);
    t.p32 = 32 * p.pitch;
    t.s_offset = (uint32_t)t.lane * p.s_pitch;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);
    t.lds = lds0 + t.wave * 1024;
    t.lds_scales = lds0 + 2 * kBigStage + t.wave * 256;
    t.wm = t.wave & 1;
    t.wn = t.wave >> 1;
    t.row = t.lane & 15;
    const int g = t.lane >> 4;
    t.c0 = ((2 * g) ^ (t.row >> 1)) * 16;
    t.c1 = ((2 * g + 1) ^ (t.row >> 1)) * 16;
    return t;
}

// the scale bytes of blocks kb..kb+3 (kb a multiple of 4): two loads
__device__ __forceinline__ void load_scales(const BigTile& t, uint32_t kb) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(t.lds_scales + (kb >> 2 & 1) * kBigScales);
    load_lds4(t.gsa + kb, t.s_offset, at);
    load_lds4(t.gsb + kb, t.s_offset, at + kBig * 4);
}

// The last matrix instructions' results are in their registers.  The compiler
// does not see that they are under way; accumulators that pass through an empty
// statement behind this one are read after it.
__device__ __forceinline__ void settle() {
    fence_order();
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    fence_order();
}

// On the scaled 8-bit instructions, by 4 waves of 128 x 128.  A wave's 8 x 8
// accumulators of 16 x 16 fill the 256 accumulation registers, so its
// fragments are read from LDS as rarely as they can be: 128 KB a block, of the
// 192 KB that 8 waves of 128 x 64 read, where LDS reads alone took 216 us of a
// product of 8192 x 8192 x 8192.  With one wave a SIMD nothing else hides a
// wait, so the order of instructions is laid down: between two matrix
// instructions stands at most one load of a fragment and one load to LDS, each
// long before its use (loads to LDS in runs of 12 blocked the wave: 403 us
// without the way out, 373 us one by one).
//
// A block of 128 is 64 matrix instructions in two halves, rows 0-3 and rows 4-7
// of the wave's 16-row fragments of A, each column by column: in the second
// half column j of B and rows 0-3 of A of the next block take the place of what
// the first half is done with; in the first half rows 4-7 of A follow.  Two
// barriers a block:
//   P, in the first half: rows 4-7 of this block have landed (before they are
//      read); B and rows 0-3 of this stage are free: 12 loads of block + 2;
//   Q, between the halves: B and rows 0-3 of the next block have landed; rows
//      4-7 of this stage are free: 4 loads of block + 2.
// At either wait 16 younger loads (18 where scale bytes came with them) are in
// flight, one and a half blocks ahead of their use.
//
// Bound by the matrix instructions at the clock that their power leaves (3.8
// PFLOP/s on random codes in registers, 4.7 on constant ones; 1.9 of 2.4 GHz
// here) for long sums, where their units are busy for 74% of the time, and for
// sums of 2048, where it is 50%, as much by a tile's first loads and by the
// results that all CUs write at the same time between two tiles.  Over cards and
// runs 8192 x 8192 x 8192 takes 375 to 425 us (2.59 to 2.93 PFLOP/s), 4096 x 8192
// x 2048 60 to 65 us, 2048 x 100352 x 2048 368 to 422 us; columns that are no
// multiple of 8 are stored one by one (2048 x 50257 x 2048 331 us, 50256 220 us).
// Loading the next tile's first blocks before the way out gave nothing (77.4
// against 78.4 us), nor did two groups of 4 waves out of step (494 against 464
// us).
template <int FA, int FB>
__global__ __launch_bounds__(256, 1) void product_big_kernel(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const BigTile t = big_tile(p, lds);
    const uint32_t kb1 = p.kb;
    auto load_first = [&](uint32_t kb, auto ST, auto E) {  // one of 12
        constexpr int e = decltype(E)::value, x = e < 8 ? e : e < 10 ? e - 8 : e - 6;
        load_lds16((e < 8 ? t.gb : t.ga) + kb * kBlkK, t.offset + x * t.p32,
                   t.lds + decltype(ST)::value * kBigStage + (e < 8 ? kBig * kBlkK : 0) + x * 4096);
    };
    auto load_second = [&](uint32_t kb, auto ST, auto E) {  // one of 4
        constexpr int e = decltype(E)::value, x = e < 2 ? e + 2 : e + 4;
        load_lds16(t.ga + kb * kBlkK, t.offset + x * t.p32, t.lds + decltype(ST)::value * kBigStage + x * 4096);
    };
    auto load_block = [&](uint32_t kb, auto ST, auto S) {
        load_first(kb, ST, Int<0>()); load_first(kb, ST, Int<1>()); load_first(kb, ST, Int<2>());
        load_first(kb, ST, Int<3>()); load_first(kb, ST, Int<4>()); load_first(kb, ST, Int<5>());
        load_first(kb, ST, Int<6>()); load_first(kb, ST, Int<7>()); load_first(kb, ST, Int<8>());
        load_first(kb, ST, Int<9>()); load_first(kb, ST, Int<10>()); load_first(kb, ST, Int<11>());
        if constexpr (decltype(S)::value) load_scales(t, kb);
        load_second(kb, ST, Int<0>()); load_second(kb, ST, Int<1>());
        load_second(kb, ST, Int<2>()); load_second(kb, ST, Int<3>());
    };
    const uint8_t* la = lds + (t.wm * 128 + t.row) * kBlkK;
    const uint8_t* lb = lds + (kBig + t.wn * 128 + t.row) * kBlkK;
    const uint32_t* sa = (const uint32_t*)(lds + 2 * kBigStage) + t.wm * 128 + t.row;
    const uint32_t* sb = (const uint32_t*)(lds + 2 * kBigStage) + kBig + t.wn * 128 + t.row;
    auto fragment = [&](const uint8_t* base, int st, int i) {
        const uint8_t* q = base + st * kBigStage + i * 16 * kBlkK;
        return __builtin_shufflevector(*(const v4i*)(q + t.c0), *(const v4i*)(q + t.c1), 0, 1, 2, 3, 4, 5, 6, 7);
    };
    v4f acc[8][8] = {};
    v8i fa[8], fb[8];
    uint32_t ea[8], eb[8];
    load_block(0, Int<0>(), Int<1>());
    if (1 < kb1) {
        load_block(1, Int<1>(), Int<0>());
        sync_loads<16>();
    } else {
        sync_loads<0>();
    }
    #pragma unroll
    for (int j = 0; j < 8; j++) fb[j] = fragment(lb, 0, j), eb[j] = sb[j * 16];
#pragma unroll
    for (int i = 0; i < 4; i++) fa[i] = fragment(la, 0, i), ea[i] = sa[i * 16];

    uint32_t kb = 0;
    // block kb, kb % 4 == Q; STEADY: at least two more follow
    auto block = [&](auto Q, auto STEADY) {
        constexpr int q = decltype(Q)::value, cur = q & 1, nxt = cur ^ 1;
        constexpr int kAfter1 = 16 + (((q + 1) & 3) == 0 ? 2 : 0), kAfter2 = 16 + (((q + 2) & 3) == 0 ? 2 : 0);
        const bool one = decltype(STEADY)::value || kb + 1 < kb1, two = decltype(STEADY)::value || kb + 2 < kb1;
        const uint32_t now = (kb >> 2 & 1) * (kBigScales / 4), then = ((kb + 1) >> 2 & 1) * (kBigScales / 4);
        auto column0 = [&](auto J) {
            constexpr int j = decltype(J)::value;
            fence_order();
#pragma unroll
            for (int i = 0; i < 4; i++) {
                mma8<FB, FA, q>(acc[i][j], fb[j], fa[i], eb[j], ea[i]);
                if constexpr (j >= 2) {
                    if (i == 0 && two) load_first(kb + 2, Int<cur>(), Int<2 * (j - 2)>());
                    if (i == 2 && two) load_first(kb + 2, Int<cur>(), Int<2 * (j - 2) + 1>());
                    if (i == 3 && j == 7 && ((q + 2) & 3) == 0 && two) load_scales(t, kb + 2);
                    if constexpr (j < 6) {
                        if (i == 1) {
                            fa[2 + j] = fragment(la, cur, 2 + j);
                            if (q == 0) ea[2 + j] = sa[now + (2 + j) * 16];
                        }
                    }
                }
                fence_order();
            }
            if constexpr (j == 1) {  // P
                if (one) sync_loads<kAfter1>();
                else sync_loads<0>();
            }
        };
        column0(Int<0>()); column0(Int<1>()); column0(Int<2>()); column0(Int<3>());
        column0(Int<4>()); column0(Int<5>()); column0(Int<6>()); column0(Int<7>());
        if (two) sync_loads<kAfter2>();  // Q
        else sync_loads<0>();
        auto column1 = [&](auto J) {
            constexpr int j = decltype(J)::value;
            fence_order();
#pragma unroll
            for (int i = 4; i < 8; i++) {
                mma8<FB, FA, q>(acc[i][j], fb[j], fa[i], eb[j], ea[i]);
                if (i == 5 && !(j & 1) && two) load_second(kb + 2, Int<cur>(), Int<(j >> 1)>());
                if (i == 5 && (j & 1)) {
                    fa[j >> 1] = fragment(la, nxt, j >> 1);
                    if (q == 3) ea[j >> 1] = sa[then + (j >> 1) * 16];
                }
                fence_order();
            }
            fb[j] = fragment(lb, nxt, j);
            if (q == 3) eb[j] = sb[then + j * 16];
        };
        column1(Int<0>()); column1(Int<1>()); column1(Int<2>()); column1(Int<3>());
        column1(Int<4>()); column1(Int<5>()); column1(Int<6>()); column1(Int<7>());
        kb++;
    };
    while (kb + 5 < kb1) {
        block(Int<0>(), Int<1>());
        block(Int<1>(), Int<1>());
        block(Int<2>(), Int<1>());
        block(Int<3>(), Int<1>());
    }
    for (;;) {
        block(Int<0>(), Int<0>());
        if (kb == kb1) break;
        block(Int<1>(), Int<0>());
        if (kb == kb1) break;
        block(Int<2>(), Int<0>());
        if (kb == kb1) break;
        block(Int<3>(), Int<0>());
        if (kb == kb1) break;
    }
    settle();
#pragma unroll
    for (int i = 0; i < 8; i++)
        asm volatile("" : "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]), "+a"(acc[i][4]),
                     "+a"(acc[i][5]), "+a"(acc[i][6]), "+a"(acc[i][7]));
    sync_loads<0>();
    finish<8, 8>(p, acc, (float*)(lds + t.wave * finish_bytes<8, 8>()), t.m0 + t.wm * 128, t.n0 + t.wn * 128, t.lo_i,
                 t.lo_j, t.lane);
}

// On the bf16 instructions, 32 x 32 x 16 (2.06 PFLOP/s on random values in
// registers, 16 x 16 x 32 1.83), by 8 waves of 128 x 64, two on a SIMD, because
// a wave by itself issues one instruction in about 8 cycles, and widening takes
// more of them than fit between the matrix instructions (by 4 waves of 128 x
// 128 as above, 1.26 PFLOP/s with the accumulators in use then).  A block of 128
// is four steps of 32 along the sum: widen the step's codes, read the next
// step's, multiply.  The two waves of a SIMD are kept out of step, one widens
// while the other multiplies: they meet at the one barrier a block, the first
// four waves before they widen the last step's codes and the others after.
// Behind it the next block has landed, nobody reads this block's stage again,
// and the loads of the block after the next go there.  8192 x 8192 x 8192 takes
// 844 to 890 us (1.24 to 1.30 PFLOP/s), in tiles of 128 969 us on the card of the
// 890; the matrix units are busy for 68% of it.
typedef float v16f __attribute__((ext_vector_type(16)));
__device__ __forceinline__ void mma16(v16f& d, const v8b& a, const v8b& b) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(d) : "v"(a), "v"(b));
}

template <int FA, int FB>
__global__ __launch_bounds__(512, 2) void product_big_wide_kernel(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t tm, tn;
    tile_of(p.tiles_m, p.tiles_n, blockIdx.x, tm, tn);
    const uint32_t lo_i = tm * kBig, lo_j = tn * kBig, m0 = min(lo_i, p.m - kBig), n0 = min(lo_j, p.n - kBig);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);
    const uint8_t* ga = p.a + (uint64_t)(m0 + 8 * wave) * p.pitch;
    const uint8_t* gb = p.b + (uint64_t)(n0 + 8 * wave) * p.pitch;
    const uint8_t* gs = wave < 4 ? p.sa + (uint64_t)(m0 + 64 * wave) * p.s_pitch
                                 : p.sb + (uint64_t)(n0 + 64 * (wave - 4)) * p.s_pitch;
    const uint32_t offset = (lane >> 3) * p.pitch + (((lane & 7) ^ (lane >> 4) ^ (wave & 1) * 4) * 16);
    const uint32_t p64 = 64 * p.pitch, s_offset = (uint32_t)lane * p.s_pitch;
    // load x of 8 of block kb, the first 4 of A
    auto load_one = [&](uint32_t kb, auto X) {
        constexpr int x = decltype(X)::value & 3, b = decltype(X)::value >> 2;
        load_lds16((b ? gb : ga) + kb * kBlkK, offset + x * p64,
                   lds0 + wave * 1024 + (kb & 1) * kBigStage + b * kBig * kBlkK + x * 8192);
    };
    auto load_bytes = [&](uint32_t kb) {
        load_lds4(gs + kb, s_offset,
                  __builtin_amdgcn_readfirstlane(lds0 + 2 * kBigStage + wave * 256 + (kb >> 2 & 1) * kBigScales));
    };
    auto load_block = [&](uint32_t kb) {
        load_one(kb, Int<0>()); load_one(kb, Int<1>()); load_one(kb, Int<2>()); load_one(kb, Int<3>());
        load_one(kb, Int<4>()); load_one(kb, Int<5>()); load_one(kb, Int<6>()); load_one(kb, Int<7>());
    };
    const int wm = wave & 1, wn = wave >> 1, row = lane & 31, h = lane >> 5;
    const uint8_t* la = lds + (wm * 128 + row) * kBlkK;
    const uint8_t* lb = lds + (kBig + wn * 64 + row) * kBlkK;
    const uint32_t* sa = (const uint32_t*)(lds + 2 * kBigStage) + wm * 128 + row;
    const uint32_t* sb = (const uint32_t*)(lds + 2 * kBigStage) + kBig + wn * 64 + row;
    v16f acc[4][2] = {};
    v4i ra[4], rb[2];
    uint32_t ea[4], eb[2];
    float ka[4], kc[2];
    // this lane's 16 codes of each fragment for step q of a block: chunk 2 q + h
    auto read_codes = [&](uint32_t stage, int q) {
        const uint32_t at = stage + ((2 * q + h) ^ (row >> 1 & 7)) * 16;
#pragma unroll
        for (int j = 0; j < 2; j++) rb[j] = *(const v4i*)(lb + at + j * 32 * kBlkK);
#pragma unroll
        for (int i = 0; i < 4; i++) ra[i] = *(const v4i*)(la + at + i * 32 * kBlkK);
    };
    load_bytes(0);
    load_block(0);
    if (p.kb > 1) {
        load_block(1);
        sync_loads<8>();
    } else {
        sync_loads<0>();
    }
    read_codes(0, 0);
    for (uint32_t kb = 0; kb < p.kb; kb++) {
        const uint32_t here = (kb & 1) * kBigStage;
        const bool two = kb + 2 < p.kb;
        if ((kb & 3) == 0) {
            const uint32_t s = (kb >> 2 & 1) * (kBigScales / 4);
#pragma unroll
            for (int i = 0; i < 4; i++) ea[i] = sa[s + i * 32];
#pragma unroll
            for (int j = 0; j < 2; j++) eb[j] = sb[s + j * 32];
        }
        const uint32_t shift = (kb & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; i++) ka[i] = scale_float(ea[i] >> shift & 255u);
#pragma unroll
        for (int j = 0; j < 2; j++) kc[j] = scale_float(eb[j] >> shift & 255u);
        auto step = [&](auto Q) {
            constexpr int q = decltype(Q)::value;
            v8b wa[4][2], wb[2][2];
            if (q == 3 && wave < 4) sync_loads<0>();
            fence_order();
#pragma unroll
            for (int j = 0; j < 2; j++) {
                wb[j][0] = widen<FB>(rb[j][0], rb[j][1], kc[j]);
                wb[j][1] = widen<FB>(rb[j][2], rb[j][3], kc[j]);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                wa[i][0] = widen<FA>(ra[i][0], ra[i][1], ka[i]);
                wa[i][1] = widen<FA>(ra[i][2], ra[i][3], ka[i]);
            }
            fence_order();
            if (q == 3 && wave >= 4) sync_loads<0>();
            read_codes(q < 3 ? here : here ^ kBigStage, (q + 1) & 3);
            fence_order();
            auto line = [&](auto I_) {
                constexpr int i = decltype(I_)::value;
#pragma unroll
                for (int j = 0; j < 2; j++) mma16(acc[i & 3][j], wb[j][i >> 2], wa[i & 3][i >> 2]);
                if constexpr (q == 3) {
                    if (two) load_one(kb + 2, I_);
                }
                fence_order();
            };
            line(Int<0>()); line(Int<1>()); line(Int<2>()); line(Int<3>());
            line(Int<4>()); line(Int<5>()); line(Int<6>()); line(Int<7>());
            if (q == 3 && two && (kb + 2 & 3) == 0) load_bytes(kb + 2);
        };
        step(Int<0>());
        step(Int<1>());
        step(Int<2>());
        step(Int<3>());
    }
    settle();
#pragma unroll
    for (int i = 0; i < 4; i++) asm volatile("" : "+a"(acc[i][0]), "+a"(acc[i][1]));
    sync_loads<0>();
    float* slab = (float*)(lds + wave * finish_bytes<2, 4>());
    finish_pieces<4, 2, 4>(p, slab, m0 + wm * 128, n0 + wn * 64, lo_i, lo_j, lane, [&](auto T) {
        constexpr int t = decltype(T)::value;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            v4f* to = (v4f*)(slab + row * 68 + j * 32 + 4 * h);
            to[0] = __builtin_shufflevector(acc[t][j], acc[t][j], 0, 1, 2, 3);
            to[2] = __builtin_shufflevector(acc[t][j], acc[t][j], 4, 5, 6, 7);
            to[4] = __builtin_shufflevector(acc[t][j], acc[t][j], 8, 9, 10, 11);
            to[6] = __builtin_shufflevector(acc[t][j], acc[t][j], 12, 13, 14, 15);
        }
    });
}

}  // namespace demo
