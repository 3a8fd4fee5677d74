// product_big.hpp -- the matrix product's kernel for large 16-bit results (gfx950):
// 256 x 256 of C by 4 waves of 128 x 128, one workgroup per CU.
//
// A wave's 8 x 8 accumulators of 16 x 16 fill the 256 accumulation registers,
// so its operands' fragments are read from LDS as rarely as they can be: 128
// KB a block of 128 along the sum, of the 192 KB that 8 waves of 128 x 64 read,
// where LDS reads alone took 216 us of a product of 8192 x 8192 x 8192.  With
// one wave per SIMD nothing else hides a wait, so the order of instructions is
// laid down: between two matrix instructions stands at most one load of a
// fragment and one load to LDS, each long before its use (loads to LDS in runs
// of 12 blocked the wave: 403 us without the way out, 373 us one by one).
// Matrix instructions stand in assembly because the compiler, given a choice,
// moves the sums between both register files (it spilled 270 registers).  They
// are volatile and in order; what reads or writes their registers otherwise is
// at least eight of them away, and the way out begins behind a wait.
//
// LDS holds two stages of 128 along the sum, as in product_kernel; loads are
// issued for the block after the next as soon as all waves have read a part of
// the stage.  Tiles that would pass the matrix' end are moved back inside, and
// write only what is theirs.
#pragma once

#include <type_traits>

#include "product.hpp"

namespace demo {

constexpr int kBig = 256;
constexpr int kBigStage = 2 * kBig * kBlkK, kBigScales = 2 * kBig * 4;
constexpr size_t kBigLds = 2 * (kBigStage + kBigScales);

template <int N>
using Int = std::integral_constant<int, N>;

__device__ __forceinline__ void fence_order() { __builtin_amdgcn_sched_barrier(0); }

// load_lds16 to lds + IMM
template <int IMM>
__device__ __forceinline__ void load_at(const uint8_t* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base),
                 "n"(IMM)
                 : "memory", "m0", "scc");
}

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
    uint32_t m0, n0, lo_i, lo_j, kb0, kb1;
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
    tile_of(p, blockIdx.x, tm, tn);
    t.lo_i = tm * kBig;
    t.lo_j = tn * kBig;
    t.m0 = min(t.lo_i, p.m - kBig);
    t.n0 = min(t.lo_j, p.n - kBig);
    t.kb0 = blockIdx.y * p.kb_split;
    t.kb1 = min(t.kb0 + p.kb_split, p.kb);
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

__device__ __forceinline__ void big_way_out(const ProductArgs& p, const BigTile& t, const v4f (&acc)[8][8], uint8_t* lds) {
    fence_order();
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __syncthreads();
    finish<8, 8>(target(p, blockIdx.y), acc, (float*)(lds + t.wave * finish_bytes<8, 8>()), t.m0 + t.wm * 128,
                 t.n0 + t.wn * 128, t.lo_i, t.lo_j, t.lane);
}

// On the scaled 8-bit instructions.  A block of 128 is 64 of them in two
// halves, rows 0-3 and rows 4-7 of the wave's 16-row fragments of A, each
// column by column: in the second half column j of B and rows 0-3 of A of the
// next block take the place of what the first half is done with; in the
// first half rows 4-7 of A follow.  Two barriers a block:
//   P, in the first half: rows 4-7 of this block have landed (before they are
//      read); B and rows 0-3 of this stage are free: 12 loads of block + 2;
//   Q, between the halves: B and rows 0-3 of the next block have landed; rows
//      4-7 of this stage are free: 4 loads of block + 2.
// At either wait 16 younger loads (18 where scale bytes came with them) are in
// flight, one and a half blocks ahead of their use.
template <int FA, int FB>
__global__ __launch_bounds__(256, 1) void product_big_kernel(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const BigTile t = big_tile(p, lds);
    const uint32_t kb1 = t.kb1;
    auto load_first = [&](uint32_t kb, auto ST, auto E) {  // one of 12
        constexpr int e = decltype(E)::value, x = e < 8 ? e : e < 10 ? e - 8 : e - 6;
        load_at<decltype(ST)::value * kBigStage + (e < 8 ? kBig * kBlkK : 0) + x * 4096>(
            (e < 8 ? t.gb : t.ga) + kb * kBlkK, t.offset + x * t.p32, t.lds);
    };
    auto load_second = [&](uint32_t kb, auto ST, auto E) {  // one of 4
        constexpr int e = decltype(E)::value, x = e < 2 ? e + 2 : e + 4;
        load_at<decltype(ST)::value * kBigStage + x * 4096>(t.ga + kb * kBlkK, t.offset + x * t.p32, t.lds);
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
    load_block(t.kb0, Int<0>(), Int<1>());
    if (t.kb0 + 1 < kb1) {
        load_block(t.kb0 + 1, Int<1>(), Int<0>());
        sync_loads<16>();
    } else {
        sync_loads<0>();
    }
    const uint32_t s0 = (t.kb0 >> 2 & 1) * (kBigScales / 4);
#pragma unroll
    for (int j = 0; j < 8; j++) fb[j] = fragment(lb, 0, j), eb[j] = sb[s0 + j * 16];
#pragma unroll
    for (int i = 0; i < 4; i++) fa[i] = fragment(la, 0, i), ea[i] = sa[s0 + i * 16];

    uint32_t kb = t.kb0;
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
                    if (i == 1 && j < 6) {
                        fa[2 + j] = fragment(la, cur, 2 + j);
                        if (q == 0) ea[2 + j] = sa[now + (2 + j) * 16];
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
    big_way_out(p, t, acc, lds);
}

}  // namespace demo
