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

// A wave's way out in pieces of 32 rows, for fp32 results in aligned accesses:
// neighbouring lanes take 16 bytes each, so that whole lines leave, where finish()
// of product.hpp stores 16 of every 32 (8192 x 8192 x 2048: 114 us, 129 so).  They go
// past the caches at every size, a split's partial sums too.
template <int SM, int SN>
struct MxLines {
    static constexpr int kRow = SN * 16 + 4, kLanes = SN * 4, kRows = 64 / kLanes, P = 32 / kRows;
    static_assert(SM % 2 == 0 && P >= 1, "pieces of 32 rows");
    v4f addend[P];

    static __device__ __forceinline__ bool fits(const ProductArgs& p) { return p.dtype == kF32 && p.wide && !p.drop.on; }
    // the addend of piece s, all loads in flight at once
    __device__ __forceinline__ void load(const ProductArgs& p, int s, uint32_t i0, uint32_t j0, uint32_t lo_i, uint32_t lo_j, int lane) {
        const uint32_t j = j0 + lane % kLanes * 4, top = i0 + s * 32 + lane / kLanes;
#pragma unroll
        for (int r = 0; r < P; r++) {
            const uint32_t i = top + r * kRows;
            addend[r] = v4f{};
            if (p.addend && j >= lo_j && j < p.n && i >= lo_i && i < p.m)
                addend[r] = *(const v4f*)((const float*)p.addend + i * p.ld_addend + j);
        }
    }
    __device__ __forceinline__ void store(const ProductArgs& p, const float* slab, int s, uint32_t i0, uint32_t j0, uint32_t lo_i,
                                          uint32_t lo_j, int lane) {
        const uint32_t j = j0 + lane % kLanes * 4, top = i0 + s * 32 + lane / kLanes;
#pragma unroll
        for (int r = 0; r < P; r++) {
            const uint32_t i = top + r * kRows;
            const v4f v = *(const v4f*)(slab + (r * kRows + lane / kLanes) * kRow + lane % kLanes * 4) + addend[r];
            if (j >= lo_j && j < p.n && i >= lo_i && i < p.m) __builtin_nontemporal_store(v, (v4f*)((float*)p.c + i * p.ldc + j));
        }
    }
};

// finish() of product.hpp, or by lines, each piece's addend loaded while the one
// before is stored (3000 x 3000 x 3000 with an addend 33.0 us, 35.7 without).  EARLY:
// `lines` holds the first piece's.
template <int SM, int SN, bool EARLY = false>
__device__ __forceinline__ void mx_finish(const ProductArgs& p, const v4f (&acc)[SM][SN], float* slab, uint32_t i0,
                                          uint32_t j0, uint32_t lo_i, uint32_t lo_j, int lane, MxLines<SM, SN>& lines) {
    typedef MxLines<SM, SN> Lines;
    if (!Lines::fits(p)) {
        finish<SM, SN>(p, acc, slab, i0, j0, lo_i, lo_j, lane);
        return;
    }
    if (!EARLY) lines.load(p, 0, i0, j0, lo_i, lo_j, lane);
#pragma unroll 1
    for (int s = 0; s < SM / 2; s++) {
        pick<SM / 2>(s, [&](auto T) {
            constexpr int t = decltype(T)::value;
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int c = 0; c < SN; c++)
                    *(v4f*)(slab + (i * 16 + (lane & 15)) * Lines::kRow + c * 16 + 4 * (lane >> 4)) = acc[t * 2 + i][c];
        });
        wave_lds_sync();
        Lines next;
        if (s + 1 < SM / 2) next.load(p, s + 1, i0, j0, lo_i, lo_j, lane);
        lines.store(p, slab, s, i0, j0, lo_i, lo_j, lane);
        lines = next;
        wave_lds_sync();
    }
}

// Places of two steps' scale bytes: of four stages three, as the steps from the one
// that is read to the last one that is loaded may begin three pairs.
template <int S>
constexpr int kMxPairs = S == 4 ? 3 : 2;

// BM x BN of C by WM x WN waves, one of the splits of the sum (grid y), loads as in
// product_kernel, S stages.  Scale bytes come 16 of a row at a time, for two steps.
// Bound by the latency of a step's loads and of the way out where tiles are few (2304
// x 768 x 2561 fp32 with an addend, 432 tiles of 64: 10.5 us, waves wait 64% of
// their time, matrix units busy 11%).  2048 x 2048 x 2048 bf16, 1024 tiles of 64, takes
// 11 us; 2048 x 2048 x 8192, 256 tiles of 128, 30.5 us.
template <int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN) void mx_kernel(ProductArgs p) {
    constexpr int NW = WM * WN, SM = BM / WM / 16, SN = BN / WN / 16;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;
    constexpr int kStage = (BM + BN) * kStepK, kScales = (BM + BN) * 2 * kStepScales;
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0 && (BM + BN) / 64 <= NW, "loads per wave");
    static_assert(S == 2 || S == 4, "a step's scale bytes behind it are none or one load");
    static_assert(NW * finish_bytes<SM, SN>() <= S * kStage, "the way out fits the stages");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint8_t* scales = lds + S * kStage;
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
    const bool has_scales = wave < (BM + BN) / 64, scale_of_a = wave * 64 < BM;
    const uint32_t srow = scale_of_a ? min((uint32_t)(wave * 64 + lane), p.m - 1 - m0)
                                     : min((uint32_t)(wave * 64 - BM + lane), p.n - 1 - n0);
    const uint8_t* gs = scale_of_a ? p.sa + (uint64_t)m0 * p.s_pitch : p.sb + (uint64_t)n0 * p.s_pitch;
    const uint32_t os = srow * p.s_pitch;

    int to = 0, to_pair = 0;  // what is filled next: the stage, and the place of two steps' scale bytes
    auto fetch = [&](uint32_t kb) {
        const uint32_t at = lds0 + to * kStage;
#pragma unroll
        for (int i = 0; i < LA; i++) load_lds16(ga + (uint64_t)kb * kStepK, oa[i], at + (wave + i * NW) * 1024);
#pragma unroll
        for (int i = 0; i < LB; i++) load_lds16(gb + (uint64_t)kb * kStepK, ob[i], at + BM * kStepK + (wave + i * NW) * 1024);
        if ((kb & 1) == 0) {
            if (has_scales) load_lds16(gs + kb * kStepScales, os, lds0 + S * kStage + to_pair * kScales + wave * 1024);
            to_pair = to_pair + 1 == kMxPairs<S> ? 0 : to_pair + 1;
        }
        to = to + 1 == S ? 0 : to + 1;
    };

    const int wm = wave % WM, wn = wave / WM, row = lane & 15, g = lane >> 4;
    const int c0 = ((2 * g) ^ (row >> 1)) * 16, c1 = ((2 * g + 1) ^ (row >> 1)) * 16;
    v4f acc[SM][SN] = {};
    uint32_t ea[SM], eb[SN];
    // a small tile's addend is loaded before anything else, and there at the end (2304 x
    // 768 x 2561: 11.9 us, 10.7 so; of a tile of 128 it stands in the way: 4096 x 2048 x 2048 24.2, 26.3 so)
    constexpr bool kEarly = SM == 2;
    const uint32_t i0 = m0 + wm * SM * 16, j0 = n0 + wn * SN * 16;
    MxLines<SM, SN> lines;
    if constexpr (kEarly) {
        const ProductArgs out = target(p, blockIdx.y);
        if (MxLines<SM, SN>::fits(out)) lines.load(out, 0, i0, j0, 0, 0, lane);
    }
    constexpr int kAfter = (S - 2) * (LA + LB);  // loads of a wave behind a step's own, its scale bytes aside
    int from = 0, from_pair = 0;
#pragma unroll
    for (int s = 0; s < S - 1; s++)
        if (kb0 + s < kb1) fetch(kb0 + s);
    for (uint32_t kb = kb0; kb < kb1; kb++) {
        // step kb has landed, and everyone has read the stage that is filled next
        if (S == 2 || kb + S - 2 >= kb1) sync_loads<0>();
        else if (has_scales) sync_loads<kAfter + 1>();  // one of the two steps has some
        else sync_loads<kAfter>();
        if (kb + S - 1 < kb1) fetch(kb + S - 1);
        const uint8_t* stage = lds + from * kStage;
        const uint8_t* sc = scales + from_pair * kScales + (kb & 1) * kStepScales + 2 * g;
        from = from + 1 == S ? 0 : from + 1;
        if (kb & 1) from_pair = from_pair + 1 == kMxPairs<S> ? 0 : from_pair + 1;
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
    mx_finish<SM, SN, kEarly>(target(p, blockIdx.y), acc, (float*)(lds + wave * finish_bytes<SM, SN>()), i0, j0, 0, 0, lane, lines);
}

// d += a b, 128 along the sum, with byte Q of the scale words.  WAIT: in steps with
// branches, whose scale bytes the compiler masks in front of it; with a wait everywhere
// 2048 x 8192 x 8192 with an addend takes 84.7 us, 81.9 so, and in mx_stream_kernel 8192
// x 8192 x 8192 249 and 236.
template <int Q, bool WAIT>
__device__ __forceinline__ void mma4(v4f& d, const v4i& a, const v4i& b, uint32_t ea, uint32_t eb) {
    if constexpr (WAIT)
        asm volatile(DEMO_MFMA_WAIT
                     "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%5,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     : "+a"(d)
                     : "v"(a), "v"(b), "v"(ea), "v"(eb), "n"(Q));
    else
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%5,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     : "+a"(d)
                     : "v"(a), "v"(b), "v"(ea), "v"(eb), "n"(Q));
}

constexpr int kMxBigScales = 2 * kBig * 2 * kStepScales;  // of two steps
constexpr size_t kMxBigLds = 2 * (kBigStage + kMxBigScales);
constexpr size_t kMxStreamLds = kMxBigLds + 4 * 4096;  // all that a CU has

// Large results: 256 x 256 of C by 4 waves of 128 x 128, one workgroup a CU, with
// the loads, halves and barriers of product_big_kernel.  A step is 128 matrix
// instructions of half the length, two for each pair of fragments; the four of a
// column's first half of the step stand before the four of the second, which add
// to the same sums.
// It takes what mx_stream_kernel does not: addends, dropouts, odd widths, an odd number
// of steps, fewer than four.  2048 x 8192 x 8192 fp32 with an addend 79 to 90 us, 66 of them without
// the addend's 67 MB, which are read when nothing multiplies; read ahead through LDS
// that nobody uses they delay the steps' own loads (90.5 against 83.0 us).
template <typename = void>
__global__ __launch_bounds__(256, 1) void mx_big_kernel(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    BigTile t = big_tile(p, lds);
    t.lds_scales += t.wave * (1024 - 256);
    const uint32_t kb1 = p.kb;
    auto load_first = [&](uint32_t kb, auto ST, auto E) {  // one of 12
        constexpr int e = decltype(E)::value, x = e < 8 ? e : e < 10 ? e - 8 : e - 6;
        load_lds16((e < 8 ? t.gb : t.ga) + kb * kStepK, t.offset + x * t.p32,
                   t.lds + decltype(ST)::value * kBigStage + (e < 8 ? kBig * kStepK : 0) + x * 4096);
    };
    auto load_second = [&](uint32_t kb, auto ST, auto E) {  // one of 4
        constexpr int e = decltype(E)::value, x = e < 2 ? e + 2 : e + 4;
        load_lds16(t.ga + kb * kStepK, t.offset + x * t.p32, t.lds + decltype(ST)::value * kBigStage + x * 4096);
    };
    auto load_scale_bytes = [&](uint32_t kb) {  // of steps kb and kb + 1, kb even: two loads
        const uint32_t at = __builtin_amdgcn_readfirstlane(t.lds_scales + (kb >> 1 & 1) * kMxBigScales);
        load_lds16(t.gsa, t.s_offset + kb * kStepScales, at);
        load_lds16(t.gsb, t.s_offset + kb * kStepScales, at + kBig * 2 * kStepScales);
    };
    auto load_step = [&](uint32_t kb, auto ST, auto S) {
        load_first(kb, ST, Int<0>()); load_first(kb, ST, Int<1>()); load_first(kb, ST, Int<2>());
        load_first(kb, ST, Int<3>()); load_first(kb, ST, Int<4>()); load_first(kb, ST, Int<5>());
        load_first(kb, ST, Int<6>()); load_first(kb, ST, Int<7>()); load_first(kb, ST, Int<8>());
        load_first(kb, ST, Int<9>()); load_first(kb, ST, Int<10>()); load_first(kb, ST, Int<11>());
        if constexpr (decltype(S)::value) load_scale_bytes(kb);
        load_second(kb, ST, Int<0>()); load_second(kb, ST, Int<1>());
        load_second(kb, ST, Int<2>()); load_second(kb, ST, Int<3>());
    };
    const int g = t.lane >> 4;
    const uint8_t* la = lds + (t.wm * 128 + t.row) * kStepK;
    const uint8_t* lb = lds + (kBig + t.wn * 128 + t.row) * kStepK;
    const uint8_t* sa = lds + 2 * kBigStage + (t.wm * 128 + t.row) * 2 * kStepScales + 2 * g;
    const uint8_t* sb = sa + (kBig + (t.wn - t.wm) * 128) * 2 * kStepScales;
    struct Fragment {
        v4i half[2];
    };
    auto fragment = [&](const uint8_t* base, int st, int i) {
        const uint8_t* q = base + st * kBigStage + i * 16 * kStepK;
        return Fragment{{*(const v4i*)(q + t.c0), *(const v4i*)(q + t.c1)}};
    };
    // this lane's two scale bytes of fragment i; at: where the step's begin
    auto scale_bytes = [&](const uint8_t* base, uint32_t at, int i) {
        return (uint32_t) * (const uint16_t*)(base + at + i * 16 * 2 * kStepScales);
    };
    v4f acc[8][8] = {};
    Fragment fa[8], fb[8];
    uint32_t ea[8], eb[8];
    load_step(0, Int<0>(), Int<1>());
    if (1 < kb1) {
        load_step(1, Int<1>(), Int<0>());
        sync_loads<16>();
    } else {
        sync_loads<0>();
    }
#pragma unroll
    for (int j = 0; j < 8; j++) fb[j] = fragment(lb, 0, j), eb[j] = scale_bytes(sb, 0, j);
#pragma unroll
    for (int i = 0; i < 4; i++) fa[i] = fragment(la, 0, i), ea[i] = scale_bytes(sa, 0, i);

    uint32_t kb = 0;
    // step kb, kb % 2 == Q; STEADY: at least two more follow
    auto step = [&](auto Q, auto STEADY) {
        constexpr int cur = decltype(Q)::value, nxt = cur ^ 1;
        constexpr int kAfter1 = nxt == 0 ? 18 : 16, kAfter2 = cur == 0 ? 18 : 16;
        const bool one = decltype(STEADY)::value || kb + 1 < kb1, two = decltype(STEADY)::value || kb + 2 < kb1;
        const uint32_t now = (kb >> 1 & 1) * kMxBigScales + cur * kStepScales;
        const uint32_t then = ((kb + 1) >> 1 & 1) * kMxBigScales + nxt * kStepScales;
        auto column0 = [&](auto J) {
            constexpr int j = decltype(J)::value;
            fence_order();
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (h == 0) mma4<0, !decltype(STEADY)::value>(acc[i][j], fb[j].half[0], fa[i].half[0], eb[j], ea[i]);
                    else mma4<1, !decltype(STEADY)::value>(acc[i][j], fb[j].half[1], fa[i].half[1], eb[j], ea[i]);
                    if constexpr (j >= 2) {
                        if (i == 0 && two) {
                            if (h == 0) load_first(kb + 2, Int<cur>(), Int<2 * (j - 2)>());
                            else load_first(kb + 2, Int<cur>(), Int<2 * (j - 2) + 1>());
                        }
                        if (h == 1 && i == 3 && j == 7 && cur == 0 && two) load_scale_bytes(kb + 2);
                        if constexpr (j < 6) {
                            if (i == 2) fa[2 + j].half[h] = *(const v4i*)(la + cur * kBigStage + (2 + j) * 16 * kStepK + (h ? t.c1 : t.c0));
                            if (h == 0 && i == 1) ea[2 + j] = scale_bytes(sa, now, 2 + j);
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
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int i = 4; i < 8; i++) {
                    if (h == 0) mma4<0, !decltype(STEADY)::value>(acc[i][j], fb[j].half[0], fa[i].half[0], eb[j], ea[i]);
                    else mma4<1, !decltype(STEADY)::value>(acc[i][j], fb[j].half[1], fa[i].half[1], eb[j], ea[i]);
                    if (h == 0 && i == 5 && !(j & 1) && two) load_second(kb + 2, Int<cur>(), Int<(j >> 1)>());
                    if ((j & 1) && i == 5) fa[j >> 1].half[h] = *(const v4i*)(la + nxt * kBigStage + (j >> 1) * 16 * kStepK + (h ? t.c1 : t.c0));
                    if ((j & 1) && h == 0 && i == 6) ea[j >> 1] = scale_bytes(sa, then, j >> 1);
                    if (h == 1 && i == 4) fb[j].half[0] = *(const v4i*)(lb + nxt * kBigStage + j * 16 * kStepK + t.c0);
                    fence_order();
                }
            fb[j].half[1] = *(const v4i*)(lb + nxt * kBigStage + j * 16 * kStepK + t.c1);
            eb[j] = scale_bytes(sb, then, j);
        };
        column1(Int<0>()); column1(Int<1>()); column1(Int<2>()); column1(Int<3>());
        column1(Int<4>()); column1(Int<5>()); column1(Int<6>()); column1(Int<7>());
        kb++;
    };
    while (kb + 3 < kb1) {
        step(Int<0>(), Int<1>());
        step(Int<1>(), Int<1>());
    }
    for (;;) {
        step(Int<0>(), Int<0>());
        if (kb == kb1) break;
        step(Int<1>(), Int<0>());
        if (kb == kb1) break;
    }
    settle();
#pragma unroll
    for (int i = 0; i < 8; i++)
        asm volatile("" : "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]), "+a"(acc[i][4]),
                     "+a"(acc[i][5]), "+a"(acc[i][6]), "+a"(acc[i][7]));
    sync_loads<0>();
    MxLines<8, 8> lines;
    mx_finish<8, 8>(p, acc, (float*)(lds + t.wave * finish_bytes<8, 8>()), t.m0 + t.wm * 128, t.n0 + t.wn * 128, t.lo_i,
                    t.lo_j, t.lane, lines);
}

// The accumulators of mx_stream_kernel: acc[i][j] is a[4 (8 i + j)] to + 3, by
// name.  Given variables, the compiler copies them where tiles follow one another
// (it spilled 200 registers).  It is told that the kernel writes all of them, but
// nothing it is told keeps it from putting a value there between two statements:
// the build reads the kernel's assembly, and fails where one of them is named
// outside these statements or anything is spilled.
__device__ __forceinline__ void all_accumulators() {
    asm volatile("" ::: "a0", "a1", "a2", "a3", "a4", "a5", "a6", "a7", "a8", "a9", "a10", "a11", "a12", "a13",
                 "a14", "a15", "a16", "a17", "a18", "a19", "a20", "a21", "a22", "a23", "a24", "a25", "a26", "a27",
                 "a28", "a29", "a30", "a31", "a32", "a33", "a34", "a35", "a36", "a37", "a38", "a39", "a40", "a41",
                 "a42", "a43", "a44", "a45", "a46", "a47", "a48", "a49", "a50", "a51", "a52", "a53", "a54", "a55",
                 "a56", "a57", "a58", "a59", "a60", "a61", "a62", "a63", "a64", "a65", "a66", "a67", "a68", "a69",
                 "a70", "a71", "a72", "a73", "a74", "a75", "a76", "a77", "a78", "a79", "a80", "a81", "a82", "a83",
                 "a84", "a85", "a86", "a87", "a88", "a89", "a90", "a91", "a92", "a93", "a94", "a95", "a96", "a97",
                 "a98", "a99", "a100", "a101", "a102", "a103", "a104", "a105", "a106", "a107", "a108", "a109",
                 "a110", "a111", "a112", "a113", "a114", "a115", "a116", "a117", "a118", "a119", "a120", "a121",
                 "a122", "a123", "a124", "a125", "a126", "a127", "a128", "a129", "a130", "a131", "a132", "a133",
                 "a134", "a135", "a136", "a137", "a138", "a139", "a140", "a141", "a142", "a143", "a144", "a145",
                 "a146", "a147", "a148", "a149", "a150", "a151", "a152", "a153", "a154", "a155", "a156", "a157",
                 "a158", "a159", "a160", "a161", "a162", "a163", "a164", "a165", "a166", "a167", "a168", "a169",
                 "a170", "a171", "a172", "a173", "a174", "a175", "a176", "a177", "a178", "a179", "a180", "a181",
                 "a182", "a183", "a184", "a185", "a186", "a187", "a188", "a189", "a190", "a191", "a192", "a193",
                 "a194", "a195", "a196", "a197", "a198", "a199", "a200", "a201", "a202", "a203", "a204", "a205",
                 "a206", "a207", "a208", "a209", "a210", "a211", "a212", "a213", "a214", "a215", "a216", "a217",
                 "a218", "a219", "a220", "a221", "a222", "a223", "a224", "a225", "a226", "a227", "a228", "a229",
                 "a230", "a231", "a232", "a233", "a234", "a235", "a236", "a237", "a238", "a239", "a240", "a241",
                 "a242", "a243", "a244", "a245", "a246", "a247", "a248", "a249", "a250", "a251", "a252", "a253",
                 "a254", "a255");
}

// acc[I][J] += a b (FIRST: = a b), 128 along the sum, with byte Q of the scale words
template <int I, int J, int Q, bool FIRST>
__device__ __forceinline__ void mma4_named(const v4i& a, const v4i& b, uint32_t ea, uint32_t eb) {
    constexpr int r = 4 * (8 * I + J);
    if constexpr (FIRST)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[%0:%1], %2, %3, 0, %4, %5 op_sel:[%6,%6,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     ::"n"(r), "n"(r + 3), "v"(a), "v"(b), "v"(ea), "v"(eb), "n"(Q));
    else
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[%0:%1], %2, %3, a[%0:%1], %4, %5 op_sel:[%6,%6,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     ::"n"(r), "n"(r + 3), "v"(a), "v"(b), "v"(ea), "v"(eb), "n"(Q));
}

template <int I, int J>
__device__ __forceinline__ v4f sums_of() {
    constexpr int r = 4 * (8 * I + J);
    float x, y, z, w;
    asm volatile("v_accvgpr_read_b32 %0, a[%4]\n\tv_accvgpr_read_b32 %1, a[%5]\n\tv_accvgpr_read_b32 %2, a[%6]\n\tv_accvgpr_read_b32 %3, a[%7]"
                 : "=v"(x), "=v"(y), "=v"(z), "=v"(w)
                 : "n"(r), "n"(r + 1), "n"(r + 2), "n"(r + 3));
    return v4f{x, y, z, w};
}

// A wave's way out: its 128 x 128 of C go through 4 KB of LDS of the wave's own in
// pieces of 16 rows x 256 bytes, so that neighbouring lanes store neighbouring
// bytes (8192 x 8192 x 1024: 53 us, 77 us with stores straight from the
// registers, whose 16 neighbouring lanes are 16 rows).  16-byte chunk c of row r
// is at c ^ r.
struct StreamOut {
    uint8_t* base;     // of C: the wave's first element
    uint32_t lane;     // bytes from there to this lane's chunk of the first four rows
    uint64_t rows4;    // bytes of four rows of C
    uint32_t put;      // LDS: this lane's row, and its lane group's place in a fragment
    uint32_t get;      // LDS: this lane's chunk of the first four rows
    uint4_v chunk[4];  // under way from LDS to C
};

typedef __attribute__((address_space(3))) uint8_t* LdsBytes;

// fragment f of piece t of the rows 64 HALF .. +63 into LDS: 8 fragments a piece of 16-bit results, 4 of fp32
template <typename T, int HALF, int t, int f>
__device__ __forceinline__ void stream_put(const StreamOut& o) {
    constexpr bool kWide = sizeof(T) == 4;
    constexpr int i = HALF * 4 + (kWide ? t / 2 : t), j = kWide ? t % 2 * 4 + f : f;
    const v4f x = sums_of<i, j>();
    if constexpr (kWide) {
        *(__attribute__((address_space(3))) v4f*)((LdsBytes)(uintptr_t)(o.put ^ f * 64)) = x;
    } else {
        typedef T t2 __attribute__((ext_vector_type(2)));
        *(__attribute__((address_space(3))) uint2_v*)((LdsBytes)(uintptr_t)(o.put ^ f * 32)) =
            uint2_v{__builtin_bit_cast(uint32_t, t2{(T)x[0], (T)x[1]}), __builtin_bit_cast(uint32_t, t2{(T)x[2], (T)x[3]})};
    }
}
// the piece back from LDS, in rows.  A wave's LDS operations are done in their order.
__device__ __forceinline__ void stream_get(StreamOut& o) {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int k = 0; k < 4; k++)  // rows 4 k + lane / 16
        o.chunk[k] = *(__attribute__((address_space(3))) const uint4_v*)((LdsBytes)(uintptr_t)((o.get ^ k * 64) + k * 1024));
    asm volatile("" ::: "memory");
}
// four rows of piece t to C
template <typename T, bool PAST, int HALF, int t, int k>
__device__ __forceinline__ void stream_store(const StreamOut& o) {
    constexpr bool kWide = sizeof(T) == 4;
    constexpr int i = HALF * 4 + (kWide ? t / 2 : t);
    uint4_v* to = (uint4_v*)(o.base + (4 * i + k) * o.rows4 + o.lane + (kWide ? t % 2 * 256 : 0));
    if (PAST) __builtin_nontemporal_store(o.chunk[k], to);
    else *to = o.chunk[k];
}

// What of a half's pieces stands behind matrix instruction s of 64.  16-bit
// results: four pieces, each 8 fragments into LDS, one read back, four stores
// in 15 slots.  fp32: eight pieces in 7 slots each, 4 fragments, one read, two
// stores at a time while the next piece's fragments go in.
template <typename T, bool PAST, int HALF, int s>
__device__ __forceinline__ void stream_slot(StreamOut& o) {
    if constexpr (sizeof(T) == 2) {
        constexpr int t = s / 15, x = s % 15;
        if constexpr (t < 4) {
            if constexpr (x < 8) stream_put<T, HALF, t, x>(o);
            else if constexpr (x == 8) stream_get(o);
        }
        constexpr int u = (s - 12) / 15, y = (s - 12) % 15;
        if constexpr (s >= 12 && u < 4 && y < 4) stream_store<T, PAST, HALF, u, y>(o);
    } else {
        constexpr int t = s / 7, x = s % 7;
        constexpr int u = (s - 6) / 7, y = (s - 6) % 7;
        if constexpr (s >= 6 && u < 8 && y < 2) stream_store<T, PAST, HALF, u, 2 * y>(o), stream_store<T, PAST, HALF, u, 2 * y + 1>(o);
        if constexpr (t < 8) {
            if constexpr (x < 4) stream_put<T, HALF, t, x>(o);
            else if constexpr (x == 4) stream_get(o);
        }
    }
}
// stores in the first 16 slots
template <typename T>
constexpr int stream_early() {
    return sizeof(T) == 2 ? 4 : 8;
}

// Large results to which nothing is added: 256 x 256 tiles by workgroups that
// stay, one a CU.  Steps follow one another across tiles without a pause: the
// first two steps of the next tile are loaded during the last two of this one,
// and a tile leaves while matrix instructions run, its upper 64 rows of each wave
// behind those of its last step's second half (which adds to the lower rows), the
// lower ones behind those of the next tile's first half.  mx_big_kernel spends 12
// us between two tiles, in which all CUs load or write and none multiplies: 4096
// x 8192 x 2048 takes 45.5 us there and 36 here, 8192 x 8192 x 8192 230 and 217 to
// 227 us beside one another; over cards, and with what ran before, 217 to 266 (4.1 to
// 5.1 PFLOP/s; from registers the instructions reach 7.1 on random codes and 9.4 on
// equal ones).
//
// Bound by the clock that the matrix instructions' power leaves, and by the
// moment when all CUs write: loads and stores come back in their order, so the
// loads behind a tile's stores wait for these (8192 x 8192 x 2048 77 us, 58 us
// without the stores).  Tiles of 256 x 128 on two sets of accumulators, whose
// stores spread over half of the next tile, read half as much again from LDS for
// a product: 48 us at 8192 x 8192 x 1024, but 78 at x 2048 and 268 at x 8192.
//
// PAST: results go past the caches.  4096 x 8192 x 2048, whose 67 MB fit the last
// cache, 40.3 us, 37.0 through them; 8192 x 8192 x 2048 77.6, 81.7 through them.
template <typename T, bool PAST>
__global__ __launch_bounds__(256, 1) void mx_stream_kernel(ProductArgs p) {
    constexpr int kStores = sizeof(T) == 4 ? 32 : 16;  // of half a tile
    constexpr int kEarly = stream_early<T>();         // of those before the first barrier
    all_accumulators();
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1, row = lane & 15, g = lane >> 4;
    const uint32_t tiles = p.tiles_m * p.tiles_n, kb1 = p.kb;
    const uint32_t offset = (lane >> 3) * p.pitch + (((lane & 7) ^ (lane >> 4) ^ (wave & 1) * 4) * 16);
    uint32_t p32 = 32 * p.pitch;
    const uint32_t s_offset = (uint32_t)lane * p.s_pitch;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);
    const uint32_t lds_codes = lds0 + wave * 1024, lds_scales = lds0 + 2 * kBigStage + wave * 1024;
    const uint32_t c0 = ((2 * g) ^ (row >> 1)) * 16, c1 = ((2 * g + 1) ^ (row >> 1)) * 16;

    // what is loaded next: step `lkb` of tile `ltile`
    uint32_t ltile = blockIdx.x, lkb = 0, lm0, ln0;
    const uint8_t *ga, *gb, *gsa, *gsb;
    auto place = [&]() __attribute__((always_inline)) {
        uint32_t tm, tn;
        tile_of(p.tiles_m, p.tiles_n, ltile, tm, tn);
        lm0 = min(tm * kBig, p.m - kBig);
        ln0 = min(tn * kBig, p.n - kBig);
        ga = p.a + (uint64_t)(lm0 + 8 * wave) * p.pitch;
        gb = p.b + (uint64_t)(ln0 + 8 * wave) * p.pitch;
        gsa = p.sa + (uint64_t)(lm0 + 64 * wave) * p.s_pitch;
        gsb = p.sb + (uint64_t)(ln0 + 64 * wave) * p.s_pitch;
    };
    auto load_first = [&](auto ST, auto E) __attribute__((always_inline)) {  // one of 12
        constexpr int e = decltype(E)::value, x = e < 8 ? e : e < 10 ? e - 8 : e - 6;
        load_lds16(e < 8 ? gb : ga, offset + x * p32, lds_codes + decltype(ST)::value * kBigStage + (e < 8 ? kBig * kStepK : 0) + x * 4096);
    };
    auto load_second = [&](auto ST, auto E) __attribute__((always_inline)) {  // one of 4
        constexpr int e = decltype(E)::value, x = e < 2 ? e + 2 : e + 4;
        load_lds16(ga, offset + x * p32, lds_codes + decltype(ST)::value * kBigStage + x * 4096);
    };
    uint32_t lpair = 0;  // which half of the scale bytes' place is filled next
    auto load_scale_bytes = [&]() __attribute__((always_inline)) {
        const uint32_t at = __builtin_amdgcn_readfirstlane(lds_scales + lpair * kMxBigScales);
        load_lds16(gsa, s_offset + lkb * kStepScales, at);
        load_lds16(gsb, s_offset + lkb * kStepScales, at + kBig * 2 * kStepScales);
        lpair ^= 1;
    };
    auto loaded = [&]() __attribute__((always_inline)) {  // the step's loads are all under way
        lkb++;
        ga += kStepK, gb += kStepK;
        if (lkb == kb1) {
            lkb = 0;
            if (ltile + gridDim.x < tiles) ltile += gridDim.x;  // behind the last tile it is loaded again, and not read
            place();
        }
    };
    auto load_step = [&](auto ST, auto S) __attribute__((always_inline)) {
        load_first(ST, Int<0>()); load_first(ST, Int<1>()); load_first(ST, Int<2>());
        load_first(ST, Int<3>()); load_first(ST, Int<4>()); load_first(ST, Int<5>());
        load_first(ST, Int<6>()); load_first(ST, Int<7>()); load_first(ST, Int<8>());
        load_first(ST, Int<9>()); load_first(ST, Int<10>()); load_first(ST, Int<11>());
        if constexpr (decltype(S)::value) load_scale_bytes();
        load_second(ST, Int<0>()); load_second(ST, Int<1>());
        load_second(ST, Int<2>()); load_second(ST, Int<3>());
        loaded();
    };
    typedef __attribute__((address_space(3))) const uint8_t* Lds;
    const Lds base = (Lds)lds;
    const uint32_t at_a = (wm * 128 + row) * kStepK, at_b = (kBig + wn * 128 + row) * kStepK;
    const uint32_t at_sa = 2 * kBigStage + (wm * 128 + row) * 2 * kStepScales + 2 * g;
    const uint32_t at_sb = at_sa + (kBig + (wn - wm) * 128) * 2 * kStepScales;
    struct Fragment {
        v4i half[2];
    };
    // this lane's codes of half h of fragment i
    auto codes = [&](uint32_t at, uint32_t stage, int i, int h) __attribute__((always_inline)) {
        return *(__attribute__((address_space(3))) const v4i*)(base + (at + (h ? c1 : c0) + stage) + i * 16 * kStepK);
    };
    auto scale_bytes = [&](uint32_t at, uint32_t half, int i) __attribute__((always_inline)) {
        return (uint32_t) * (__attribute__((address_space(3))) const uint16_t*)(base + (at + half) + i * 16 * 2 * kStepScales);
    };
    Fragment fa[8], fb[8];
    uint32_t ea[8], eb[8];
    StreamOut out;
    out.base = nullptr;
    out.rows4 = 4 * p.ldc * sizeof(T);
    out.lane = (uint32_t)((lane >> 4) * p.ldc * sizeof(T)) + (lane & 15) * 16;
    const uint32_t slab = lds0 + kMxBigLds + wave * 4096;
    out.put = slab + row * 256 + (sizeof(T) == 4 ? (g ^ row) * 16 : ((g >> 1) ^ row) * 16 + (g & 1) * 8);
    out.get = slab + (lane >> 4) * 256 + ((lane & 15) ^ (lane >> 4)) * 16;
    place();
    uint32_t m0 = lm0, n0 = ln0;
    load_step(Int<0>(), Int<1>());
    load_step(Int<1>(), Int<0>());
    sync_loads<16>();
#pragma unroll
    for (int j = 0; j < 8; j++) fb[j] = Fragment{{codes(at_b, 0, j, 0), codes(at_b, 0, j, 1)}}, eb[j] = scale_bytes(at_sb, 0, j);
#pragma unroll
    for (int i = 0; i < 4; i++) fa[i] = Fragment{{codes(at_a, 0, i, 0), codes(at_a, 0, i, 1)}}, ea[i] = scale_bytes(at_sa, 0, i);

    auto place_of_c = [&]() __attribute__((always_inline)) { return (uint8_t*)p.c + ((uint64_t)(m0 + wm * 128) * p.ldc + n0 + wn * 128) * sizeof(T); };
    uint32_t pair = 0;     // which half of the scale bytes' place this step's are in
    // Q: the step's parity.  PLACE: 0 the tile's first step, 1 the second, 2 one
    // in between, 3 the last.  BEFORE: another tile's rows 64..127 are stored
    // in the first step.
    auto step = [&](auto Q, auto PLACE, auto BEFORE) __attribute__((always_inline)) {
        constexpr int cur = decltype(Q)::value, nxt = cur ^ 1;
        constexpr bool first = decltype(PLACE)::value == 0, second = decltype(PLACE)::value == 1;
        constexpr bool last = decltype(PLACE)::value == 3, before = decltype(BEFORE)::value;
        constexpr int kAfter1 = nxt == 0 ? 18 : 16, kAfter2 = cur == 0 ? 18 : 16;
        // sums with these are made where they are used, or they would take registers that are not there
        uint32_t here = cur * kBigStage, there = nxt * kBigStage;
        asm volatile("" : "+s"(p32), "+s"(here), "+s"(there));
        const uint32_t now = pair * kMxBigScales + cur * kStepScales;
        const uint32_t then = (cur ? pair ^ 1 : pair) * kMxBigScales + nxt * kStepScales;
        // matrix instruction (I, J, H), H the half of the step, and what stands behind it
        auto slot0 = [&](auto J, auto H, auto I) __attribute__((always_inline)) {
            constexpr int j = decltype(J)::value, h = decltype(H)::value, i = decltype(I)::value;
            mma4_named<i, j, h, first && h == 0>(fb[j].half[h], fa[i].half[h], eb[j], ea[i]);
            if constexpr (j >= 2) {
                if constexpr (i == 0) load_first(Int<cur>(), Int<2 * (j - 2) + h>());
                if constexpr (h == 1 && i == 3 && j == 7 && cur == 0) load_scale_bytes();
                if constexpr (j < 6 && i == 2) fa[2 + j].half[h] = codes(at_a, here, 2 + j, h);
                if constexpr (j < 6 && h == 0 && i == 1) ea[2 + j] = scale_bytes(at_sa, now, 2 + j);
            }
            if constexpr (first && before) stream_slot<T, PAST, 1, 8 * j + 4 * h + i>(out);
            fence_order();
        };
        auto column0 = [&](auto J) __attribute__((always_inline)) {
            fence_order();
            slot0(J, Int<0>(), Int<0>()); slot0(J, Int<0>(), Int<1>()); slot0(J, Int<0>(), Int<2>()); slot0(J, Int<0>(), Int<3>());
            slot0(J, Int<1>(), Int<0>()); slot0(J, Int<1>(), Int<1>()); slot0(J, Int<1>(), Int<2>()); slot0(J, Int<1>(), Int<3>());
            if constexpr (decltype(J)::value == 1) {  // P
                if constexpr (first && before) sync_loads<(kAfter1 + kStores + kEarly < 63 ? kAfter1 + kStores + kEarly : 63)>();
                else if constexpr (second && before) sync_loads<kAfter1 + kStores>();
                else sync_loads<kAfter1>();
            }
        };
        column0(Int<0>()); column0(Int<1>()); column0(Int<2>()); column0(Int<3>());
        column0(Int<4>()); column0(Int<5>()); column0(Int<6>()); column0(Int<7>());
        if constexpr (first && before) sync_loads<(kAfter2 + 2 * kStores < 63 ? kAfter2 + 2 * kStores : 63)>();
        else sync_loads<kAfter2>();
        if constexpr (last) out.base = place_of_c();
        auto slot1 = [&](auto J, auto H, auto I) __attribute__((always_inline)) {
            constexpr int j = decltype(J)::value, h = decltype(H)::value, i = decltype(I)::value;
            mma4_named<i, j, h, first && h == 0>(fb[j].half[h], fa[i].half[h], eb[j], ea[i]);
            if constexpr (h == 0 && i == 5 && !(j & 1)) load_second(Int<cur>(), Int<(j >> 1)>());
            if constexpr ((j & 1) && i == 5) fa[j >> 1].half[h] = codes(at_a, there, j >> 1, h);
            if constexpr ((j & 1) && h == 0 && i == 6) ea[j >> 1] = scale_bytes(at_sa, then, j >> 1);
            if constexpr (h == 1 && i == 4) fb[j].half[0] = codes(at_b, there, j, 0);
            if constexpr (last) stream_slot<T, PAST, 0, 8 * j + 4 * h + i - 4>(out);
            fence_order();
        };
        auto column1 = [&](auto J) __attribute__((always_inline)) {
            constexpr int j = decltype(J)::value;
            fence_order();
            slot1(J, Int<0>(), Int<4>()); slot1(J, Int<0>(), Int<5>()); slot1(J, Int<0>(), Int<6>()); slot1(J, Int<0>(), Int<7>());
            slot1(J, Int<1>(), Int<4>()); slot1(J, Int<1>(), Int<5>()); slot1(J, Int<1>(), Int<6>()); slot1(J, Int<1>(), Int<7>());
            fb[j].half[1] = codes(at_b, there, j, 1);
            eb[j] = scale_bytes(at_sb, then, j);
        };
        column1(Int<0>()); column1(Int<1>()); column1(Int<2>()); column1(Int<3>());
        column1(Int<4>()); column1(Int<5>()); column1(Int<6>()); column1(Int<7>());
        loaded();
        if (cur) pair ^= 1;
    };
    step(Int<0>(), Int<0>(), Int<0>());
    step(Int<1>(), Int<1>(), Int<0>());
    for (uint32_t tile = blockIdx.x;;) {
        for (uint32_t kb = 4; kb < kb1; kb += 2) {
            step(Int<0>(), Int<2>(), Int<0>());
            step(Int<1>(), Int<2>(), Int<0>());
        }
        const uint32_t next_m0 = lm0, next_n0 = ln0;
        step(Int<0>(), Int<2>(), Int<0>());
        step(Int<1>(), Int<3>(), Int<0>());
        tile += gridDim.x;
        if (tile >= tiles) break;
        m0 = next_m0, n0 = next_n0;
        step(Int<0>(), Int<0>(), Int<1>());
        step(Int<1>(), Int<1>(), Int<1>());
    }
    settle();
    auto rest = [&](auto X) __attribute__((always_inline)) {
        constexpr int x = 8 * decltype(X)::value;
        stream_slot<T, PAST, 1, x>(out), stream_slot<T, PAST, 1, x + 1>(out), stream_slot<T, PAST, 1, x + 2>(out), stream_slot<T, PAST, 1, x + 3>(out);
        stream_slot<T, PAST, 1, x + 4>(out), stream_slot<T, PAST, 1, x + 5>(out), stream_slot<T, PAST, 1, x + 6>(out), stream_slot<T, PAST, 1, x + 7>(out);
    };
    rest(Int<0>()); rest(Int<1>()); rest(Int<2>()); rest(Int<3>()); rest(Int<4>()); rest(Int<5>()); rest(Int<6>()); rest(Int<7>());
    all_accumulators();
}

// Few rows: 16 columns of C for up to 16 rows by NW waves that share the sum
// among them, each taking every NW-th step straight from memory, eight steps' loads
// under way at a time.  The waves' sums are added in their order.  Bound by the
// latency of those loads: 16 x 2048 x 8192 takes 7.8 us (8.2 with one step's loads
// and eight waves), 16 x 8192 x 2048 5.2, 16 x 100352 x 2048 32 us (3.6 TB/s; 40 us
// where a load took 16 bytes of every 32), 8 x 4096 x 14336 10.3 to 12 us.
template <int NW>
__global__ __launch_bounds__(64 * NW) void mx_few_kernel(ProductArgs p) {
    constexpr int U = 8;
    __shared__ __attribute__((aligned(16))) float sums[NW][16 * 20];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row = lane & 15, g = lane >> 4;
    const uint32_t n0 = blockIdx.x * 16;
    const uint32_t ra = min((uint32_t)row, p.m - 1), rb = min(n0 + row, p.n - 1);
    // chunks g and 4 + g of a step: a load takes 64 bytes of a row
    const uint8_t *qa = p.a + (uint64_t)ra * p.pitch + g * 16, *xa = p.sa + (uint64_t)ra * p.s_pitch;
    const uint8_t *qb = p.b + (uint64_t)rb * p.pitch + g * 16, *xb = p.sb + (uint64_t)rb * p.s_pitch;
    v4f acc[1][1] = {};
    auto steps = [&](uint32_t kb, auto N) {
        constexpr int n = decltype(N)::value;
        uint2_v ea[n], eb[n];
        v4i a[n][2][1], b[n][2][1];
#pragma unroll
        for (int u = 0; u < n; u++) {
            const uint32_t k = kb + u * NW;
            b[u][0][0] = *(const v4i*)(qb + k * kStepK), b[u][1][0] = *(const v4i*)(qb + k * kStepK + 64);
            a[u][0][0] = *(const v4i*)(qa + k * kStepK), a[u][1][0] = *(const v4i*)(qa + k * kStepK + 64);
            eb[u] = *(const uint2_v*)(xb + k * kStepScales);
            ea[u] = *(const uint2_v*)(xa + k * kStepScales);
        }
#pragma unroll
        for (int u = 0; u < n; u++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t x[1] = {ea[u][h] >> 8 * g}, y[1] = {eb[u][h] >> 8 * g};
                mx_multiply<0>(acc, a[u][h], b[u][h], x, y);
            }
    };
    uint32_t kb = wave;
    for (; kb + (U - 1) * NW < p.kb; kb += U * NW) steps(kb, Int<U>());
    if (kb + 3 * NW < p.kb) steps(kb, Int<4>()), kb += 4 * NW;
    if (kb + NW < p.kb) steps(kb, Int<2>()), kb += 2 * NW;
    if (kb < p.kb) steps(kb, Int<1>());
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

// One or two rows, as a token at a time makes them: a wave for each column of C,
// whose loads take 1 KB of it in one piece.  Lane l takes block l of 64 blocks of
// 32 codes, of the rows and of the column alike, so the "rows" that the matrix
// instruction multiplies are sixteen parts of the sum: their products are its
// diagonal, and the rest of the result is nobody's.  Bound by the loads' latency
// and, where there are many columns, by memory: calls back to back, one row x 2048 x 8192 takes
// 4.2 us (mx_few_kernel 5.8), x 16384 x 8192 15.7 us (18.5); two or four columns a
// wave 4.9 and 16.6 us, 5.7 and 17.6 us.  The kernel alone takes 3.6 and 12.5 us (5.7
// TB/s).
template <int M>
__global__ __launch_bounds__(256) void mx_rows_kernel(ProductArgs p) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t j = blockIdx.x * 4 + wave;
    if (j >= p.n) return;
    const uint8_t *qb = p.b + (uint64_t)j * p.pitch, *xb = p.sb + (uint64_t)j * p.s_pitch;
    const uint32_t blocks = p.kb * kStepScales;
    v4f acc[M][1] = {};
    auto step = [&](uint32_t k, bool on) {  // matrix instructions heed no mask: what is off multiplies zeros
        v4i a[M] = {}, b[1] = {};
        uint32_t ea[M] = {}, eb[1] = {};
        if (on) {
            b[0] = *(const v4i*)(qb + k * 16);
            eb[0] = xb[k];
#pragma unroll
            for (int i = 0; i < M; i++) {
                a[i] = *(const v4i*)(p.a + (uint64_t)i * p.pitch + k * 16);
                ea[i] = p.sa[(uint64_t)i * p.s_pitch + k];
            }
        }
        mx_multiply<0>(acc, a, b, ea, eb);
    };
    uint32_t k0 = 0;
    for (; k0 + 64 <= blocks; k0 += 64) step(k0 + lane, true);
    if (k0 < blocks) step(k0 + lane, k0 + lane < blocks);
    const int d = (lane & 15) - 4 * (lane >> 4);  // which of this lane's four sums is on the diagonal
    float sum[M];
#pragma unroll
    for (int i = 0; i < M; i++) {
        sum[i] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; q++) sum[i] = d == q ? acc[i][0][q] : sum[i];
#pragma unroll
        for (int x = 32; x; x >>= 1) sum[i] += __shfl_xor(sum[i], x);
    }
    if (lane < M) {
        float v[8] = {M > 1 && lane ? sum[M - 1] : sum[0]};
        if (p.drop.on) drop8(p.drop, (uint64_t)lane * p.n + j, v);
        if (p.dtype == kF32) put_row<float>(p, lane, j, 0, 1, v, false);
        else if (p.dtype == kF16) put_row<f16_t>(p, lane, j, 0, 1, v, false);
        else put_row<bf16_t>(p, lane, j, 0, 1, v, false);
    }
}

}  // namespace demo
