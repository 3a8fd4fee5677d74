// mx.hip -- host side of the linear layer on 4-bit operands: quantisation,
// values and the matrix product.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "demo.h"
#include "linear_host.hpp"
#include "mx_product.hpp"
#include "mx_quantize.hpp"

namespace {

using demo::aligned16;
using demo::aligned_to;
using demo::drop_of;
using demo::elem_bytes;
using demo::launch;
using demo::overlap;
using demo::pitch_ok;
using demo::sides_ok;
using demo::status_of;
using demo::up;

constexpr uint64_t kStep = 256;  // codes of a step, 128 bytes

demo_operand mx_operand_of(uint64_t rows, uint64_t cols) {
    demo_operand o{};
    o.pitch = up(cols, kStep) / 2;
    o.scale_pitch = up(o.pitch * 2 / DEMO_MX_BLOCK, 16);
    o.scale_off = demo::up256(rows * o.pitch);
    o.total_bytes = demo::up256(o.scale_off + rows * o.scale_pitch);
    return o;
}

int check(const demo_mx_cfg* cfg, bool quantiser) {
    if (!cfg) return DEMO_EINVAL;
    if (cfg->abi_version != DEMO_ABI_VERSION) return DEMO_EABI;
    if (cfg->tile > (quantiser ? 1u : 0u) || cfg->dtype > DEMO_DTYPE_BF16 || cfg->reserved != 0) return DEMO_EINVAL;
    return DEMO_OK;
}

int check_product(const demo_mx_cfg* cfg, uint64_t m, uint64_t n, uint64_t k) {
    if (const int rc = check(cfg, false)) return rc;
    if (!sides_ok(m, n) || k < 1) return DEMO_EINVAL;
    if (k > DEMO_BLOCK_MAX_K) return DEMO_EUNSUPPORTED;
    if (!sides_ok(m, k) || !sides_ok(n, k)) return DEMO_EINVAL;
    return DEMO_OK;
}

template <typename F>
hipError_t with_type(uint32_t dtype, F f) {
    switch (dtype) {
    case DEMO_DTYPE_F32: return f(0.f);
    case DEMO_DTYPE_F16: return f((demo::f16_t)0);
    default: return f((demo::bf16_t)0);
    }
}

template <typename T, bool TILE>
hipError_t launch_quantize(const demo::MxArgs& a, bool wide, dim3 grid, hipStream_t s) {
    if (a.drop.on)
        return launch(wide ? demo::mx_quantize_kernel<T, TILE, true, true> : demo::mx_quantize_kernel<T, TILE, true, false>,
                      grid, dim3(256), 0, s, a);
    return launch(wide ? demo::mx_quantize_kernel<T, TILE, false, true> : demo::mx_quantize_kernel<T, TILE, false, false>,
                  grid, dim3(256), 0, s, a);
}

constexpr uint64_t kMaxSquares = (uint64_t)1 << 24;  // of 256 work-items: a grid has less than 2^32 of them

// the kernel for few rows, and the columns that its grid holds (below 2^32 work-items)
constexpr uint64_t kFewRows = 16, kFewRowsMaxCols = (uint64_t)1 << 25;

constexpr uint32_t kCus = 256;

// Results of mx_stream_kernel up to this many bytes stay in the caches for who reads
// them next, larger ones go past them.  (The other tiles'
// 16-bit results in aligned accesses, and fp32 ones through no dropout, go past them at
// every size.)
constexpr uint64_t kCached = (uint64_t)96 << 20;

// How a product is cut: tiles of `tile` x `tile` and `splits` of the sum, or
// (tile 0) the kernel for few rows.
struct Plan {
    uint32_t tile;
    uint32_t splits;
    uint32_t kb_split;
};

// The card runs 256 tiles of 256 x 256 at a time, 512 of 128 x 128 or 1024 of 64
// x 64 (one, two and four workgroups a CU).  Measured:
//  * a round of 256 tiles costs 1.6 rounds of 128 tiles (4096 x 4096 x 1024: 16.3
//    against 18.3 us; 5120 x 5120 x 2048: 36.6 against 40.6; 4096 x 2048 x 2048, half
//    a round: 24.9 against 17.1), so they are taken where rounds say so;
//  * up to 256 tiles of 128, tiles of 64 fill the card better (1024 x 2048 x 2048:
//    8.3 against 10.8 us), unless there are more than 192 of them with a sum of
//    4096 or more (2048 x 2048 x 8192: 34.0 against 30.0; 300 x 10000 x 5000: 24.3
//    against 20.7);
//  * the sum is split where there are fewer than 512 workgroups, down to 10 steps
//    (256 x 2048 x 8192: 15.9 us in 3, 18.8 in one, 16.7 in 2 or 4; 768 x 768 x
//    16384: 22.0 in 3, 35.3 in one; 64 x 16384 x 4096: 12.7 in one, 14.5 in 2).
Plan plan_of(uint64_t m, uint64_t n, uint64_t k) {
    const uint64_t kb = up(k, kStep) / kStep;
    if (m <= kFewRows && n <= kFewRowsMaxCols) return {0, 1, (uint32_t)kb};
    const auto tiles = [&](uint64_t t) { return up(m, t) / t * (up(n, t) / t); };
    const auto rounds = [](uint64_t count, uint64_t at_once) { return (count + at_once - 1) / at_once; };
    if (m >= 256 && n >= 256 && 33 * rounds(tiles(256), 256) <= 20 * rounds(tiles(128), 512))
        return {256, 1, (uint32_t)up(kb, 2)};
    const uint64_t tile = tiles(128) > (kb >= 16 ? 192u : 256u) ? 128 : 64, least = tile == 128 ? 32 : 10;
    uint64_t splits = 512 / tiles(tile);
    if (splits > kb / least) splits = kb / least;
    if (splits < 1) splits = 1;
    const uint64_t each = up((kb + splits - 1) / splits, 2);
    return {(uint32_t)tile, (uint32_t)((kb + each - 1) / each), (uint32_t)each};
}
// the partial sums of up to 512 tiles of 128 x 128
static_assert(512 * 128 * 128 * 4 <= DEMO_BLOCK_MAX_WORKSPACE, "workspace");

template <int TILE, int STAGES>
hipError_t launch_tiles(const demo::ProductArgs& a, dim3 grid, hipStream_t s) {
    constexpr size_t lds = 2 * TILE * (STAGES * demo::kStepK + demo::kMxPairs<STAGES> * 2 * demo::kStepScales);
    return launch(demo::mx_kernel<TILE, TILE, 2, 2, STAGES>, grid, dim3(256), lds, s, a);
}

template <typename T>
hipError_t launch_stream(const demo::ProductArgs& a, hipStream_t s) {
    const uint32_t tiles = a.tiles_m * a.tiles_n;
    const bool past = (uint64_t)a.m * a.n * sizeof(T) > kCached;
    return launch(past ? demo::mx_stream_kernel<T, true> : demo::mx_stream_kernel<T, false>,
                  dim3(tiles < kCus ? tiles : kCus), dim3(256), demo::kMxStreamLds, s, a);
}

// 256 x 256 tiles: by workgroups that stay where nothing but the sums goes to C
hipError_t launch_big(const demo::ProductArgs& a, hipStream_t s) {
    const bool plain = a.wide && !a.addend && !a.drop.on && a.kb % 2 == 0 && a.kb >= 4 && a.ldc < ((uint64_t)1 << 25);
    if (plain) {
        if (a.dtype == DEMO_DTYPE_F32) return launch_stream<float>(a, s);
        return a.dtype == DEMO_DTYPE_F16 ? launch_stream<demo::f16_t>(a, s) : launch_stream<demo::bf16_t>(a, s);
    }
    return launch(demo::mx_big_kernel<>, dim3(a.tiles_m * a.tiles_n), dim3(256), demo::kMxBigLds, s, a);
}

hipError_t launch_product(demo::ProductArgs a, const Plan& plan, void* workspace, hipStream_t s) {
    if (plan.tile == 0) {
        // a wave a column, unless the columns are many and short (1 x 100352 x 2048: 27.0 us, 24.9 in the kernel for few rows)
        if (a.m <= 2 && (a.kb > 8 || a.n <= 32768))
            return launch(a.m == 1 ? demo::mx_rows_kernel<1> : demo::mx_rows_kernel<2>, dim3((a.n + 3) / 4), dim3(256), 0, s, a);
        return launch(demo::mx_few_kernel<4>, dim3((a.n + 15) / 16), dim3(256), 0, s, a);
    }
    a.kb_split = plan.kb_split;
    a.partial = plan.splits > 1 ? static_cast<float*>(workspace) : nullptr;
    a.tiles_m = (a.m + plan.tile - 1) / plan.tile;
    a.tiles_n = (a.n + plan.tile - 1) / plan.tile;
    const dim3 grid(a.tiles_m * a.tiles_n, plan.splits);
    // where a CU has one workgroup at most, three steps' loads are under way instead of one
    // (64 x 16384 x 4096: 10.4 us, 12.4 with two stages; 32 x 4096 x 4096: 9.5 and 11.3; but 512 x
    // 6144 x 1024, three a CU, 9.2 and 7.3)
    const hipError_t e = plan.tile == 64    ? grid.x * grid.y <= kCus ? launch_tiles<64, 4>(a, grid, s) : launch_tiles<64, 2>(a, grid, s)
                         : plan.tile == 128 ? launch_tiles<128, 2>(a, grid, s)
                                            : launch_big(a, s);
    if (e != hipSuccess || plan.splits == 1) return e;
    const uint64_t blocks = ((uint64_t)a.m * ((a.n + 7) / 8) + 255) / 256;
    return launch(demo::product_join_kernel<>, dim3((unsigned)(blocks < (1u << 20) ? blocks : (1u << 20))), dim3(256), 0, s,
                  a, plan.splits);
}

}  // namespace

extern "C" {

int demo_mx_layout(uint64_t rows, uint64_t cols, demo_operand* out) {
    if (!out || !sides_ok(rows, cols)) return DEMO_EINVAL;
    *out = mx_operand_of(rows, cols);
    return DEMO_OK;
}

int demo_mx_quantize(const demo_mx_cfg* cfg, uint64_t rows, uint64_t cols, const void* src, uint64_t ld,
                     const demo_dropout_cfg* dropout, void* operand, void* operand_t, void* hip_stream) {
    if (const int rc = check(cfg, true)) return rc;
    if (!sides_ok(rows, cols) || !pitch_ok(rows, cols, ld)) return DEMO_EINVAL;
    demo::MxArgs a{};
    if (const int rc = drop_of(dropout, rows * cols, &a.drop)) return rc;
    if (!src || (!operand && !operand_t)) return DEMO_EINVAL;
    const uint64_t eb = elem_bytes(cfg->dtype);
    if (!aligned_to(src, eb) || !aligned16(operand) || !aligned16(operand_t)) return DEMO_EALIGN;
    const demo_operand o = mx_operand_of(rows, cols), t = mx_operand_of(cols, rows);
    const uint64_t nb = ((rows - 1) * ld + cols) * eb;
    if (overlap(src, nb, operand, o.total_bytes) || overlap(src, nb, operand_t, t.total_bytes) ||
        overlap(operand, o.total_bytes, operand_t, t.total_bytes))
        return DEMO_EINVAL;
    a.src = src;
    a.ld = ld;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    // squares of 128 x 128; a pitch has an even number of them, and those behind the matrix write its zeros
    a.tiles_r = (uint32_t)(up(rows, 128) / 128);
    a.tiles_c = (uint32_t)(up(cols, 128) / 128);
    if (operand) {
        a.q = static_cast<uint8_t*>(operand);
        a.s = a.q + o.scale_off;
        a.pitch = o.pitch;
        a.s_pitch = (uint32_t)o.scale_pitch;
        a.tiles_c = (uint32_t)(o.pitch / 64);
    }
    if (operand_t) {
        a.qt = static_cast<uint8_t*>(operand_t);
        a.st = a.qt + t.scale_off;
        a.pitch_t = t.pitch;
        a.s_pitch_t = (uint32_t)t.scale_pitch;
        a.tiles_r = (uint32_t)(t.pitch / 64);
    }
    const uint64_t squares = (uint64_t)a.tiles_r * a.tiles_c;
    if (squares >= kMaxSquares) return DEMO_EUNSUPPORTED;
    const bool wide = aligned16(src) && ld * eb % 16 == 0 && cols % 8 == 0;
    const dim3 grid((unsigned)squares);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    return status_of(with_type(cfg->dtype, [&](auto type) {
        typedef decltype(type) T;
        return cfg->tile ? launch_quantize<T, true>(a, wide, grid, s) : launch_quantize<T, false>(a, wide, grid, s);
    }));
}

int demo_mx_dequantize(const demo_mx_cfg* cfg, uint64_t rows, uint64_t cols, const void* operand, void* dst,
                       uint64_t ld, void* hip_stream) {
    if (const int rc = check(cfg, false)) return rc;
    if (!sides_ok(rows, cols) || !pitch_ok(rows, cols, ld) || !operand || !dst) return DEMO_EINVAL;
    const uint64_t eb = elem_bytes(cfg->dtype);
    if (!aligned16(operand) || !aligned_to(dst, eb)) return DEMO_EALIGN;
    const demo_operand o = mx_operand_of(rows, cols);
    if (overlap(operand, o.total_bytes, dst, ((rows - 1) * ld + cols) * eb)) return DEMO_EINVAL;
    demo::MxValuesArgs a{};
    a.q = static_cast<const uint8_t*>(operand);
    a.s = a.q + o.scale_off;
    a.pitch = o.pitch;
    a.ld = ld;
    a.s_pitch = (uint32_t)o.scale_pitch;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.dst = dst;
    const bool wide = aligned16(dst) && ld * eb % 16 == 0 && cols % 8 == 0;
    const uint64_t blocks = (rows * ((cols + 7) / 8) + 255) / 256;
    const dim3 grid((unsigned)(blocks < (1u << 22) ? blocks : (1u << 22)));
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    return status_of(with_type(cfg->dtype, [&](auto type) {
        typedef decltype(type) T;
        return launch(wide ? demo::mx_values_kernel<T, true> : demo::mx_values_kernel<T, false>, grid, dim3(256), 0, s, a);
    }));
}

int demo_mx_workspace(const demo_mx_cfg* cfg, uint64_t m, uint64_t n, uint64_t k, uint64_t* bytes) {
    if (const int rc = check_product(cfg, m, n, k)) return rc;
    if (!bytes) return DEMO_EINVAL;
    const Plan plan = plan_of(m, n, k);
    *bytes = plan.splits > 1 ? plan.splits * m * n * 4 : 0;
    return DEMO_OK;
}

int demo_mx_matmul(const demo_mx_cfg* cfg, uint64_t m, uint64_t n, uint64_t k, const void* a, const void* b, void* c,
                   uint64_t ldc, const void* addend, uint64_t ld_addend, const demo_dropout_cfg* dropout,
                   void* workspace, uint64_t workspace_bytes, void* hip_stream) {
    if (const int rc = check_product(cfg, m, n, k)) return rc;
    if (!pitch_ok(m, n, ldc) || (addend && !pitch_ok(m, n, ld_addend))) return DEMO_EINVAL;
    demo::ProductArgs p{};
    if (const int rc = drop_of(dropout, m * n, &p.drop)) return rc;
    if (!a || !b || !c) return DEMO_EINVAL;
    const uint64_t eb = elem_bytes(cfg->dtype);
    if (!aligned16(a) || !aligned16(b) || !aligned_to(c, eb) || !aligned_to(addend, eb) || !aligned16(workspace))
        return DEMO_EALIGN;
    const demo_operand oa = mx_operand_of(m, k), ob = mx_operand_of(n, k);
    const uint64_t cb = ((m - 1) * ldc + n) * eb, db = addend ? ((m - 1) * ld_addend + n) * eb : 0;
    const bool in_place = addend == c && ld_addend == ldc;
    if (overlap(c, cb, a, oa.total_bytes) || overlap(c, cb, b, ob.total_bytes) || (!in_place && overlap(c, cb, addend, db)))
        return DEMO_EINVAL;
    const Plan plan = plan_of(m, n, k);
    const uint64_t need = plan.splits > 1 ? plan.splits * m * n * 4 : 0;
    if (need && (!workspace || workspace_bytes < need)) return DEMO_EINVAL;
    if (need && (overlap(workspace, need, a, oa.total_bytes) || overlap(workspace, need, b, ob.total_bytes) ||
                 overlap(workspace, need, c, cb) || overlap(workspace, need, addend, db)))
        return DEMO_EINVAL;
    p.a = static_cast<const uint8_t*>(a);
    p.b = static_cast<const uint8_t*>(b);
    p.sa = p.a + oa.scale_off;
    p.sb = p.b + ob.scale_off;
    p.m = (uint32_t)m;
    p.n = (uint32_t)n;
    p.kb = (uint32_t)(oa.pitch / demo::kStepK);
    p.pitch = (uint32_t)oa.pitch;
    p.s_pitch = (uint32_t)oa.scale_pitch;
    p.c = c;
    p.addend = addend;
    p.ldc = ldc;
    p.ld_addend = addend ? ld_addend : 0;
    p.dtype = cfg->dtype;
    p.wide = n % 8 == 0 && aligned16(c) && ldc * eb % 16 == 0 && aligned16(addend) && p.ld_addend * eb % 16 == 0;
    return status_of(launch_product(p, plan, workspace, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
