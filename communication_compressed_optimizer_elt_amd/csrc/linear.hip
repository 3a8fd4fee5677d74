// linear.hip -- host side of the low-precision linear layer: dropout,
// block-scaled quantisation and the block-scaled matrix product.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "demo.h"
#include "host.hpp"
#include "product_big.hpp"
#include "quantize.hpp"

namespace {

using demo::aligned16;
using demo::launch;
using demo::overlap;
using demo::status_of;

constexpr uint64_t kMaxSide = (uint64_t)1 << 30;  // grids stay below 2^32 work-items, indices below 2^32

uint64_t up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }

uint64_t elem_bytes(uint32_t dtype) { return dtype == DEMO_DTYPE_F32 ? 4 : 2; }

bool aligned_to(const void* p, uint64_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool sides_ok(uint64_t rows, uint64_t cols) {
    return rows >= 1 && cols >= 1 && rows <= kMaxSide && cols <= kMaxSide && rows * cols <= DEMO_MAX_ELEMS;
}

// a row pitch that keeps every index of the matrix in 64 bits with room to spare
bool pitch_ok(uint64_t rows, uint64_t cols, uint64_t ld) {
    return ld >= cols && ld <= DEMO_MAX_ELEMS && rows - 1 <= ((uint64_t)1 << 40) / ld;
}

demo_operand operand_of(uint64_t rows, uint64_t cols) {
    demo_operand o{};
    o.pitch = up(cols, DEMO_BLOCK);
    o.scale_pitch = up(o.pitch / DEMO_BLOCK, 4);
    o.scale_off = demo::up256(rows * o.pitch);
    o.total_bytes = demo::up256(o.scale_off + rows * o.scale_pitch);
    return o;
}

// demo::Drop of a configuration for n elements, or an error code
int drop_of(const demo_dropout_cfg* cfg, uint64_t n, demo::Drop* d) {
    *d = demo::Drop{};
    if (!cfg) return DEMO_OK;
    if (cfg->abi_version != DEMO_ABI_VERSION) return DEMO_EABI;
    if (!(cfg->p >= 0.f && cfg->p <= 1.f) || cfg->site >= (1u << 24) || cfg->reserved != 0) return DEMO_EINVAL;
    const uint64_t last = (uint64_t)1 << 59;  // the element's number fits 64 bits
    if (cfg->chunk_offset > last || cfg->chunk_offset + (n + 31) / 32 > last) return DEMO_EINVAL;
    d->first = cfg->chunk_offset * (DEMO_CHUNK / 8);
    d->k0 = (uint32_t)cfg->seed;
    d->k1 = (uint32_t)(cfg->seed >> 32);
    d->step = (uint32_t)cfg->step;
    d->c3 = (demo::kTagDropout << 24) | cfg->site;
    d->threshold = (uint32_t)std::floor((double)cfg->p * 65536.0 + 0.5);
    d->scale = d->threshold == 65536u ? 0.f : (float)(65536.0 / (65536.0 - (double)d->threshold));
    d->on = 1;
    return DEMO_OK;
}

template <typename T>
hipError_t launch_dropout(const demo::DropoutArgs& a, hipStream_t s) {
    const uint64_t blocks = (a.n + 2047) / 2048;
    const dim3 grid((unsigned)(blocks < (1u << 22) ? blocks : (1u << 22)));
    return launch(a.residual ? demo::dropout_kernel<T, true> : demo::dropout_kernel<T, false>, grid, dim3(256), 0, s, a);
}

int dropout_impl(const demo_dropout_cfg* cfg, uint32_t dtype, uint64_t n, const void* x, const void* residual, void* y,
                 void* hip_stream) {
    if (!cfg) return DEMO_EINVAL;
    demo::DropoutArgs a{};
    if (n == 0 || n > DEMO_MAX_ELEMS) return DEMO_EINVAL;
    if (const int rc = drop_of(cfg, n, &a.drop)) return rc;
    if (dtype > DEMO_DTYPE_BF16 || !x || !y) return DEMO_EINVAL;
    if (!aligned16(x) || !aligned16(y) || (residual && !aligned16(residual))) return DEMO_EALIGN;
    const uint64_t nb = n * elem_bytes(dtype);
    if ((x != y && overlap(x, nb, y, nb)) || (residual != y && overlap(residual, nb, y, nb))) return DEMO_EINVAL;
    a.x = x;
    a.residual = residual;
    a.y = y;
    a.n = n;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    switch (dtype) {
    case DEMO_DTYPE_F32: return status_of(launch_dropout<float>(a, s));
    case DEMO_DTYPE_F16: return status_of(launch_dropout<demo::f16_t>(a, s));
    default: return status_of(launch_dropout<demo::bf16_t>(a, s));
    }
}

// least magnitude of a 16-bit type, as its bits, whose product with `scale` (0
// or at least 1) is infinite or NaN in fp32
uint32_t odd_from(uint32_t dtype, float scale) {
    if (dtype != DEMO_DTYPE_BF16) return 0x7C00u;  // fp16 times 65536 is far below fp32's largest
    const auto value = [](uint32_t u) {
        u <<= 16;
        float f;
        std::memcpy(&f, &u, 4);
        return f;
    };
    uint32_t u = 0x7F80u;
    while (u && !std::isfinite(value(u - 1) * scale)) u--;
    return u;
}

template <typename T, int FMT, bool TILE>
hipError_t launch_quantize(const demo::QuantArgs& a, bool wide, dim3 grid, hipStream_t s) {
    if (a.drop.on)
        return launch(wide ? demo::quantize_kernel<T, FMT, TILE, true, true> : demo::quantize_kernel<T, FMT, TILE, true, false>,
                      grid, dim3(256), 0, s, a);
    return launch(wide ? demo::quantize_kernel<T, FMT, TILE, false, true> : demo::quantize_kernel<T, FMT, TILE, false, false>,
                  grid, dim3(256), 0, s, a);
}

template <typename T>
hipError_t launch_quantize(const demo::QuantArgs& a, const demo_block_cfg* cfg, dim3 grid, hipStream_t s) {
    const bool wide = aligned16(a.src) && a.ld * sizeof(T) % 16 == 0 && a.cols % 8 == 0;
    if (cfg->fmt == DEMO_FMT_E4M3)
        return cfg->tile ? launch_quantize<T, demo::kE4M3, true>(a, wide, grid, s)
                         : launch_quantize<T, demo::kE4M3, false>(a, wide, grid, s);
    return cfg->tile ? launch_quantize<T, demo::kE5M2, true>(a, wide, grid, s)
                     : launch_quantize<T, demo::kE5M2, false>(a, wide, grid, s);
}

int check_product(const demo_product_cfg* cfg, uint64_t m, uint64_t n, uint64_t k) {
    if (!cfg) return DEMO_EINVAL;
    if (cfg->abi_version != DEMO_ABI_VERSION) return DEMO_EABI;
    if (cfg->fmt_a > DEMO_FMT_E5M2 || cfg->fmt_b > DEMO_FMT_E5M2 || cfg->dtype > DEMO_DTYPE_BF16) return DEMO_EINVAL;
    if (!sides_ok(m, n) || k < 1) return DEMO_EINVAL;
    if (k > DEMO_BLOCK_MAX_K) return DEMO_EUNSUPPORTED;
    if (!sides_ok(m, k) || !sides_ok(n, k)) return DEMO_EINVAL;
    return DEMO_OK;
}

// the kernels for few rows, and the columns that their grids hold (below 2^32
// work-items)
constexpr uint64_t kFewRows = 16, kFewRowsMaxCols = (uint64_t)1 << 22;

// How a product is cut: tiles of `tile` x `tile` and `splits` of the sum, or
// (tile 0) the kernels for few rows.
struct Plan {
    uint32_t tile;
    uint32_t splits;
    uint32_t kb_split;
};

// The card runs 256 tiles of 256 x 256 at a time, 512 of 128 x 128 or 1024 of 64
// x 64 (one, two and four workgroups a CU).  Measured, 16-bit result:
//  * a round of 256 tiles costs 1.6 to 1.8 rounds of 128 tiles (8192 x 2048 x
//    2048: 32.2 against 38.3 us; 6144 x 4096 x 2048, where the second round is
//    half empty: 56.3 against 53.9 us; 4096 x 2048 x 2048, half a round: 25.6
//    against 19.9 us), so they are taken where rounds say so at 1.65;
//  * up to 256 tiles of 128, tiles of 64 fill the card better (1024 x 2048 x
//    2048: 9.2 against 14.6 us; 2048 x 2048 x 2048, 256 tiles: 15.8 against 16.6
//    us, 24.1 against 28.7 us with an fp32 result); 16-bit results with a sum of
//    8192 or more up to 192 (2048 x 2048 x 8192: 54 against 53 us, but 75 against
//    85 us with an fp32 result);
//  * the sum is split where there are fewer than 512 workgroups: down to 16
//    blocks of 128 for tiles of 64 (256 x 2048 x 8192: 16.4 us in 4, 23.8 in one;
//    128 x 2048 x 2048: 7.6 us in one, 9.7 in 2), to 64 for tiles of 128 (2048 x
//    2048 x 16384: 80 us in 2, 90 in one).  Up to 1024 workgroups, which tiles of
//    64 would fill, measured no better: 512 x 2048 x 8192 23.7 us in 4, 23.9 in 2
//    (fp32 result: 28.9 and 26.6); 768 x 768 x 16384 28.0 us in 7, 29.8 in 3
//    (33.2 and 31.7).  Nor did 8 blocks: 256 x 2048 x 2048 11.6 us in 2, 10.1 in
//    one; 256 x 2048 x 8192 18.5 us in 8, 16.7 in 4.
// With an fp32 result a round of 256 tiles costs 1.75 to 1.87 of 128 (8192 x
// 8192 x 8192: 890 against 969 us; 4096 x 8192 x 2048: 148 against 158 us).
Plan plan_of(uint64_t m, uint64_t n, uint64_t k, bool wide) {
    const uint64_t kb = up(k, DEMO_BLOCK) / DEMO_BLOCK;
    if (m <= kFewRows && n <= kFewRowsMaxCols) return {0, 1, (uint32_t)kb};
    const auto tiles = [&](uint64_t t) { return up(m, t) / t * (up(n, t) / t); };
    const auto rounds = [](uint64_t count, uint64_t at_once) { return (count + at_once - 1) / at_once; };
    if (m >= 256 && n >= 256 && (wide ? 37 : 33) * rounds(tiles(256), 256) <= 20 * rounds(tiles(128), 512))
        return {256, 1, (uint32_t)up(kb, 4)};
    const uint64_t tile = tiles(128) > (kb >= 64 && !wide ? 192u : 256u) ? 128 : 64, least = tile == 128 ? 64 : 16;
    uint64_t splits = 512 / tiles(tile);
    if (splits > kb / least) splits = kb / least;
    if (splits < 1) splits = 1;
    const uint64_t each = up((kb + splits - 1) / splits, 4);
    return {(uint32_t)tile, (uint32_t)((kb + each - 1) / each), (uint32_t)each};
}
// the partial sums of up to 512 tiles of 128 x 128
static_assert(512 * 128 * 128 * 4 <= DEMO_BLOCK_MAX_WORKSPACE, "workspace");

template <int FA, int FB, bool WIDE, int TILE>
hipError_t launch_tiles(const demo::ProductArgs& a, dim3 grid, hipStream_t s) {
    const size_t lds = 2 * 2 * TILE * (DEMO_BLOCK + 4);
    if constexpr (WIDE && TILE == 64) return launch(demo::product_shared_kernel<FA, FB>, grid, dim3(256), lds, s, a);
    else return launch(demo::product_kernel<FA, FB, WIDE, TILE, TILE, 2, 2>, grid, dim3(256), lds, s, a);
}

template <int FA, int FB, bool WIDE>
hipError_t launch_product(demo::ProductArgs a, const Plan& plan, void* workspace, hipStream_t s) {
    if (plan.tile == 0) {
        if (a.m == 1) return launch(demo::product_rows_kernel<FA, FB, 1>, dim3((a.n + 3) / 4), dim3(256), 0, s, a);
        if (a.m == 2) return launch(demo::product_rows_kernel<FA, FB, 2>, dim3((a.n + 3) / 4), dim3(256), 0, s, a);
        return launch(demo::product_few_kernel<FA, FB, WIDE, 8>, dim3((a.n + 15) / 16), dim3(512), 0, s, a);
    }
    a.kb_split = plan.kb_split;
    a.partial = plan.splits > 1 ? static_cast<float*>(workspace) : nullptr;
    a.tiles_m = (a.m + plan.tile - 1) / plan.tile;
    a.tiles_n = (a.n + plan.tile - 1) / plan.tile;
    const dim3 grid(a.tiles_m * a.tiles_n, plan.splits);
    hipError_t e;
    if (plan.tile == 64) e = launch_tiles<FA, FB, WIDE, 64>(a, grid, s);
    else if (plan.tile == 128) e = launch_tiles<FA, FB, WIDE, 128>(a, grid, s);
    else if (WIDE) e = launch(demo::product_big_wide_kernel<FA, FB>, grid, dim3(512), demo::kBigLds, s, a);
    else e = launch(demo::product_big_kernel<FA, FB>, grid, dim3(256), demo::kBigLds, s, a);
    if (e != hipSuccess || plan.splits == 1) return e;
    const uint64_t blocks = ((uint64_t)a.m * ((a.n + 7) / 8) + 255) / 256;
    return launch(demo::product_join_kernel, dim3((unsigned)(blocks < (1u << 20) ? blocks : (1u << 20))), dim3(256), 0, s,
                  a, plan.splits);
}

template <int FA, int FB>
hipError_t launch_product(const demo::ProductArgs& a, const Plan& plan, void* workspace, hipStream_t s) {
    return a.dtype == DEMO_DTYPE_F32 ? launch_product<FA, FB, true>(a, plan, workspace, s)
                                     : launch_product<FA, FB, false>(a, plan, workspace, s);
}

}  // namespace

extern "C" {

int demo_dropout(const demo_dropout_cfg* cfg, uint32_t dtype, uint64_t n_elems, const void* x, const void* residual,
                 void* y, void* hip_stream) {
    return dropout_impl(cfg, dtype, n_elems, x, residual, y, hip_stream);
}

int demo_dropout_backward(const demo_dropout_cfg* cfg, uint32_t dtype, uint64_t n_elems, const void* dy, void* dx,
                          void* hip_stream) {
    return dropout_impl(cfg, dtype, n_elems, dy, nullptr, dx, hip_stream);
}

int demo_block_layout(uint64_t rows, uint64_t cols, demo_operand* out) {
    if (!out || !sides_ok(rows, cols)) return DEMO_EINVAL;
    *out = operand_of(rows, cols);
    return DEMO_OK;
}

int demo_block_quantize(const demo_block_cfg* cfg, uint64_t rows, uint64_t cols, const void* src, uint64_t ld,
                        const demo_dropout_cfg* dropout, void* operand, void* operand_t, void* hip_stream) {
    if (!cfg) return DEMO_EINVAL;
    if (cfg->abi_version != DEMO_ABI_VERSION) return DEMO_EABI;
    if (cfg->fmt > DEMO_FMT_E5M2 || cfg->tile > 1 || cfg->dtype > DEMO_DTYPE_BF16) return DEMO_EINVAL;
    if (!sides_ok(rows, cols) || !pitch_ok(rows, cols, ld)) return DEMO_EINVAL;
    demo::QuantArgs a{};
    if (const int rc = drop_of(dropout, rows * cols, &a.drop)) return rc;
    if (!src || (!operand && !operand_t)) return DEMO_EINVAL;
    const uint64_t eb = elem_bytes(cfg->dtype);
    if (!aligned_to(src, eb) || !aligned16(operand) || !aligned16(operand_t)) return DEMO_EALIGN;
    const demo_operand o = operand_of(rows, cols), t = operand_of(cols, rows);
    const uint64_t nb = ((rows - 1) * ld + cols) * eb;
    if (overlap(src, nb, operand, o.total_bytes) || overlap(src, nb, operand_t, t.total_bytes) ||
        overlap(operand, o.total_bytes, operand_t, t.total_bytes))
        return DEMO_EINVAL;
    a.src = src;
    a.ld = ld;
    a.odd_from = odd_from(cfg->dtype, a.drop.scale);
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    if (operand) {
        a.q = static_cast<uint8_t*>(operand);
        a.s = a.q + o.scale_off;
        a.pitch = o.pitch;
        a.s_pitch = (uint32_t)o.scale_pitch;
    }
    if (operand_t) {
        a.qt = static_cast<uint8_t*>(operand_t);
        a.st = a.qt + t.scale_off;
        a.pitch_t = t.pitch;
        a.s_pitch_t = (uint32_t)t.scale_pitch;
    }
    a.tiles_c = (uint32_t)(o.pitch / DEMO_BLOCK);
    const dim3 grid(a.tiles_c * (uint32_t)((rows + DEMO_BLOCK - 1) / DEMO_BLOCK));
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    switch (cfg->dtype) {
    case DEMO_DTYPE_F32: return status_of(launch_quantize<float>(a, cfg, grid, s));
    case DEMO_DTYPE_F16: return status_of(launch_quantize<demo::f16_t>(a, cfg, grid, s));
    default: return status_of(launch_quantize<demo::bf16_t>(a, cfg, grid, s));
    }
}

int demo_block_workspace(const demo_product_cfg* cfg, uint64_t m, uint64_t n, uint64_t k, uint64_t* bytes) {
    if (const int rc = check_product(cfg, m, n, k)) return rc;
    if (!bytes) return DEMO_EINVAL;
    const Plan plan = plan_of(m, n, k, cfg->dtype == DEMO_DTYPE_F32);
    *bytes = plan.splits > 1 ? plan.splits * m * n * 4 : 0;
    return DEMO_OK;
}

int demo_block_matmul(const demo_product_cfg* cfg, uint64_t m, uint64_t n, uint64_t k, const void* a, const void* b,
                      void* c, uint64_t ldc, const void* addend, uint64_t ld_addend, const demo_dropout_cfg* dropout,
                      void* workspace, uint64_t workspace_bytes, void* hip_stream) {
    if (const int rc = check_product(cfg, m, n, k)) return rc;
    if (!pitch_ok(m, n, ldc) || (addend && !pitch_ok(m, n, ld_addend))) return DEMO_EINVAL;
    demo::ProductArgs p{};
    if (const int rc = drop_of(dropout, m * n, &p.drop)) return rc;
    if (!a || !b || !c) return DEMO_EINVAL;
    const uint64_t eb = elem_bytes(cfg->dtype);
    if (!aligned16(a) || !aligned16(b) || !aligned_to(c, eb) || !aligned_to(addend, eb) || !aligned16(workspace))
        return DEMO_EALIGN;
    const demo_operand oa = operand_of(m, k), ob = operand_of(n, k);
    const uint64_t cb = ((m - 1) * ldc + n) * eb, db = addend ? ((m - 1) * ld_addend + n) * eb : 0;
    const bool in_place = addend == c && ld_addend == ldc;
    if (overlap(c, cb, a, oa.total_bytes) || overlap(c, cb, b, ob.total_bytes) || (!in_place && overlap(c, cb, addend, db)))
        return DEMO_EINVAL;
    uint64_t need = 0;
    if (const int rc = demo_block_workspace(cfg, m, n, k, &need)) return rc;
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
    p.kb = (uint32_t)(oa.pitch / DEMO_BLOCK);
    p.pitch = (uint32_t)oa.pitch;
    p.s_pitch = (uint32_t)oa.scale_pitch;
    p.c = c;
    p.addend = addend;
    p.ldc = ldc;
    p.ld_addend = addend ? ld_addend : 0;
    p.dtype = cfg->dtype;
    p.wide = n % 8 == 0 && aligned16(c) && ldc * eb % 16 == 0 && aligned16(addend) && p.ld_addend * eb % 16 == 0;
    const Plan plan = plan_of(m, n, k, cfg->dtype == DEMO_DTYPE_F32);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (cfg->fmt_a == DEMO_FMT_E4M3)
        return status_of(cfg->fmt_b == DEMO_FMT_E4M3 ? launch_product<demo::kE4M3, demo::kE4M3>(p, plan, workspace, s)
                                                     : launch_product<demo::kE4M3, demo::kE5M2>(p, plan, workspace, s));
    return status_of(cfg->fmt_b == DEMO_FMT_E4M3 ? launch_product<demo::kE5M2, demo::kE4M3>(p, plan, workspace, s)
                                                 : launch_product<demo::kE5M2, demo::kE5M2>(p, plan, workspace, s));
}

}  // extern "C"
