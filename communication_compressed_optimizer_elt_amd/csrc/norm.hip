// norm.hip -- host side of the root-mean-square norm.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "demo.h"
#include "linear_host.hpp"
#include "norm.hpp"

namespace {

using demo::aligned16;
using demo::aligned_to;
using demo::elem_bytes;
using demo::launch;
using demo::operand_of;
using demo::overlap;
using demo::pitch_ok;
using demo::sides_ok;
using demo::status_of;

int check(const demo_norm_cfg* cfg, uint64_t rows, uint64_t cols) {
    if (!cfg) return DEMO_EINVAL;
    if (cfg->abi_version != DEMO_ABI_VERSION) return DEMO_EABI;
    if (cfg->dtype > DEMO_DTYPE_BF16 || cfg->fmt > DEMO_FMT_E5M2) return DEMO_EINVAL;
    if (!(cfg->eps >= 0.f) || !std::isfinite(cfg->eps) || !sides_ok(rows, cols)) return DEMO_EINVAL;
    return cols > DEMO_NORM_MAX_COLS ? DEMO_EUNSUPPORTED : DEMO_OK;
}

// memory of a call: a matrix of rows with a pitch, or (ld 0) `bytes` of it
struct Span {
    const void* at;
    uint64_t ld, bytes;
};

// a matrix that is written may be one that is read, row by row in the same
// place; otherwise what is written meets nothing
template <size_t R, size_t W>
bool apart(const Span (&read)[R], const Span (&written)[W]) {
    for (size_t i = 0; i < W; i++) {
        for (const Span& r : read)
            if (overlap(written[i].at, written[i].bytes, r.at, r.bytes) &&
                !(written[i].ld && written[i].at == r.at && written[i].ld == r.ld))
                return false;
        for (size_t j = 0; j < i; j++)
            if (overlap(written[i].at, written[i].bytes, written[j].at, written[j].bytes)) return false;
    }
    return true;
}

// whether rows begin at aligned addresses, eight values at a time
bool rows_aligned(const Span& m, uint64_t eb) { return aligned16(m.at) && m.ld * eb % 16 == 0; }

template <int W, int NV>
struct Shape {
    static constexpr int kWaves = W, kVectors = NV;
};

// Waves that share a row: 512 columns each, and twice that for the longest rows.
template <typename F>
hipError_t with_shape(uint64_t cols, F f) {
    switch ((cols + 511) / 512) {
    case 1: return f(Shape<1, 1>());
    case 2: return f(Shape<2, 1>());
    case 3: return f(Shape<3, 1>());
    case 4: return f(Shape<4, 1>());
    case 5: return f(Shape<5, 1>());
    case 6: return f(Shape<6, 1>());
    case 7:
    case 8: return f(Shape<8, 1>());
    case 9:
    case 10: return f(Shape<10, 1>());
    case 11:
    case 12: return f(Shape<12, 1>());
    case 13:
    case 14:
    case 15:
    case 16: return f(Shape<16, 1>());
    default: return f(Shape<16, 2>());
    }
}
static_assert(DEMO_NORM_MAX_COLS == 16 * 2 * 512, "the longest row");

uint32_t grid_of(uint64_t rows, uint64_t each, uint32_t most) {
    const uint64_t blocks = (rows + each - 1) / each;
    return (uint32_t)(blocks < most ? blocks : most);
}

// The backward pass' workgroups, each with a sum for each column: two a CU, or
// one where a row is more than eight waves' (16384 x 2048 bf16: 53.2 us, 56 to 61
// with 384, 640 or 768 of them; 4096 x 8192: 57.4 us, 64 with 512).
constexpr uint32_t kBackGrid = 512;
template <typename S>
uint32_t back_grid(uint64_t rows) {
    return grid_of(rows, demo::kBackRows<S::kWaves>, S::kWaves <= 8 ? kBackGrid : kBackGrid / 2);
}
uint32_t back_grid(uint64_t rows, uint64_t cols) {
    uint32_t grid = 0;
    (void)with_shape(cols, [&](auto shape) {
        grid = back_grid<decltype(shape)>(rows);
        return hipSuccess;
    });
    return grid;
}
static_assert((uint64_t)kBackGrid * DEMO_NORM_MAX_COLS * 4 <= DEMO_BLOCK_MAX_WORKSPACE, "workspace");

// The forward pass' workgroups: up to six waves one for each row (or four rows of one
// wave), so that nothing is loaded ahead below a million of them; up to eight waves 4096,
// beyond 512.  Microseconds a call, bf16 with residual, h, y and r, of the same build with
// 1024, 2048, 4096, 8192 workgroups and one a row:
//   65536 x 1024   94    100   105   101   91
//   16384 x 2048   52.5  53.8  51.8  49.2  49.0
//   16384 x 4096   106   103   99    94.6  93.2
//   8192 x 3600    49.2  47.4  45.2  45.9  45.8
// and with 256, 512, 1024, 2048 and one a row:
//   4096 x 8192    48.7 49.3  51.0  53.0  57.0
//   16384 x 5120   117  130   138   130   124
//   4096 x 16384   99.4 98.0  98.1  98.4  100.6
template <typename T>
hipError_t launch_norm(const demo::NormArgs& a, bool wide, hipStream_t s) {
    return with_shape(a.cols, [&](auto shape) {
        typedef decltype(shape) S;
        constexpr int W = S::kWaves, NV = S::kVectors;
        return launch(wide ? demo::norm_kernel<T, W, NV, true> : demo::norm_kernel<T, W, NV, false>,
                      dim3(grid_of(a.rows, demo::kNormWaves<W> / W, W <= 6 ? 1u << 20 : W <= 8 ? 4096 : 512)),
                      dim3(64 * demo::kNormWaves<W>), 0, s, a);
    });
}

template <typename T>
hipError_t launch_turn(const demo::NormTurnArgs& a, uint32_t fmt, bool wide, hipStream_t s) {
    // below 2^32 work-items: the most of 256 are 16519106 workgroups, of DEMO_MAX_ELEMS / 65 rows of 65 columns
    const dim3 grid(a.tiles_c * ((a.rows + DEMO_BLOCK - 1) / DEMO_BLOCK));
    if (fmt == DEMO_FMT_E4M3)
        return launch(wide ? demo::norm_turn_kernel<T, demo::kE4M3, true> : demo::norm_turn_kernel<T, demo::kE4M3, false>,
                      grid, dim3(256), 0, s, a);
    return launch(wide ? demo::norm_turn_kernel<T, demo::kE5M2, true> : demo::norm_turn_kernel<T, demo::kE5M2, false>,
                  grid, dim3(256), 0, s, a);
}

template <typename T>
hipError_t launch_back(const demo::NormBackArgs& a, bool wide, hipStream_t s) {
    return with_shape(a.cols, [&](auto shape) {
        typedef decltype(shape) S;
        constexpr int W = S::kWaves, NV = S::kVectors;
        return launch(wide ? demo::norm_back_kernel<T, W, NV, true> : demo::norm_back_kernel<T, W, NV, false>,
                      dim3(back_grid<S>(a.rows)), dim3(64 * W * demo::kBackRows<W>), 0, s, a);
    });
}

template <typename F>
hipError_t with_type(uint32_t dtype, F f) {
    switch (dtype) {
    case DEMO_DTYPE_F32: return f(0.f);
    case DEMO_DTYPE_F16: return f((demo::f16_t)0);
    default: return f((demo::bf16_t)0);
    }
}

}  // namespace

extern "C" {

int demo_rms_norm(const demo_norm_cfg* cfg, uint64_t rows, uint64_t cols, const void* x, uint64_t ld_x,
                  const void* residual, uint64_t ld_residual, const float* weight, void* h, uint64_t ld_h, void* y,
                  uint64_t ld_y, float* rstd, void* operand, void* operand_t, void* hip_stream) {
    if (const int rc = check(cfg, rows, cols)) return rc;
    if (!pitch_ok(rows, cols, ld_x) || (residual && !pitch_ok(rows, cols, ld_residual)) ||
        (h && !pitch_ok(rows, cols, ld_h)) || (y && !pitch_ok(rows, cols, ld_y)))
        return DEMO_EINVAL;
    if (!x || !weight || (!h && !y && !rstd && !operand && !operand_t)) return DEMO_EINVAL;
    if (operand_t && (!rstd || (residual && !h))) return DEMO_EINVAL;
    const uint64_t eb = elem_bytes(cfg->dtype);
    if (!aligned_to(x, eb) || !aligned_to(residual, eb) || !aligned_to(h, eb) || !aligned_to(y, eb) ||
        !aligned_to(weight, 4) || !aligned_to(rstd, 4) || !aligned16(operand) || !aligned16(operand_t))
        return DEMO_EALIGN;
    const auto matrix = [&](const void* p, uint64_t ld) {
        return Span{p, p ? ld : 0, p ? ((rows - 1) * ld + cols) * eb : 0};
    };
    const demo_operand o = operand_of(rows, cols), ot = operand_of(cols, rows);
    const Span read[] = {matrix(x, ld_x), matrix(residual, ld_residual), {weight, 0, 4 * cols}};
    const Span written[] = {matrix(h, ld_h),
                            matrix(y, ld_y),
                            {rstd, 0, rstd ? 4 * rows : 0},
                            {operand, 0, operand ? o.total_bytes : 0},
                            {operand_t, 0, operand_t ? ot.total_bytes : 0}};
    if (!apart(read, written)) return DEMO_EINVAL;
    if (operand_t && !h && y == x) return DEMO_EINVAL;  // x is read again
    demo::NormArgs a{};
    a.x = x;
    a.res = residual;
    a.w = weight;
    a.h = h;
    a.y = y;
    a.rstd = rstd;
    a.ld_x = ld_x;
    a.ld_res = ld_residual;
    a.ld_h = ld_h;
    a.ld_y = ld_y;
    a.fmt = cfg->fmt;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.eps = cfg->eps;
    if (operand) {
        a.q = static_cast<uint8_t*>(operand);
        a.s = a.q + o.scale_off;
        a.pitch = o.pitch;
        a.s_pitch = (uint32_t)o.scale_pitch;
    }
    const bool wide = cols % 8 == 0 && aligned16(weight) && rows_aligned(read[0], eb) && rows_aligned(read[1], eb) &&
                      rows_aligned(written[0], eb) && rows_aligned(written[1], eb);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    return status_of(with_type(cfg->dtype, [&](auto type) {
        typedef decltype(type) T;
        const hipError_t e = launch_norm<T>(a, wide, s);
        if (e != hipSuccess || !operand_t) return e;
        demo::NormTurnArgs t{};
        t.h = h ? h : x;
        t.w = weight;
        t.rstd = rstd;
        t.qt = static_cast<uint8_t*>(operand_t);
        t.st = t.qt + ot.scale_off;
        t.ld_h = h ? ld_h : ld_x;
        t.pitch_t = ot.pitch;
        t.s_pitch_t = (uint32_t)ot.scale_pitch;
        t.rows = a.rows;
        t.cols = a.cols;
        t.tiles_c = (a.cols + 63) / 64;
        return launch_turn<T>(t, cfg->fmt, wide && aligned16(rstd), s);
    }));
}

int demo_rms_norm_workspace(const demo_norm_cfg* cfg, uint64_t rows, uint64_t cols, uint64_t* bytes) {
    if (const int rc = check(cfg, rows, cols)) return rc;
    if (!bytes) return DEMO_EINVAL;
    *bytes = back_grid(rows, cols) * cols * 4;
    return DEMO_OK;
}

int demo_rms_norm_backward(const demo_norm_cfg* cfg, uint64_t rows, uint64_t cols, const void* dy, uint64_t ld_dy,
                           const void* h, uint64_t ld_h, const float* weight, const float* rstd, const void* dresidual,
                           uint64_t ld_dresidual, void* dx, uint64_t ld_dx, float* dweight, const float* addend,
                           void* workspace, uint64_t workspace_bytes, void* hip_stream) {
    if (const int rc = check(cfg, rows, cols)) return rc;
    if (!pitch_ok(rows, cols, ld_dy) || !pitch_ok(rows, cols, ld_h) || !pitch_ok(rows, cols, ld_dx) ||
        (dresidual && !pitch_ok(rows, cols, ld_dresidual)))
        return DEMO_EINVAL;
    if (!dy || !h || !weight || !rstd || !dx || (addend && !dweight)) return DEMO_EINVAL;
    const uint64_t eb = elem_bytes(cfg->dtype);
    if (!aligned_to(dy, eb) || !aligned_to(h, eb) || !aligned_to(dresidual, eb) || !aligned_to(dx, eb) ||
        !aligned_to(weight, 4) || !aligned_to(rstd, 4) || !aligned_to(dweight, 4) || !aligned_to(addend, 4) ||
        !aligned16(workspace))
        return DEMO_EALIGN;
    const uint64_t grid = back_grid(rows, cols), need = dweight ? grid * cols * 4 : 0;
    if (need && (!workspace || workspace_bytes < need)) return DEMO_EINVAL;
    const auto matrix = [&](const void* p, uint64_t ld) {
        return Span{p, p ? ld : 0, p ? ((rows - 1) * ld + cols) * eb : 0};
    };
    // the weight's gradient may be its addend: both are vectors, rows of pitch `cols`
    const Span read[] = {matrix(dy, ld_dy),          matrix(h, ld_h),     matrix(dresidual, ld_dresidual),
                         {weight, 0, 4 * cols},      {rstd, 0, 4 * rows}, {addend, addend ? cols : 0, addend ? 4 * cols : 0}};
    const Span written[] = {matrix(dx, ld_dx), {dweight, dweight ? cols : 0, dweight ? 4 * cols : 0}, {workspace, 0, need}};
    if (!apart(read, written) || (dweight && (const void*)dweight == dy) || (dweight && (const void*)dweight == h) ||
        (dweight && (const void*)dweight == dresidual) || (addend && (const void*)addend == dx))
        return DEMO_EINVAL;
    demo::NormBackArgs a{};
    a.dy = dy;
    a.h = h;
    a.dres = dresidual;
    a.w = weight;
    a.rstd = rstd;
    a.dx = dx;
    a.partial = need ? static_cast<float*>(workspace) : nullptr;
    a.ld_dy = ld_dy;
    a.ld_h = ld_h;
    a.ld_dres = ld_dresidual;
    a.ld_dx = ld_dx;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    const bool wide = cols % 8 == 0 && aligned16(weight) && rows_aligned(read[0], eb) && rows_aligned(read[1], eb) &&
                      rows_aligned(read[2], eb) && rows_aligned(written[0], eb);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const hipError_t e = with_type(cfg->dtype, [&](auto type) { return launch_back<decltype(type)>(a, wide, s); });
    if (e != hipSuccess || !need) return status_of(e);
    return status_of(launch(demo::norm_join_kernel, dim3((a.cols + demo::kJoinCols - 1) / demo::kJoinCols), dim3(1024), 0, s, a.partial,
                            (uint32_t)grid, a.cols, addend, dweight));
}

}  // extern "C"
