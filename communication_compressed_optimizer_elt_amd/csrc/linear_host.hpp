// linear_host.hpp -- what the entry points of the linear layer, of its norm and
// of its 4-bit form check alike: sizes, pitches, alignment, dropouts.
#pragma once

#include <cmath>
#include <cstdint>

#include "demo.h"
#include "dropout.hpp"
#include "host.hpp"

namespace demo {

constexpr uint64_t kMaxSide = (uint64_t)1 << 30;  // grids stay below 2^32 work-items, indices below 2^32

inline uint64_t up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }

inline uint64_t elem_bytes(uint32_t dtype) { return dtype == DEMO_DTYPE_F32 ? 4 : 2; }

inline bool aligned_to(const void* p, uint64_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool sides_ok(uint64_t rows, uint64_t cols) {
    return rows >= 1 && cols >= 1 && rows <= kMaxSide && cols <= kMaxSide && rows * cols <= DEMO_MAX_ELEMS;
}

// a row pitch that keeps every index of the matrix in 64 bits with room to spare
inline bool pitch_ok(uint64_t rows, uint64_t cols, uint64_t ld) {
    return ld >= cols && ld <= DEMO_MAX_ELEMS && rows - 1 <= ((uint64_t)1 << 40) / ld;
}

inline demo_operand operand_of(uint64_t rows, uint64_t cols) {
    demo_operand o{};
    o.pitch = up(cols, DEMO_BLOCK);
    o.scale_pitch = up(o.pitch / DEMO_BLOCK, 4);
    o.scale_off = up256(rows * o.pitch);
    o.total_bytes = up256(o.scale_off + rows * o.scale_pitch);
    return o;
}

// Drop of a configuration for n elements, or an error code
inline int drop_of(const demo_dropout_cfg* cfg, uint64_t n, Drop* d) {
    *d = Drop{};
    if (!cfg) return DEMO_OK;
    if (cfg->abi_version != DEMO_ABI_VERSION) return DEMO_EABI;
    if (!(cfg->p >= 0.f && cfg->p <= 1.f) || cfg->site >= (1u << 24) || cfg->reserved != 0) return DEMO_EINVAL;
    const uint64_t last = (uint64_t)1 << 59;  // the element's number fits 64 bits
    if (cfg->chunk_offset > last || cfg->chunk_offset + (n + 31) / 32 > last) return DEMO_EINVAL;
    d->first = cfg->chunk_offset * (DEMO_CHUNK / 8);
    d->k0 = (uint32_t)cfg->seed;
    d->k1 = (uint32_t)(cfg->seed >> 32);
    d->step = (uint32_t)cfg->step;
    d->c3 = (kTagDropout << 24) | cfg->site;
    d->threshold = (uint32_t)std::floor((double)cfg->p * 65536.0 + 0.5);
    d->scale = d->threshold == 65536u ? 0.f : (float)(65536.0 / (65536.0 - (double)d->threshold));
    d->on = 1;
    return DEMO_OK;
}

}  // namespace demo
