// grad.hip -- host side of the gradient's norm and clipping.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "demo.h"
#include "grad.hpp"
#include "linear_host.hpp"

namespace {

using demo::aligned16;
using demo::aligned_to;
using demo::elem_bytes;
using demo::GradArgs;
using demo::kTable;
using demo::launch;
using demo::overlap;
using demo::status_of;

// Copies up to this many bytes stay in the caches for who reads them next,
// larger ones go past them.
constexpr uint64_t kCached = (uint64_t)96 << 20;

// A list of at most this many elements is one workgroup's, without partial sums:
// norm and copy of 65536 11.7 us, of 131072 14.4 us (16.6 by one workgroup).
constexpr uint64_t kSmall = 1u << 16;

int check(uint32_t count, const demo_tensor* t) {
    if (count > DEMO_MAX_TENSORS || (count && !t)) return DEMO_EINVAL;
    for (uint32_t i = 0; i < count; i++) {
        if (t[i].dtype > DEMO_DTYPE_BF16 || t[i].reserved != 0 || t[i].n_elems > DEMO_MAX_ELEMS) return DEMO_EINVAL;
        if (t[i].n_elems && !t[i].data) return DEMO_EINVAL;
        if (!aligned_to(t[i].data, elem_bytes(t[i].dtype))) return DEMO_EALIGN;
    }
    return DEMO_OK;
}

uint64_t bytes_of(const demo_tensor& t) { return t.n_elems * elem_bytes(t.dtype); }

// Elements of a chunk, which is a wave's: as few as 2048, but no more than `most`
// chunks where `most` allows that many, and below 2^31 of them.
uint32_t chunk_of(uint64_t elems, uint64_t most) {
    uint64_t chunk = 2048;
    while (elems / chunk >= most) chunk *= 2;
    return (uint32_t)chunk;
}
// The norm's sums, one for four chunks, are added up by one workgroup: 32768
// chunks (44 tensors of 268 million bf16: 349 us with the copy, 359 and 353 with
// half and twice as many).  The copy has none: 2048 elements a wave (640 million
// fp32 794 us, 882 in chunks of four times that).
constexpr uint64_t kNormChunks = 1 << 15, kScaleChunks = 1 << 22;

// f(arguments, their number of elements) for every launch: up to kTable tensors that hold something
template <typename F>
int each_launch(uint32_t count, const demo_tensor* src, const demo_tensor* dst, uint64_t most, F f) {
    for (uint32_t i = 0; i < count;) {
        GradArgs a;
        a.count = 0;
        uint64_t elems = 0;
        uint32_t from = i;
        for (; i < count && a.count < kTable; i++) {
            if (!src[i].n_elems) continue;
            elems += src[i].n_elems;
            a.count++;
        }
        if (!a.count) continue;
        a.chunk = chunk_of(elems, most);
        a.count = 0;
        uint64_t chunks = 0;
        for (; from < i; from++) {
            const demo_tensor &x = src[from], &y = dst ? dst[from] : x;
            if (!x.n_elems) continue;
            const uint32_t k = a.count++;
            a.src[k] = x.data;
            a.dst[k] = y.data;
            a.n[k] = x.n_elems;
            a.first[k] = (uint32_t)chunks;
            a.kind[k] = x.dtype | y.dtype << 2 | (aligned16(x.data) && aligned16(y.data) ? 16u : 0u);
            chunks += (x.n_elems + a.chunk - 1) / a.chunk;
        }
        a.chunks = (uint32_t)chunks;
        if (const int rc = f(a, elems)) return rc;
    }
    return DEMO_OK;
}

uint32_t grid_of(uint32_t chunks) { return (chunks + 3) / 4; }  // workgroups of four waves

// sums of a norm's workgroups over all its launches; 0: one workgroup does it all
uint64_t sums_of(uint32_t count, const demo_tensor* t) {
    uint64_t sums = 0, total = 0;
    uint32_t launches = 0;
    for (uint32_t i = 0; i < count; launches++) {
        uint64_t elems = 0, chunks = 0;
        uint32_t from = i, held = 0;
        for (; i < count && held < kTable; i++)
            if (t[i].n_elems) elems += t[i].n_elems, held++;
        const uint32_t chunk = chunk_of(elems, kNormChunks);
        for (; from < i; from++) chunks += (t[from].n_elems + chunk - 1) / chunk;
        sums += grid_of((uint32_t)chunks);
        total += elems;
    }
    return launches <= 1 && total <= kSmall ? 0 : sums;
}

// whether what is written meets anything else that is read or written; a
// tensor may be its own destination
int disjoint(uint32_t count, const demo_tensor* src, const demo_tensor* dst, const void* sumsq, const float* norm) {
    // The usual calls need no sorting: pieces that ascend, in place or all of them
    // away from what is read.
    uintptr_t end = 0, first = UINTPTR_MAX, src_first = UINTPTR_MAX, src_end = 0;
    bool ascending = true, in_place = true;
    for (uint32_t i = 0; i < count; i++) {
        if (!dst[i].n_elems) continue;
        const uintptr_t d = (uintptr_t)dst[i].data, s = (uintptr_t)src[i].data;
        ascending = ascending && d >= end;
        in_place = in_place && d == s;
        first = std::min(first, d);
        end = d + bytes_of(dst[i]);
        src_first = std::min(src_first, s);
        src_end = std::max(src_end, s + bytes_of(src[i]));
    }
    const auto apart = [](uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) { return a1 <= b0 || b1 <= a0; };
    const uintptr_t q = (uintptr_t)sumsq, r = (uintptr_t)norm;
    if (ascending && (in_place || apart(first, end, src_first, src_end)) && apart(first, end, q, q + 8) &&
        (!norm || (apart(first, end, r, r + 4) && apart(src_first, src_end, r, r + 4) && apart(q, q + 8, r, r + 4))))
        return DEMO_OK;
    struct Span {
        uintptr_t from, to;
        bool written;
    };
    try {
        std::vector<Span> spans;
        spans.reserve(2 * (size_t)count + 2);
        const auto add = [&](const void* p, uint64_t n, bool written) {
            if (n) spans.push_back({(uintptr_t)p, (uintptr_t)p + n, written});
        };
        for (uint32_t i = 0; i < count; i++) {
            add(dst[i].data, bytes_of(dst[i]), true);
            if (src[i].data != dst[i].data) add(src[i].data, bytes_of(src[i]), false);
        }
        add(sumsq, sizeof(double), false);
        if (norm) add(norm, sizeof(float), true);
        std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.from < b.from; });
        uintptr_t read = 0, written = 0;  // how far what begins before reaches
        for (const Span& s : spans) {
            if (s.from < written || (s.written && s.from < read)) return DEMO_EINVAL;
            (s.written ? written : read) = std::max(s.written ? written : read, s.to);
        }
    } catch (const std::bad_alloc&) {
        return DEMO_EINVAL;
    }
    return DEMO_OK;
}

}  // namespace

extern "C" {

int demo_grad_workspace(uint32_t count, const demo_tensor* tensors, uint64_t* bytes) {
    if (const int rc = check(count, tensors)) return rc;
    if (!bytes) return DEMO_EINVAL;
    *bytes = sums_of(count, tensors) * sizeof(double);
    return DEMO_OK;
}

int demo_grad_norm(uint32_t count, const demo_tensor* tensors, double* sumsq, void* workspace,
                   uint64_t workspace_bytes, void* hip_stream) {
    if (const int rc = check(count, tensors)) return rc;
    if (!sumsq) return DEMO_EINVAL;
    if (!aligned_to(sumsq, 8) || !aligned16(workspace)) return DEMO_EALIGN;
    const uint64_t sums = sums_of(count, tensors), need = sums * sizeof(double);
    if (need && (!workspace || workspace_bytes < need || overlap(workspace, need, sumsq, 8))) return DEMO_EINVAL;
    for (uint32_t i = 0; i < count; i++)
        if (overlap(sumsq, 8, tensors[i].data, bytes_of(tensors[i])) ||
            overlap(workspace, need, tensors[i].data, bytes_of(tensors[i])))
            return DEMO_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    double* partial = need ? static_cast<double*>(workspace) : sumsq;
    bool any = false;
    const int rc = each_launch(count, tensors, nullptr, kNormChunks, [&](GradArgs& a, uint64_t) {
        any = true;
        a.partial = partial;
        partial += grid_of(a.chunks);
        return status_of(need ? launch(demo::grad_norm_kernel<4>, dim3(grid_of(a.chunks)), dim3(256), 0, s, a)
                              : launch(demo::grad_norm_kernel<16>, dim3(1), dim3(1024), 0, s, a));
    });
    if (rc || (any && !need)) return rc;
    return status_of(launch(demo::grad_join_kernel, dim3(1), dim3(1024), 0, s, static_cast<const double*>(workspace),
                            (uint32_t)sums, sumsq));
}

int demo_grad_clip(uint32_t count, const demo_tensor* src, const demo_tensor* dst, const double* sumsq, double max_norm,
                   float* norm, void* hip_stream) {
    if (!dst) dst = src;
    if (const int rc = check(count, src)) return rc;
    if (const int rc = check(count, dst)) return rc;
    for (uint32_t i = 0; i < count; i++)
        if (dst[i].n_elems != src[i].n_elems || (dst[i].dtype != src[i].dtype && dst[i].dtype != DEMO_DTYPE_F32) ||
            (dst[i].data == src[i].data && dst[i].dtype != src[i].dtype && src[i].n_elems))
            return DEMO_EINVAL;
    if (!sumsq || !(max_norm >= 0)) return DEMO_EINVAL;
    if (!aligned_to(sumsq, 8) || !aligned_to(norm, 4)) return DEMO_EALIGN;
    if (const int rc = disjoint(count, src, dst, sumsq, norm)) return rc;
    uint64_t bytes = 0;
    for (uint32_t i = 0; i < count; i++) bytes += bytes_of(dst[i]);
    const bool past = bytes > kCached;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const auto go = [&](GradArgs& a) {
        a.sumsq = sumsq;
        a.max_norm = max_norm;
        a.norm = norm;
        norm = nullptr;  // the first launch writes it
        return status_of(launch(past ? demo::grad_scale_kernel<true> : demo::grad_scale_kernel<false>,
                                dim3(std::max(grid_of(a.chunks), 1u)), dim3(256), 0, s, a));
    };
    if (const int rc = each_launch(count, src, dst, kScaleChunks, [&](GradArgs& a, uint64_t) { return go(a); })) return rc;
    if (!norm) return DEMO_OK;
    GradArgs a{};  // no tensor holds anything: the norm alone
    return go(a);
}

}  // extern "C"
