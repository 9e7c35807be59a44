// Checks that the block operators' entry points share (block_plan.cpp, linattn_plan.cpp): the launch
// description, strides, alignment, the extents of arrays and whether they meet, the workspace.
#ifndef VIMSCAN_CALL_CHECKS_H
#define VIMSCAN_CALL_CHECKS_H

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "vimscan.h"

namespace vimscan_host {

// Rows of a tile (128 at most) lie within the 2^31 bytes that one buffer resource's offsets span.
constexpr int64_t kMaxRowStride = int64_t(1) << 22;
constexpr int64_t kMaxTokens = int64_t(1) << 31;

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool positive(float v) { return std::isfinite(v) && v > 0.0f; }

// A byte range; a NULL pointer is an empty one.
struct Span {
    const void* p;
    size_t n;
};

// The whole extent of rows of width elements, ld elements apart.
inline Span rows_span(const void* p, int64_t rows, int64_t ld, int64_t width, size_t e) {
    if (!p || rows <= 0 || width <= 0) return {nullptr, 0};
    return {p, (static_cast<size_t>(rows - 1) * ld + width) * e};
}

inline Span dense_span(const void* p, int64_t rows, int64_t width, size_t e) { return rows_span(p, rows, width, width, e); }

inline bool meet(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// Whether two arrays of equally many rows of d elements of e bytes, ld_* elements apart, share an element. Slices of
// one array may be interleaved: their rows have the same distance and lie beside each other. (Of rows at different
// distances only the first ones are compared.)
inline bool rows_meet(const void* a, int64_t ld_a, const void* b, int64_t ld_b, int64_t rows, int64_t d, size_t e) {
    if (!meet(rows_span(a, rows, ld_a, d, e), rows_span(b, rows, ld_b, d, e))) return false;
    if (ld_a != ld_b) return meet(dense_span(a, 1, d, e), dense_span(b, 1, d, e));
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const size_t beside = (x > y ? x - y : y - x) % (static_cast<size_t>(ld_a) * e), row = static_cast<size_t>(d) * e;
    return beside < row || static_cast<size_t>(ld_a) * e - beside < row;
}

template <size_t N, size_t M>
inline bool any_meet(const Span (&a)[N], const Span (&b)[M]) {
    for (const Span& x : a)
        for (const Span& y : b)
            if (meet(x, y)) return true;
    return false;
}

// The checks that every launch of these operators shares.
inline int check_launch(const vimscan_launch* l, int64_t d_state, int32_t flags) {
    if (!l) return VIMSCAN_ERR_NULL;
    if (l->batch < 0 || l->seqlen < 0 || l->d_inner < 0 || l->d_state != d_state) return VIMSCAN_ERR_SHAPE;
    if (l->d_inner >= (int64_t(1) << 22)) return VIMSCAN_ERR_SHAPE;
    if (l->batch >= kMaxTokens || l->seqlen >= kMaxTokens || l->batch * l->seqlen >= kMaxTokens)
        return VIMSCAN_ERR_SHAPE;
    if (l->io_dtype != VIMSCAN_F32 && l->io_dtype != VIMSCAN_BF16) return VIMSCAN_ERR_DTYPE;
    if (l->chunk_len != 0) return VIMSCAN_ERR_CHUNK;
    if (l->flags & ~flags) return VIMSCAN_ERR_FLAGS;
    return VIMSCAN_OK;
}

inline size_t io_bytes(const vimscan_launch* l) { return l->io_dtype == VIMSCAN_F32 ? 4 : 2; }

inline bool good_stride(int64_t ld, int64_t d) { return ld >= d && ld < kMaxRowStride; }

// The workspace: there, large enough, aligned, apart from every array of the call.
template <size_t N, size_t M>
inline int check_workspace(const vimscan_launch* l, size_t need, const Span (&ins)[N], const Span (&outs)[M]) {
    if (need == 0) return VIMSCAN_OK;
    if (!l->workspace || l->workspace_bytes < need) return VIMSCAN_ERR_WORKSPACE;
    if (!is_aligned(l->workspace, 16)) return VIMSCAN_ERR_ALIGN;
    const Span w[] = {{l->workspace, need}};
    return any_meet(w, ins) || any_meet(w, outs) ? VIMSCAN_ERR_ALIAS : VIMSCAN_OK;
}

}  // namespace vimscan_host

#endif  // VIMSCAN_CALL_CHECKS_H
