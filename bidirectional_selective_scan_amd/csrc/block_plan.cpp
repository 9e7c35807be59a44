// Host side of the gated recurrence and the block norm (see block_plan.h).

#include "block_plan.h"

#include <cmath>
#include <cstring>

namespace vimscan_host {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 31;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool positive(float v) { return std::isfinite(v) && v > 0.0f; }

// A byte range; a NULL pointer is an empty one.
struct Span {
    const void* p;
    size_t n;
};

// The whole extent of rows of width elements, ld elements apart.
Span rows_span(const void* p, int64_t rows, int64_t ld, int64_t width, size_t e) {
    if (!p || rows <= 0 || width <= 0) return {nullptr, 0};
    return {p, (static_cast<size_t>(rows - 1) * ld + width) * e};
}

Span dense_span(const void* p, int64_t rows, int64_t width, size_t e) { return rows_span(p, rows, width, width, e); }

bool meet(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// Whether two arrays of equally many rows of d elements of e bytes, ld_* elements apart, share an element. Slices of
// one array may be interleaved: their rows have the same distance and lie beside each other. (Of rows at different
// distances only the first ones are compared.)
bool rows_meet(const void* a, int64_t ld_a, const void* b, int64_t ld_b, int64_t rows, int64_t d, size_t e) {
    if (!meet(rows_span(a, rows, ld_a, d, e), rows_span(b, rows, ld_b, d, e))) return false;
    if (ld_a != ld_b) return meet(dense_span(a, 1, d, e), dense_span(b, 1, d, e));
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const size_t beside = (x > y ? x - y : y - x) % (static_cast<size_t>(ld_a) * e), row = static_cast<size_t>(d) * e;
    return beside < row || static_cast<size_t>(ld_a) * e - beside < row;
}

template <size_t N, size_t M>
bool any_meet(const Span (&a)[N], const Span (&b)[M]) {
    for (const Span& x : a)
        for (const Span& y : b)
            if (meet(x, y)) return true;
    return false;
}

// The checks that every launch of these operators shares.
int check_launch(const vimscan_launch* l, int64_t d_state, int32_t flags) {
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

size_t io_bytes(const vimscan_launch* l) { return l->io_dtype == VIMSCAN_F32 ? 4 : 2; }

bool good_stride(int64_t ld, int64_t d) { return ld >= d && ld < kMaxRowStride; }

// The workspace: there, large enough, aligned, apart from every array of the call.
template <size_t N, size_t M>
int check_workspace(const vimscan_launch* l, size_t need, const Span (&ins)[N], const Span (&outs)[M]) {
    if (need == 0) return VIMSCAN_OK;
    if (!l->workspace || l->workspace_bytes < need) return VIMSCAN_ERR_WORKSPACE;
    if (!is_aligned(l->workspace, 16)) return VIMSCAN_ERR_ALIGN;
    const Span w[] = {{l->workspace, need}};
    return any_meet(w, ins) || any_meet(w, outs) ? VIMSCAN_ERR_ALIAS : VIMSCAN_OK;
}

// Tile of the forward pass. Long tiles hand on half as often and share the work per tile among twice the
// elements; short ones give more and lighter workgroups. Measured (bf16, us, 128 / 64 tokens): sequences
// of 65537 x 1536 188 / 235, 16384 x 768 29.0 / 38.3, 512 x 197 x 768 125 / 131; but 1 x 1024 x 768
// 9.3 / 6.9, 128 x 197 x 384 23.1 / 21.3, 4 x 1025 x 768 12.9 / 11.3 and, where sequences end with
// the tile, 1024 x 64 x 768 85 / 76. Near its border the rule can be a few percent off: 8 x 1025 x 768 takes 64
// tokens, 16.0 / 17.0. In fp32 the same shapes choose alike.
int64_t fwd_tile(int64_t tokens, int64_t length, int64_t ncb) {
    const int64_t wgs = (tokens + kGatedFwdTile - 1) / kGatedFwdTile * ncb;
    return length <= kGatedFwdTileSmall || (length <= 2048 && wgs < 2048) ? kGatedFwdTileSmall : kGatedFwdTile;
}

// Rows of D channels that a workgroup of a block norm works on at once.
template <size_t N>
int64_t rows_at_once(const NormSpread (&spreads)[N], int64_t D) {
    for (const NormSpread& s : spreads)
        if (D <= s.width()) return s.rows();
    return 1;
}

}  // namespace

int make_gated_plan(const vimscan_launch* l, int64_t seg_len, bool packed, int64_t nseq, bool backward, GatedPlan* p) {
    const int rc = check_launch(l, 1, VIMSCAN_FLAG_REVERSE);
    if (rc != VIMSCAN_OK) return rc;
    if (seg_len < 0 || (seg_len > 0 && l->seqlen % seg_len != 0)) return VIMSCAN_ERR_SEGLEN;
    if (packed && seg_len != 0) return VIMSCAN_ERR_PARAM;
    if (packed && (nseq < 0 || nseq >= kMaxTokens)) return VIMSCAN_ERR_SHAPE;
    std::memset(p, 0, sizeof(*p));
    p->packed = packed;
    p->tokens = l->batch * l->seqlen;
    if (packed && nseq == 0 && p->tokens > 0) return VIMSCAN_ERR_SHAPE;
    p->Lp = packed ? 0 : (seg_len > 0 ? seg_len : l->seqlen);
    // uniform sequences of no tokens: one per batch row
    p->nseq = packed ? nseq : (p->tokens > 0 ? p->tokens / p->Lp : l->batch);
    if (l->d_inner == 0 || p->nseq == 0) return VIMSCAN_OK;
    p->ncb = (l->d_inner + kGatedBlock - 1) / kGatedBlock;
    p->tile = backward ? kGatedBwdTile : fwd_tile(p->tokens, p->packed ? (p->tokens + nseq - 1) / nseq : p->Lp, p->ncb);
    // a call without tokens still writes the states of its empty sequences
    p->tiles = p->tokens > 0 ? (p->tokens + p->tile - 1) / p->tile : 1;
    if (p->tiles > kMaxGatedWgs / p->ncb) return VIMSCAN_ERR_SHAPE;
    p->wgs = p->tiles * p->ncb;
    p->groups = (p->tiles + kGatedGroup - 1) / kGatedGroup;
    // no sequence crosses a tile boundary: nothing to hand on
    p->chain = p->tiles > 1 && (packed || p->tile % p->Lp != 0);
    const size_t width = static_cast<size_t>(p->ncb) * kGatedBlock;
    if (p->chain) {
        p->off_inc = up256(static_cast<size_t>(p->tiles) * width * 2 * sizeof(uint64_t));
        p->off_part = p->off_inc + up256(static_cast<size_t>(p->groups) * width * 2 * sizeof(uint64_t));
        p->ws = p->off_part;
    }
    if (backward && p->tokens > 0) p->ws += up256(static_cast<size_t>(p->tiles) * width * sizeof(float));
    return VIMSCAN_OK;
}

int check_gated_call(const vimscan_gated* g, const void* y, const float* h_last, const float* states,
                     const vimscan_gated_grad* grad, const vimscan_launch* l, const GatedPlan& p) {
    const int64_t n = p.tokens, d = l->d_inner;
    const size_t e = io_bytes(l);
    if (!positive(g->c)) return VIMSCAN_ERR_PARAM;
    if (!good_stride(g->ld_x, d) || !good_stride(g->ld_r, d) || !good_stride(g->ld_i, d)) return VIMSCAN_ERR_PARAM;
    if (grad && (!good_stride(grad->ld_dx, d) || (grad->dy && !good_stride(grad->ld_dy, d)) ||
                 (grad->dr && !good_stride(grad->ld_dr, d)) || (grad->di && !good_stride(grad->ld_di, d))))
        return VIMSCAN_ERR_PARAM;
    if (!g->lam && (n > 0 || (grad && grad->dlam))) return VIMSCAN_ERR_NULL;
    if (n > 0) {
        if (!g->x || !g->r || !g->i) return VIMSCAN_ERR_NULL;
        if (grad ? (!grad->states || !grad->dx) : !y) return VIMSCAN_ERR_NULL;
    }
    const void* io[] = {g->x, g->r, g->i, y, grad ? grad->dy : nullptr, grad ? grad->dx : nullptr,
                        grad ? grad->dr : nullptr, grad ? grad->di : nullptr};
    for (const void* q : io)
        if (!is_aligned(q, e)) return VIMSCAN_ERR_ALIGN;
    const void* w4[] = {g->lam, g->h0, g->offsets, h_last, states, grad ? grad->dh_last : nullptr,
                        grad ? grad->states : nullptr, grad ? grad->dlam : nullptr, grad ? grad->dh0 : nullptr};
    for (const void* q : w4)
        if (!is_aligned(q, 4)) return VIMSCAN_ERR_ALIGN;
    const int64_t groups = (n + kGatedStride - 1) / kGatedStride;
    const Span none = {nullptr, 0};
    const Span ins[] = {rows_span(g->x, n, g->ld_x, d, e),
                        rows_span(g->r, n, g->ld_r, d, e),
                        rows_span(g->i, n, g->ld_i, d, e),
                        dense_span(g->lam, 1, d, 4),
                        dense_span(g->h0, p.nseq, d, 4),
                        p.packed ? dense_span(g->offsets, p.nseq + 1, 1, 4) : none,
                        grad ? rows_span(grad->dy, n, grad->ld_dy, d, e) : none,
                        grad ? dense_span(grad->dh_last, p.nseq, d, 4) : none,
                        grad ? dense_span(grad->states, groups, d, 4) : none};
    if (!grad) {
        const Span outs[] = {dense_span(y, n, d, e), dense_span(h_last, p.nseq, d, 4), dense_span(states, groups, d, 4)};
        if (any_meet(outs, ins) || meet(outs[0], outs[1]) || meet(outs[0], outs[2]) || meet(outs[1], outs[2]))
            return VIMSCAN_ERR_ALIAS;
        return check_workspace(l, p.ws, ins, outs);
    }
    const Span outs[] = {rows_span(grad->dx, n, grad->ld_dx, d, e), rows_span(grad->dr, n, grad->ld_dr, d, e),
                         rows_span(grad->di, n, grad->ld_di, d, e), dense_span(grad->dlam, 1, d, 4),
                         dense_span(grad->dh0, p.nseq, d, 4)};
    if (any_meet(outs, ins) || meet(outs[3], outs[4])) return VIMSCAN_ERR_ALIAS;
    if (rows_meet(grad->dx, grad->ld_dx, grad->dr, grad->ld_dr, n, d, e) ||
        rows_meet(grad->dx, grad->ld_dx, grad->di, grad->ld_di, n, d, e) ||
        rows_meet(grad->dr, grad->ld_dr, grad->di, grad->ld_di, n, d, e))
        return VIMSCAN_ERR_ALIAS;
    for (int k = 0; k < 3; ++k)
        if (meet(outs[k], outs[3]) || meet(outs[k], outs[4])) return VIMSCAN_ERR_ALIAS;
    return check_workspace(l, p.ws, ins, outs);
}

int check_gated_step(const vimscan_gated* g, const float* state, int64_t nslots, const int32_t* slots_in,
                     const int32_t* slots_out, const void* y, const vimscan_launch* l) {
    if (!g) return VIMSCAN_ERR_NULL;
    const int rc = check_launch(l, 1, 0);
    if (rc != VIMSCAN_OK) return rc;
    if (l->seqlen != 1 || nslots < 0 || nslots >= kMaxTokens) return VIMSCAN_ERR_SHAPE;
    const int64_t n = l->batch, d = l->d_inner;
    if (!positive(g->c)) return VIMSCAN_ERR_PARAM;
    if (!good_stride(g->ld_x, d) || !good_stride(g->ld_r, d) || !good_stride(g->ld_i, d)) return VIMSCAN_ERR_PARAM;
    if (n == 0 || d == 0) return VIMSCAN_OK;
    if (n > kMaxStepParts / ((d + 63) / 64)) return VIMSCAN_ERR_SHAPE;
    if (!g->x || !g->r || !g->i || !g->lam || !y || (nslots > 0 && !state)) return VIMSCAN_ERR_NULL;
    const size_t e = io_bytes(l);
    const void* io[] = {g->x, g->r, g->i, y};
    for (const void* q : io)
        if (!is_aligned(q, e)) return VIMSCAN_ERR_ALIGN;
    const void* w4[] = {g->lam, state, slots_in, slots_out};
    for (const void* q : w4)
        if (!is_aligned(q, 4)) return VIMSCAN_ERR_ALIGN;
    const Span ins[] = {rows_span(g->x, n, g->ld_x, d, e), rows_span(g->r, n, g->ld_r, d, e),
                        rows_span(g->i, n, g->ld_i, d, e), dense_span(g->lam, 1, d, 4),
                        dense_span(slots_in, n, 1, 4),     dense_span(slots_out, n, 1, 4)};
    const Span outs[] = {dense_span(y, n, d, e), dense_span(state, nslots, d, 4)};
    return any_meet(outs, ins) || meet(outs[0], outs[1]) ? VIMSCAN_ERR_ALIAS : VIMSCAN_OK;
}

int make_norm_plan(const vimscan_launch* l, bool backward, NormPlan* p) {
    const int rc = check_launch(l, 0, VIMSCAN_FLAG_GATE_AFTER);
    if (rc != VIMSCAN_OK) return rc;
    if (l->d_inner > kNormMaxWidth) return VIMSCAN_ERR_SHAPE;
    std::memset(p, 0, sizeof(*p));
    p->rows = l->batch * l->seqlen;
    p->D = l->d_inner;
    if (p->rows == 0 || p->D == 0) return VIMSCAN_OK;
    // enough workgroups for every CU's waves; fewer, each with more rows, where every one leaves three rows
    // of partial weight gradients
    const int64_t most = p->D <= 256 ? 2048 : 512;
    const int64_t at_once = l->io_dtype == VIMSCAN_F32 && p->D % 4 != 0 ? rows_at_once(kNormSingles, p->D)
                            : backward                                  ? rows_at_once(kNormBackward, p->D)
                                                                        : rows_at_once(kNormForward, p->D);
    const int64_t turns = (p->rows + at_once - 1) / at_once;
    p->wgs = turns < most ? turns : most;
    p->rows_per_wg = (turns + p->wgs - 1) / p->wgs * at_once;
    if (backward) p->ws = up256(static_cast<size_t>(p->wgs) * 3 * p->D * sizeof(float));
    return VIMSCAN_OK;
}

int check_norm_call(const vimscan_norm* n, const void* sum, const void* out, const vimscan_norm_grad* g,
                    const vimscan_launch* l, const NormPlan& p) {
    const int64_t rows = p.rows, d = l->d_inner;
    const size_t e = io_bytes(l);
    if (n->res_dtype != VIMSCAN_F32 && n->res_dtype != l->io_dtype) return VIMSCAN_ERR_DTYPE;
    const size_t re = n->res_dtype == VIMSCAN_F32 ? 4 : 2;
    if (!positive(n->eps)) return VIMSCAN_ERR_PARAM;
    if (!good_stride(n->ld_x, d) || (n->z && !good_stride(n->ld_z, d))) return VIMSCAN_ERR_PARAM;
    if (rows == 0 || d == 0) {  // pointers may be NULL; an empty backward pass still zeroes weight gradients
        if (!g || d == 0) return VIMSCAN_OK;
    } else if (!n->x) {
        return VIMSCAN_ERR_NULL;
    }
    if ((l->flags & VIMSCAN_FLAG_GATE_AFTER) && rows > 0 && (!n->z || !n->w_post)) return VIMSCAN_ERR_PARAM;
    if (!g) {
        if ((out != nullptr) != (n->w_pre != nullptr)) return VIMSCAN_ERR_PARAM;
        if (!sum && !out) return VIMSCAN_ERR_NULL;
    } else {
        if ((g->dn && !n->w_pre) || (g->dw_pre && !n->w_pre) || (g->dgamma && !n->gamma) || (g->dw_post && !n->w_post))
            return VIMSCAN_ERR_PARAM;
        if (rows > 0 && ((g->dz && !n->z) || (g->dresidual && !n->residual))) return VIMSCAN_ERR_PARAM;
        if ((g->dx && !good_stride(g->ld_dx, d)) || (g->dz && !good_stride(g->ld_dz, d))) return VIMSCAN_ERR_PARAM;
    }
    const void* io[] = {n->x, n->z, out, g ? g->dn : nullptr, g ? g->dx : nullptr, g ? g->dz : nullptr};
    for (const void* q : io)
        if (!is_aligned(q, e)) return VIMSCAN_ERR_ALIGN;
    const void* rs[] = {n->residual, sum, g ? g->dsum : nullptr, g ? g->dresidual : nullptr};
    for (const void* q : rs)
        if (!is_aligned(q, re)) return VIMSCAN_ERR_ALIGN;
    const void* w4[] = {n->w_post, n->gamma, n->w_pre, g ? g->dw_post : nullptr, g ? g->dgamma : nullptr,
                        g ? g->dw_pre : nullptr};
    for (const void* q : w4)
        if (!is_aligned(q, 4)) return VIMSCAN_ERR_ALIGN;
    const Span none = {nullptr, 0};
    const Span res = dense_span(n->residual, rows, d, re);
    const Span ins[] = {rows_span(n->x, rows, n->ld_x, d, e), rows_span(n->z, rows, n->ld_z, d, e),
                        dense_span(n->w_post, 1, d, 4), dense_span(n->gamma, 1, d, 4), dense_span(n->w_pre, 1, d, 4),
                        g ? dense_span(g->dn, rows, d, e) : none};
    if (!g) {
        const Span outs[] = {dense_span(sum, rows, d, re), dense_span(out, rows, d, e)};
        if (any_meet(outs, ins) || meet(outs[0], outs[1]) || meet(outs[1], res)) return VIMSCAN_ERR_ALIAS;
        if (sum != n->residual && meet(outs[0], res)) return VIMSCAN_ERR_ALIAS;
        return VIMSCAN_OK;
    }
    const Span dsum = dense_span(g->dsum, rows, d, re), dres = dense_span(g->dresidual, rows, d, re);
    const Span rin[] = {res, dsum};
    const Span outs[] = {rows_span(g->dx, rows, g->ld_dx, d, e), rows_span(g->dz, rows, g->ld_dz, d, e),
                         dense_span(g->dw_post, 1, d, 4), dense_span(g->dgamma, 1, d, 4), dense_span(g->dw_pre, 1, d, 4)};
    const Span rout[] = {dres};
    if (any_meet(outs, ins) || any_meet(outs, rin) || any_meet(outs, rout) || any_meet(rout, ins) || meet(dres, res))
        return VIMSCAN_ERR_ALIAS;
    if (g->dresidual != g->dsum && meet(dres, dsum)) return VIMSCAN_ERR_ALIAS;
    if (rows_meet(g->dx, g->ld_dx, g->dz, g->ld_dz, rows, d, e)) return VIMSCAN_ERR_ALIAS;
    for (int k = 2; k < 5; ++k)
        for (int j = 0; j < k; ++j)
            if (meet(outs[k], outs[j])) return VIMSCAN_ERR_ALIAS;
    if (!g->dw_post && !g->dgamma && !g->dw_pre) return VIMSCAN_OK;
    const int rc = check_workspace(l, p.ws, ins, outs);
    if (rc != VIMSCAN_OK || p.ws == 0) return rc;
    const Span w[] = {{l->workspace, p.ws}};
    return any_meet(w, rin) || any_meet(w, rout) ? VIMSCAN_ERR_ALIAS : VIMSCAN_OK;
}

}  // namespace vimscan_host

using namespace vimscan_host;

extern "C" {

int vimscan_gated_plan(const vimscan_launch* launch, int64_t seg_len, int packed, int64_t nseq, int backward,
                       vimscan_plan* plan) {
    if (!plan) return VIMSCAN_ERR_NULL;
    GatedPlan p;
    const int rc = make_gated_plan(launch, seg_len, packed != 0, nseq, backward != 0, &p);
    if (rc != VIMSCAN_OK) return rc;
    std::memset(plan, 0, sizeof(*plan));
    plan->sequences = p.nseq;
    plan->seq_tokens = p.Lp;
    plan->chunk_len = p.tile;
    plan->chunks = p.tiles;
    plan->workgroups = p.wgs;
    plan->kernels = p.wgs == 0 ? 0 : (backward ? 2 : 1);
    plan->workspace_bytes = p.ws;
    return VIMSCAN_OK;
}

int vimscan_norm_plan(const vimscan_launch* launch, int backward, vimscan_plan* plan) {
    if (!plan) return VIMSCAN_ERR_NULL;
    NormPlan p;
    const int rc = make_norm_plan(launch, backward != 0, &p);
    if (rc != VIMSCAN_OK) return rc;
    std::memset(plan, 0, sizeof(*plan));
    plan->sequences = p.rows;
    plan->seq_tokens = p.rows > 0 ? 1 : 0;
    plan->chunk_len = p.rows_per_wg;
    plan->chunks = p.rows > 0 ? 1 : 0;
    plan->workgroups = p.wgs;
    plan->kernels = p.wgs == 0 ? 0 : (backward ? 2 : 1);
    plan->workspace_bytes = p.ws;
    return VIMSCAN_OK;
}

}  // extern "C"
