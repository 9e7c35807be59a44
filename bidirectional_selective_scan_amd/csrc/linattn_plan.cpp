// Host side of linear attention (see linattn_plan.h).

#include "linattn_plan.h"

#include <cmath>
#include <cstring>

#include "call_checks.h"

namespace vimscan_host {
namespace {

// heads and groups, and the head sizes that the launch gives with them
int check_dims(const vimscan_launch* l, int64_t heads, int64_t groups) {
    if (heads < 1 || groups < 1 || heads > l->d_inner || heads % groups != 0 || l->d_inner % heads != 0)
        return VIMSCAN_ERR_SHAPE;
    if (l->d_state < 1 || l->d_state > kLinMaxDim || l->d_inner / heads > kLinMaxDim) return VIMSCAN_ERR_SHAPE;
    // (rows of the gradients by head lie within a buffer resource, as those of d_inner channels)
    if (heads * l->d_state >= (int64_t(1) << 22)) return VIMSCAN_ERR_SHAPE;
    return VIMSCAN_OK;
}

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens per segment, or 0: sequences stay whole. A wave for each SIMD of the chip (1024): more, shorter segments cost more
// in their states than they gain (heads of 64 x 64 bf16, forward, us, chunks of 32 tokens per segment; 8 x 1025 x 12, 2: 51, 4: 47, 5: 48, 9: 62,
// whole 105; 1 x 4096 x 24, 2: 55, 4: 48, 6: 52, 9: 63, whole 388; 1 x 65537 x 24, 17: 324, 25: 305, 33: 296 to 308, 49: 298 to 308).
// Two where packed sequences differ in length (16 x up to 2000 x 24, 9: 108, 13: 127, 17: 148, 25: 170, whole 195; 64 x up to
// 1025 x 12, whose heads alone are 768 waves, hardly gains, in training 9: 491, 17: 582, whole 508), and twice as many in fp32, whose chunks take
// longer (packed 32 x up to 513 x 6 of 40 x 56 in training 2: 214, 3: 216, 4: 231, 9: 292, whole 290).
// Where sequences and heads alone are more than half as many waves, they stay whole, however long (64 x 4097 x 24 whole 788, 64: 1233, 128: 1300;
// 43 x 8200 x 24 1219, 1571, 1790; 22 x 8200 x 24 812, 900, 931).
// The fold walks a sequence's segments one behind the other, eight at a time, so with few heads a segment is no shorter than the square root of
// chunks / 32, where a segment's chunks and the fold cost alike (1 x 65537 x 1 head, 3: 119, 4: 99, 8: 84, 12: 91; 1 x 16385 x 1,
// 2: 59, 4: 52, 6: 55; 4 x 8192 x 2, 2: 50, 3: 47, 4: 46; 1 x 65537 x 2 in training 5: 334, 8: 309, 12: 327).
// Segments are of nearly equal length (16 x 8200 x 24, 257 chunks: three of 86 657, two of 128 and a single chunk 817). Their own states and
// the fold cost about as much as 0.6 of the pass and three chunks: where that is not less than the chunks saved, sequences stay whole.
int64_t segment(int64_t length, int64_t waves, bool packed, int bytes) {
    constexpr int64_t kLeast = 2, kMost = 128;   // chunks
    const int64_t chunks = up(length, kLinChunk), parts = 1024 * (packed ? 2 : 1) * (bytes == 4 ? 2 : 1) / waves;
    if (parts < (packed ? 3 : 2) || chunks <= kLeast) return 0;
    int64_t seg = up(chunks, parts);
    if (seg < kLeast) seg = kLeast;
    if (seg > kMost) seg = kMost;
    while (32 * seg * seg < chunks) ++seg;
    seg = up(chunks, up(chunks, seg));
    return 10 * chunks <= 16 * seg + 30 ? 0 : seg * kLinChunk;
}

// The whole extent of [tokens][heads][d] with strides.
Span heads_span(const void* p, int64_t tokens, int64_t heads, int64_t ld, int64_t hs, int64_t d, size_t e) {
    if (!p || tokens <= 0 || heads <= 0) return {nullptr, 0};
    return {p, (static_cast<size_t>(tokens - 1) * ld + static_cast<size_t>(heads - 1) * hs + d) * e};
}

bool good_head_stride(int64_t hs) { return hs >= 0 && hs < kMaxHeadStride; }

int check_strides(const vimscan_linattn* a, int64_t dk, int64_t dv) {
    if (!std::isfinite(a->scale)) return VIMSCAN_ERR_PARAM;
    if (!good_stride(a->ld_q, dk) || !good_stride(a->ld_k, dk) || !good_stride(a->ld_v, dv)) return VIMSCAN_ERR_PARAM;
    if (!good_head_stride(a->hs_q) || !good_head_stride(a->hs_k) || !good_head_stride(a->hs_v)) return VIMSCAN_ERR_PARAM;
    if (a->ld_decay != 0 && !good_stride(a->ld_decay, a->heads)) return VIMSCAN_ERR_PARAM;
    return VIMSCAN_OK;
}

Span decay_span(const vimscan_linattn* a, int64_t tokens) {
    return a->ld_decay == 0 ? dense_span(a->log_decay, 1, a->heads, 4)
                            : rows_span(a->log_decay, tokens, a->ld_decay, a->heads, 4);
}

}  // namespace

int make_linattn_plan(const vimscan_launch* l, int64_t seg_len, int64_t heads, int64_t groups, bool packed, int64_t nseq,
                      bool backward, LinPlan* p) {
    if (!l) return VIMSCAN_ERR_NULL;
    int rc = check_launch(l, l->d_state, VIMSCAN_FLAG_REVERSE);
    if (rc != VIMSCAN_OK) return rc;
    rc = check_dims(l, heads, groups);
    if (rc != VIMSCAN_OK) return rc;
    if (seg_len < 0 || (seg_len > 0 && l->seqlen % seg_len != 0)) return VIMSCAN_ERR_SEGLEN;
    if (packed && seg_len != 0) return VIMSCAN_ERR_PARAM;
    if (packed && (nseq < 0 || nseq >= kMaxTokens)) return VIMSCAN_ERR_SHAPE;
    std::memset(p, 0, sizeof(*p));
    p->packed = packed;
    p->tokens = l->batch * l->seqlen;
    if (packed && nseq == 0 && p->tokens > 0) return VIMSCAN_ERR_SHAPE;
    p->Lp = packed || p->tokens == 0 ? 0 : (seg_len > 0 ? seg_len : l->seqlen);
    // uniform sequences of no tokens: one per batch row (cut at seg_len: none)
    p->nseq = packed ? nseq : p->tokens > 0 ? p->tokens / p->Lp : seg_len > 0 ? 0 : l->batch;
    p->H = heads;
    p->G = groups;
    p->dk = l->d_state;
    p->dv = l->d_inner / heads;
    if (p->nseq == 0) return VIMSCAN_OK;
    // (packed sequences: the longest is taken to be twice the mean)
    const int64_t twice = packed ? 2 * up(p->tokens, p->nseq) : 0, length = !packed ? p->Lp : twice < p->tokens ? twice : p->tokens;
    const int bytes = static_cast<int>(io_bytes(l));
    const int64_t blocks = lin_blocks(bytes, p->dk, p->dv), qblocks = lin_blocks(bytes, p->dv, p->dk);
    // (up to three passes of the backward pass are one launch)
    const int64_t most_waves = kMaxLinWaves / ((blocks > qblocks ? blocks : qblocks) * heads * (backward ? 3 : 1));
    if (p->nseq > most_waves) return VIMSCAN_ERR_SHAPE;
    p->seg = segment(length, p->nseq * heads * blocks, packed, bytes);
    // packed sequences that are whole by that: any that is longer than they are taken to be is cut, if it could be a long chain
    // (24 heads of 64 x 64 bf16, forward and backward, us: 65537 + 63 x 1 tokens 763 + 2610, whole 6320 + 20900; 12 heads, 20000 + 200 x 100
    // 494 + 1200, whole 1926 + 6010). Where none is cut the two launches cost some 10 us (256 x up to 513 x 12 138 + 495, whole 127 + 455;
    // 64 x up to 65 x 12 23 + 56, whole 14 + 40, which at most 8192 tokens stay).
    if (packed && p->seg == 0 && p->tokens > kLinLongest) {
        const int64_t most = length > kLinLongest / 4 ? up(length, kLinChunk) * kLinChunk : kLinLongest / 4;
        if (p->tokens > most && p->tokens / most + p->nseq <= most_waves) p->seg = most;
    }
    p->split = p->seg > 0;
    p->segs = p->split && !packed ? up(p->Lp, p->seg) : 1;
    p->slots = !p->split ? p->nseq : packed ? p->tokens / p->seg + p->nseq : p->nseq * p->segs;
    if (!p->split) p->seg = p->Lp;
    if (p->slots > most_waves) return VIMSCAN_ERR_SHAPE;
    p->waves = p->slots * heads * blocks;
    const size_t per_head = static_cast<size_t>(p->slots) * heads, state = per_head * p->dk * p->dv * sizeof(float);
    auto take = [&](size_t bytes) {
        const size_t at = p->ws;
        p->ws += up256(bytes);
        return at;
    };
    if (p->split) {
        p->off_s = take(state);
        p->off_tot = take(per_head * sizeof(float));
    }
    if (!backward || p->tokens == 0) return VIMSCAN_OK;
    if (p->split) p->off_e = take(state);
    const size_t rows = static_cast<size_t>(p->tokens) * heads;
    p->off_rq = take(rows * qblocks * sizeof(float));
    p->off_rk = take(rows * qblocks * sizeof(float));
    p->off_cd = take(per_head * qblocks * sizeof(float));
    p->off_hs = take(per_head * sizeof(float));
    if (groups != heads) {
        p->off_pq = take(rows * p->dk * sizeof(float));
        p->off_pk = take(rows * p->dk * sizeof(float));
    }
    p->ws_plain = p->ws;
    // (packed: a segment of n tokens from walking position t on has (n - 1) / window borders from t / window on, at most those before
    // the next's)
    p->seg_borders = packed ? 0 : (p->seg - 1) / kLinWindow;
    p->borders = packed ? p->tokens / kLinWindow : p->slots * p->seg_borders;
    const size_t at_borders = static_cast<size_t>(p->borders) * heads, marks = at_borders * lin_state_floats(bytes, p->dv, p->dk) * sizeof(float);
    p->off_ms = take(marks);
    p->off_me = take(marks);
    p->off_bd = take(at_borders * qblocks * sizeof(float));
    return VIMSCAN_OK;
}

int check_linattn_call(const vimscan_linattn* a, const void* y, const float* h_last, const vimscan_linattn_grad* g,
                       const vimscan_launch* l, const LinPlan& p) {
    const int64_t n = p.tokens;
    const size_t e = io_bytes(l);
    int rc = check_strides(a, p.dk, p.dv);
    if (rc != VIMSCAN_OK) return rc;
    if (g && g->dy && (!good_stride(g->ld_dy, p.dv) || !good_head_stride(g->hs_dy))) return VIMSCAN_ERR_PARAM;
    if (n > 0) {
        if (!a->q || !a->k || !a->v || !a->log_decay) return VIMSCAN_ERR_NULL;
        if (g ? (!g->dq || !g->dk || !g->dv) : !y) return VIMSCAN_ERR_NULL;
    }
    const void* io[] = {a->q, a->k, a->v, y, g ? g->dy : nullptr, g ? g->dq : nullptr, g ? g->dk : nullptr,
                        g ? g->dv : nullptr};
    for (const void* q : io)
        if (!is_aligned(q, e)) return VIMSCAN_ERR_ALIGN;
    const void* w4[] = {a->log_decay, a->h0, a->offsets, h_last, g ? g->dh_last : nullptr, g ? g->dlog_decay : nullptr,
                        g ? g->dh0 : nullptr};
    for (const void* q : w4)
        if (!is_aligned(q, 4)) return VIMSCAN_ERR_ALIGN;
    const int64_t hstate = p.nseq * p.H, state = p.dk * p.dv;
    const Span none = {nullptr, 0};
    const Span ins[] = {heads_span(a->q, n, p.G, a->ld_q, a->hs_q, p.dk, e),
                        heads_span(a->k, n, p.G, a->ld_k, a->hs_k, p.dk, e),
                        heads_span(a->v, n, p.H, a->ld_v, a->hs_v, p.dv, e),
                        decay_span(a, n),
                        dense_span(a->h0, hstate, state, 4),
                        p.packed ? dense_span(a->offsets, p.nseq + 1, 1, 4) : none,
                        g ? heads_span(g->dy, n, p.H, g->ld_dy, g->hs_dy, p.dv, e) : none,
                        g ? dense_span(g->dh_last, hstate, state, 4) : none};
    if (!g) {
        const Span outs[] = {dense_span(y, n, p.H * p.dv, e), dense_span(h_last, hstate, state, 4)};
        if (any_meet(outs, ins) || meet(outs[0], outs[1])) return VIMSCAN_ERR_ALIAS;
        return check_workspace(l, p.ws, ins, outs);
    }
    const Span outs[] = {dense_span(g->dq, n, p.G * p.dk, e), dense_span(g->dk, n, p.G * p.dk, e),
                         dense_span(g->dv, n, p.H * p.dv, e),
                         a->ld_decay ? dense_span(g->dlog_decay, n, p.H, 4) : dense_span(g->dlog_decay, 1, p.H, 4),
                         dense_span(g->dh0, hstate, state, 4)};
    if (any_meet(outs, ins)) return VIMSCAN_ERR_ALIAS;
    for (int k = 1; k < 5; ++k)
        for (int j = 0; j < k; ++j)
            if (meet(outs[k], outs[j])) return VIMSCAN_ERR_ALIAS;
    return check_workspace(l, g->dlog_decay ? p.ws : p.ws_plain, ins, outs);
}

int check_linattn_step(const vimscan_linattn* a, const float* state, int64_t nslots, const int32_t* slots_in,
                       const int32_t* slots_out, const void* y, const vimscan_launch* l) {
    if (!a || !l) return VIMSCAN_ERR_NULL;
    int rc = check_launch(l, l->d_state, 0);
    if (rc != VIMSCAN_OK) return rc;
    rc = check_dims(l, a->heads, a->groups);
    if (rc != VIMSCAN_OK) return rc;
    if (l->seqlen != 1 || nslots < 0 || nslots >= kMaxTokens) return VIMSCAN_ERR_SHAPE;
    const int64_t n = l->batch, H = a->heads, dk = l->d_state, dv = l->d_inner / H;
    rc = check_strides(a, dk, dv);
    if (rc != VIMSCAN_OK) return rc;
    if (n == 0) return VIMSCAN_OK;
    if (n > kMaxLinWgs / (H * up(dv, 64))) return VIMSCAN_ERR_SHAPE;
    if (!a->q || !a->k || !a->v || !a->log_decay || !y || (nslots > 0 && !state)) return VIMSCAN_ERR_NULL;
    const size_t e = io_bytes(l);
    const void* io[] = {a->q, a->k, a->v, y};
    for (const void* q : io)
        if (!is_aligned(q, e)) return VIMSCAN_ERR_ALIGN;
    const void* w4[] = {a->log_decay, state, slots_in, slots_out};
    for (const void* q : w4)
        if (!is_aligned(q, 4)) return VIMSCAN_ERR_ALIGN;
    const Span ins[] = {heads_span(a->q, n, a->groups, a->ld_q, a->hs_q, dk, e),
                        heads_span(a->k, n, a->groups, a->ld_k, a->hs_k, dk, e),
                        heads_span(a->v, n, H, a->ld_v, a->hs_v, dv, e),
                        decay_span(a, n),
                        dense_span(slots_in, n, 1, 4),
                        dense_span(slots_out, n, 1, 4)};
    const Span outs[] = {dense_span(y, n, H * dv, e), dense_span(state, nslots, H * dk * dv, 4)};
    return any_meet(outs, ins) || meet(outs[0], outs[1]) ? VIMSCAN_ERR_ALIAS : VIMSCAN_OK;
}

}  // namespace vimscan_host

using namespace vimscan_host;

extern "C" {

int vimscan_linattn_plan(const vimscan_launch* launch, int64_t seg_len, int64_t heads, int64_t groups, int packed,
                         int64_t nseq, int backward, vimscan_plan* plan) {
    if (!plan) return VIMSCAN_ERR_NULL;
    LinPlan p;
    const int rc = make_linattn_plan(launch, seg_len, heads, groups, packed != 0, nseq, backward != 0, &p);
    if (rc != VIMSCAN_OK) return rc;
    std::memset(plan, 0, sizeof(*plan));
    plan->sequences = p.nseq;
    plan->seq_tokens = p.Lp;
    plan->chunk_len = p.seg;
    plan->chunks = p.nseq == 0 ? 0 : p.split && packed ? p.slots : p.segs;
    plan->workgroups = p.waves;
    // forward: the pass, where it is split after the segments' states and their fold; backward: the same
    // states and those of the gradients, the passes of dq and dk in one launch and that of dv, the values at
    // the windows' borders, the decays' gradient and its sum over the tokens (without it passes that are alike are one launch), the sums over shared heads
    const bool decays = backward != 2;
    if (p.waves > 0) {
        if (!backward) plan->kernels = p.split ? 3 : 1;
        else if (p.tokens == 0) plan->kernels = decays ? 2 : 1;
        else plan->kernels = (p.split ? 4 : 0) + (decays ? 4 + (p.borders > 0) : lin_alike(static_cast<int>(io_bytes(launch)), p.dk, p.dv) ? 1 : 2) +
                             (p.G != p.H ? 2 : 0);
    }
    plan->workspace_bytes = backward && !decays && p.tokens > 0 ? p.ws_plain : p.ws;
    return VIMSCAN_OK;
}

}  // extern "C"
