// The host side of linear attention and the layer norm (csrc/linattn_plan.cpp, block_plan.cpp) driven through sizes at and
// past every limit and random argument structures, for a build with the address and undefined-behaviour sanitizers.
#include <cstdio>
#include <cstring>
#include <limits>
#include <random>

#include "../../bidirectional_selective_scan_amd/csrc/block_plan.h"
#include "../../bidirectional_selective_scan_amd/csrc/linattn_plan.h"

using namespace vimscan_host;

namespace {

std::mt19937_64 rng(11);
int failures = 0;

void expect(bool ok, const char* what, int64_t a, int64_t b) {
    if (ok) return;
    if (++failures < 10) std::printf("FAILED: %s (%lld, %lld)\n", what, static_cast<long long>(a), static_cast<long long>(b));
}

int64_t any_size() {
    static const int64_t special[] = {0, 1, 2, 31, 32, 33, 64, 128, 129, 1024, 32768, 32769, (1 << 22) - 1, 1 << 22,
                                      (int64_t(1) << 31) - 1, int64_t(1) << 31, -1, std::numeric_limits<int64_t>::max(),
                                      std::numeric_limits<int64_t>::min()};
    const uint64_t r = rng();
    if (r % 3 == 0) return special[(r >> 8) % (sizeof(special) / sizeof(special[0]))];
    return static_cast<int64_t>((r >> 8) >> (8 + (r >> 2) % 46));
}
const void* any_ptr() {
    const uint64_t r = rng();
    if (r % 8 == 0) return nullptr;
    return reinterpret_cast<const void*>((uint64_t(1) << 40) + ((r >> 8) % 64 << 30) + (r % 16 == 1 ? (r >> 40) % 16 : 0));
}
template <typename T>
T* as(const void* p) { return static_cast<T*>(const_cast<void*>(p)); }

vimscan_launch any_launch() {
    vimscan_launch l;
    std::memset(&l, 0, sizeof(l));
    l.batch = any_size();
    l.seqlen = any_size();
    l.d_inner = any_size();
    l.d_state = rng() % 4 ? static_cast<int64_t>(rng() % 140) : any_size();
    l.io_dtype = rng() % 16 ? static_cast<int32_t>(rng() % 2) : 2;
    l.flags = rng() % 4 ? 0 : static_cast<int32_t>(rng() % 64);
    l.chunk_len = rng() % 16 ? 0 : any_size();
    l.workspace = as<void>(any_ptr());
    l.workspace_bytes = static_cast<size_t>(rng() >> (rng() % 60));
    return l;
}

void check_plan(const vimscan_launch& l, int64_t seg, int64_t heads, int64_t groups, bool packed, int64_t nseq, bool back) {
    LinPlan p;
    const int rc = make_linattn_plan(&l, seg, heads, groups, packed, nseq, back, &p);
    expect(rc <= 0 && rc >= VIMSCAN_ERR_PARAM, "status", rc, l.batch);
    vimscan_plan q;
    expect(vimscan_linattn_plan(&l, seg, heads, groups, packed, nseq, back, &q) == rc, "the plan entry point agrees", l.batch, l.seqlen);
    if (rc != VIMSCAN_OK || p.nseq == 0) return;
    expect(p.H * p.dv == l.d_inner && p.dk <= kLinMaxDim && p.dv <= kLinMaxDim && p.H * p.dk < (1 << 22), "dimensions", p.H, p.dv);
    const int bytes = l.io_dtype == VIMSCAN_F32 ? 4 : 2;
    const int64_t blocks = lin_blocks(bytes, p.dk, p.dv), qblocks = lin_blocks(bytes, p.dv, p.dk);
    expect(blocks * 16 * lin_output_tiles(bytes, p.dk, p.dv) >= p.dv && 16 * lin_contract_tiles(p.dk) >= p.dk, "tiles hold a head", p.dk, p.dv);
    expect(p.waves == p.slots * p.H * blocks && p.waves <= kMaxLinWaves && p.slots * p.H * qblocks <= kMaxLinWaves, "waves", p.waves, p.slots);
    if (!packed && p.tokens > 0) expect(p.nseq * p.Lp == p.tokens, "sequences", p.nseq, p.Lp);
    if (p.split) {
        expect(p.seg > 0 && p.seg % kLinChunk == 0, "segments are chunks", p.seg, p.Lp);
        if (!packed) expect(p.segs * p.seg >= p.Lp && (p.segs - 1) * p.seg < p.Lp && p.slots == p.nseq * p.segs, "segments", p.segs, p.seg);
        else expect(p.slots == p.tokens / p.seg + p.nseq, "slots", p.slots, p.nseq);
        const size_t state = static_cast<size_t>(p.slots) * p.H * p.dk * p.dv * 4;
        expect(p.off_tot - p.off_s >= state && p.ws > p.off_tot, "states fit", p.slots, p.H);
        if (back && p.tokens > 0) expect(p.off_rq - p.off_e >= state, "gradients of states fit", p.slots, p.H);
    }
    if (back && p.tokens > 0) {
        const size_t rows = static_cast<size_t>(p.tokens) * p.H;
        expect(p.off_rk - p.off_rq >= rows * qblocks * 4 && p.off_cd - p.off_rk >= rows * qblocks * 4, "terms fit", p.tokens, p.H);
        expect(p.off_hs - p.off_cd >= static_cast<size_t>(p.slots) * p.H * qblocks * 4, "ends fit", p.slots, p.H);
        if (p.G != p.H) expect(p.off_pk - p.off_pq >= rows * p.dk * 4 && p.ws - p.off_pk >= rows * p.dk * 4, "parts fit", p.tokens, p.H);
    }
}

}  // namespace

int main() {
    for (int k = 0; k < 300000; ++k) {
        vimscan_launch l = any_launch();
        int64_t heads = any_size(), groups = any_size();
        if (rng() % 2) {
            heads = 1 + rng() % 32;
            groups = rng() % 2 ? heads : 1;
            l.d_inner = heads * (1 + rng() % 128);
            l.batch = rng() % 300;
            l.flags = 0;
            l.chunk_len = 0;
        }
        check_plan(l, rng() % 2 ? 0 : any_size(), heads, groups, rng() % 2, any_size(), rng() % 2);
        l.d_state = rng() % 8 ? 0 : l.d_state;
        NormPlan n;
        const bool back = rng() % 2;
        if (make_layernorm_plan(&l, back, &n) == VIMSCAN_OK && n.wgs > 0) {
            expect(n.wgs * n.rows_per_wg >= n.rows, "rows", n.wgs, n.rows);
            if (back) expect(static_cast<int64_t>(n.ws) >= n.wgs * 2 * n.D * 4, "partial gradients fit", n.wgs, n.D);
        }
    }
    // the slots of packed sequences: base(q) = offsets[q] / seg + q gives each its own, all below the count
    for (int k = 0; k < 20000; ++k) {
        const int64_t nseq = 1 + rng() % 20, seg = 32 * (1 + rng() % 6);
        int64_t at = 0, next = 0;
        for (int64_t q = 0; q < nseq; ++q) {
            const int64_t len = rng() % 3 ? static_cast<int64_t>(rng() % 700) : 0, base = at / seg + q;
            expect(base >= next, "slots of their own", base, next);
            next = base + (len > 0 ? (len + seg - 1) / seg : 1);
            at += len;
        }
        expect(next <= at / seg + nseq, "slots in all", next, at / seg + nseq);
    }
    int refused = 0, accepted = 0;
    for (int k = 0; k < 300000; ++k) {
        vimscan_launch l = any_launch();
        vimscan_linattn a;
        std::memset(&a, 0, sizeof(a));
        a.heads = 1 + rng() % 8;
        a.groups = rng() % 2 ? a.heads : 1;
        if (rng() % 4) {
            l.batch = rng() % 4;
            l.seqlen = rng() % 300;
            l.d_inner = a.heads * (1 + rng() % 64);
            l.d_state = 1 + rng() % 64;
            l.flags = l.chunk_len = 0;
            l.io_dtype = rng() % 2;
        }
        a.q = any_ptr();
        a.k = any_ptr();
        a.v = any_ptr();
        a.ld_q = rng() % 8 ? 1024 : any_size();
        a.ld_k = rng() % 8 ? 1000 : any_size();
        a.ld_v = rng() % 8 ? l.d_inner : any_size();
        a.hs_q = rng() % 8 ? l.d_state : any_size();
        a.hs_k = rng() % 8 ? l.d_state : any_size();
        a.hs_v = rng() % 8 ? l.d_inner / a.heads : any_size();
        a.log_decay = as<const float>(any_ptr());
        a.ld_decay = rng() % 2 ? 0 : rng() % 8 ? a.heads : any_size();
        a.h0 = as<const float>(any_ptr());
        a.offsets = rng() % 2 ? nullptr : as<const int32_t>(any_ptr());
        a.nseq = any_size();
        a.scale = rng() % 8 ? 1.0f : std::numeric_limits<float>::infinity();
        vimscan_linattn_grad g;
        std::memset(&g, 0, sizeof(g));
        g.dy = any_ptr();
        g.ld_dy = rng() % 8 ? l.d_inner : any_size();
        g.hs_dy = rng() % 8 ? 64 : any_size();
        g.dh_last = as<const float>(any_ptr());
        g.dq = as<void>(any_ptr());
        g.dk = as<void>(any_ptr());
        g.dv = as<void>(any_ptr());
        g.dlog_decay = as<float>(any_ptr());
        g.dh0 = as<float>(any_ptr());
        LinPlan p;
        const bool back = rng() % 2;
        if (make_linattn_plan(&l, 0, a.heads, a.groups, a.offsets != nullptr, a.nseq, back, &p) == VIMSCAN_OK)
            (check_linattn_call(&a, any_ptr(), as<const float>(any_ptr()), back ? &g : nullptr, &l, p) == VIMSCAN_OK ? accepted : refused) += 1;
        l.seqlen = 1;
        check_linattn_step(&a, as<const float>(any_ptr()), any_size(), as<const int32_t>(any_ptr()), as<const int32_t>(any_ptr()), any_ptr(), &l);
        l.d_state = 0;
        vimscan_layernorm n;
        std::memset(&n, 0, sizeof(n));
        n.x = any_ptr();
        n.ld_x = rng() % 8 ? l.d_inner : any_size();
        n.residual = any_ptr();
        n.weight = as<const float>(any_ptr());
        n.bias = as<const float>(any_ptr());
        n.eps = rng() % 8 ? 1e-5f : -1.0f;
        n.res_dtype = static_cast<int32_t>(rng() % 3);
        vimscan_layernorm_grad ng;
        std::memset(&ng, 0, sizeof(ng));
        ng.dsum = any_ptr();
        ng.dn = any_ptr();
        ng.dx = as<void>(any_ptr());
        ng.ld_dx = rng() % 8 ? l.d_inner : any_size();
        ng.dresidual = as<void>(any_ptr());
        ng.dweight = as<float>(any_ptr());
        ng.dbias = as<float>(any_ptr());
        NormPlan np;
        if (make_layernorm_plan(&l, back, &np) == VIMSCAN_OK)
            (check_layernorm_call(&n, any_ptr(), any_ptr(), back ? &ng : nullptr, &l, np) == VIMSCAN_OK ? accepted : refused) += 1;
    }
    expect(accepted > 100 && refused > 100, "both outcomes were reached", accepted, refused);
    if (failures) return 1;
    std::printf("linattn driver ok (%d accepted, %d refused)\n", accepted, refused);
    return 0;
}
