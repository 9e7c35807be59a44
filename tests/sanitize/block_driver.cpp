// Drives the host side of the gated recurrence and the block norm (csrc/block_plan.cpp: plans and
// argument checks) through many shapes, sizes at and past every limit and random argument structures,
// for a build with the address and undefined-behaviour sanitizers. No HIP call is involved.
// Exit status 0 and "block driver ok" on success.
#include <cinttypes>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <random>

#include "../../bidirectional_selective_scan_amd/csrc/block_plan.h"
#include "vimscan.h"

using namespace vimscan_host;

namespace {

int failures = 0;

void expect(bool ok, const char* what, int64_t a, int64_t b) {
    if (!ok) {
        ++failures;
        std::printf("FAIL %s (%" PRId64 ", %" PRId64 ")\n", what, a, b);
    }
}

std::mt19937_64 rng(7);

int64_t any_size() {
    static const int64_t special[] = {0, 1, 2, 63, 64, 65, 127, 128, 129, 197, 1024, 32768, 32769, (1 << 22) - 1, 1 << 22,
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

vimscan_launch any_launch(int64_t d_state) {
    vimscan_launch l;
    std::memset(&l, 0, sizeof(l));
    l.batch = any_size();
    l.seqlen = any_size();
    l.d_inner = any_size();
    l.d_state = rng() % 16 ? d_state : any_size();
    l.io_dtype = rng() % 16 ? static_cast<int32_t>(rng() % 2) : 2;
    l.flags = rng() % 4 ? 0 : static_cast<int32_t>(rng() % 64);
    l.chunk_len = rng() % 16 ? 0 : any_size();
    l.workspace = const_cast<void*>(any_ptr());
    l.workspace_bytes = static_cast<size_t>(rng() >> (rng() % 60));
    return l;
}

void check_gated(const vimscan_launch& l, int64_t seg, bool packed, int64_t nseq, bool back) {
    GatedPlan p;
    const int rc = make_gated_plan(&l, seg, packed, nseq, back, &p);
    expect(rc <= 0 && rc >= VIMSCAN_ERR_PARAM, "status", rc, l.batch);
    vimscan_plan q;
    expect(vimscan_gated_plan(&l, seg, packed, nseq, back, &q) == rc, "the plan entry point agrees", l.batch, l.seqlen);
    if (rc != VIMSCAN_OK || p.wgs == 0) return;
    const int64_t width = p.ncb * kGatedBlock;
    expect(width >= l.d_inner && width - l.d_inner < kGatedBlock, "width", width, l.d_inner);
    expect(p.wgs == p.tiles * p.ncb && p.wgs <= kMaxGatedWgs, "workgroups", p.wgs, p.tiles);
    expect(p.tokens == 0 ? p.tiles == 1 : (p.tiles - 1) * p.tile < p.tokens && p.tokens <= p.tiles * p.tile, "tiles", p.tiles,
           p.tokens);
    if (!packed && p.tokens > 0) expect(p.nseq * p.Lp == p.tokens, "sequences", p.nseq, p.Lp);
    if (p.chain) {
        expect(static_cast<int64_t>(p.off_inc) >= p.tiles * 2 * width * 8, "tile maps fit", p.tiles, width);
        expect(static_cast<int64_t>(p.off_part - p.off_inc) >= p.groups * 2 * width * 8, "group states fit", p.groups, width);
        expect(p.groups * kGatedGroup >= p.tiles, "groups", p.groups, p.tiles);
    }
    if (back && p.tokens > 0)
        expect(static_cast<int64_t>(p.ws - p.off_part) >= p.tiles * width * 4, "partial sums fit", p.tiles, width);
}

void check_norm(const vimscan_launch& l, bool back) {
    NormPlan p;
    const int rc = make_norm_plan(&l, back, &p);
    vimscan_plan q;
    expect(vimscan_norm_plan(&l, back, &q) == rc, "the plan entry point agrees", l.batch, l.seqlen);
    if (rc != VIMSCAN_OK || p.wgs == 0) return;
    expect(p.wgs * p.rows_per_wg >= p.rows, "rows", p.wgs, p.rows);
    if (back) expect(static_cast<int64_t>(p.ws) >= p.wgs * 3 * p.D * 4, "partial gradients fit", p.wgs, p.D);
}

template <typename T>
T* cast(const void* p) { return static_cast<T*>(const_cast<void*>(p)); }

}  // namespace

int main() {
    for (int k = 0; k < 400000; ++k) {
        const vimscan_launch l = any_launch(1);
        check_gated(l, rng() % 2 ? 0 : any_size(), rng() % 2, any_size(), rng() % 2);
        check_norm(any_launch(0), rng() % 2);
    }
    int refused = 0, accepted = 0;
    for (int k = 0; k < 400000; ++k) {
        vimscan_launch l = any_launch(1);
        if (rng() % 2) {  // mostly sensible sizes, so that the later checks are reached
            l.batch = rng() % 4;
            l.seqlen = rng() % 300;
            l.d_inner = rng() % 100;
            l.chunk_len = l.flags = 0;
            l.io_dtype = rng() % 2;
        }
        const int64_t d = l.d_inner;
        vimscan_gated g;
        std::memset(&g, 0, sizeof(g));
        g.x = any_ptr();
        g.r = any_ptr();
        g.i = any_ptr();
        g.ld_x = rng() % 8 ? d : any_size();
        g.ld_r = rng() % 8 ? d : any_size();
        g.ld_i = rng() % 8 ? d : any_size();
        g.lam = cast<const float>(any_ptr());
        g.h0 = cast<const float>(any_ptr());
        g.offsets = rng() % 2 ? nullptr : cast<const int32_t>(any_ptr());
        g.nseq = any_size();
        g.c = rng() % 8 ? 8.0f : static_cast<float>(any_size()) / 3.0f;
        vimscan_gated_grad gr;
        std::memset(&gr, 0, sizeof(gr));
        gr.dy = any_ptr();
        gr.dh_last = cast<const float>(any_ptr());
        gr.states = cast<const float>(any_ptr());
        gr.dx = cast<void>(any_ptr());
        gr.dr = cast<void>(any_ptr());
        gr.di = cast<void>(any_ptr());
        gr.ld_dy = gr.ld_dx = gr.ld_dr = gr.ld_di = rng() % 8 ? d : any_size();
        gr.dlam = cast<float>(any_ptr());
        gr.dh0 = cast<float>(any_ptr());
        GatedPlan p;
        const bool back = rng() % 2;
        if (make_gated_plan(&l, 0, g.offsets != nullptr, g.nseq, back, &p) == VIMSCAN_OK) {
            const int rc = check_gated_call(&g, any_ptr(), cast<const float>(any_ptr()), cast<const float>(any_ptr()),
                                            back ? &gr : nullptr, &l, p);
            (rc == VIMSCAN_OK ? accepted : refused) += 1;
        }
        l.seqlen = 1;
        check_gated_step(&g, cast<const float>(any_ptr()), any_size(), cast<const int32_t>(any_ptr()),
                         cast<const int32_t>(any_ptr()), any_ptr(), &l);
        l.d_state = 0;
        vimscan_norm n;
        std::memset(&n, 0, sizeof(n));
        n.x = any_ptr();
        n.z = any_ptr();
        n.ld_x = n.ld_z = rng() % 8 ? d : any_size();
        n.w_post = cast<const float>(any_ptr());
        n.residual = any_ptr();
        n.gamma = cast<const float>(any_ptr());
        n.w_pre = cast<const float>(any_ptr());
        n.eps = rng() % 8 ? 1e-5f : -1.0f;
        n.res_dtype = static_cast<int32_t>(rng() % 3);
        vimscan_norm_grad ng;
        std::memset(&ng, 0, sizeof(ng));
        ng.dsum = any_ptr();
        ng.dn = any_ptr();
        ng.dx = cast<void>(any_ptr());
        ng.dz = cast<void>(any_ptr());
        ng.ld_dx = ng.ld_dz = rng() % 8 ? d : any_size();
        ng.dresidual = cast<void>(any_ptr());
        ng.dw_post = cast<float>(any_ptr());
        ng.dgamma = cast<float>(any_ptr());
        ng.dw_pre = cast<float>(any_ptr());
        NormPlan np;
        if (make_norm_plan(&l, back, &np) == VIMSCAN_OK) {
            const int rc = check_norm_call(&n, any_ptr(), any_ptr(), back ? &ng : nullptr, &l, np);
            (rc == VIMSCAN_OK ? accepted : refused) += 1;
        }
    }
    expect(accepted > 100 && refused > 100, "both outcomes were reached", accepted, refused);
    if (failures) return 1;
    std::printf("block driver ok (%d accepted, %d refused)\n", accepted, refused);
    return 0;
}
