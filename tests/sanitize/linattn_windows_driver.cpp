// The windows of the decays' gradient of linear attention (csrc/linattn_plan.cpp): every border between two windows of a segment has
// a place of its own among those that the workspace holds. For a build with the address and undefined-behaviour sanitizers.
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "../../bidirectional_selective_scan_amd/csrc/linattn_plan.h"

using namespace vimscan_host;

namespace {

std::mt19937_64 rng(5);
int failures = 0, cut = 0, whole = 0;

void expect(bool ok, const char* what, int64_t a, int64_t b) {
    if (ok) return;
    if (++failures < 10) std::printf("FAILED: %s (%lld, %lld)\n", what, static_cast<long long>(a), static_cast<long long>(b));
}

void one() {
    const bool packed = rng() % 2;
    const int64_t nseq = 1 + rng() % (rng() % 4 ? 12 : 700), heads = int64_t(1) << rng() % 6, most = rng() % 5 ? 600 : 9000;
    std::vector<int64_t> len(nseq, 1 + static_cast<int64_t>(rng() % most));
    int64_t tokens = 0;
    for (int64_t& v : len) {
        if (packed) v = rng() % 4 ? static_cast<int64_t>(rng() % most) : static_cast<int64_t>(rng() % 5) * 64;
        tokens += v;
    }
    vimscan_launch l;
    std::memset(&l, 0, sizeof(l));
    l.batch = packed ? 1 : nseq;
    l.seqlen = packed ? tokens : len[0];
    l.d_state = 1 + rng() % 128;
    const int64_t dv = 1 + rng() % 128;
    l.d_inner = heads * dv;
    l.io_dtype = rng() % 2;
    LinPlan p;
    const int rc = make_linattn_plan(&l, 0, heads, heads, packed, nseq, true, &p);
    expect(rc == VIMSCAN_OK, "plan", rc, tokens);
    if (rc != VIMSCAN_OK || tokens == 0) return;
    const int bytes = l.io_dtype == VIMSCAN_F32 ? 4 : 2;
    const size_t places = static_cast<size_t>(p.borders) * heads, state = lin_state_floats(bytes, p.dv, p.dk) * 4;
    expect(p.off_me - p.off_ms >= places * state && p.off_bd - p.off_me >= places * state, "states at the borders fit", p.borders, heads);
    expect(p.ws - p.off_bd >= places * lin_blocks(bytes, p.dv, p.dk) * 4 && p.ws_plain <= p.off_ms, "products fit", p.borders, heads);
    expect(state >= static_cast<size_t>(p.dk * p.dv) * 4, "a state fits", p.dk, p.dv);
    (p.split ? cut : whole) += 1;
    // the device's numbering of segments, in the order of their slots
    std::vector<char> taken(p.borders);
    int64_t at = 0;
    for (int64_t q = 0; q < nseq; ++q) {
        const int64_t parts = p.split && len[q] > 0 ? (len[q] + p.seg - 1) / p.seg : 1;
        for (int64_t j = 0; j < parts; ++j) {
            const int64_t w0 = p.split ? j * p.seg : 0, n = p.split && len[q] - w0 > p.seg ? p.seg : len[q] - w0;
            const int64_t first = packed ? (at + w0) / kLinWindow : (q * p.segs + j) * p.seg_borders;
            for (int64_t b = 0; b < (n > 0 ? (n - 1) / kLinWindow : 0); ++b) {
                const bool in = first + b >= 0 && first + b < p.borders;
                expect(in, "a border inside the workspace", first + b, p.borders);
                if (!in) continue;
                expect(!taken[first + b], "a border of its own", first + b, q);
                taken[first + b] = 1;
            }
        }
        at += len[q];
    }
}

}  // namespace

int main() {
    for (int k = 0; k < 20000; ++k) one();
    if (cut < 100 || whole < 100) ++failures;
    std::printf("%d failures, %d cut, %d whole\n", failures, cut, whole);
    return failures != 0;
}
