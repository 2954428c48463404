// The split of paged attention (csrc/ra_paged_split.h) run on the host: a
// family of segments planned, walked by every CTA, and looked up as the join does.
#include <vector>

#include "ra_paged_split.h"

using namespace ra;
using namespace ra::dev;

namespace {

struct Split {
    PagedArgs a{};
    PagedFamily f{};
    std::vector<PagedSeg> seg;
    long long W = 0, R = 0, per = 0;

    Split(int S, const int *n, const int *len, int G, int Hkv, int rt, int kt, int halves, int least, int ctas) {
        a.G = G;
        a.Hkv = Hkv;
        f.S = S;
        f.rt = rt;
        f.kt = kt;
        f.n = ctas;
        f.halves = halves;
        f.least = least;
        while (1 << f.rt_log < rt) ++f.rt_log;
        while (1 << f.kt_log < kt) ++f.kt_log;
        int tok = 0;
        for (int s = 0; s < S; ++s) {
            PagedSeg g{tok, n[s], len[s], n[s] > 0 ? (len[s] + kt - 1) >> f.kt_log : 0, W, R};
            W += paged_tiles(a, f, g);
            R += paged_rows(a, f, g);
            tok += n[s];
            seg.push_back(g);
        }
        per = paged_per(f, W);
    }
};

}  // namespace

extern "C" {

// Units of all CTAs, 10 numbers each: CTA, segment, head, first row, rows, first tile, end tile, first partial row,
// tokens, keys.  Returns their count (at most `room` are written), and W, R and per.
long long split_walk(int S, const int *n, const int *len, int G, int Hkv, int rt, int kt, int halves, int least,
                     int ctas, long long *out, long long room, long long *sums) {
    Split p(S, n, len, G, Hkv, rt, kt, halves, least, ctas);
    sums[0] = p.W;
    sums[1] = p.R;
    sums[2] = p.per;
    long long count = 0;
    for (int c = 0; c < ctas; ++c) {
        PagedWalk k{};
        k.x = c * p.per;
        k.x1 = lesser(p.W, k.x + p.per);
        if (k.x >= k.x1) continue;
        for (int s = 0; s < S; ++s)  // the segment with tiles at the run's first place
            if (k.x >= p.seg[s].W0 && k.x < p.seg[s].W0 + paged_tiles(p.a, p.f, p.seg[s])) k.s = s;
        k.g = p.seg[k.s];
        for (PagedUnit u; paged_walk(p.a, p.f, k, u, [&](PagedWalk &w, long long) { w.g = p.seg[++w.s]; }); ++count) {
            if (count >= room) continue;
            long long *o = out + count * 10;
            o[0] = c, o[1] = u.s, o[2] = u.h, o[3] = u.r0, o[4] = u.rows, o[5] = u.t0, o[6] = u.t1;
            o[7] = u.base + (long long)c * rt, o[8] = u.n, o[9] = u.len;
        }
    }
    return count;
}

// The partial rows of query row `r` of segment s and head h, as the join finds them.
int split_parts(int S, const int *n, const int *len, int G, int Hkv, int rt, int kt, int halves, int least, int ctas,
                int s, int r, int h, long long *out, int room) {
    Split p(S, n, len, G, Hkv, rt, kt, halves, least, ctas);
    const PagedParts q = paged_parts(p.a, p.f, p.seg[s], p.per, r, h);
    int count = 0;
    for (int i = 0; i < q.cnt; ++i) {
        const long long row = paged_part(p.f, q, p.per, i);
        if (row >= 0 && count++ < room) out[count - 1] = row;
    }
    return count;
}

// The segment search with its 32 probes in turn.
int split_search(const int *ends, int n, long long t) {
    return search32(n, [&](int lo, int step, int left) {
        int c = 0;
        for (int lane = 0; lane < 32; ++lane) {
            const int q = (lane + 1) * step - 1;
            c += q < left && ends[lo + q] <= t;
        }
        return c;
    });
}

}  // extern "C"
