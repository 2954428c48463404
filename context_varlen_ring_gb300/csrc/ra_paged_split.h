// ra_paged_split.h -- how paged attention splits its work: units on a line,
// the CTAs' runs along it, and the partial rows that the join finds again.
// The same code on the device and on the host, where the tests run it.
#pragma once

#include <cstdint>

#include "ra_kernels.h"

#ifdef __CUDACC__
#define RA_HD __host__ __device__ __forceinline__
#else
#define RA_HD inline
#endif

namespace ra {
namespace dev {

template <typename T>
RA_HD T lesser(T a, T b) {
    return b < a ? b : a;
}
template <typename T>
RA_HD T greater(T a, T b) {
    return a < b ? b : a;
}

// How many of the n non-decreasing ends are <= some t, by 32 probes a round:
// below(at, step, n) says how many of the 32 ends at, at + step, ... that lie
// ahead of n are.  With ends that decrease the result is still in [0, n].
template <typename Below>
RA_HD int search32(int n, Below below) {
    int lo = 0;
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int c = below(lo, step, n);
        lo += c * step;
        n = lesser(step - 1, n - c * step);
    }
    return lo;
}

// x / y of non-negative numbers, in 32 bits wherever they fit (a 64-bit
// division is some hundred instructions).
RA_HD long long paged_div(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// Partial rows of a tile of `rows` query rows.
RA_HD int paged_alloc(const PagedFamily &f, int rows) { return f.halves && 2 * rows <= f.rt ? 2 * rows : rows; }

struct PagedUnit {
    int s, tok0, n, len; // its segment
    int r0, rows, h;     // first query row in the segment, query rows, KV head
    int t0, t1;          // the CTA's key tiles in it
    long long base;      // first partial row (of CTA 0)
};

// What a unit and its key tiles weigh, in sixteenths of a warp-level tile: a
// unit takes its own cost (queries, join, partial) and then its tiles, so a run
// that goes on into another unit has fewer tiles for it.  Of the tcgen05 kernel,
// a tile for two row tiles takes 1.75 us, one of alternating tiles for a single
// row tile 1.0 to 1.4 (bound by its softmax, or by memory), a unit about 4.
struct PagedCost {
    int tile, unit;
};
RA_HD PagedCost paged_cost(const PagedArgs &a, const PagedFamily &f, const PagedSeg &g) {
    return PagedCost{!f.halves ? 16 : g.n * a.G * 2 > f.rt ? 48 : 32, f.halves ? 96 : 32};
}
RA_HD int paged_all(const PagedSeg &g, const PagedCost &c) {  // (at most 2^24 tiles)
    return g.w ? g.w * c.tile + c.unit : 0;
}
// The first tile of a unit that begins at or behind place `at` of it: a tile
// belongs to the run in which it begins.
RA_HD int paged_tile(int at, const PagedCost &c) {
    const unsigned x = (unsigned)greater(at - c.unit + c.tile - 1, 0) >> 4;
    return (int)(c.tile == 48 ? x / 3 : c.tile == 32 ? x >> 1 : x);
}
// The weight of all its units, and its partial rows.  (n * G < 2^31.)
RA_HD long long paged_tiles(const PagedArgs &a, const PagedFamily &f, const PagedSeg &g) {
    return (long long)((g.n * a.G + f.rt - 1) >> f.rt_log) * a.Hkv * paged_all(g, paged_cost(a, f, g));
}
RA_HD long long paged_rows(const PagedArgs &a, const PagedFamily &f, const PagedSeg &g) {
    const int R = g.n * a.G, full = R & -f.rt;
    return (long long)a.Hkv * (full + paged_alloc(f, R - full));
}
// The weight of a CTA's run.
RA_HD long long paged_per(const PagedFamily &f, long long W) {
    return greater((long long)f.least, paged_div(W + f.n - 1, f.n));
}

// A CTA's run of the line, and its place in it: the segment and the unit.
struct PagedWalk {
    long long x, x1;
    int s;
    PagedSeg g;
};

// The CTA's next unit and its tiles there; false where its run has no more.
// next(k, end) moves k to the next segment, whose place in the line is `end`.
// Row tiles are outermost in a segment, so CTAs an equal share of the line
// apart read the same keys for different rows at about the same time (from L2).
template <typename Next>
RA_HD bool paged_walk(const PagedArgs &a, const PagedFamily &f, PagedWalk &k, PagedUnit &u, Next next) {
    while (k.x < k.x1) {
        for (long long end; (end = k.g.W0 + paged_tiles(a, f, k.g)) <= k.x;) next(k, end);
        const long long rel = k.x - k.g.W0;
        const PagedCost cost = paged_cost(a, f, k.g);
        const int all = paged_all(k.g, cost);
        const int lu = (int)paged_div(rel, all), rtile = lu < a.Hkv ? 0 : lu / a.Hkv;
        const int from = (int)(rel - (long long)lu * all), to = (int)lesser((long long)all, from + (k.x1 - k.x));
        k.x += to - from;
        u.t0 = paged_tile(from, cost);
        u.t1 = paged_tile(to, cost);
        if (u.t0 >= u.t1) continue;  // the run ends inside a tile that another one began
        u.s = k.s;
        u.tok0 = k.g.tok0;
        u.n = k.g.n;
        u.len = k.g.len;
        u.h = lu - rtile * a.Hkv;
        u.r0 = rtile << f.rt_log;
        u.rows = lesser(f.rt, k.g.n * a.G - u.r0);
        u.base = k.g.R0 + (long long)u.r0 * a.Hkv + (long long)u.h * paged_alloc(f, u.rows);
        return true;
    }
    return false;
}

// The partials of a token and query head in a family: cnt of them, the i-th
// (of CTA c0 + (i >> two)) at partial row  at + (i >> two) * rt + (i & two) * second.
struct PagedParts {
    long long at, x;  // x: the unit's place in the line
    int cnt, two, second, c0, all;
    PagedCost cost;
};
// Of query row `r` of segment `sg`.
RA_HD PagedParts paged_parts(const PagedArgs &a, const PagedFamily &f, const PagedSeg &sg, long long per, int r, int h) {
    PagedParts p{};
    if (sg.w == 0) return p;
    const int rtile = r >> f.rt_log;
    const int rows = lesser(f.rt, sg.n * a.G - rtile * f.rt), alloc = paged_alloc(f, rows);
    p.cost = paged_cost(a, f, sg);
    p.all = paged_all(sg, p.cost);
    p.x = sg.W0 + (long long)(rtile * a.Hkv + h) * p.all;
    const int c1 = (int)paged_div(p.x + p.all - 1, per);
    p.c0 = (int)paged_div(p.x, per);
    p.at = sg.R0 + (long long)rtile * f.rt * a.Hkv + (long long)h * alloc + (long long)p.c0 * f.rt + (r & (f.rt - 1));
    p.two = alloc > rows ? 1 : 0;
    p.second = rows;
    p.cnt = (c1 - p.c0 + 1) << p.two;
    return p;
}
// The partial row of the i-th of them, or -1 where its CTA began no tile of the unit.
RA_HD long long paged_part(const PagedFamily &f, const PagedParts &p, long long per, int i) {
    const long long run = (p.c0 + (i >> p.two)) * per - p.x;  // its CTA's place in the unit
    const int from = (int)greater(0ll, run), to = (int)lesser((long long)p.all, run + per);
    if (i >= p.cnt || paged_tile(from, p.cost) >= paged_tile(to, p.cost)) return -1;
    return p.at + (long long)(i >> p.two) * f.rt + (i & p.two) * p.second;
}

}  // namespace dev
}  // namespace ra
