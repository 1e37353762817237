// How the work of mla_key_weight is cut: (sequence, block of key tiles, group of rows, key tile) in that order, into equal
// shares by cost. Plain arithmetic, on the device and, for its tests, on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVR_HD __host__ __device__ __forceinline__
#else
#define KVR_HD inline
#endif

namespace kvr {

constexpr int KW_KEYS = 256;    // keys of a tile
constexpr int KW_BLOCK = 24;    // tiles of a block: its sums stay in shared memory while the groups pass
// What a group costs beside its tiles, in tiles: its queries.
constexpr double KW_GROUP_COST = 0.5;

struct KwPos {
    int n, kb, g, kt;   // sequence, block, group, tile of the block
};

// A sequence's rows in groups of `rows`, its keys in tiles and blocks.
struct KwShape {
    int L, K, H, rows;
    bool causal;

    KVR_HD int groups() const { return int((unsigned(L) * unsigned(H) + unsigned(rows) - 1u) / unsigned(rows)); }
    KVR_HD int tiles() const { return (K + KW_KEYS - 1) / KW_KEYS; }
    KVR_HD int blocks() const { return (tiles() + KW_BLOCK - 1) / KW_BLOCK; }
    KVR_HD int block_tiles(int kb) const {
        const int left = tiles() - kb * KW_BLOCK;
        return left < KW_BLOCK ? left : KW_BLOCK;
    }
    // Tiles of a block that the group's last row sees.
    KVR_HD int seen_tiles(int kb, int g) const {
        const int most = block_tiles(kb);
        if (!causal) return most;
        const unsigned last = unsigned(g) * unsigned(rows) + unsigned(rows) - 1u;
        const int t = int(last / unsigned(H)) < L - 1 ? int(last / unsigned(H)) : L - 1;
        const int64_t see = int64_t(K) - L + t + 1, before = int64_t(kb) * (KW_BLOCK * KW_KEYS);
        if (see <= before) return 0;
        const int64_t n = (see - before + KW_KEYS - 1) / KW_KEYS;
        return n < most ? int(n) : most;
    }
    // Whether every group sees all tiles (but for a fraction of the last ones).
    KVR_HD bool even() const { return !causal || groups() == 1; }
    // Cost of a block's first x groups: x grows by KW_GROUP_COST at least from group to group. Where the rows see more and
    // more keys, the integral over the groups of what their ends see, and half a tile, as tiles are whole.
    KVR_HD double cost(int kb, int x) const {
        const double most = block_tiles(kb);
        if (even()) return x * (most + KW_GROUP_COST);
        const double step = double(rows) / (double(H) * KW_KEYS), first = (double(K) - L) / KW_KEYS + step + 0.5 - double(kb) * KW_BLOCK;
        double x1 = -first / step, x2 = (most - first) / step;   // where it leaves 0, where it reaches `most`
        x1 = x1 < 0 ? 0 : (x1 > x ? x : x1);
        x2 = x2 < x1 ? x1 : (x2 > x ? x : x2);
        return (x2 - x1) * (first + step * (x1 + x2) * 0.5) + (x - x2) * most + x * KW_GROUP_COST;
    }
    KVR_HD double cost() const {
        if (L == 0 || K == 0) return 0;
        if (even()) return groups() * (tiles() + KW_GROUP_COST * blocks());
        double sum = 0;
        for (int kb = 0; kb < blocks(); ++kb) sum += cost(kb, groups());
        return sum;
    }
    // Where the share that begins at `off` of the sequence's cost begins. Grows with `off`: shares neither overlap nor leave gaps.
    KVR_HD KwPos locate(int n, double off) const {
        const int G = groups(), B = blocks();
        int kb = 0;
        if (even()) {
            const double each = G * (KW_BLOCK + KW_GROUP_COST);
            const double at = off / each;
            kb = at < B - 1 ? int(at) : B - 1;
            off -= kb * each;
        } else {
            for (; kb < B - 1; ++kb) {
                const double each = cost(kb, G);
                if (off < each) break;
                off -= each;
            }
        }
        if (off < 0) off = 0;
        int lo = 0, hi = G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (cost(kb, mid) <= off) lo = mid;
            else hi = mid - 1;
        }
        const double c0 = cost(kb, lo), c1 = cost(kb, lo + 1);
        const int kn = seen_tiles(kb, lo);
        const double f = (off - c0) / (c1 - c0) * kn + 0.5;
        const int kt = f < 0 ? 0 : (f < kn ? int(f) : kn);
        return {n, kb, lo, kt};
    }
};

// Whether a position lies inside a block, behind its begin.
KVR_HD bool kw_inside(const KwPos& p) { return p.g > 0 || p.kt > 0; }
KVR_HD bool kw_same_block(const KwPos& a, const KwPos& b) { return a.n == b.n && a.kb == b.kb; }
KVR_HD bool kw_same(const KwPos& a, const KwPos& b) { return kw_same_block(a, b) && a.g == b.g && a.kt == b.kt; }

// CTA pairs that get work: at most one a tile and a half, so that a pair has more to do than to begin.
KVR_HD int kw_active(double total, int pairs) {
    const double most = total / 1.5;
    return most < 1 ? 1 : (most < pairs ? int(most) : pairs);
}

// The parts of a share, block by block. `shape(n)` gives a sequence's KwShape.
template <class Shapes>
struct KwWalk {
    Shapes shapes;
    KwPos at, end;
    int N;
    // the current block
    KwShape s;
    int n, kb, tiles;
    int g_at, g_end, kt_first, kt_last;   // groups left; tiles of the first and of the last one where the share cuts it
    // the current part
    int g, kt0, kt1;
    bool begun = false;

    KVR_HD KwWalk(const Shapes& sh, const KwPos& a, const KwPos& e, int count) : shapes(sh), at(a), end(e), N(count) {}
    KVR_HD bool next_block() {
        if (begun) at = {n, kb + 1, 0, 0};
        for (;;) {
            if (at.n >= N || at.n > end.n || (at.n == end.n && (at.kb > end.kb || (at.kb == end.kb && (at.g > end.g || (at.g == end.g && at.kt >= end.kt)))))) return false;
            if (!begun || at.n != n) s = shapes(at.n);
            begun = true;
            n = at.n;
            if (s.L == 0 || at.kb >= s.blocks()) {
                at = {n + 1, 0, 0, 0};
                continue;
            }
            kb = at.kb;
            tiles = s.block_tiles(kb);
            const bool last = end.n == n && end.kb == kb;
            g_at = at.g;
            kt_first = at.kt;
            g_end = last ? (end.kt > 0 ? end.g + 1 : end.g) : s.groups();
            kt_last = last && end.kt > 0 ? end.kt : KW_BLOCK;
            return true;
        }
    }
    KVR_HD bool next_part() {
        while (g_at < g_end) {
            g = g_at++;
            kt0 = kt_first;
            kt_first = 0;
            kt1 = s.seen_tiles(kb, g);
            if (g_at == g_end && kt1 > kt_last) kt1 = kt_last;
            if (kt0 < kt1) return true;
        }
        return false;
    }
    // Whether the share has all of the block.
    KVR_HD bool whole(const KwPos& begin) const {
        return !(begin.n == n && begin.kb == kb && kw_inside(begin)) && !(end.n == n && end.kb == kb);
    }
};

}  // namespace kvr
