// How the work of mla_key_weight is cut: (sequence, key tile, group of rows) in that order, into equal shares by cost. Plain
// arithmetic, on the device and, for its tests, on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVR_HD __host__ __device__ __forceinline__
#else
#define KVR_HD inline
#endif

namespace kvr {

constexpr int KW_KEYS = 256;    // keys of a tile
struct KwPos {
    int n, kt, g;   // sequence, tile, group
    int cut;        // whether groups of the tile come before it
};

// A sequence's rows in groups of 2^shift, its keys in tiles.
struct KwShape {
    int L, K, H, shift;
    bool causal;

    KVR_HD int groups() const { return int((unsigned(L) * unsigned(H) + (1u << shift) - 1u) >> shift); }
    KVR_HD int tiles() const { return (K + KW_KEYS - 1) / KW_KEYS; }
    // The first group with a row that sees a key of the tile.
    KVR_HD int first_group(int kt) const {
        if (!causal) return 0;
        const int64_t token = int64_t(kt) * KW_KEYS - (int64_t(K) - L);
        return token <= 0 ? 0 : int(token * H >> shift);
    }
    // Cost of the first x tiles, in groups; a tile costs one more, for bringing its keys, so that this grows by one at least
    // from tile to tile. Where tiles lie behind the first token's keys, fewer and fewer groups see them: with the last tile's
    // first key d tokens behind, d H / 2^shift of its groups do not, and the integral over d is taken off; groups of tokens that
    // are too many for the keys see no tile. (d < L, so that d^2 H < 2^62. Whole numbers: an SM has few units for doubles, and a
    // call's first microseconds count.)
    KVR_HD int64_t cost(int x) const {
        const int none = causal && L > K ? int(int64_t(L - K) * H >> shift) : 0;
        const int64_t all = int64_t(x) * (groups() - none + 1), d = int64_t(x - 1) * KW_KEYS - (K > L ? K - L : 0);
        return !causal || d <= 0 ? all : all - (d * d * H >> (9 + shift));
    }
    KVR_HD int64_t cost() const { return L == 0 || K == 0 ? 0 : cost(tiles()); }
    // Where the share that begins at `off` of the sequence's cost begins. Grows with `off`: shares neither overlap nor leave gaps.
    KVR_HD KwPos locate(int n, int64_t off) const {
        const int G = groups(), T = tiles();
        if (G == 1) {   // whole tiles, of cost 2
            const int64_t x = (off + 1) / 2;
            return {n, x < T ? int(x) : T, 0, 0};
        }
        int lo = 0, hi = T - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (cost(mid) <= off) lo = mid;
            else hi = mid - 1;
        }
        const int64_t c0 = cost(lo), c1 = cost(lo + 1);
        const int g0 = first_group(lo), count = G - g0;
        const float f = float(off - c0) / float(c1 - c0) * float(count) + 0.5f;
        const int g = f < 0 ? 0 : (f < float(count) ? int(f) : count);
        return {n, lo, g0 + g, g > 0};
    }
};

// Where share `which` of `active` begins.
KVR_HD int64_t kw_share(int64_t total, int which, int active) {
    if (which >= active) return total;
    if (total < (int64_t(1) << 31) / 256) return unsigned(total) * unsigned(which) / unsigned(active);
    const int64_t each = total / active;
    return each * which + (total - each * active) * which / active;
}

KVR_HD bool kw_same_tile(const KwPos& a, const KwPos& b) { return a.n == b.n && a.kt == b.kt; }
KVR_HD bool kw_same(const KwPos& a, const KwPos& b) { return kw_same_tile(a, b) && a.g == b.g; }

// Seconds that a wait may take beyond the first. A tile's keys are in use while all groups of a sequence pass, and a group that stays
// keeps its place for all of a sequence's tiles. Measured: a row takes 11 ns in groups of 256 and 50 in
// groups of 32, over codes with scales per channel 20 and 101; a tile of one row 5 us at most.
KVR_HD int kw_patience(int64_t rows, int64_t keys) { return int((rows >> 22) + (keys >> 22)); }

// CTA pairs that get work: none less than a tile of one group.
KVR_HD int kw_active(int64_t total, int pairs) { return total < 2 ? 1 : (total / 2 < pairs ? int(total / 2) : pairs); }

// The runs of a share: some tiles of a sequence with one group, or the groups [ga, gb) of one tile.
template <class Shapes>
struct KwWalk {
    Shapes shapes;
    KwPos at, end;
    int N, loaded = -1;
    KwShape s;
    // the current run
    int n, kt0, kt1, ga, gb;
    bool whole;   // the share has all groups that see its tiles

    KVR_HD KwWalk(const Shapes& sh, const KwPos& a, const KwPos& e, int count) : shapes(sh), at(a), end(e), N(count) {}
    KVR_HD bool next() {
        for (;;) {
            if (at.n >= N || at.n > end.n ||
                (at.n == end.n && (at.kt > end.kt || (at.kt == end.kt && (at.cut ? at.g >= end.g : !end.cut)))))
                return false;
            if (loaded != at.n) {
                s = shapes(at.n);
                loaded = at.n;
            }
            const int T = s.L == 0 ? 0 : s.tiles();
            if (at.kt >= T) {
                at = {at.n + 1, 0, 0, 0};
                continue;
            }
            n = at.n;
            kt0 = at.kt;
            if (s.groups() == 1) {
                kt1 = end.n == n && end.kt < T ? end.kt : T;
                ga = 0;
                gb = 1;
                whole = true;
            } else {
                kt1 = kt0 + 1;
                ga = at.cut ? at.g : s.first_group(kt0);
                const bool last = end.n == n && end.kt == kt0;
                gb = last ? end.g : s.groups();
                whole = !at.cut && !last;
            }
            at = {n, kt1, 0, 0};
            return true;
        }
    }
};

}  // namespace kvr
