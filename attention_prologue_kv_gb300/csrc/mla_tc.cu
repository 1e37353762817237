// Latent attention on the tensor cores: rows of up to 512 + 64 channels.
//
// For the rows (token, head) of a sequence and its keys:
//   S = scale (Qn C^T + Qr K^T),  O = softmax(S) C,
// computed key tile by key tile with the running maximum m and sum l of each
// row: O = O 2^(m - m') + P C with P = 2^(S - m').
//
// What bounds it: each (row, key) pair costs 2 (2 Dv + Dk) flops and each key
// 1152 bytes (bf16): below about 128 rows per key the cache's bytes, above it
// the tensor cores. A row's output sum alone is 2 KB, so 128 rows of it would
// fill the whole TMEM of an SM.
//
// Tiling: a CTA pair (cta_group::2) owns 128 rows, 64 in each CTA, and 64 keys a
// step. With 64 rows of its own, a CTA's sum takes 256 of its 512 TMEM columns
// (M = 128 over a pair puts the second half of the columns on the upper 64
// lanes), and the pair runs at the full rate of M = 128 per SM while each SM
// reads only its half of the second operand: S splits the keys between the CTAs,
// P C splits the channels (CTA r has channels [128 r, 128 r + 128) of each 256).
//
// A key step in a CTA, up to four in flight:
//   load   its 32 keys, all channels, into 9 boxes [32 keys x 64 channels];
//   S      128 x 64 by the pair; the other CTA's keys come from its shared memory;
//   swap   the boxes of channels that the other CTA sums are dead now: they take
//          this CTA's channels of the other 32 keys, so that the second product
//          finds all 64 keys of its channels in the same 9 boxes;
//   softmax in 128 threads (row, half of the keys); P to shared memory;
//   O += P C.
//
// Work: (sequence, row tile) items in a row, cut into equal parts by cost over the
// CTA pairs, wherever that falls inside an item. A part of an item leaves
// its O, m and l in the workspace, and a second kernel joins them in a fixed
// order, so results do not change from run to run.
//
// Measured: 512 tokens x 128 heads over 16384 keys 1540 us (1.5 PFLOP/s, 80% of the measured bf16 rate; a step takes
// 0.82 us; the unit that runs tcgen05 is busy 92% of the time, 68% with the products themselves); 256 sequences of one
// token, 128 heads, 1-4095 keys 159 us (4.5 TB/s, 66% of the copy rate; a step 0.89 us, a part's queries and output 5 us);
// 61 sequences of one token over up to 16384 keys in E4M3 170 us (that unit 59%, no counter above: the chain load, decode,
// scores, swap, softmax, second product of its three steps in flight); one sequence of 1000 keys, 16 heads 14.9 us. Steps
// of 128 keys with two of them in flight were slower (1826 us): a stage's load, scores, softmax and second product follow
// one another. Paths without TMA, with codes or with small blocks, at 65536 keys, us a step: blocks of 16 keys 1.8, of
// 8 2.6, of 100 3.5, of 1 3.9; rotary codes over 16-bit latent rows 4.0 (blocks of 1: 5.0); latent codes 1.2 (blocks of 1: 1.4).
#include <mutex>
#include <type_traits>

#include "tcgen05.cuh"

namespace kvr {

namespace {

constexpr int ROWS = 128, CROWS = 64;    // rows of a pair, of a CTA
constexpr int KEYS = 64, CKEYS = 32;     // keys of a step, of a CTA
constexpr uint32_t QBOX = CROWS * 128, KBOX = CKEYS * 128;
constexpr uint32_t STAGE_BYTES = 9 * KBOX, PBUF = CROWS * 128;
constexpr uint32_t OFF_Q = 0, OFF_P = 9 * QBOX, OFF_K = OFF_P + PBUF;
constexpr int MAX_STAGES = 4;
// Steps in flight: 4 fill the shared memory; with codes 3, which leaves room for the scales.
template <bool C8>
constexpr int stages_of() { return C8 ? 3 : 4; }
constexpr uint32_t TMEM_COLS = 512, COL_S = 256;   // O: columns 0..255, S: two buffers of 32 + 32
// An item's own cost, in keys (its queries, first scores and output: about 7 steps). With 192, 448 and 768: chunks of 33-129
// tokens of 8 sequences, 128 heads, 292, 268 and 279 us; chunks of 5-17 tokens of 30, 64 heads, 68.3, 63.9 and 64.8; one
// token of 256 sequences, 1-4095 keys, 164, 154 and 155; of 64, 300-900 keys, 40.1, 37.4 and 37.4; 1-7 tokens of 33, 20
// heads, 35.9, 35.5 and 35.2.
constexpr int64_t ITEM_COST = 448;
// Least work of a pair, in keys: the join of more parts costs more than they save. One token, 16 heads, with 192, 320, 512
// and 768: 300 keys 13.0, 13.5, 14.6 and 14.6 us; 1000 keys 15.3, 14.9, 17.9 and 23.9; 2300 keys 15.3, 15.3, 16.7 and 19.8;
// 4000 keys 20.1, 18.8, 20.0 and 22.9; 9000 keys 28.2, 23.6, 22.5 and 23.9; 20000 keys 39.3, 34.8, 31.8 and 29.9 (where
// fewer parts to join would be better). Calls that fill the grid do not depend on it. (Both sweeps with the caches in L2.)
constexpr int64_t MIN_KEYS = 320;

struct Bound {
    int n, i, kt, pad;   // sequence, row tile, key tile
};
struct alignas(16) Start {   // a pair's begin, as the join reads it: with its sequence's first row and its tokens
    int n, i, kt, L;
    int64_t q0, pad;
};

struct Seq {
    int64_t q0;
    int L, K;   // L = 0: nothing to do
};

struct alignas(16) Misc {
    uint64_t k_full[MAX_STAGES], v_full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t h_full[MAX_STAGES];   // `held` of a stage is written: within the CTA
    uint64_t s_full[2], p_full, pv_done, q_full, q_free, k_fix, v_fix, drain;
    uint32_t tmem;
    int abort, large;
    Bound begin, end;
    Seq first;               // the sequence of `begin`
    int64_t wsum[17];
    float red[2][256];
    uint32_t held[MAX_STAGES][2];   // keys of a step that exist: bit i of a half for its key i
    float inv_k[64], lift;   // 1 / scale of the rotary channels; a power of two taken out of their queries
};
struct alignas(16) Scales {   // behind Misc, with codes
    float inv_v[512];         // 1 / scale of a channel
};
template <bool C8>
constexpr uint32_t smem_of() {
    return OFF_K + stages_of<C8>() * STAGE_BYTES + uint32_t(sizeof(Misc)) + (C8 ? uint32_t(sizeof(Scales)) : 0u);
}
static_assert(smem_of<false>() <= 232448 && smem_of<true>() <= 232448, "shared memory of a CTA");

// Workspace: header, the pairs' begins, (m, l) and O of two parts a pair.
struct Space {
    int32_t* active;
    Start* starts;
    float2* ml;
    float* o;
};
__host__ __device__ inline int64_t ws_ml(int pairs) { return 256 + (int64_t(pairs) * 32 + 255) / 256 * 256; }
__host__ __device__ inline int64_t ws_o(int pairs) { return ws_ml(pairs) + int64_t(pairs) * 2 * ROWS * 8; }
__host__ __device__ inline int64_t ws_bytes(int pairs, int Dv) { return ws_o(pairs) + int64_t(pairs) * 2 * ROWS * Dv * 4; }
__device__ __forceinline__ Space ws_space(const MlaParams& p) {
    char* w = static_cast<char*>(p.workspace);
    return {reinterpret_cast<int32_t*>(w), reinterpret_cast<Start*>(w + 256), reinterpret_cast<float2*>(w + ws_ml(p.pairs)),
            reinterpret_cast<float*>(w + ws_o(p.pairs))};
}

__device__ __forceinline__ Seq load_seq(const MlaParams& p, int n, int* bits = nullptr) {
    const int64_t a = p.query_start[n], b = p.query_start[n + 1], K = p.key_length[n];
    if (a < 0 || b < a || b > p.T) {
        if (bits != nullptr) *bits |= KVR_DEVERR_QUERY;
        return {0, 0, 0};
    }
    if (a == b) return {0, 0, 0};
    if (K < 0 || K > p.max_keys) {
        if (bits != nullptr) *bits |= KVR_DEVERR_KEY_LENGTH;
        return {0, 0, 0};
    }
    return {a, int(b - a), int(K)};
}
__device__ __forceinline__ int row_tiles(const MlaParams& p, int L) { return int((unsigned(L) * unsigned(p.H) + (ROWS - 1)) / ROWS); }
// Keys that token t of the sequence sees.
__device__ __forceinline__ int seen(const MlaParams& p, int L, int K, int t) {
    return p.causal ? min(max(K - L + t + 1, 0), K) : K;
}
__device__ __forceinline__ int key_tiles(const MlaParams& p, int L, int K, int i) {
    const int t1 = min(L - 1, int((unsigned(i) * ROWS + (ROWS - 1)) / unsigned(p.H)));
    return max(1, (seen(p, L, K, t1) + KEYS - 1) / KEYS);   // one step even without keys: it writes the zeros
}
// Cost of the first i row tiles, times H (so that it is whole): a causal tile
// sees 128 / H more keys than the one before.
__device__ __forceinline__ int64_t cost(const MlaParams& p, int L, int K, int64_t i) {
    if (p.causal) return i * (p.H * (max(K - L, 0) + ITEM_COST) + ROWS / 2 * i);
    return i * p.H * (K + ITEM_COST);
}

// Where the share that begins at `off` of a sequence's cost begins.
__device__ Bound locate(const MlaParams& p, int n, const Seq& s, int64_t off) {
    int lo = 0, hi = row_tiles(p, s.L) - 1;
#pragma unroll 1
    while (lo < hi) {   // (one row tile, as in a decode step, needs no search)
        const int mid = (lo + hi + 1) / 2;
        if (cost(p, s.L, s.K, mid) <= off) lo = mid;
        else hi = mid - 1;
    }
    const int64_t c0 = cost(p, s.L, s.K, lo), c1 = cost(p, s.L, s.K, lo + 1);
    const int kn = key_tiles(p, s.L, s.K, lo);
    const int kt = int(float(off - c0) / float(c1 - c0) * float(kn));   // monotonic in off: shares neither overlap nor leave gaps
    return {n, lo, min(kt, kn - 1), 0};
}

// The parts of items between two bounds, in order.
struct Walk {
    const MlaParams& p;
    Bound at, end;
    int loaded;
    Seq s;
    // the current part
    int n, i, kt0, kt1;
    bool whole;
    __device__ Walk(const MlaParams& q, const Misc* m) : p(q), at(m->begin), end(m->end), loaded(m->begin.n), s(m->first) {}
    __device__ bool next() {
        for (;;) {
            if (at.n >= p.N || at.n > end.n || (at.n == end.n && (at.i > end.i || (at.i == end.i && at.kt >= end.kt)))) return false;
            if (loaded != at.n) {
                s = load_seq(p, at.n);
                loaded = at.n;
            }
            if (at.i >= row_tiles(p, s.L)) {
                at = {at.n + 1, 0, 0, 0};
                continue;
            }
            const int kn = key_tiles(p, s.L, s.K, at.i);
            n = at.n;
            i = at.i;
            kt0 = at.kt;
            kt1 = (at.n == end.n && at.i == end.i) ? min(end.kt, kn) : kn;
            whole = kt0 == 0 && kt1 == kn;
            at = {at.n, at.i + 1, 0, 0};
            if (kt0 < kt1) return true;
        }
    }
};

// Where share `which` of `active` begins, in cost: total * which / active, which the product may not fit. Out of line where
// it takes 64-bit divisions of about 100 instructions each: in line they moved the loops and cost a long chunk 1%.
__device__ __noinline__ int64_t long_share(int64_t total, int which, int active) {
    const int64_t each = total / active;
    return each * which + unsigned(total - each * active) * unsigned(which) / unsigned(active);
}
__device__ __forceinline__ int64_t share(int64_t total, int which, int active) {
    if (which >= active) return total;
    if (total < (int64_t(1) << 31) / 256) return unsigned(total) * unsigned(which) / unsigned(active);
    return long_share(total, which, active);
}
// Pairs that get work: equal shares, but none below MIN_KEYS.
__device__ __forceinline__ int active_pairs(const MlaParams& p, int64_t total) {
    const int64_t least = int64_t(p.H) * MIN_KEYS;
    return total >= least * p.pairs ? p.pairs : max(1, int(unsigned(total) / unsigned(least)));
}

// A pair's share where a warp holds all sequences and their cost is small (a few conversations: latency counts): one warp
// for its begin, one for its end, without a word between warps. A kernel's first instructions come from far, up to 100
// cycles each, so the few steps here took 9800 cycles by the way below. False: that way is to be taken.
__device__ __forceinline__ bool schedule_small(const MlaParams& p, Misc* m, int pair) {
    const int lane = threadIdx.x & 31, half = threadIdx.x >> 5;
    Seq s = {0, 0, 0};
    int bits = 0;
    if (lane < p.N) s = load_seq(p, lane, &bits);
    const int64_t mine = s.L > 0 ? cost(p, s.L, s.K, row_tiles(p, s.L)) : 0;
    if (__any_sync(0xFFFFFFFFu, mine >= 1 << 18)) return false;
    int scan = int(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    const int total = __shfl_sync(0xFFFFFFFFu, scan, 31), active = active_pairs(p, total);
    const int u = int(share(total, pair + half, active)), base = scan - int(mine);
    if (u >= base && u < scan) {
        const Bound b = locate(p, lane, s, u - base);
        if (half) {
            m->end = b;
        } else {
            m->begin = b;
            m->first = s;
        }
    } else if (u == total && lane == 0) {
        (half ? m->end : m->begin) = {int(p.N), 0, 0, 0};
    }
    if (half == 0) {
        if (bits != 0 && blockIdx.x == 0 && p.status != nullptr) atomicOr(p.status, bits);
        if (lane == 0 && pair == 0 && cluster_rank() == 0) *ws_space(p).active = active;
    }
    return true;
}

// This pair's share of the work: every CTA scans all sequences' costs, twice side by side: the first half of the warps
// for the share's begin, the second for its end.
template <int THREADS>
__device__ void schedule(const MlaParams& p, Misc* m, int pair) {
    constexpr int HALF = THREADS / 64;   // warps of a half (one may be left over)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = warp < HALF ? 0 : 1, first = half * HALF, id = tid - first * 32;
    const bool works = warp < 2 * HALF;
    const int N = int(p.N), per = (N + HALF * 32 - 1) / (HALF * 32);
    const int n0 = works ? min(id * per, N) : N, n1 = works ? min(n0 + per, N) : N;
    int64_t sum = 0;
    int bits = 0;
    Seq s = {0, 0, 0};
#pragma unroll 1
    for (int n = n0; n < n1; ++n) {
        s = load_seq(p, n, &bits);
        if (s.L > 0) sum += cost(p, s.L, s.K, row_tiles(p, s.L));
    }
    if (bits != 0 && blockIdx.x == 0 && half == 0 && p.status != nullptr) atomicOr(p.status, bits);
    int64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) m->wsum[warp] = scan;
    if (tid == 0) m->begin = m->end = {N, 0, 0, 0};
    __syncthreads();
    if (works) {
        // Sums of the warps before this one and of all: lane i has warp i's.
        int64_t of = lane < HALF ? m->wsum[first + lane] : 0, before = lane < warp - first ? of : 0;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            of += __shfl_xor_sync(0xFFFFFFFFu, of, o);
            before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        }
        const int64_t total = __shfl_sync(0xFFFFFFFFu, of, 0);
        int64_t base = scan - sum + __shfl_sync(0xFFFFFFFFu, before, 0);
        const int active = active_pairs(p, total);
        const int64_t u = share(total, pair + half, active);
        if (u >= base && u < base + sum) {
            int n = n0;
            if (per > 1)
#pragma unroll 1
                for (; n < n1; ++n) {
                    s = load_seq(p, n);
                    const int64_t c = s.L > 0 ? cost(p, s.L, s.K, row_tiles(p, s.L)) : 0;
                    if (u < base + c) break;
                    base += c;
                }
            const Bound b = locate(p, n, s, u - base);
            if (half) {
                m->end = b;
            } else {
                m->begin = b;
                m->first = s;
            }
        }
        if (tid == 0 && pair == 0 && cluster_rank() == 0) *ws_space(p).active = active;
    }
}

// Four 8-bit codes of kind K to halves, exactly.
template <int K>
__device__ __forceinline__ uint2 codes_to_halves(uint32_t u) {
    uint32_t h[2];
    if constexpr (K == OUT_I8) {   // 1024 + (code + 128) as a half, less 1152
        u ^= 0x80808080u;
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t x = __byte_perm(u, 0x64646464u, k ? 0x4342 : 0x4140);
            __half2 r = __hsub2(*reinterpret_cast<__half2*>(&x), off);
            h[k] = *reinterpret_cast<uint32_t*>(&r);
        }
    } else if constexpr (K == OUT_E5M2) {   // the upper byte of a half
        h[0] = __byte_perm(u, 0, 0x1404);
        h[1] = __byte_perm(u, 0, 0x3424);
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(h[0]), "=r"(h[1])
            : "r"(u));
    }
    return make_uint2(h[0], h[1]);
}
template <int K>
__device__ __forceinline__ uint4 codes_to_halves(uint32_t a, uint32_t b) {
    const uint2 x = codes_to_halves<K>(a), y = codes_to_halves<K>(b);
    return make_uint4(x.x, x.y, y.x, y.y);
}
// Eight codes of a runtime kind to values of type IT (the rotary part's).
template <class IT>
__device__ __forceinline__ uint4 dec8x8(int kind, uint32_t a, uint32_t b) {
    const uint4 h = kind == OUT_I8 ? codes_to_halves<OUT_I8>(a, b)
                                   : (kind == OUT_E5M2 ? codes_to_halves<OUT_E5M2>(a, b) : codes_to_halves<OUT_E4M3>(a, b));
    if constexpr (!is_bf16<IT>) return h;
    return make_uint4(BF16::pack(F16::lo(h.x), F16::hi(h.x)), BF16::pack(F16::lo(h.y), F16::hi(h.y)),
                      BF16::pack(F16::lo(h.z), F16::hi(h.z)), BF16::pack(F16::lo(h.w), F16::hi(h.w)));
}

// Cache row of a key, or -1 where there is none to read.
__device__ __forceinline__ int64_t key_row(const MlaParams& p, int n, int K, int key) {
    if (key >= K) return -1;
    if (p.table == nullptr) return n * p.d1 + key;
    const unsigned d1 = unsigned(p.d1 < (1 << 30) ? p.d1 : (1 << 30));   // keys stay below 2^30
    const unsigned q = unsigned(key) / d1;
    const int64_t e = p.table[n * p.max_blocks + q];
    if (e < 0 || e >= p.d0) {
        if (e != -1 && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_INDEX);
        return -1;
    }
    return e * p.d1 + (unsigned(key) - q * d1);
}

// Cache rows of the keys of a part, for one warp. Where blocks hold whole halves of a step (a multiple of 32 keys, or
// Norm mode) lane i looks up the first row of steps base + i, once for 32 steps: a lookup and its division a step, even
// one step ahead, cost the lone warp that brings the keys about 1000 cycles. Else each lane looks up its key k, one
// step ahead.
struct Rows {
    const MlaParams& p;
    int n = 0, K = 0, base = 0;
    int64_t r[2];        // of the halves: first row of step base + lane, or this lane's row of the step asked for next
    __device__ __forceinline__ explicit Rows(const MlaParams& q) : p(q) {}
    __device__ __forceinline__ void look(int step, int k, int halves) {
#pragma unroll
        for (int h = 0; h < 2; ++h) r[h] = halves >> h & 1 ? key_row(p, n, K, step * KEYS + h * CKEYS + k) : -1;
    }
    __device__ __forceinline__ void begin(const Walk& w, int lane, int k, int halves) {
        n = w.n;
        K = w.s.K;
        base = w.kt0;
        look(p.runs ? base + lane : base, p.runs ? 0 : k, halves);
    }
    // This lane's row of key k in a half of step kt, -1 where there is none; next() before going on to step kt + 1.
    template <int H>
    __device__ __forceinline__ int64_t row(int kt, int k) const {
        if (!p.runs) return r[H];
        const int64_t f = __shfl_sync(0xFFFFFFFFu, r[H], kt - base);
        return f >= 0 && kt * KEYS + H * CKEYS + k < K ? f + k : -1;
    }
    __device__ __forceinline__ void next(int kt, int lane, int k, int halves) {
        if (!p.runs) {
            look(kt + 1, k, halves);
        } else if (kt + 1 - base >= 32) {
            base = kt + 1;
            look(base + lane, 0, halves);
        }
    }
};

__device__ __forceinline__ uint32_t box_at(uint32_t box, int row, int chunk) {
    return box + uint32_t(row) * 128u + (uint32_t(chunk ^ (row & 7)) << 4);
}

// Cache rows through TMA, seen as [64-channel box][row][channel], so that one copy brings 32 rows of several
// boxes: all boxes of the latent part, two of them (the swap), the rotary part. Where a block ends inside 32 rows, a
// copy brings R rows of one box. One copy a box took the key warp 2200 cycles a step (32 rows of all: 2 copies).
struct Maps {
    CUtensorMap all, two, rope;
};

// The rest of a wait, out of line: the roles' loops have to stay in the instruction cache. `more`: seconds beyond the first.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, int more) {
    while (*abort == 0) {
        if (mbar_wait(bar, parity, abort)) return true;
        if (--more < 0) *abort = 1;
    }
    return false;
}

// What every role has.
struct Ctx {
    const MlaParams& p;
    Misc* m;
    Scales* sc;
    uint32_t base, tmem, rank;
    int lane, nb;        // nb: 64-channel boxes of the latent part
    volatile int* abort;
    bool ok;

    // A wait that gives up (after one second, or one and `more`) poisons the CTA: the others give up at their first look.
    // The warps that start TMA copies then stop; every other role runs its loops to the end without waiting, so that no
    // barrier is left with threads missing.
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, int more = 0) {
        if (!mbar_try_wait(bar, parity)) ok = wait_on(bar, parity, abort, more) && ok;
        __syncwarp();
    }
    __device__ __forceinline__ bool gone() const { return __any_sync(0xFFFFFFFFu, !ok); }
    __device__ __forceinline__ uint32_t stage(int st) const { return base + OFF_K + uint32_t(st) * STAGE_BYTES; }
    // This warp's shared-memory writes are done: tell the MMA warp of the pair.
    __device__ __forceinline__ void arrive(uint64_t* bar) {
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(bar, 0);
    }
};

// One warp brings a CTA's 16-bit cache rows, step by step: SWAP = false its own
// 32 keys (all channels, rotary part in box 8), SWAP = true the other CTA's keys
// (this CTA's channels, into the boxes that the scores are done with).
// Rows that do not exist become zeros: a NaN there would reach the sum through
// its zero weight.
template <class IT, bool K8, bool SWAP>
__device__ __forceinline__ void key_warp(Ctx& c, const Maps& maps) {
    constexpr int STAGES = stages_of<false>();
    const MlaParams& p = c.p;
    Misc* m = c.m;
    const int lane = c.lane, R = p.box_rows;
    // Boxes: latent ones first; the place of box b, its 64 channels.
    const int nl = SWAP ? min(2, max(0, c.nb - 2 * int(c.rank))) + min(2, max(0, c.nb - 4 - 2 * int(c.rank))) : c.nb;
    auto place = [&](int b) {
        if (SWAP) return (b >> 1) * 4 + int(c.rank ^ 1) * 2 + (b & 1);
        return b < nl ? b : 8;
    };
    auto channels = [&](int b) { return SWAP ? (b >> 1) * 4 + int(c.rank) * 2 + (b & 1) : b; };
    uint64_t* fix = SWAP ? &m->v_fix : &m->k_fix;
    uint64_t* full = SWAP ? m->v_full : m->k_full;
    int j = 0, fixed = 0, pend = -1;
    const int mine = int(SWAP ? c.rank ^ 1 : c.rank), halves = SWAP ? 1 << mine : 3;
    Rows rows(p);
    Walk w(p, m);
#pragma unroll 1
    while (w.next() && !c.gone()) {
        rows.begin(w, lane, lane, halves);
#pragma unroll 1
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++j) {
            const int st = j % STAGES;
            const uint32_t stage = c.stage(st);
            const int64_t lo = rows.row<0>(kt, lane), hi = rows.row<1>(kt, lane), slot = mine ? hi : lo;
            rows.next(kt, lane, lane, halves);
            const uint32_t live = __ballot_sync(0xFFFFFFFFu, slot >= 0);
            uint2 codes[8];
            if (K8 && !SWAP) {   // rotary codes: 8 of each row (lane >> 3) + 4 rr, decoded below
#pragma unroll
                for (int rr = 0; rr < 8; ++rr) {
                    const int64_t row = __shfl_sync(0xFFFFFFFFu, slot, rr * 4 + (lane >> 3));
                    codes[rr] = row >= 0 && (lane & 7) < p.Dk / 8
                                    ? ld_stream_v2(static_cast<const uint8_t*>(p.kc) + row * p.Dk + (lane & 7) * 8)
                                    : make_uint2(0, 0);
                }
            }
            uint64_t* bar = SWAP ? &m->s_full[j & 1] : &m->empty[st];
            const uint32_t parity = SWAP ? (j >> 1) & 1 : ((j / STAGES) & 1) ^ 1;
            if (SWAP || j >= STAGES) {
                if (pend >= 0 && !__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) {
                    cp_async_wait<0>();
                    c.arrive(&full[pend]);
                    pend = -1;
                }
                c.wait(bar, parity);
                if (c.gone()) break;
            }
            if (!SWAP) {
                const uint32_t theirs = __ballot_sync(0xFFFFFFFFu, (mine ? lo : hi) >= 0);
                if (lane == 0) {
                    m->held[st][mine] = live;
                    m->held[st][mine ^ 1] = theirs;
                    mbar_arrive(&m->h_full[st]);
                }
            }
            if (R > 0) {
                const bool whole = live == 0xFFFFFFFFu;
                const int groups = CKEYS / R;
                const int boxes = SWAP ? 2 * ((c.nb + 3) / 4) : c.nb + 1;   // a pair that lies behind the row is zeros
                uint64_t* done = whole ? &full[st] : fix;
                const uint32_t to = whole ? 0 : c.rank;
                if (whole) {
                    if (lane == 0) mbar_expect_at(done, 0, uint32_t(boxes) * KBOX);
                } else if (live != 0) {
                    // Groups of R rows with one that exists; their other rows are cleared below.
                    uint32_t some = 0;
#pragma unroll 1
                    for (int g = 0; g < groups; ++g) some += live >> (g * R) & 1;
                    if (lane == 0) mbar_arrive_expect_tx(fix, uint32_t(boxes) * some * uint32_t(R) * 128u);
                }
                __syncwarp();
                // A box at a time: a copy of several would put them R rows apart.
#pragma unroll 1
                for (int q0 = 0; q0 < boxes * groups; q0 += 32) {
                    const int q = q0 + lane, g = min(q / boxes, groups - 1), b = q - g * boxes;
                    const int row = __shfl_sync(0xFFFFFFFFu, int(slot), g * R);
                    const bool rope = !SWAP && b == c.nb;
                    if (q < boxes * groups && row >= 0)
                        tma_box_at(stage + uint32_t(place(b)) * KBOX + uint32_t(g * R) * 128u, rope ? &maps.rope : &maps.all, 0, row,
                                   rope ? 0 : channels(b), done, to);
                }
                if (!whole) {
                    if (live != 0) {
                        c.wait(fix, fixed & 1);
                        ++fixed;
                    }
                    if (slot < 0)
#pragma unroll 1
                        for (int b = 0; b < boxes; ++b)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                st_shared_v4(stage + uint32_t(place(b)) * KBOX + uint32_t(lane) * 128u + k * 16u, make_uint4(0, 0, 0, 0));
                    c.arrive(&full[st]);
                }
            } else {
                const int nc = p.Dv / 8, nr = p.Dk / 8, ch = lane & 7;
#pragma unroll
                for (int rr = 0; rr < 8; ++rr) {
                    const int r = rr * 4 + (lane >> 3);
                    const int64_t row = __shfl_sync(0xFFFFFFFFu, slot, r);
                    const uint16_t* v = static_cast<const uint16_t*>(p.ckv) + (row < 0 ? 0 : row) * p.Dv;
#pragma unroll 1
                    for (int b = 0; b < nl; ++b) {
                        const int q = channels(b) * 8 + ch;
                        const bool in = row >= 0 && q < nc;
                        cp_async16(box_at(stage + uint32_t(place(b)) * KBOX, r, ch), in ? v + q * 8 : v, in);
                    }
                    if (K8 && !SWAP) {
                        st_shared_v4(box_at(stage + 8 * KBOX, r, ch), dec8x8<IT>(p.k_kind, codes[rr].x, codes[rr].y));
                    } else if (!SWAP) {
                        const uint16_t* k = static_cast<const uint16_t*>(p.kc) + (row < 0 ? 0 : row) * p.Dk;
                        const bool in = row >= 0 && ch < nr;
                        cp_async16(box_at(stage + 8 * KBOX, r, ch), in ? k + ch * 8 : k, in);
                    }
                }
                cp_async_commit();
                if (pend >= 0) {
                    cp_async_wait<1>();
                    c.arrive(&full[pend]);
                }
                pend = st;
            }
        }
    }
    if (pend >= 0) {
        cp_async_wait<0>();
        c.arrive(&full[pend]);
    }
}

// key_warp where a TMA copy takes the whole half of a step. One thread's instructions set the pace here (about 5 cycles
// each): the step's path is kept short.
template <bool SWAP>
__device__ __forceinline__ void key_warp_tma(Ctx& c, const Maps& maps) {
    constexpr int STAGES = stages_of<false>();
    static_assert((STAGES & (STAGES - 1)) == 0, "stages are counted by masks");
    const MlaParams& p = c.p;
    Misc* m = c.m;
    const int lane = c.lane;
    const int mine = int(SWAP ? c.rank ^ 1 : c.rank);
    const int boxes = SWAP ? 2 * ((c.nb + 3) / 4) : c.nb + 1;   // a pair that lies behind the row is zeros
    const uint32_t place = (SWAP ? uint32_t(c.rank ^ 1) * 2 : 0) * KBOX;
    uint64_t* fix = SWAP ? &m->v_fix : &m->k_fix;
    uint64_t* full = SWAP ? m->v_full : m->k_full;
    auto copy = [&](uint32_t stage, int row, uint64_t* done, uint32_t to) {
        if (SWAP) {
            tma_box_at(stage + place, &maps.two, 0, row, int(c.rank) * 2, done, to);
            if (boxes > 2) tma_box_at(stage + place + 4 * KBOX, &maps.two, 0, row, int(c.rank) * 2 + 4, done, to);
        } else {
            tma_box_at(stage, &maps.all, 0, row, 0, done, to);
            tma_box_at(stage + 8 * KBOX, &maps.rope, 0, row, 0, done, to);
        }
    };
    int j = 0, fixed = 0;
    Walk w(p, m);
#pragma unroll 1
    while (w.next() && !c.gone()) {
        const int n = w.n, K = w.s.K;
        int base = w.kt0 - 32, own = -1, other = -1;   // first rows of this lane's step, base + lane
#pragma unroll 1
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++j) {
            if (kt - base >= 32) {
                base = kt;
                own = int(key_row(p, n, K, (base + lane) * KEYS + mine * CKEYS));
                if (!SWAP) other = int(key_row(p, n, K, (base + lane) * KEYS + (mine ^ 1) * CKEYS));
            }
            const int row = __shfl_sync(0xFFFFFFFFu, own, kt - base), row2 = SWAP ? 0 : __shfl_sync(0xFFFFFFFFu, other, kt - base);
            const int left = K - kt * KEYS - mine * CKEYS, left2 = K - kt * KEYS - (mine ^ 1) * CKEYS;
            const uint32_t live = row < 0 ? 0u : (left >= CKEYS ? 0xFFFFFFFFu : (1u << left) - 1u);
            const int st = j & (STAGES - 1);
            const uint32_t stage = c.stage(st);
            if (SWAP) c.wait(&m->s_full[j & 1], (j >> 1) & 1);
            else if (j >= STAGES) c.wait(&m->empty[st], ((j / STAGES) & 1) ^ 1);
            if (c.gone()) break;
            if (live == 0xFFFFFFFFu) {
                if (lane == 0) {
                    mbar_expect_at(&full[st], 0, uint32_t(boxes) * KBOX);
                    copy(stage, row, &full[st], 0);
                }
                __syncwarp();
            } else {   // the last keys of a sequence, or a hole: clear the rows that do not exist
                if (live != 0) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(fix, uint32_t(boxes) * KBOX);
                        copy(stage, row, fix, c.rank);
                    }
                    __syncwarp();
                    c.wait(fix, fixed & 1);
                    ++fixed;
                }
                if (!(live >> lane & 1))
#pragma unroll 1
                    for (int b = 0; b < boxes; ++b) {
                        const uint32_t box = stage + (SWAP ? place + uint32_t((b >> 1) * 4 + (b & 1)) * KBOX : uint32_t(b < c.nb ? b : 8) * KBOX);
#pragma unroll
                        for (int k = 0; k < 8; ++k) st_shared_v4(box + uint32_t(lane) * 128u + k * 16u, make_uint4(0, 0, 0, 0));
                    }
                c.arrive(&full[st]);
            }
            if (!SWAP && lane == 0) {   // behind the copy, which is what the step waits for
                m->held[st][mine] = live;
                m->held[st][mine ^ 1] = row2 < 0 ? 0u : (left2 >= CKEYS ? 0xFFFFFFFFu : (1u << left2) - 1u);
                mbar_arrive(&m->h_full[st]);
            }
        }
    }
}

// 8-bit latent rows, decoded into halves (the rotary part into q's type): a lane has 16 codes, a quarter of a box, of one
// of 8 rows, so that a warp's stores fill the banks. The next step's loads are in flight meanwhile. Where blocks hold whole
// groups of 8 keys, lane i looks up a group's first row for step base + i, once for 32 steps.
struct Group {
    int first;   // of step base + lane
    __device__ __forceinline__ void look(const MlaParams& p, int n, int K, int step, int key) { first = int(key_row(p, n, K, step * KEYS + key)); }
    __device__ __forceinline__ int of(int i) const { return __shfl_sync(0xFFFFFFFFu, first, i); }
};
// Of 8 keys, which exist, given the first one's row and the keys that are left from it on.
__device__ __forceinline__ uint32_t group_bits(int first, int left) {
    return first < 0 ? 0u : (left >= 8 ? 0xFFu : (1u << max(left, 0)) - 1u);
}

// Eight warps bring a CTA's own 32 keys: warp & 3 has 8 of them, warp >> 2 half of the channels.
template <class IT, int CK>
__device__ __forceinline__ void code_keys(Ctx& c, int v) {
    constexpr int STAGES = stages_of<true>();
    const MlaParams& p = c.p;
    Misc* m = c.m;
    const int lane = c.lane, wp = v >> 5 & 3, half = v >> 7, sub = lane >> 2, tk = wp * 8 + sub, c4 = lane & 3;
    const int mine = int(c.rank) * CKEYS + wp * 8, theirs = mine ^ CKEYS;   // first keys of the groups
    const int nc = p.Dv / 16, nr = p.k_kind == OUT16 ? p.Dk / 8 : p.Dk / 16, nb = c.nb - half * 4;
    const uint32_t at0 = box_at(0, tk, 2 * c4), at1 = box_at(0, tk, 2 * c4 + 1);   // this lane's places in a box
    const bool full = half * 16 + 16 <= nc && half * 4 + 4 <= nr;   // all this lane's pieces exist
    const int kbytes = p.Dk * (p.k_kind == OUT16 ? 2 : 1);
    const uint8_t* codes = static_cast<const uint8_t*>(p.ckv) + half * 256 + c4 * 16;
    const uint8_t* ropes = static_cast<const uint8_t*>(p.kc) + (half * 4 + c4) * 16;
    int st = 0, turn = 0;
    Walk w(p, m);
#pragma unroll 1
    while (w.next()) {
        const int n = w.n, K = w.s.K, kt0 = w.kt0, kt1 = w.kt1;
        int base = kt0 - 32;
        Group own, other;
        struct Load {
            uint4 x[4], rope;
            uint32_t held;   // which keys of a group exist: of this CTA's (half 0) or of the other's (half 1)
        };
        auto load = [&](int kt, Load& a) {
            int64_t slot;
            if (p.groups) {
                if (kt - base >= 32) {
                    base = kt;
                    own.look(p, n, K, base + lane, mine);
                    if (half) other.look(p, n, K, base + lane, theirs);
                }
                const int f = own.of(kt - base), left = K - kt * KEYS;
                if (half) a.held = group_bits(other.of(kt - base), left - theirs);
                else a.held = group_bits(f, left - mine);
                slot = f >= 0 && sub < left - mine ? f + sub : -1;
            } else {
                slot = key_row(p, n, K, kt * KEYS + mine + sub);
                // Every fourth bit.
                uint32_t b = __ballot_sync(0xFFFFFFFFu, (half ? key_row(p, n, K, kt * KEYS + theirs + sub) : slot) >= 0) & 0x11111111u;
                b = (b | b >> 3) & 0x03030303u;
                b = (b | b >> 6) & 0x000F000Fu;
                a.held = (b | b >> 12) & 0xFFu;
            }
            const uint8_t* src = codes + slot * p.Dv;
            const uint8_t* k = ropes + slot * kbytes;
            if (full && slot >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) a.x[i] = ld_ahead_v4(src + 64 * i);
                a.rope = ld_ahead_v4(k);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) a.x[i] = slot >= 0 && half * 16 + c4 + 4 * i < nc ? ld_ahead_v4(src + 64 * i) : make_uint4(0, 0, 0, 0);
                a.rope = slot >= 0 && half * 4 + c4 < nr ? ld_ahead_v4(k) : make_uint4(0, 0, 0, 0);
            }
        };
        auto store = [&](const Load& a) {
            const uint32_t stage = c.stage(st);
            if (turn > 0) c.wait(&m->empty[st], (turn & 1) ^ 1);
            const uint32_t to = stage + half * (4 * KBOX), box = stage + 8 * KBOX;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < nb) {
                    st_shared_v4(to + i * KBOX + at0, codes_to_halves<CK>(a.x[i].x, a.x[i].y));
                    st_shared_v4(to + i * KBOX + at1, codes_to_halves<CK>(a.x[i].z, a.x[i].w));
                }
            if (p.k_kind == OUT16) {   // eight pieces a row: four of each half
                st_shared_v4(box_at(box, tk, half * 4 + c4), a.rope);
            } else if (half == 0) {    // four pieces a row
                st_shared_v4(box + at0, dec8x8<IT>(p.k_kind, a.rope.x, a.rope.y));
                st_shared_v4(box + at1, dec8x8<IT>(p.k_kind, a.rope.z, a.rope.w));
            }
            if (lane == 0) {
                reinterpret_cast<uint8_t*>(&m->held[st][int(c.rank) ^ half])[wp] = uint8_t(a.held);
                mbar_arrive(&m->h_full[st]);
            }
            c.arrive(&m->k_full[st]);
            if (++st == STAGES) st = 0, ++turn;
        };
        Load x, y;
        load(kt0, x);
#pragma unroll 1
        for (int kt = kt0; kt < kt1; kt += 2) {   // two steps a turn: the loads in flight need no copies
            if (kt + 1 < kt1) load(kt + 1, y);
            store(x);
            if (kt + 1 == kt1) break;
            if (kt + 2 < kt1) load(kt + 2, x);
            store(y);
        }
    }
}

// Three warps bring the other CTA's keys of a part (this CTA's four boxes of channels): warp w has box w of the four
// groups of 8 rows and, in turn, their box 3 (groups 0 and 3, group 1, group 2).
template <int CK>
__device__ __forceinline__ void code_swaps(Ctx& c, int v, const Walk& w, int& j) {
    constexpr int STAGES = stages_of<true>();
    const MlaParams& p = c.p;
    Misc* m = c.m;
    const int lane = c.lane, wp = v >> 5, theirs = int(c.rank ^ 1), sub = lane >> 2;
    const int n = w.n, K = w.s.K, kt0 = w.kt0, kt1 = w.kt1;
    int base = kt0 - 32;
    Group group[4];
    auto channel = [&](int b) { return ((b >> 1) * 4 + int(c.rank) * 2 + (b & 1)) * 64; };
    const int qa = channel(wp), qb = channel(3);
    const uint32_t boxa = uint32_t((wp >> 1) * 4 + theirs * 2 + (wp & 1)) * KBOX, boxb = uint32_t(4 + theirs * 2 + 1) * KBOX;
    auto load = [&](int kt, uint4 (&a)[6]) {
        int64_t slot[4];
        if (p.groups) {
            if (kt - base >= 32) {
                base = kt;
#pragma unroll
                for (int g = 0; g < 4; ++g) group[g].look(p, n, K, base + lane, theirs * CKEYS + g * 8);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int f = group[g].of(kt - base);
                slot[g] = f >= 0 && kt * KEYS + theirs * CKEYS + g * 8 + sub < K ? f + sub : -1;
            }
        } else {
            const int64_t s = key_row(p, n, K, kt * KEYS + theirs * CKEYS + lane);
#pragma unroll
            for (int g = 0; g < 4; ++g) slot[g] = __shfl_sync(0xFFFFFFFFu, s, g * 8 + sub);
        }
        const int64_t extra = wp == 0 ? slot[0] : (wp == 1 ? slot[1] : slot[2]);
        const uint8_t* src = static_cast<const uint8_t*>(p.ckv) + (lane & 3) * 16;
#pragma unroll
        for (int g = 0; g < 4; ++g) a[g] = slot[g] >= 0 && qa + (lane & 3) * 16 < p.Dv ? ld_ahead_v4(src + slot[g] * p.Dv + qa) : make_uint4(0, 0, 0, 0);
        a[4] = extra >= 0 && qb + (lane & 3) * 16 < p.Dv ? ld_ahead_v4(src + extra * p.Dv + qb) : make_uint4(0, 0, 0, 0);
        a[5] = wp == 0 && slot[3] >= 0 && qb + (lane & 3) * 16 < p.Dv ? ld_ahead_v4(src + slot[3] * p.Dv + qb) : make_uint4(0, 0, 0, 0);
    };
    auto put = [&](uint32_t box, int g, const uint4& x) {
        st_shared_v4(box_at(box, g * 8 + sub, 2 * (lane & 3)), codes_to_halves<CK>(x.x, x.y));
        st_shared_v4(box_at(box, g * 8 + sub, 2 * (lane & 3) + 1), codes_to_halves<CK>(x.z, x.w));
    };
    auto store = [&](const uint4 (&a)[6]) {
        const int st = j % STAGES;
        const uint32_t stage = c.stage(st);
        c.wait(&m->s_full[j & 1], (j >> 1) & 1);
#pragma unroll
        for (int g = 0; g < 4; ++g) put(stage + boxa, g, a[g]);
        put(stage + boxb, wp, a[4]);
        if (wp == 0) put(stage + boxb, 3, a[5]);
        c.arrive(&m->v_full[st]);
        ++j;
    };
    uint4 x[6], y[6];
    load(kt0, x);
#pragma unroll 1
    for (int kt = kt0; kt < kt1; kt += 2) {
        if (kt + 1 < kt1) load(kt + 1, y);
        store(x);
        if (kt + 1 == kt1) break;
        if (kt + 2 < kt1) load(kt + 2, x);
        store(y);
    }
}

// The query warps (four; three with codes) bring the queries of a part: lane v & 7 has chunk v & 7 of each box of a row.
template <bool C8>
__device__ __forceinline__ void load_queries(Ctx& c, int v, const Walk& w, int part, int steps) {
    constexpr int AT_ONCE = C8 ? 12 : 16, TURNS = C8 ? 6 : 4;   // rows of a turn
    const MlaParams& p = c.p;
    Misc* m = c.m;
    const int nc = p.Dv / 8, nr = p.Dk / 8, ch = v & 7;
    const uint16_t *qn[TURNS], *qr[TURNS];
    uint32_t lives = 0;
    const unsigned rows = unsigned(w.s.L) * unsigned(p.H), row0 = unsigned(w.i) * ROWS + c.rank * CROWS + (v >> 3);
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const unsigned row = row0 + i * AT_ONCE;
        const bool live = i * AT_ONCE + (v >> 3) < CROWS && row < rows;
        if (p.q_flat) {   // head after head, token after token
            const int64_t at = live ? w.s.q0 * p.H + row : 0;
            qn[i] = static_cast<const uint16_t*>(p.qn) + at * p.qn_hs + ch * 8;
            qr[i] = static_cast<const uint16_t*>(p.qr) + at * p.qr_hs + ch * 8;
        } else {
            const int64_t t = live ? w.s.q0 + row / unsigned(p.H) : 0, head = live ? row % unsigned(p.H) : 0;
            qn[i] = static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + head * p.qn_hs + ch * 8;
            qr[i] = static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + head * p.qr_hs + ch * 8;
        }
        lives |= uint32_t(live) << i;
    }
    // This wait alone lasts as long as a part, the `steps` of the one before: 2^24 keys take 0.2 s over TMA rows and 1.3 s
    // where blocks of one key and rotary codes make a step 5.0 us, so it has another second for every 2^16 of them.
    if (part > 0) c.wait(&m->q_free, (part - 1) & 1, steps >> 16);
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int r = i * AT_ONCE + (v >> 3);
        const bool live = lives >> i & 1;
        if (C8 && r >= CROWS) break;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const bool in = live && b * 8 + ch < nc;
            if (b < c.nb) cp_async16(box_at(c.base + OFF_Q + b * QBOX, r, ch), in ? qn[i] + b * 64 : qn[i], in);
        }
        cp_async16(box_at(c.base + OFF_Q + 8 * QBOX, r, ch), qr[i], live && ch < nr);
    }
    cp_async_commit();
    cp_async_wait<0>();
    c.arrive(&m->q_full);
}

// Brings the queries of the next part into L2 meanwhile.
__device__ __forceinline__ void prefetch_queries(Ctx& c, int v, const Walk& w) {
    const MlaParams& p = c.p;
    const unsigned row = unsigned(w.i) * ROWS + c.rank * CROWS + (v >> 1);
    if (row >= unsigned(w.s.L) * unsigned(p.H)) return;
    const int64_t t = w.s.q0 + row / unsigned(p.H), head = row % unsigned(p.H);
    const uint16_t* qn = static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + head * p.qn_hs;
#pragma unroll 1
    for (int ch = (v & 1) * 64; ch < p.Dv; ch += 128) prefetch_l2(qn + ch);
    if ((v & 1) == 0) prefetch_l2(static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + head * p.qr_hs);
}

// Groups of four softmax warps: a lone warp of a scheduler goes at about 5 cycles an instruction, so what a warp has to do
// sets the time of a step's softmax and of a part's output. With codes the warps are needed more for decoding.
template <bool C8>
constexpr int groups_of() { return C8 ? 1 : 2; }
template <bool C8>
__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(128 * groups_of<C8>()) : "memory");
}

// Output of a part (a row tile of a sequence), by the softmax warps: thread (row r, half h of the channels; group g has
// half of the 256 columns). Each thread writes its row's sectors itself, with few instructions: through shared memory, for
// whole lines, took more of them and longer (7000 cycles a part against 5000).
template <class IT, bool C8>
__device__ __forceinline__ void output_part(Ctx& c, int tid, int pair, int part, const Walk& w, unsigned row, bool live, float2 ml) {
    constexpr int G = groups_of<C8>();
    const MlaParams& p = c.p;
    const int r = tid & 63, h = tid >> 6 & 1, g = tid >> 7;
    const uint32_t lanes = c.tmem + (uint32_t(tid >> 5 & 3) << 21);
    const bool none = ml.y == 0.f;
    const int64_t t = w.s.q0 + row / unsigned(p.H), head = row % unsigned(p.H);
    const int q0 = g * 128, q1 = min(q0 + 256 / G, p.Dv > 256 ? 256 : 128);
    if (!w.whole) {
        const Space ws = ws_space(p);
        const int64_t slot = int64_t(pair) * 2 + (part ? 1 : 0);
        const int in = c.rank * CROWS + r;
        if (live && h == 0 && g == 0) ws.ml[slot * ROWS + in] = ml;
        float* po = ws.o + slot * ROWS * p.Dv + in * 8;   // [8 channels of all rows]: a warp's stores are whole lines
#pragma unroll 1
        for (int q = q0; q < q1; q += 32) {   // (a row without keys leaves what it may: the join skips it)
            float o[32];
            __syncwarp();
            tmem_ld32(lanes + q, o);
            tmem_wait_ld();
            const int ch = (q >> 7) * 256 + h * 128 + (q & 127);
            if (C8) {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= c.sc->inv_v[ch + k];
            }
            if (live && ch + 32 <= p.Dv) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) st_global_v8(po + (ch + k) * ROWS, reinterpret_cast<const uint32_t*>(o) + k);
            } else if (live) {
#pragma unroll
                for (int k = 0; k < 32; k += 8)
                    if (ch + k < p.Dv) st_global_v8(po + (ch + k) * ROWS, reinterpret_cast<const uint32_t*>(o) + k);
            }
        }
    } else {
        if (live && h == 0 && g == 0 && p.lse != nullptr)
            p.lse[t * p.H + head] = none ? -INFINITY : (ml.x + log2f(ml.y)) * 0.6931471805599453f;
        uint16_t* out = static_cast<uint16_t*>(p.out) + t * p.o_ts + head * p.o_hs;
        const float inv = none ? 0.f : 1.f / ml.y;
        const bool zero = __any_sync(0xFFFFFFFFu, none);   // a row without keys: zeros, whatever the others' keys hold
#pragma unroll 1
        for (int q = q0; q < q1; q += 32) {
            float o[32];
            __syncwarp();
            tmem_ld32(lanes + q, o);
            tmem_wait_ld();
            const int ch = (q >> 7) * 256 + h * 128 + (q & 127);
            if (C8) {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= c.sc->inv_v[ch + k];
            }
            uint32_t u[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float2 x = __fmul2_rn(make_float2(o[2 * k], o[2 * k + 1]), make_float2(inv, inv));
                u[k] = IT::pack(x.x, x.y);
            }
            if (zero) {
#pragma unroll
                for (int k = 0; k < 16; ++k) u[k] = none ? 0u : u[k];
            }
            if (live && p.out_wide && ch + 32 <= p.Dv) {
                st_global_v8(out + ch, u);
                st_global_v8(out + ch + 16, u + 8);
            } else if (live) {
#pragma unroll
                for (int k = 0; k < 16; k += 4)
                    if (ch + 2 * k < p.Dv) *reinterpret_cast<uint4*>(out + ch + 2 * k) = make_uint4(u[k], u[k + 1], u[k + 2], u[k + 3]);
            }
        }
    }
    tc_fence_before();
}

// Over the threads of row r (two a group), always in this order.
template <int G>
__device__ __forceinline__ float row_max(const float* x, int r) {
    const float v = fmaxf(x[r], x[r + 64]);
    return G == 1 ? v : fmaxf(v, fmaxf(x[r + 128], x[r + 192]));
}
template <int G>
__device__ __forceinline__ float row_sum(const float* x, int r) {
    const float v = x[r] + x[r + 64];
    return G == 1 ? v : v + (x[r + 128] + x[r + 192]);
}

// Octaves by which weights are held above their reference where they are rounded to halves: a half's spacing stops
// shrinking at 2^-24, so that a weight below 2^-14 of the reference would lose bits and one below 2^-25 be lost from O,
// while l counts it (an attention sink and 10^5 keys 17 nats below it: the output off by a third). 7 is the most there is
// room for: weights below 2^(8 + 7), a half ends at 65504. What is lost of a weight then is 2^-32 of the row's largest.
template <class PT>
constexpr float LIFT = is_bf16<PT> ? 0.f : 7.f;
// The exponent that weights are taken to. Where scores are so large (2^24) that a float cannot be 7 lower, it may not be
// more than 7 lower either, or weights would overflow.
template <class PT>
__device__ __forceinline__ float reference(float mx) {
    if (LIFT<PT> == 0.f) return mx;
    const float r = mx - LIFT<PT>;
    return mx - r <= LIFT<PT> ? r : mx;   // (infinities stay)
}

// Softmax: thread (row r, half h of the keys, group g: half of that half).
template <class IT, bool C8, bool K8>
__device__ __forceinline__ void softmax_warps(Ctx& c, int tid, int pair) {
    using PT = typename std::conditional<C8, F16, IT>::type;   // type of the weights and the decoded codes
    constexpr int G = groups_of<C8>(), NK = CKEYS / G;          // keys of a thread
    const MlaParams& p = c.p;
    Misc* m = c.m;
    const int r = tid & 63, h = tid >> 6 & 1, g = tid >> 7;
    const uint32_t lanes = c.tmem + (uint32_t(tid >> 5 & 3) << 21);
    constexpr bool split = C8 || K8;
    // Score = fn * (latent product) + fr * (rotary product), in powers of two.
    const float l2 = p.scale * 1.4426950408889634f;
    float fn = l2, fr = l2;
    if (K8) fr = l2 * (p.k_scale_per_ch ? m->lift : m->inv_k[0]);
    int j = 0, part = 0;
    Walk w(p, m);
#pragma unroll 1
    while (w.next()) {
        const unsigned row = unsigned(w.i) * ROWS + c.rank * CROWS + r;
        const bool live = row < unsigned(w.s.L) * unsigned(p.H);
        const int vis = live ? seen(p, w.s.L, w.s.K, int(row / unsigned(p.H))) : 0;
        int wmin = live ? vis : 0x7FFFFFFF;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) wmin = min(wmin, __shfl_xor_sync(0xFFFFFFFFu, wmin, o));
        if (C8) {
            fn = l2 * (p.ckv_scale_per_ch ? 1.f : c.sc->inv_v[0]);
            if (p.row_mul != nullptr && live) fn *= p.row_mul[(w.s.q0 + row / unsigned(p.H)) * p.H + row % unsigned(p.H)];
        }
        float mx = -INFINITY, at = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++j) {
            const int key0 = kt * KEYS + h * CKEYS + g * NK;
            float* red = m->red[j & 1];
            // Keys that exist: bit i for key0 + i. They come over a barrier of this CTA, as the arrivals that start the
            // scores order nothing for these warps. (The word is written anew once this step's weights have gone into O,
            // and they depend on it.)
            constexpr int STAGES = stages_of<C8>();
            c.wait(&m->h_full[j % STAGES], (j / STAGES) & 1);
            const uint32_t held = m->held[j % STAGES][h] >> (g * NK);
            c.wait(&m->s_full[j & 1], (j >> 1) & 1);
            tc_fence_after();
            float s[NK];
            tmem_ld(lanes + COL_S + uint32_t(j & 1) * 64 + g * NK, s);
            if (split) {
                float s2[NK];
                tmem_ld(lanes + COL_S + uint32_t(j & 1) * 64 + 32 + g * NK, s2);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < NK; ++i) s[i] = fmaf(s2[i], fr, s[i] * fn);
            } else {
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < NK; ++i) s[i] *= fn;
            }
            constexpr uint32_t all = NK == 32 ? 0xFFFFFFFFu : 0xFFFFu;
            if ((held & all) != all || key0 + NK > wmin) {
                const int left = vis - key0;
#pragma unroll
                for (int i = 0; i < NK; ++i)
                    if (i >= left || !(held >> i & 1)) s[i] = -INFINITY;
            }
            float top = s[0];
#pragma unroll
            for (int i = 1; i < NK; ++i) top = fmaxf(top, s[i]);
            red[tid] = top;
            softmax_sync<C8>();
            top = fmaxf(row_max<G>(red, r), mx);
            // The sum is rescaled only when the maximum grows by more than 2^8: weights then stay below 2^(8 + LIFT).
            const bool grow = top - mx > 8.f;
            float f = 1.f;
            if (grow) {
                const float next = reference<PT>(top);
                f = exp2_approx(at - next);
                mx = top;
                at = next;
                sum *= f;
            }
            const float ref = mx == -INFINITY ? 0.f : at;
            uint32_t pk[NK / 2];
            float step = 0.f;   // of its own: one addition a step to the long sum, which rounds small weights beside a large one
#pragma unroll
            for (int i = 0; i < NK / 2; ++i) {
                const float a = exp2_approx(s[2 * i] - ref), b = exp2_approx(s[2 * i + 1] - ref);
                step += a + b;
                pk[i] = PT::pack(a, b);
            }
            sum += step;
            // The product before this one is done: P's buffer is free and O at rest.
            if (j > 0) c.wait(&m->pv_done, (j - 1) & 1);
            if (__any_sync(0xFFFFFFFFu, grow) && kt > w.kt0) {
                tc_fence_after();
                const int q1 = min(g * 128 + 256 / G, p.Dv > 256 ? 256 : 128);
#pragma unroll 1
                for (int q = g * 128; q < q1; q += 32) {
                    float o[32];
                    tmem_ld32(lanes + q, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= f;
                    tmem_st32(lanes + q, o);
                }
                tmem_wait_st();
            }
#pragma unroll
            for (int q = 0; q < NK / 8; ++q)
                st_shared_v4(box_at(c.base + OFF_P, r, h * 4 + g * (NK / 8) + q),
                             make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]));
            tc_fence_before();
            c.arrive(&m->p_full);
        }
        // The rows' m and l for the output.
        float* red = m->red[j & 1];
        red[tid] = sum;   // the next step's buffer: its own maxima come after the second barrier
        softmax_sync<C8>();
        const float2 ml = make_float2(at, row_sum<G>(red, r));   // the exponent that l and O are taken to
        softmax_sync<C8>();
        c.wait(&m->pv_done, (j - 1) & 1);
        tc_fence_after();
        output_part<IT, C8>(c, tid, pair, part, w, row, live, ml);
        ++part;
    }
}

// The query warps: queries of a part and, with codes, its swaps.
template <int CK>
__device__ __forceinline__ void query_warps(Ctx& c, int v) {
    constexpr bool C8 = CK != OUT16;
    Walk w(c.p, c.m);
    int j = 0, steps = 0;
    bool more = w.next();
#pragma unroll 1
    for (int part = 0; more; ++part) {
        load_queries<C8>(c, v, w, part, steps);
        steps = w.kt1 - w.kt0;
        if constexpr (C8) code_swaps<CK>(c, v, w, j);
        more = w.next();
        if (!C8 && more) prefetch_queries(c, v, w);   // (with codes they were just written)
    }
}

// The MMA warp of CTA 0: S of a step is issued before O of the one before, which waits for its softmax.
template <class IT, bool C8, bool K8>
__device__ __forceinline__ void mma_warp(Ctx& c) {
    const MlaParams& p = c.p;
    Misc* m = c.m;
    constexpr int STAGES = stages_of<C8>();
    constexpr bool half = C8 || !is_bf16<IT>;   // type of the latent operands
    constexpr uint32_t id_n = tc_idesc(ROWS, KEYS, !half, false), id_r = tc_idesc(ROWS, KEYS, is_bf16<IT>, false),
                       id_o = tc_idesc(ROWS, 256, !half, true);
    constexpr bool split = C8 || K8;
    const bool leader = elect_one(), two = p.Dv > 256;
    const uint64_t qd = tc_desc(c.base + OFF_Q, 16, 1024), pd = tc_desc(c.base + OFF_P, 16, 1024);
    int j = 0, parts = 0;
    bool prev = false, prev_first = false;
    auto issue_o = [&](int i, bool first) {
        c.wait(&m->p_full, i & 1);
        c.wait(&m->v_full[i % STAGES], (i / STAGES) & 1);
        tc_fence_after();
        const uint64_t vd = tc_desc(c.stage(i % STAGES), KBOX, 1024);
        if (leader) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
                if (a == 0 || two)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        tc_mma_pair(c.tmem + a * 128, pd + s * 2, vd + ((a * 4 + (s >> 1) * 2) * KBOX + (s & 1) * 2048) / 16, id_o,
                                    !(first && s == 0));
            tc_commit_pair(&m->pv_done);
            tc_commit_pair(&m->empty[i % STAGES]);
        }
        __syncwarp();
    };
    Walk w(p, m);
#pragma unroll 1
    while (w.next()) {
        if (prev) issue_o(j - 1, prev_first);
        prev = false;
        c.wait(&m->q_full, parts & 1);
        ++parts;
#pragma unroll 1
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++j) {
            const int st = j % STAGES;
            c.wait(&m->k_full[st], (j / STAGES) & 1);
            tc_fence_after();
            const uint64_t kd = tc_desc(c.stage(st), 16, 1024);
            const uint32_t d = c.tmem + COL_S + uint32_t(j & 1) * 64;
            if (leader) {
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (b < c.nb)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            tc_mma_pair(d, qd + (b * QBOX) / 16 + s * 2, kd + (b * KBOX) / 16 + s * 2, id_n, b > 0 || s > 0);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    tc_mma_pair(d + (split ? 32 : 0), qd + (8 * QBOX) / 16 + s * 2, kd + (8 * KBOX) / 16 + s * 2, id_r, !split || s > 0);
                tc_commit_pair(&m->s_full[j & 1]);
                if (kt + 1 == w.kt1) tc_commit_pair(&m->q_free);
            }
            __syncwarp();
            if (prev) issue_o(j - 1, prev_first);
            prev = true;
            prev_first = kt == w.kt0;
        }
    }
    if (prev) issue_o(j - 1, prev_first);
    if (!c.ok) {   // let what was issued finish before TMEM goes
        if (leader) {
            tc_commit_pair(&m->drain);
            mbar_wait(&m->drain, 0, nullptr);
        }
        __syncwarp();
    }
}

// Warps. 16-bit latent rows: 0-7 softmax, 8 keys, 9 swap, 10 MMA, 12-15 queries; codes: 0-3 softmax, 4-11 keys, 12-14
// queries and swap, 15 MMA.
constexpr int NT = 512;

// CK: OutKind of the latent rows; K8: the rotary ones are codes.
template <class IT, int CK, bool K8>
__global__ void __launch_bounds__(NT, 1) __cluster_dims__(2, 1, 1)
    mla_tc_kernel(const __grid_constant__ MlaParams p, const __grid_constant__ Maps maps) {
    constexpr bool C8 = CK != OUT16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];   // the swizzle repeats every 1024 bytes
    constexpr int MMA_WARP = C8 ? 15 : 10;
    const uint32_t base = smem_u32(smem_raw);
    constexpr int STAGES = stages_of<C8>();
    Misc* m = reinterpret_cast<Misc*>(smem_raw + OFF_K + STAGES * STAGE_BYTES);
    Scales* sc = reinterpret_cast<Scales*>(m + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;

    if (base % 1024 != 0) {   // the declaration's alignment was not kept: nothing below would be right
        if (tid == 0 && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
#pragma unroll 1
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&m->k_full[s], C8 ? 16 : 2);
            mbar_init(&m->v_full[s], C8 ? 6 : 2);
            mbar_init(&m->empty[s], 1);
            mbar_init(&m->h_full[s], C8 ? 8 : 1);
        }
        mbar_init(&m->s_full[0], 1);
        mbar_init(&m->s_full[1], 1);
        mbar_init(&m->p_full, 8 * groups_of<C8>());
        mbar_init(&m->pv_done, 1);
        mbar_init(&m->q_full, C8 ? 6 : 8);
        mbar_init(&m->q_free, 1);
        mbar_init(&m->k_fix, 1);
        mbar_init(&m->v_fix, 1);
        mbar_init(&m->drain, 1);
        m->abort = 0;
        m->large = 0;
        fence_mbar_init();
    }
    if (warp == MMA_WARP) tmem_alloc_pair(&m->tmem, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();   // barriers and TMEM are set up; the other half is below, behind the schedule
    pdl_wait();
    pdl_launch_dependents();
    if (p.N <= 32) {
        if (warp < 2 && !schedule_small(p, m, pair) && lane == 0) m->large = 1;
        __syncthreads();
    }
    if (p.N > 32 || m->large) {
        schedule<NT>(p, m, pair);
        __syncthreads();
    }
    if (tid == 0 && rank == 0) ws_space(p).starts[pair] = {m->begin.n, m->begin.i, m->begin.kt, m->first.L, m->first.q0, 0};
    if (C8) {
#pragma unroll 1
        for (int ch = tid; ch < 512; ch += NT) sc->inv_v[ch] = ch >= p.Dv ? 1.f : 1.f / p.ckv_scale[p.ckv_scale_per_ch ? ch : 0];
    }
    if (K8 && warp == 0) {
        float v = 0.f;
#pragma unroll 1
        for (int ch = lane; ch < 64; ch += 32) {
            const float x = ch >= p.Dk ? 0.f : 1.f / p.k_scale[p.k_scale_per_ch ? ch : 0];
            m->inv_k[ch] = x;
            v = fmaxf(v, fabsf(x));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        if (lane == 0) m->lift = exp2f(ceilf(log2f(v)));
    }
    __syncthreads();
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = m->tmem;
    Ctx c{p, m, sc, base, tmem, rank, lane, (p.Dv + 63) / 64, &m->abort, true};

    if (warp < 4 * groups_of<C8>()) {
        softmax_warps<IT, C8, K8>(c, tid, pair);
    } else if (warp == MMA_WARP) {
        if (rank == 0) mma_warp<IT, C8, K8>(c);
    } else if constexpr (C8) {
        if (warp < 12) code_keys<IT, CK>(c, tid - 128);
        else query_warps<CK>(c, tid - 384);
    } else {
        if (warp == 8) {
            if (!K8 && p.box_rows == CKEYS) key_warp_tma<false>(c, maps);
            else key_warp<IT, K8, false>(c, maps);
        } else if (warp == 9) {
            if (!K8 && p.box_rows == CKEYS) key_warp_tma<true>(c, maps);
            else key_warp<IT, K8, true>(c, maps);
        } else if (warp >= 12) {
            query_warps<CK>(c, tid - 384);
        }
    }
    if (!c.ok) {
        if (p.status != nullptr) atomicOr(p.status, KVR_DEVERR_TIMEOUT);
        const uint64_t t0 = globaltimer_ns();   // copies in flight land in microseconds
        while (globaltimer_ns() - t0 < 10000000) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == MMA_WARP) tmem_free_pair(tmem, TMEM_COLS);
}

// Queries for a cache of codes. A scale per channel goes into the query, q / scale, rounded once: to halves, whose 11 bits
// keep that rounding small (the products with the codes, exact as halves, then run on halves whatever q's type). A power
// of two per row, put back into its scores, keeps q / scale below 2^14: it comes from the row's largest |q| and the largest
// 1 / scale, and float16's range then reaches 2^-38 below. The rotary part keeps q's type, with the scale per channel
// over a power of two of the largest 1 / scale: that is 8 bits in bf16, as its own rounding was, and no more accurate than
// that. 4 tokens of 32 heads over 900 keys, bf16: root-mean-square error of the output 0.0023 with a rotary scale per channel,
// 0.0022 with one scale, lse off by 6e-4 and 2e-6. One warp a row.
template <class IT>
__global__ void __launch_bounds__(256) mla_queries_kernel(const __grid_constant__ MlaParams p, uint16_t* qn_out, float* mul_out, uint16_t* qr_out) {
    __shared__ float inv[512], invk[64], most[2];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (qn_out != nullptr)
        for (int c = threadIdx.x; c < p.Dv; c += 256) inv[c] = p.ckv_scale_per_ch ? 1.f / p.ckv_scale[c] : 1.f;
    if (qr_out != nullptr && threadIdx.x < p.Dk) invk[threadIdx.x] = 1.f / p.k_scale[threadIdx.x];
    __syncthreads();
    if (warp < 2) {
        float v = 0.f;
        if (warp == 0 && qn_out != nullptr)
            for (int c = lane; c < p.Dv; c += 32) v = fmaxf(v, fabsf(inv[c]));
        if (warp == 1 && qr_out != nullptr)
            for (int c = lane; c < p.Dk; c += 32) v = fmaxf(v, fabsf(invk[c]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        if (lane == 0) most[warp] = exp2f(ceilf(log2f(v)));
    }
    __syncthreads();
    const float lift = most[0], g_rope = 1.f / most[1];
    const int64_t rows = p.T * p.H;
    for (int64_t row = int64_t(blockIdx.x) * 8 + warp; row < rows; row += int64_t(gridDim.x) * 8) {
        const int64_t t = row / p.H, head = row - t * p.H;
        if (qn_out != nullptr) {
            const uint16_t* q = static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + head * p.qn_hs;
            uint4 x[2];
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int ch = (k * 32 + lane) * 8;
                x[k] = ch < p.Dv ? ld_stream_v4(q + ch) : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(IT::lo(u[i])), fabsf(IT::hi(u[i]))));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const int e = top > 0.f && top <= 3.0e38f ? min(max(ilogbf(top) + ilogbf(lift) - 13, -113), 113) : 0;
            const float g = ldexpf(1.f, -e);
            if (lane == 0) mul_out[row] = ldexpf(1.f, e);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int ch = (k * 32 + lane) * 8;
                if (ch >= p.Dv) break;
                const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                uint32_t z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = F16::pack(IT::lo(u[i]) * inv[ch + 2 * i] * g, IT::hi(u[i]) * inv[ch + 2 * i + 1] * g);
                *reinterpret_cast<uint4*>(qn_out + row * p.Dv + ch) = make_uint4(z[0], z[1], z[2], z[3]);
            }
        }
        if (qr_out != nullptr && lane * 8 < p.Dk) {
            const uint4 x = ld_stream_v4(static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + head * p.qr_hs + lane * 8);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
            uint32_t z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                z[i] = IT::pack(IT::lo(u[i]) * (invk[lane * 8 + 2 * i] * g_rope), IT::hi(u[i]) * (invk[lane * 8 + 2 * i + 1] * g_rope));
            *reinterpret_cast<uint4*>(qr_out + row * p.Dk + lane * 8) = make_uint4(z[0], z[1], z[2], z[3]);
        }
    }
}

// Joins the parts of the items that were cut: the blocks x take the item that the begin of pair x + 1 is in, if that is
// the first one inside it. A warp has 32 rows, a lane 16 channels of its row. Latency is what it costs, of two rounds of
// loads: it follows the last part.
constexpr int JOIN_WARPS = 4;   // of a block: 32 rows, 64 channels
template <class IT>
__global__ void __launch_bounds__(32 * JOIN_WARPS) mla_join_kernel(const __grid_constant__ MlaParams p) {
    const Space ws = ws_space(p);
    const int lane = threadIdx.x & 31, b = blockIdx.x + 1;
    const int r = blockIdx.z * 32 + lane, ch = (blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5)) * 16;
    auto start = [&](int q) {
        Start v = {-1, 0, 0, 0, 0, 0};
        if (q < p.pairs) v = ws.starts[q];
        return v;
    };
    pdl_wait();
    pdl_launch_dependents();
    // Lane q has pair b - 1 + q and the one after it.
    const int active = *ws.active;
    Start me = start(b - 1 + lane), nx = start(b + lane);
    const int n = __shfl_sync(0xFFFFFFFFu, nx.n, 0), i = __shfl_sync(0xFFFFFFFFu, nx.i, 0), kt = __shfl_sync(0xFFFFFFFFu, nx.kt, 0);
    const unsigned L = __shfl_sync(0xFFFFFFFFu, nx.L, 0);
    const int64_t q0 = __shfl_sync(0xFFFFFFFFu, nx.q0, 0);
    const bool same = __shfl_sync(0xFFFFFFFFu, me.n == n && me.i == i, 0), cut = __shfl_sync(0xFFFFFFFFu, me.kt > 0, 0);
    const unsigned row = unsigned(i) * ROWS + r, rows = L * unsigned(p.H);
    if (b >= active || n >= p.N || kt == 0 || (same && cut) || ch >= p.Dv || unsigned(i) * ROWS + (r & ~31) >= rows) return;
    const bool live = row < rows, two = ch + 8 < p.Dv;
    // Parts: the last of pair b - 1, then the first of each pair that begins inside the item, but for pairs without
    // work (the next one begins where they do).
    struct Part {
        float2 ml;
        float o[16];
    };
    float mx = -INFINITY, l = 0.f, o[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) o[c] = 0.f;
    auto fetch = [&](int slot, Part& x) {
        x.ml = make_float2(-INFINITY, 0.f);
        if (live && slot >= 0) {
            x.ml = ws.ml[int64_t(slot) * ROWS + r];
            const float* from = ws.o + int64_t(slot) * ROWS * p.Dv + (ch * ROWS + r * 8);
            ld_global_v8(from, x.o);
            if (two) ld_global_v8(from + 8 * ROWS, x.o + 8);
        }
    };
    auto take = [&](const Part& x) {   // in order; a part whose keys the row does not see has left nothing
        if (x.ml.y == 0.f) return;
        const float top = fmaxf(mx, x.ml.x);
        const float back = mx == top ? 1.f : exp2_approx(mx - top), f = x.ml.x == top ? 1.f : exp2_approx(x.ml.x - top);
        mx = top;
        l = l * back + x.ml.y * f;
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] = o[c] * back + x.o[c] * f;
    };
#pragma unroll 1
    for (int at = b - 1;; at += 32) {
        const int q = at + lane;
        const bool in = q == b - 1 || (q < active && me.n == n && me.i == i && me.kt > 0);
        const uint32_t run = __ballot_sync(0xFFFFFFFFu, in);
        const int count = run == 0xFFFFFFFFu ? 32 : __ffs(~run) - 1;
        const bool work = lane < count && !(q + 1 < active && me.n == nx.n && me.i == nx.i && me.kt == nx.kt);
        const int slot = work ? q * 2 + (q == b - 1 && !same ? 1 : 0) : -1;
        Part x[2];   // a part, the next one on its way
        fetch(__shfl_sync(0xFFFFFFFFu, slot, 0), x[0]);
#pragma unroll 1
        for (int k = 0; k < count; k += 2) {
            if (k + 1 < count) fetch(__shfl_sync(0xFFFFFFFFu, slot, k + 1), x[1]);
            take(x[0]);
            if (k + 1 == count) break;
            if (k + 2 < count) fetch(__shfl_sync(0xFFFFFFFFu, slot, k + 2), x[0]);
            take(x[1]);
        }
        if (count < 32) break;
        me = start(at + 32 + lane);
        nx = start(at + 33 + lane);
    }
    if (!live) return;
    const int64_t t = q0 + row / unsigned(p.H), head = row % unsigned(p.H);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* out = static_cast<uint16_t*>(p.out) + t * p.o_ts + head * p.o_hs + ch;
    uint32_t u[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) u[c] = IT::pack(o[2 * c] * inv, o[2 * c + 1] * inv);
    *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
    if (two) *reinterpret_cast<uint4*>(out + 8) = make_uint4(u[4], u[5], u[6], u[7]);
    if (ch == 0 && p.lse != nullptr) p.lse[t * p.H + head] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

// The kernel for a type and cache kinds, as a launch takes it.
using MlaKernel = void (*)(MlaParams, Maps);
template <class IT, int CK>
static MlaKernel kernel_of_k(bool k8) { return k8 ? MlaKernel(mla_tc_kernel<IT, CK, true>) : MlaKernel(mla_tc_kernel<IT, CK, false>); }
template <class IT>
static MlaKernel kernel_of_ck(int ck, bool k8) {
    switch (ck) {
        case OUT_I8: return kernel_of_k<IT, OUT_I8>(k8);
        case OUT_E4M3: return kernel_of_k<IT, OUT_E4M3>(k8);
        case OUT_E5M2: return kernel_of_k<IT, OUT_E5M2>(k8);
        default: return kernel_of_k<IT, OUT16>(k8);
    }
}
static MlaKernel kernel_of(int dtype, int ck, bool k8) { return dtype == KVR_BF16 ? kernel_of_ck<BF16>(ck, k8) : kernel_of_ck<F16>(ck, k8); }
static uint32_t smem_for(int ck) { return ck == OUT16 ? smem_of<false>() : smem_of<true>(); }

// CTA pairs that fit on the current device at once (a GPC with an odd number of
// SMs leaves one over); looked up once per device, as is the shared memory allowed.
static int mla_tc_pairs() {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return 1;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == 0) {
        int n = 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(sm_count_current_device()) / 2 * 2);
        cfg.blockDim = dim3(NT);
        cfg.dynamicSmemBytes = smem_for(OUT16);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        bool good = true;
        for (int dtype : {KVR_BF16, KVR_F16})
            for (int ck : {OUT16, OUT_I8, OUT_E4M3, OUT_E5M2})
                for (bool k8 : {false, true})
                    good = good && cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel_of(dtype, ck, k8)),
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem_for(ck))) == cudaSuccess;
        good = good && cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(kernel_of(KVR_BF16, OUT16, false)), &cfg) == cudaSuccess && n > 0;
        if (!good) {
            (void)cudaGetLastError();
            return 1;
        }
        cache[dev] = n;
    }
    return cache[dev];
}

// Queries that a cache of codes needs prepared: the latent part unless q has halves and the scale is one, the rotary
// part where its scale is per channel.
static bool prepares_nope(const MlaParams& p, int dtype) { return p.ckv_kind != OUT16 && (p.ckv_scale_per_ch || dtype != KVR_F16); }
static bool prepares_rope(const MlaParams& p) { return p.k_kind != OUT16 && p.k_scale_per_ch; }
static int64_t round_up(int64_t x) { return (x + 255) / 256 * 256; }

bool mla_tc_fits(const MlaParams& p) {
    // cost() of one sequence is at most row tiles * (H * (keys + ITEM_COST) + ROWS / 2 * row tiles), row tiles <= 2^24, and N
    // of them, which may share rows, are added up in 64 bits.
    const int64_t tiles = (p.T * p.H + ROWS - 1) / ROWS, each = p.H * (p.max_keys + ITEM_COST) + ROWS / 2 * tiles;
    return each <= (int64_t(1) << 62) / tiles / p.N;
}

int64_t mla_tc_workspace(const MlaParams& p, int dtype) {
    int64_t n = round_up(ws_bytes(mla_tc_pairs(), p.Dv));
    if (prepares_nope(p, dtype)) n += round_up(p.T * p.H * p.Dv * 2) + round_up(p.T * p.H * 4);
    if (prepares_rope(p)) n += round_up(p.T * p.H * p.Dk * 2);
    return n;
}

// The driver's tensor-map encoder, found through the runtime (no link to libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}
static bool encode_rows(CUtensorMap* map, const void* base, bool bf16, int64_t rows, int width, int box_rows, int boxes) {
    const cuuint64_t dims[3] = {64, cuuint64_t(rows), cuuint64_t(width) / 64}, strides[2] = {cuuint64_t(width) * 2, 128};
    const cuuint32_t box[3] = {64, cuuint32_t(box_rows), cuuint32_t(boxes)}, one[3] = {1, 1, 1};
    return encoder()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
                     dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_mla_tc(MlaParams p, int dtype, cudaStream_t s) {
    p.pairs = mla_tc_pairs();
    p.out_wide = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.o_ts % 16 == 0 && p.o_hs % 16 == 0;
    // TMA boxes of R rows, R the largest power of two (8 to 32) that divides the block: a box never crosses one, and
    // its rows keep their place in the 8-row swizzle. Other blocks, codes and narrow rows take 16-byte copies.
    Maps maps = {};
    p.box_rows = 0;
    p.runs = p.table == nullptr || p.d1 % CKEYS == 0;
    const int64_t rows = p.d0 * p.d1;
    p.groups = (p.table == nullptr || p.d1 % 8 == 0) && rows < int64_t(1) << 31;
    if (p.ckv_kind == OUT16 && p.k_kind == OUT16 && p.Dv % 64 == 0 && p.Dk == 64 && rows < (int64_t(1) << 31) - 64) {
        int r = 32;
        while (p.table != nullptr && r > 1 && p.d1 % r != 0) r /= 2;
        const bool bf = dtype == KVR_BF16;
        if (r >= 8 && encoder() != nullptr && encode_rows(&maps.all, p.ckv, bf, rows, p.Dv, r, r == 32 ? p.Dv / 64 : 1) &&
            encode_rows(&maps.two, p.ckv, bf, rows, p.Dv, r, 2) && encode_rows(&maps.rope, p.kc, bf, rows, p.Dk, r, 1))
            p.box_rows = r;
    }
    const bool nope = prepares_nope(p, dtype), rope = prepares_rope(p);
    if (nope || rope) {
        char* at = static_cast<char*>(p.workspace) + round_up(ws_bytes(p.pairs, p.Dv));
        uint16_t *qn = nullptr, *qr = nullptr;
        float* mul = nullptr;
        if (nope) {
            qn = reinterpret_cast<uint16_t*>(at);
            mul = reinterpret_cast<float*>(at + round_up(p.T * p.H * p.Dv * 2));
            at += round_up(p.T * p.H * p.Dv * 2) + round_up(p.T * p.H * 4);
        }
        if (rope) qr = reinterpret_cast<uint16_t*>(at);
        const int64_t cap = int64_t(sm_count_current_device()) * 8, need = (p.T * p.H + 7) / 8;
        const dim3 grid(unsigned(need < cap ? need : cap));
        const cudaError_t e = dtype == KVR_BF16 ? launch_pdl(mla_queries_kernel<BF16>, grid, dim3(256), 0, s, p, qn, mul, qr)
                                                : launch_pdl(mla_queries_kernel<F16>, grid, dim3(256), 0, s, p, qn, mul, qr);
        if (e != cudaSuccess) return e;
        if (nope) {
            p.qn = qn;
            p.row_mul = mul;
            p.qn_ts = int64_t(p.H) * p.Dv;
            p.qn_hs = p.Dv;
        }
        if (rope) {
            p.qr = qr;
            p.qr_ts = int64_t(p.H) * p.Dk;
            p.qr_hs = p.Dk;
        }
    }
    p.q_flat = p.qn_ts == p.H * p.qn_hs && p.qr_ts == p.H * p.qr_hs;
    const cudaError_t e = launch_pdl(kernel_of(dtype, p.ckv_kind, p.k_kind != OUT16), dim3(unsigned(p.pairs * 2)), dim3(NT),
                                     smem_for(p.ckv_kind), s, p, maps);
    if (e != cudaSuccess || p.pairs == 1) return e;
    // (no item has more rows than the call)
    const int64_t groups = (p.T * p.H + 31) / 32;
    const dim3 grid(unsigned(p.pairs - 1), unsigned(p.Dv + 63) / 64, unsigned(groups < ROWS / 32 ? groups : ROWS / 32)), block(32 * JOIN_WARPS);
    return dtype == KVR_BF16 ? launch_pdl(mla_join_kernel<BF16>, grid, block, 0, s, p) : launch_pdl(mla_join_kernel<F16>, grid, block, 0, s, p);
}

}  // namespace kvr
