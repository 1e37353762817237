// The attention weight of each key on the tensor cores: rows of up to 512 + 64 channels.
//
// For the keys of a sequence and its rows (token, head):
//   S = K Q^T,  w[i] = decay past[i] + sum over the rows r that see key i of 2^(f_r S[i, r] - l_r),
// f = scale log2 e and l_r = lse_r log2 e. The logarithms are given, so that no pass over the keys has to come first.
//
// Keys are the product's first operand: a key's scores then lie in one TMEM lane, and the sum over rows is a sum within a
// thread: no shuffles, no atomics, one number a key and share of the work. What is not a key (a hole, the end of a block)
// only spoils its own lane, which is left out at the end.
//
// Tiling: a CTA pair (cta_group::2, M = 256) has 256 keys, 128 in each CTA, in 9 boxes of 64 channels that stay in shared
// memory while the sequence's rows pass in groups of up to 256, half of them through each CTA, box by box through a ring.
// A box of keys is brought, and codes are decoded, once for all rows. It is free, and the next tile's box on its way, once the
// last group's product with it is done. Where a sequence has one group (a decode step) whose boxes fit the ring, its
// queries stay there for all its tiles. Scores take turns over two halves of TMEM: the exponentials of a group run beside
// the products of the next one.
//
// Caches of codes: eight warps decode them into halves (every code is exact there). The queries are divided by scales per channel
// before and held as the sum of two halves each, 22 bits, as a weight is a float32: one half alone was off by 2e-4 of it. One
// scale for all latent channels goes into the row's factor instead.
//
// Work is cut into equal shares by cost over the pairs (key_weight_plan.cuh). A tile that the cut goes through leaves its
// sums in the workspace, and a second kernel adds them up in a fixed order.
//
// What bounds it, at 6786 GB/s and 1914 TFLOP/s: the cache's bytes below some 280 rows a key in 16 bits, 80 over codes with scales per
// channel and 140 with one; above, the tensor cores. Measured: 256 sequences of one token, 128 heads, 1-4095 keys 108 to 111 us
// (6.1 TB/s, 90% of the copy rate); 512 tokens x 128 heads over 16384 keys 625 to 640 us alone (1.9 PFLOP/s, the rate of a library
// product) and 690 to 712 in a long run at the power limit; windows of 17-32 tokens, 8 sequences of 3000-8192 keys in E4M3, 164 to
// 168 us (twice the latent products, for the second halves; windows of 32 over 4096 keys 190, with one scale 120 to 124); one token
// of 16 heads over 1000 keys 6.8 us. The sums on the tensor cores are cut off at each addition of 16 products: a weight is 1.4e-6
// of itself too small in bf16, 2.6e-6 over codes with scales per channel, 0.9e-6 with one.
#include <mutex>

#include "cache_ops.cuh"
#include "key_weight_plan.cuh"
#include "latent_tiles.cuh"

namespace kvr {

namespace {

constexpr int CKEYS = KW_KEYS / 2;   // keys of a CTA
constexpr uint32_t BOX = CKEYS * 128;
constexpr int KBOXES = 9, ROPE = 8;   // boxes of a tile; the rotary part's
constexpr uint32_t OFF_Q = KBOXES * BOX, Q_BYTES = 73728, OFF_LSE = OFF_Q + Q_BYTES;   // the queries' ring
constexpr int MAX_SLOTS = 18;        // of that ring: all boxes of a row in two halves
constexpr int LSE_SLOTS = 4;         // groups whose logarithms are in shared memory
constexpr uint32_t LSE_SLOT = 2048, OFF_MISC = OFF_LSE + LSE_SLOTS * LSE_SLOT;
constexpr uint32_t TMEM_COLS = 512, COL_D = 256;   // a group's scores: 256 columns at most

struct alignas(16) Misc {
    uint64_t k_full[KBOXES], k_empty[KBOXES], q_full[MAX_SLOTS], q_empty[MAX_SLOTS];
    uint64_t d_full[2], d_free[2], lse_full[LSE_SLOTS], lse_free[LSE_SLOTS], drain;
    uint32_t tmem;
    int abort;
    KwPos begin, end;
    int64_t wsum[32];
    float other[2][CKEYS];   // sums of the second half of the sum warps
};
constexpr uint32_t SMEM = OFF_MISC + uint32_t(sizeof(Misc));
static_assert(SMEM <= 232448, "shared memory of a CTA");

struct Tc {
    KeyWeightParams w;       // its queries: row t * H + h at that times qn_hs, qr_hs (those of codes prepared)
    const float* row_mul;    // power of two per row that prepared queries lack, or NULL
    int pairs, rows, shift, slots, box_rows;   // rows = 2^shift
    int lo_n, lo_r;          // the latent, the rotary part's queries have a second half
    int patience;            // seconds of a wait beyond the first
};
struct Maps {
    CUtensorMap qn, qr, qn_lo, qr_lo, latent, rope;
};

// Workspace: header, the pairs' begins, sums of two tiles a pair.
struct alignas(16) Start {
    KwPos at;
    int L, K, pad[2];
};
__host__ __device__ inline int64_t ws_sums(int pairs) { return 256 + (int64_t(pairs) * int64_t(sizeof(Start)) + 255) / 256 * 256; }
__host__ __device__ inline int64_t ws_bytes(int pairs) { return ws_sums(pairs) + int64_t(pairs) * 2 * KW_KEYS * 4; }
struct Space {
    int32_t* active;
    Start* starts;
    float* sums;
};
__device__ __forceinline__ Space ws_space(const Tc& p) {
    char* w = static_cast<char*>(p.w.m.workspace);
    return {reinterpret_cast<int32_t*>(w), reinterpret_cast<Start*>(w + 256), reinterpret_cast<float*>(w + ws_sums(p.pairs))};
}

struct Shapes {
    const Tc& p;
    __device__ __forceinline__ KwShape operator()(int n, int* bits = nullptr) const {
        const Seq s = load_seq(p.w.m, n, bits);
        return {s.L, s.K, p.w.m.H, p.shift, p.w.m.causal != 0};
    }
};
using Walk = KwWalk<Shapes>;

// This pair's share: every CTA adds up all sequences' costs in the same order.
template <int THREADS>
__device__ void schedule(const Tc& p, Misc* m, int pair) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = int(p.w.m.N);
    const int per = (N - 1) / THREADS + 1, n0 = min(int64_t(tid) * per, int64_t(N)), n1 = min(int64_t(n0) + per, int64_t(N));
    const Shapes shapes{p};
    int64_t sum = 0;
    int bits = 0;
    KwShape s = {0, 0, 1, 5, false};
    for (int n = n0; n < n1; ++n) {
        s = shapes(n, &bits);
        sum += s.cost();
    }
    if (bits != 0 && blockIdx.x == 0 && p.w.m.status != nullptr) atomicOr(p.w.m.status, bits);
    int64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) m->wsum[warp] = scan;
    if (tid == 0) m->begin = m->end = {N, 0, 0, 0};
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int q = 0; q < WARPS; ++q) {
        const int64_t v = m->wsum[q];
        if (q < warp) before += v;
        total += v;
    }
    const int64_t upto = before + scan, base = upto - sum;
    const int active = kw_active(total, p.pairs);
    for (int h = 0; h < 2; ++h) {
        int64_t at = kw_share(total, pair + h, active);
        if (at < base || at >= upto) continue;
        at -= base;
        for (int n = n0;; ++n) {   // (one of them holds it)
            if (per > 1) s = shapes(n);
            const int64_t c = s.cost();
            if (at < c) {
                (h ? m->end : m->begin) = s.locate(n, at);
                break;
            }
            at -= c;
        }
    }
    if (tid == 0 && pair == 0 && cluster_rank() == 0) *ws_space(p).active = active;
}

// The same where a lane can have a sequence each (a few conversations: latency counts): one warp for the share's begin, one for its
// end, without a word between warps.
__device__ __forceinline__ void schedule_small(const Tc& p, Misc* m, int pair) {
    const int lane = threadIdx.x & 31, half = threadIdx.x >> 5, N = int(p.w.m.N);
    int bits = 0;
    KwShape s = {0, 0, 1, 5, false};
    if (lane < N) s = Shapes{p}(lane, &bits);
    const int64_t mine = s.cost();
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    const int64_t total = __shfl_sync(0xFFFFFFFFu, scan, 31);
    const int active = kw_active(total, p.pairs);
    const int64_t at = kw_share(total, pair + half, active);
    KwPos* to = half ? &m->end : &m->begin;
    if (at >= scan - mine && at < scan) *to = s.locate(lane, at - (scan - mine));
    if (at == total && lane == 0) *to = {N, 0, 0, 0};
    if (half == 0) {
        if (bits != 0 && blockIdx.x == 0 && p.w.m.status != nullptr) atomicOr(p.w.m.status, bits);
        if (lane == 0 && pair == 0 && cluster_rank() == 0) *ws_space(p).active = active;
    }
}

// What every role has.
struct Ctx {
    const Tc& p;
    Misc* m;
    uint32_t base, tmem, rank;
    int lane, nb;   // nb: 64-channel boxes of the latent part
    float* lse;
    volatile int* abort;
    bool ok;

    // As in the attention kernel: a wait that gives up (after one second and `patience`) poisons the CTA; the roles that start TMA
    // copies then stop, the others run their loops to the end without waiting.
    __device__ __forceinline__ void wait_alone(uint64_t* bar, uint32_t parity) {   // by one thread of a warp
        if (ok && !mbar_try_wait(bar, parity)) ok = wait_on(bar, parity, abort, p.patience);
    }
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
        wait_alone(bar, parity);
        __syncwarp();
    }
    __device__ __forceinline__ bool gone() const { return __any_sync(0xFFFFFFFFu, !ok); }
    __device__ __forceinline__ uint32_t k_box(int b) const { return base + uint32_t(b) * BOX; }
    __device__ __forceinline__ uint32_t q_slot(int s) const { return base + OFF_Q + uint32_t(s) * uint32_t(p.rows) * 64u; }
    // This warp's shared-memory writes are done: tell the MMA warp of the pair.
    __device__ __forceinline__ void arrive(uint64_t* bar) {
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(bar, 0);
    }
    __device__ __forceinline__ Walk walk() const { return Walk(Shapes{p}, m->begin, m->end, int(p.w.m.N)); }
    __device__ __forceinline__ int q_boxes() const { return (nb << p.lo_n) + (1 << p.lo_r); }
    // Whether a run's queries stay in the ring for its tiles.
    __device__ __forceinline__ bool stays(const Walk& w) const { return w.kt1 - w.kt0 > 1 && q_boxes() <= p.slots; }
};

// A key's row, looked up in two steps: the load of the block table, and what needs it.
struct Look {
    int64_t e;
    unsigned off;
    bool in;
    __device__ __forceinline__ void begin(const MlaParams& p, int n, int K, int key) {
        in = key < K;
        off = unsigned(key);
        e = n;
        if (in && p.table != nullptr) {
            const unsigned d1 = unsigned(p.d1 < (1 << 30) ? p.d1 : (1 << 30)), q = off / d1;
            off -= q * d1;
            e = p.table[n * p.max_blocks + q];
        }
    }
    __device__ __forceinline__ int64_t row(const MlaParams& p) const {
        if (!in) return -1;
        if (e < 0 || e >= p.d0) {
            if (e != -1 && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_INDEX);
            return -1;
        }
        return e * p.d1 + off;
    }
};

// Two warps bring the CTA's 16-bit keys through TMA, every other box each: a box is 128 / R copies of R rows, R what divides the
// cache's blocks. (One warp: blocks of 16 keys, 64 sequences of 4096, 64 to 69 us, by how its copies were compiled; two 58. Blocks
// of 128 take 57 with either.)
__device__ __forceinline__ void key_warp(Ctx& c, const Maps& maps, int which) {
    const MlaParams& p = c.p.w.m;
    const int R = c.p.box_rows, copies = CKEYS / R;
    int tile = 0;
    Walk w = c.walk();
    while (w.next()) {
        if (w.ga >= w.gb) continue;
        Look next;
        auto look = [&](int kt) {   // (a lane without a copy, and what lies behind the run, has no key)
            next.begin(p, w.n, c.lane < copies && kt < w.kt1 ? w.s.K : 0, kt * KW_KEYS + int(c.rank) * CKEYS + c.lane * R);
        };
        look(w.kt0);
#pragma unroll 1
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++tile) {
            const int row = int(next.row(p));
            look(kt + 1);
            const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xFFFFFFFFu, row >= 0))) * uint32_t(R) * 128u;
#pragma unroll 1
            for (int b = which; b <= c.nb; b += 2) {
                const int at = b < c.nb ? b : ROPE;
                if (tile > 0) c.wait(&c.m->k_empty[at], (tile & 1) ^ 1);
                if (c.gone()) return;
                if (c.lane == 0) mbar_expect_at(&c.m->k_full[at], 0, bytes);
                __syncwarp();
                if (row >= 0)
                    tma_tile_at(c.k_box(at) + uint32_t(c.lane * R) * 128u, b < c.nb ? &maps.latent : &maps.rope, b < c.nb ? b * 64 : 0,
                                row, &c.m->k_full[at], 0);
            }
        }
    }
}

// One thread brings the queries, half of a group's rows, box by box in the order of the products. Rows behind the sequence's
// last one are another's, or none: their columns are left out of the sums.
__device__ __forceinline__ void query_thread(Ctx& c, const Maps& maps) {
    const Tc& p = c.p;
    const MlaParams& a = p.w.m;
    const int half = p.rows / 2, slots = p.slots;
    const uint32_t bytes = uint32_t(half) * 128u;
    const int64_t all = a.T * a.H;
    int slot = 0;
    uint32_t turn = 0;
    Walk w = c.walk();
    while (w.next()) {
        const int64_t first = a.query_start[w.n] * a.H + int64_t(c.rank) * half;
        const int turns = c.stays(w) ? 1 : w.kt1 - w.kt0;
#pragma unroll 1
        for (int t = 0; t < turns; ++t)
#pragma unroll 1
            for (int g = w.ga; g < w.gb; ++g) {
                const int64_t at = first + int64_t(g) * p.rows;
                const int row = int(at < all ? at : all);
                auto box = [&](const CUtensorMap* map, int x) {
                    if (turn > 0) c.wait_alone(&c.m->q_empty[slot], (turn & 1) ^ 1);
                    if (!c.ok) return;
                    mbar_expect_at(&c.m->q_full[slot], 0, bytes);
                    tma_tile_at(c.q_slot(slot), map, x, row, &c.m->q_full[slot], 0);
                    if (++slot == slots) slot = 0, ++turn;
                };
#pragma unroll 1
                for (int b = 0; b < c.nb; ++b) {
                    box(&maps.qn, b * 64);
                    if (p.lo_n) box(&maps.qn_lo, b * 64);
                }
                box(&maps.qr, 0);
                if (p.lo_r) box(&maps.qr_lo, 0);
                if (!c.ok) return;
            }
    }
}

// One warp brings the groups' logarithms, times log2 e and negative, as they are added; -inf (a row that saw nothing, or padding) as
// -inf, so that the row adds 2^-inf. With prepared queries each row's factor stands beside.
template <bool PREP>
__device__ __forceinline__ void lse_warp(Ctx& c) {
    const MlaParams& p = c.p.w.m;
    const int rows = c.p.rows;
    constexpr float LOG2E = 1.4426950408889634f;
    int item = 0;
    Walk w = c.walk();
    while (w.next()) {
        const int64_t first = p.query_start[w.n] * p.H;
        const unsigned all = unsigned(w.s.L) * unsigned(p.H);
        for (int kt = w.kt0; kt < w.kt1; ++kt)
#pragma unroll 1
            for (int g = w.ga; g < w.gb; ++g, ++item) {
                const int slot = item % LSE_SLOTS;
                float l[8], f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int i = k * 32 + c.lane;
                    const unsigned row = unsigned(g) * unsigned(rows) + i;
                    const bool live = i < rows && row < all;
                    l[k] = live ? p.lse[first + row] : 0.f;
                    f[k] = PREP && live ? c.p.row_mul[first + row] * (p.scale * LOG2E) : 0.f;
                }
                if (item >= LSE_SLOTS) c.wait(&c.m->lse_free[slot], ((item / LSE_SLOTS) & 1) ^ 1);
                float* lse = c.lse + slot * (LSE_SLOT / 4);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int i = k * 32 + c.lane;
                    if (i >= rows) break;
                    const float x = l[k] == -INFINITY ? -INFINITY : -l[k] * LOG2E;
                    if (PREP) *reinterpret_cast<float2*>(lse + 2 * i) = make_float2(f[k], x);
                    else lse[i] = x;
                }
                __syncwarp();
                if (c.lane == 0) mbar_arrive(&c.m->lse_full[slot]);
            }
    }
}

// The tiles of a share as the loading warps go over them: a thread looks up NL rows of each, `step` apart.
template <int NL>
struct Tiles {
    const Ctx& c;
    Walk w;
    int kt = 0, r0, step;
    bool in = false;
    Look look[NL];
    int64_t slot[NL];
    __device__ __forceinline__ Tiles(const Ctx& x, int first, int apart) : c(x), w(x.walk()), r0(first), step(apart) {}
    __device__ __forceinline__ void begin(int t) {
        const int key = t * KW_KEYS + int(c.rank) * CKEYS + r0;
#pragma unroll
        for (int i = 0; i < NL; ++i) look[i].begin(c.p.w.m, w.n, w.s.K, key + i * step);
    }
    __device__ __forceinline__ bool next() {
        if (!in || ++kt >= w.kt1) {
            do {
                if (!w.next()) return false;
            } while (w.ga >= w.gb);
            in = true;
            kt = w.kt0;
            begin(kt);
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) slot[i] = look[i].row(c.p.w.m);
        if (kt + 1 < w.kt1) begin(kt + 1);   // one tile ahead
        return true;
    }
};

// Eight warps bring 16-bit latent rows that TMA does not take (blocks that no 8 keys divide, rotary codes): 16-byte copies,
// three boxes in flight. A thread has pieces c4 and c4 + 4 of its rows; odd rows take them the other way round, so that eight
// lanes write to all banks.
__device__ __forceinline__ void copy_warps(Ctx& c, int v) {
    const MlaParams& p = c.p.w.m;
    const int c4 = v & 3, r0 = v >> 2, nc = p.Dv / 8, nr = p.Dk / 8;
    const bool k8 = p.k_kind != OUT16;
    int tile = 0;
    Tiles<2> t(c, r0, 64);
    for (; t.next(); ++tile) {
        uint4 codes[2];
        if (k8)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                codes[h] = t.slot[h] >= 0 && c4 < p.Dk / 16 ? ld_ahead_v4(static_cast<const uint8_t*>(p.kc) + t.slot[h] * p.Dk + c4 * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int b = 0; b <= c.nb; ++b) {
            const bool rope = b == c.nb;
            const int at = rope ? ROPE : b;
            if (tile > 0) c.wait(&c.m->k_empty[at], (tile & 1) ^ 1);
            const uint32_t box = c.k_box(at);
            if (rope && k8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    st_shared_v4(box_at(box, r0 + 64 * h, 2 * c4), dec8x8<F16>(p.k_kind, codes[h].x, codes[h].y));
                    st_shared_v4(box_at(box, r0 + 64 * h, 2 * c4 + 1), dec8x8<F16>(p.k_kind, codes[h].z, codes[h].w));
                }
            } else {
                const uint16_t* from = static_cast<const uint16_t*>(rope ? p.kc : p.ckv);
                const int width = rope ? p.Dk : p.Dv, count = rope ? nr : nc, first = rope ? 0 : b * 8;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int piece = c4 + 4 * (k ^ (r0 & 1));
                        const bool ok = t.slot[h] >= 0 && first + piece < count;
                        cp_async16(box_at(box, r0 + 64 * h, piece), ok ? from + t.slot[h] * width + (first + piece) * 8 : from, ok);
                    }
            }
            cp_async_commit();
            if (b >= 3) {
                cp_async_wait<3>();
                c.arrive(&c.m->k_full[b - 3]);
            }
        }
        // The tile's last boxes: the next one's first is free only when the products have had all of this one.
        cp_async_wait<0>();
        for (int b = max(0, c.nb - 2); b <= c.nb; ++b) c.arrive(&c.m->k_full[b < c.nb ? b : ROPE]);
    }
}

// Eight warps decode a cache of codes: two have two of a tile's latent boxes, 64 rows each, a lane 16 pieces of 16 codes. Each
// half's next loads start as soon as it is stored, so that they have a tile's time. 64 sequences of 8192 keys in int8 take 139
// to 142 us with 16 heads (E4M3 with scales per channel and 128 heads: 145 to 149), the same from L2 as from DRAM; without any load
// 85. Both move by as much as 15% with the order of the roles in the code, which share the instruction cache. Tried, when int8 took
// 145 to 151: all eight warps at each pair of boxes in turn, four arrivals a tile 162; sixteen warps of half the rows 136, but 190
// instead of 155 with 128 heads; half of the codes decoded ahead of the wait 189; the next rows prefetched into L2 164; whole
// lines a load 178.
template <int CK>
__device__ __forceinline__ void code_warps(Ctx& c, int v) {
    const MlaParams& p = c.p.w.m;
    const int lane = c.lane, c4 = lane & 3, r = lane >> 2, u = v >> 6, row0 = (v >> 5 & 1) * 64;
    if (2 * u >= c.nb) return;
    const uint32_t box = c.k_box(2 * u) + uint32_t(row0) * 128u, at0 = box_at(box, r, 2 * c4), at1 = box_at(box, r, 2 * c4 + 1);
    const int first = u * 8 + c4, nc = p.Dv / 16, done = min(2 * u + 1, c.nb - 1);
    const bool in0 = first < nc, in1 = first + 4 < nc, two = 2 * u + 1 < c.nb;
    const uint8_t* base = static_cast<const uint8_t*>(p.ckv) + (in0 ? first : 0) * 16;
    const bool whole = u * 8 + 8 <= nc;   // (the same in all lanes)
    const int second = in1 ? 64 : 0;
    int tile = 0;
    Tiles<2> t(c, row0 + lane, 32);
    // Rows half * 32 + 8 k + r. In the place of a key that does not exist, row 0: what it holds spoils that key's sums alone, which
    // are left out, and a branch a load took 250 cycles each. Channels that do not exist are zeros.
    auto load = [&](int half, uint4 (&x)[8]) {
        const uint8_t* src[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) src[k] = base + max(__shfl_sync(0xFFFFFFFFu, t.slot[half], 8 * k + r), int64_t(0)) * p.Dv;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = ld_ahead_v4(src[k]);
            x[2 * k + 1] = ld_ahead_v4(src[k] + second);
        }
        if (!whole) {
            const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (!(k & 1 ? in1 : in0)) x[k] = none;
        }
    };
    auto store = [&](int half, const uint4 (&x)[8]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t to = uint32_t(half * 32 + 8 * k) * 128u;
            st_shared_v4(at0 + to, codes_to_halves<CK>(x[2 * k].x, x[2 * k].y));
            st_shared_v4(at1 + to, codes_to_halves<CK>(x[2 * k].z, x[2 * k].w));
            if (two) {
                st_shared_v4(at0 + to + BOX, codes_to_halves<CK>(x[2 * k + 1].x, x[2 * k + 1].y));
                st_shared_v4(at1 + to + BOX, codes_to_halves<CK>(x[2 * k + 1].z, x[2 * k + 1].w));
            }
        }
    };
    uint4 x[8], y[8];
    bool more = t.next();
    if (!more) return;
    load(0, x);
    load(1, y);
    for (; more; ++tile) {
        // (the products have had a tile's boxes in order)
        more = t.next();
        if (tile > 0) c.wait(&c.m->k_empty[done], (tile & 1) ^ 1);
        store(0, x);
        if (more) load(0, x);
        store(1, y);
        if (more) load(1, y);
        c.arrive(&c.m->k_full[2 * u]);
    }
}

// Beside them, one warp brings the rotary part: 16-bit rows by 16-byte copies, codes decoded.
__device__ __forceinline__ void rope_warp(Ctx& c) {
    const MlaParams& p = c.p.w.m;
    const bool k8 = p.k_kind != OUT16;
    const int lane = c.lane, per = k8 ? 4 : 8, ch = lane & (per - 1), r = lane / per;   // lanes a row
    const bool in = ch < p.Dk / (k8 ? 16 : 8);
    const uint8_t* base = static_cast<const uint8_t*>(p.kc) + ch * 16;
    const int bytes = p.Dk * (k8 ? 1 : 2);
    const uint32_t box = c.k_box(ROPE);
    int tile = 0;
    Tiles<4> t(c, lane, 32);
    for (; t.next(); ++tile) {
        if (tile > 0) c.wait(&c.m->k_empty[ROPE], (tile & 1) ^ 1);
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // 32 rows
            if (k8) {
                uint4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t row = __shfl_sync(0xFFFFFFFFu, t.slot[q], 8 * k + r);
                    x[k] = row >= 0 && in ? ld_ahead_v4(base + row * bytes) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    st_shared_v4(box_at(box, 32 * q + 8 * k + r, 2 * ch), dec8x8<F16>(p.k_kind, x[k].x, x[k].y));
                    st_shared_v4(box_at(box, 32 * q + 8 * k + r, 2 * ch + 1), dec8x8<F16>(p.k_kind, x[k].z, x[k].w));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int64_t row = __shfl_sync(0xFFFFFFFFu, t.slot[q], 4 * k + r);
                    const bool ok = row >= 0 && in;
                    cp_async16(box_at(box, 32 * q + 4 * k + r, ch), ok ? base + row * bytes : base, ok);
                }
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
        c.arrive(&c.m->k_full[ROPE]);
    }
}

// The MMA warp of CTA 0: one thread goes over the boxes. It has about 250 cycles for each (64 channels of 128 rows), at about 5
// an instruction: nothing is worked out in the loop that need not be, and no other lane is waited for.
template <class IT, bool C8>
__device__ __forceinline__ void mma_thread(Ctx& c) {
    const Tc& p = c.p;
    Misc* m = c.m;
    const uint32_t id_it = tc_idesc(KW_KEYS, p.rows, is_bf16<IT>, false), id_half = tc_idesc(KW_KEYS, p.rows, false, false);
    const uint32_t id_n = C8 ? id_half : id_it, id_r = p.w.m.k_kind != OUT16 ? id_half : id_it;
    const uint64_t keys = tc_desc(c.base, 16, 1024), queries = tc_desc(c.q_slot(0), 16, 1024);
    const uint32_t q_step = uint32_t(p.rows) * 64u / 16u;
    const bool lo_n = p.lo_n;
    int tile = 0, item = 0, slot = 0, slots = p.slots, nb = c.nb;
    uint32_t turn = 0;
    Walk w = c.walk();
    while (w.next()) {
        if (w.ga >= w.gb) continue;
        const bool stay = c.stays(w);
        const int slot0 = slot;
        const uint32_t turn0 = turn;
#pragma unroll 1
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++tile) {
            if (stay) slot = slot0, turn = turn0;
            const bool fresh = !stay || kt == w.kt0, free = !stay || kt + 1 == w.kt1;   // the queries come, and go
#pragma unroll 1
            for (int g = w.ga; g < w.gb; ++g, ++item) {
                const int h = item & 1;
                const uint32_t d = c.tmem + uint32_t(h) * COL_D;
                const bool first = g == w.ga, last = g + 1 == w.gb;
                if (item > 1) c.wait_alone(&m->d_free[h], ((item >> 1) & 1) ^ 1);
                auto box = [&](int at, uint32_t id, bool accumulate) {   // one box of queries with the keys' box `at`
                    if (fresh) c.wait_alone(&m->q_full[slot], turn & 1);
                    tc_fence_after();
                    const uint64_t kd = keys + uint32_t(at) * (BOX / 16), qd = queries + uint32_t(slot) * q_step;
                    tc_mma_pair(d, kd, qd, id, accumulate);
#pragma unroll
                    for (int s = 1; s < 4; ++s) tc_mma_pair(d, kd + s * 2, qd + s * 2, id, true);
                    if (free) tc_commit_pair(&m->q_empty[slot]);
                    if (++slot == slots) slot = 0, ++turn;
                };
#pragma unroll 1
                for (int b = 0; b < nb; ++b) {
                    if (first && (!C8 || b % 2 == 0)) c.wait_alone(&m->k_full[b], tile & 1);   // (codes: a barrier for two boxes)
                    box(b, id_n, b > 0);
                    if (C8 && lo_n) box(b, id_n, true);
                    if (last) tc_commit_pair(&m->k_empty[b]);
                }
                if (first) c.wait_alone(&m->k_full[ROPE], tile & 1);
#pragma unroll 1
                for (int lo = 0; lo <= p.lo_r; ++lo) box(ROPE, id_r, true);
                if (last) tc_commit_pair(&m->k_empty[ROPE]);
                tc_commit_pair(&m->d_full[h]);
            }
        }
    }
    if (!c.ok) {   // let what was issued finish before TMEM goes
        tc_commit_pair(&m->drain);
        mbar_wait(&m->drain, 0, nullptr);
    }
}

// 2^(f s - l) of 32 columns, added up.
template <bool PREP>
__device__ __forceinline__ float2 column_sum(const float (&s)[32], const float* lse, float f, float2 sum) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        float2 a, b;
        if (PREP) {
            const float4 u = *reinterpret_cast<const float4*>(lse + 2 * i), v = *reinterpret_cast<const float4*>(lse + 2 * i + 4);
            a = make_float2(fmaf(s[i], u.x, u.y), fmaf(s[i + 1], u.z, u.w));
            b = make_float2(fmaf(s[i + 2], v.x, v.y), fmaf(s[i + 3], v.z, v.w));
        } else {
            const float4 u = *reinterpret_cast<const float4*>(lse + i);
            a = __ffma2_rn(make_float2(s[i], s[i + 1]), make_float2(f, f), make_float2(u.x, u.y));
            b = __ffma2_rn(make_float2(s[i + 2], s[i + 3]), make_float2(f, f), make_float2(u.z, u.w));
        }
        sum = __fadd2_rn(sum, make_float2(exp2_approx(a.x), exp2_approx(a.y)));
        sum = __fadd2_rn(sum, make_float2(exp2_approx(b.x), exp2_approx(b.y)));
    }
    return sum;
}
// The same over the columns [from, upto) alone.
template <bool PREP>
__device__ __forceinline__ float2 masked_sum(const float (&s)[32], const float* lse, float f, float2 sum, int from, int upto) {
    uint32_t see = from <= 0 ? 0xFFFFFFFFu : (from < 32 ? 0xFFFFFFFFu << from : 0u);
    if (upto < 32) see &= upto <= 0 ? 0u : (1u << upto) - 1u;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float a = exp2_approx(PREP ? fmaf(s[i], lse[2 * i], lse[2 * i + 1]) : fmaf(s[i], f, lse[i]));
        const float b = exp2_approx(PREP ? fmaf(s[i + 1], lse[2 * i + 2], lse[2 * i + 3]) : fmaf(s[i + 1], f, lse[i + 1]));
        sum.x += see >> i & 1 ? a : 0.f;
        sum.y += see >> (i + 1) & 1 ? b : 0.f;
    }
    return sum;
}

// A group's sum anew, rows of 2^-inf left out: with a score that is not finite (a padded row's query may hold anything) they have
// made it NaN, the only thing but 0 that they can add. Looked for afterwards and out of line, so that the sums' loop stays as it
// is: masks of such rows, written and looked at with every group, cost 64 tokens of a chunk 1% and int8 codes 3%. The additions
// keep their order.
template <bool PREP>
__device__ __noinline__ float counted_sum(uint32_t d, const float* lse, float f, int rows, int from, int upto) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int q = 0; q < rows; q += 16) {
        float s[16];
        tmem_ld16(d + q, s);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float by = PREP ? lse[2 * (q + i)] : f, l = PREP ? lse[2 * (q + i) + 1] : lse[q + i];
            const float a = l == -INFINITY || q + i < from || q + i >= upto ? 0.f : exp2_approx(fmaf(s[i], by, l));
            if (i & 1) sum.y += a;
            else sum.x += a;
        }
    }
    return sum.x + sum.y;
}

// Four warps a half of TMEM (EG = 2), or four for both: thread r has key r of the CTA's half of a tile.
template <bool PREP, int EG>
__device__ __forceinline__ void sum_warps(Ctx& c, int tid, int pair) {
    const Tc& p = c.p;
    const MlaParams& a = p.w.m;
    Misc* m = c.m;
    const int mine = EG == 2 ? tid >> 7 : 0, r = tid & 127, rows = p.rows;
    const uint32_t lanes = c.tmem + (uint32_t(tid >> 5 & 3) << 21);
    const float f = a.scale * 1.4426950408889634f;
    int item = 0, joined = 0;
    Walk w = c.walk();
    while (w.next()) {
        const unsigned all = unsigned(w.s.L) * unsigned(a.H);
        const int slot = pair * 2 + (m->begin.n == w.n && m->begin.kt == w.kt0 ? 0 : 1);
        const float* past = p.w.past == nullptr ? nullptr : p.w.past + w.n * p.w.past_stride;
        float* weight = p.w.weight + w.n * p.w.weight_stride;
#pragma unroll 1
        for (int kt = w.kt0; kt < w.kt1; ++kt) {
            const int key0 = kt * KW_KEYS + int(c.rank) * CKEYS, key = key0 + r;
            const int old_keys = a.causal ? w.s.K - w.s.L : 0x40000000, own = min(key - old_keys, w.s.L);
            const bool writes = EG == 1 || (w.gb - w.ga == 1 ? (item & 1) == mine : mine == 0);
            float old = 0.f, total = 0.f;
            if (writes && w.whole && past != nullptr && key < w.s.K) old = past[key];
            const bool held = writes && key_row(a, w.n, w.s.K, key) >= 0;
#pragma unroll 1
            for (int g = w.ga; g < w.gb; ++g, ++item) {
                const int h = item & 1, ls = item % LSE_SLOTS;
                if (EG == 2 && h != mine) continue;
                // Columns [from, left) are rows that see the key: those of its own token, where it is a new one, and behind.
                const unsigned first = unsigned(g) * unsigned(rows);
                const int left = int(min(all - first, unsigned(rows)));
                const int from = own <= 0 ? 0 : int(min(int64_t(own) * a.H - first, int64_t(rows)));
                const bool masked = (key0 + CKEYS - 1 - old_keys) > 0 || left < rows;
                const float* lse = c.lse + ls * (LSE_SLOT / 4);
                c.wait(&m->lse_full[ls], (item / LSE_SLOTS) & 1);
                c.wait(&m->d_full[h], (item >> 1) & 1);
                tc_fence_after();
                const uint32_t d = lanes + uint32_t(h) * COL_D;
                float2 sum = make_float2(0.f, 0.f);
                float x[32], y[32];
                tmem_ld32(d, y);
#pragma unroll 1
                for (int q = 0; q < rows; q += 32) {   // (once in the code: instructions come from far)
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = y[i];
                    if (q + 32 < rows) tmem_ld32(d + q + 32, y);
                    const float* l = lse + q * (PREP ? 2 : 1);
                    if (masked && !__all_sync(0xFFFFFFFFu, from <= q && left >= q + 32)) sum = masked_sum<PREP>(x, l, f, sum, from - q, left - q);
                    else sum = column_sum<PREP>(x, l, f, sum);
                }
                float part = sum.x + sum.y;
                if (__any_sync(0xFFFFFFFFu, part != part && key < w.s.K)) part = counted_sum<PREP>(d, lse, f, rows, from, left);
                tc_fence_before();
                __syncwarp();
                if (c.lane == 0) {
                    mbar_arrive_at(&m->d_free[h], 0);
                    mbar_arrive(&m->lse_free[ls]);
                }
                total += part;
            }
            if (EG == 2 && w.gb - w.ga > 1) {
                float* other = &m->other[joined & 1][r];
                ++joined;
                if (mine == 1) *other = total;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (mine == 0) total += *other;
            }
            if (!writes) continue;
            if (!held) total = 0.f;   // whatever lay in its place
            if (!w.whole) ws_space(p).sums[int64_t(slot) * KW_KEYS + int(c.rank) * CKEYS + r] = total;
            else if (key < w.s.K) weight[key] = past == nullptr ? total : fmaf(p.w.decay, old, total);
        }
    }
}

// TMA: the latent rows come through it. Warps: 0 to 4 EG - 1 sums, then MMA, queries, logarithms, and 2 for TMA, 8 that copy, or
// 8 that decode and 1 for the rotary part; at most 16, so that each thread may have 128 registers.
template <bool TMA>
struct Roles {
    static constexpr int EG = TMA ? 2 : 1;
    static constexpr int MMA = 4 * EG, QUERY = MMA + 1, LSE = MMA + 2, LOAD = MMA + 3, LOADERS = TMA ? 2 : 9;
    static constexpr int THREADS = (LOAD + LOADERS) * 32;
};

// CK: OutKind of the latent rows.
template <class IT, int CK, bool TMA>
__global__ void __launch_bounds__(Roles<TMA>::THREADS, 1) __cluster_dims__(2, 1, 1)
    key_weight_tc_kernel(const __grid_constant__ Tc p, const __grid_constant__ Maps maps) {
    using R = Roles<TMA>;
    constexpr bool C8 = CK != OUT16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];   // the swizzle repeats every 1024 bytes
    const uint32_t base = smem_u32(smem_raw);
    float* lse = reinterpret_cast<float*>(smem_raw + OFF_LSE);
    Misc* m = reinterpret_cast<Misc*>(smem_raw + OFF_MISC);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pair = blockIdx.x >> 1;
    const uint32_t rank = cluster_rank();
    if (base % 1024 != 0) {   // the declaration's alignment was not kept: nothing below would be right
        if (tid == 0 && p.w.m.status != nullptr) atomicOr(p.w.m.status, KVR_DEVERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int b = 0; b < KBOXES; ++b) {
            mbar_init(&m->k_full[b], TMA ? 2 : (C8 ? (b == ROPE ? 2 : 4) : 16));
            mbar_init(&m->k_empty[b], 1);
        }
        for (int s = 0; s < MAX_SLOTS; ++s) {
            mbar_init(&m->q_full[s], 2);
            mbar_init(&m->q_empty[s], 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&m->d_full[h], 1);
            mbar_init(&m->d_free[h], 8);
        }
        for (int s = 0; s < LSE_SLOTS; ++s) {
            mbar_init(&m->lse_full[s], 1);
            mbar_init(&m->lse_free[s], 4);
        }
        mbar_init(&m->drain, 1);
        m->abort = 0;
        fence_mbar_init();
    }
    if (warp == R::MMA) tmem_alloc_pair(&m->tmem, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();   // barriers and TMEM are set up; the other half is below, behind the schedule
    pdl_wait();
    pdl_launch_dependents();
    if (p.w.m.N > 32) schedule<R::THREADS>(p, m, pair);
    else if (warp < 2) schedule_small(p, m, pair);
    __syncthreads();
    if (tid == 0 && rank == 0) {
        Seq s = {0, 0, 0};
        if (m->begin.n < p.w.m.N) s = load_seq(p.w.m, m->begin.n);
        ws_space(p).starts[pair] = {m->begin, s.L, s.K, {0, 0}};
    }
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = m->tmem;
    Ctx c{p, m, base, tmem, rank, lane, (p.w.m.Dv + 63) / 64, lse, &m->abort, true};
    const bool prep = C8 || (!TMA && p.row_mul != nullptr);   // (rotary codes alone come without TMA)
    if (warp < R::MMA) {
        if (prep) sum_warps<true, R::EG>(c, tid, pair);
        else if (!C8) sum_warps<false, R::EG>(c, tid, pair);
    } else if (warp == R::MMA) {
        if (rank == 0 && elect_one()) mma_thread<IT, C8>(c);
    } else if (warp == R::QUERY) {
        if (elect_one()) query_thread(c, maps);
    } else if (warp == R::LSE) {
        if (prep) lse_warp<true>(c);
        else if (!C8) lse_warp<false>(c);
    } else if constexpr (TMA) {
        key_warp(c, maps, warp - R::LOAD);
    } else if constexpr (C8) {
        if (warp < R::LOAD + 8) code_warps<CK>(c, tid - R::LOAD * 32);
        else rope_warp(c);
    } else {
        if (warp < R::LOAD + 8) copy_warps(c, tid - R::LOAD * 32);
    }
    if (!c.ok) {
        if (p.w.m.status != nullptr) atomicOr(p.w.m.status, KVR_DEVERR_TIMEOUT);
        const uint64_t t0 = globaltimer_ns();   // copies in flight land in microseconds
        while (globaltimer_ns() - t0 < 10000000) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == R::MMA) tmem_free_pair(tmem, TMEM_COLS);
}

// Queries for a cache of codes: z = q / scale (q itself for a part that is 16-bit), over a power of two per row that keeps all
// of the row's z below 2^14, as halves hi = half(z) and lo = half(z - hi): 22 bits of z, or of 2^-24 where z is smaller.
// One scale for all latent channels goes into the row's factor instead: z = q, which a half holds exactly (or to 2^-38 of the
// row's largest), and the rotary part is multiplied by that scale, in two parts of its cache's type: 9 + 1 box products
// instead of 16 + 1. A 16-bit part keeps its type, over the same power. Without `mul` the rows are laid out densely as they
// are, for queries whose rows lie unevenly over tokens and heads (TMA takes them by rows). One warp a row.
template <class IT>
__global__ void __launch_bounds__(256, 6) key_weight_queries_kernel(const __grid_constant__ MlaParams p, uint16_t* qn, uint16_t* qn_lo, uint16_t* qr,
                                                                 uint16_t* qr_lo, float* mul) {
    __shared__ __align__(16) float inv[512], invk[64];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool half_n = p.ckv_kind != OUT16, half_r = p.k_kind != OUT16;
    const float one = half_n && qn_lo == nullptr ? p.ckv_scale[0] : 1.f;   // the one scale
    for (int c = threadIdx.x; c < 512; c += 256) inv[c] = qn_lo == nullptr || c >= p.Dv ? 1.f : 1.f / p.ckv_scale[c];
    if (threadIdx.x < 64)
        invk[threadIdx.x] = one * (!half_r || threadIdx.x >= p.Dk ? 1.f : 1.f / p.k_scale[p.k_scale_per_ch ? threadIdx.x : 0]);
    __syncthreads();
    const int64_t rows = p.T * p.H;
    for (int64_t row = int64_t(blockIdx.x) * 8 + warp; row < rows; row += int64_t(gridDim.x) * 8) {
        const int64_t t = row / p.H, head = row - t * p.H;
        const uint16_t* from[2] = {static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + head * p.qn_hs,
                                   static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + head * p.qr_hs};
        uint4 x[3];   // two pieces of the latent part, one of the rotary part
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int ch = (k == 1 ? 32 + lane : lane) * 8;
            x[k] = ch < (k < 2 ? p.Dv : p.Dk) ? ld_stream_v4(from[k >> 1] + ch) : make_uint4(0, 0, 0, 0);
        }
        // z of a word's two channels.
        auto pair = [&](int k, int i) {
            const float* by = (k < 2 ? inv : invk) + (k == 1 ? 32 + lane : lane & (k < 2 ? 31 : 7)) * 8 + 2 * i;
            const uint32_t u = i == 0 ? x[k].x : (i == 1 ? x[k].y : (i == 2 ? x[k].z : x[k].w));
            const float2 b = *reinterpret_cast<const float2*>(by);
            return make_float2(IT::lo(u) * b.x, IT::hi(u) * b.y);
        };
        float top = 0.f;
        if (mul != nullptr) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 z = pair(k, i);
                    top = fmaxf(top, fmaxf(fabsf(z.x), fabsf(z.y)));
                }
            top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));   // (not negative: ordered as its bits)
        }
        const int e = top > 0.f && top <= 3.0e38f ? min(max(ilogbf(top) - 13, -113), 113) : 0;
        const float g = ldexpf(1.f, -e);
        if (lane == 0 && mul != nullptr) mul[row] = ldexpf(1.f, e) / one;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int ch = (k == 1 ? 32 + lane : lane) * 8, width = k < 2 ? p.Dv : p.Dk;
            if (ch >= width) continue;
            uint16_t* hi = (k < 2 ? qn : qr) + row * width + ch;
            uint16_t* lo = k < 2 ? qn_lo : qr_lo;
            const bool half = k < 2 ? half_n : half_r;
            uint32_t a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 z = pair(k, i);
                const float u = z.x * g, v = z.y * g;
                if (half) {
                    a[i] = F16::pack(u, v);
                    b[i] = F16::pack(u - F16::lo(a[i]), v - F16::hi(a[i]));
                } else {
                    a[i] = IT::pack(u, v);
                    b[i] = IT::pack(u - IT::lo(a[i]), v - IT::hi(a[i]));
                }
            }
            *reinterpret_cast<uint4*>(hi) = make_uint4(a[0], a[1], a[2], a[3]);
            if (lo != nullptr) *reinterpret_cast<uint4*>(lo + row * width + ch) = make_uint4(b[0], b[1], b[2], b[3]);
        }
    }
}

// Adds up the sums of a tile that the cut goes through, in the pairs' order: block x takes the one that the begin of pair
// x + 1 is in, if that is the first inside it. A thread has a key.
__global__ void __launch_bounds__(KW_KEYS) key_weight_join_kernel(const __grid_constant__ Tc p) {
    const Space ws = ws_space(p);
    const int lane = threadIdx.x & 31, b = blockIdx.x + 1, i = threadIdx.x;
    auto start = [&](int q) {
        Start v = {{-1, 0, 0, 0}, 0, 0, {0, 0}};
        if (q < p.pairs) v = ws.starts[q];
        return v;
    };
    pdl_wait();
    pdl_launch_dependents();
    const int active = *ws.active;
    const Start here = start(b), before = start(b - 1);
    if (b >= active || here.at.n >= p.w.m.N || !here.at.cut) return;
    const bool same = kw_same_tile(before.at, here.at);
    if (same && before.at.cut) return;
    const int n = here.at.n, key = here.at.kt * KW_KEYS + i;
    float sum = 0.f;
    auto add = [&](int slot) { sum += ws.sums[int64_t(slot) * KW_KEYS + i]; };
    // The last tile of pair b - 1, then the first of each pair that begins inside; none of a pair without work.
    if (!kw_same(before.at, here.at)) add((b - 1) * 2 + (same ? 0 : 1));
    for (int at = b;; at += 31) {
        const Start x = start(at + lane);   // lane i has pair at + i; its end is lane i + 1's begin
        const KwPos y = {__shfl_down_sync(0xFFFFFFFFu, x.at.n, 1), __shfl_down_sync(0xFFFFFFFFu, x.at.kt, 1),
                         __shfl_down_sync(0xFFFFFFFFu, x.at.g, 1), 0};
        const bool in = at + lane < active && kw_same_tile(x.at, here.at);
        const uint32_t run = __ballot_sync(0xFFFFFFFFu, in), works = __ballot_sync(0xFFFFFFFFu, in && !(at + lane + 1 < active && kw_same(x.at, y)));
        const int count = min(31, run == 0xFFFFFFFFu ? 32 : __ffs(~run) - 1);
#pragma unroll 4
        for (int q = 0; q < count; ++q)
            if (works >> q & 1) add((at + q) * 2);
        if (count < 31) break;
    }
    if (key >= here.K) return;
    float* to = p.w.weight + n * p.w.weight_stride + key;
    *to = p.w.past == nullptr ? sum : fmaf(p.w.decay, p.w.past[n * p.w.past_stride + key], sum);
}

using Kernel = void (*)(Tc, Maps);
template <class IT>
Kernel kernel_of_t(int ck, bool tma) {
    switch (ck) {
        case OUT_I8: return key_weight_tc_kernel<IT, OUT_I8, false>;
        case OUT_E4M3: return key_weight_tc_kernel<IT, OUT_E4M3, false>;
        case OUT_E5M2: return key_weight_tc_kernel<IT, OUT_E5M2, false>;
        default: return tma ? Kernel(key_weight_tc_kernel<IT, OUT16, true>) : Kernel(key_weight_tc_kernel<IT, OUT16, false>);
    }
}
Kernel kernel_of(int dtype, int ck, bool tma) { return dtype == KVR_BF16 ? kernel_of_t<BF16>(ck, tma) : kernel_of_t<F16>(ck, tma); }
int threads_of(bool tma) { return tma ? Roles<true>::THREADS : Roles<false>::THREADS; }

// CTA pairs that fit on the current device at once; looked up once per device, as is the shared memory allowed.
int pairs_of_device() {
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
        cfg.blockDim = dim3(threads_of(true));
        cfg.dynamicSmemBytes = SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        bool good = true;
        for (int dtype : {KVR_BF16, KVR_F16})
            for (int ck : {OUT16, OUT_I8, OUT_E4M3, OUT_E5M2})
                for (bool tma : {false, true})
                    good = good && cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel_of(dtype, ck, tma)),
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM)) == cudaSuccess;
        good = good && cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(kernel_of(KVR_BF16, OUT16, true)), &cfg) == cudaSuccess && n > 0;
        if (!good) {
            (void)cudaGetLastError();
            return 1;
        }
        cache[dev] = n;
    }
    return cache[dev];
}

int64_t round_up(int64_t x) { return (x + 255) / 256 * 256; }
// Which queries are held in two parts.
bool two_n(const MlaParams& p) { return p.ckv_kind != OUT16 && p.ckv_scale_per_ch; }
bool two_r(const MlaParams& p) { return p.k_kind != OUT16 || (p.ckv_kind != OUT16 && !p.ckv_scale_per_ch); }
bool codes_in(const MlaParams& p) { return p.ckv_kind != OUT16 || p.k_kind != OUT16; }
// Whether the queries' rows, (token, head) in order, are evenly spaced, as TMA takes them.
bool q_flat(const MlaParams& p) {
    const int64_t far = int64_t(1) << 38;
    return (p.T == 1 && p.H == 1) || ((p.T == 1 || (p.qn_ts == p.H * p.qn_hs && p.qr_ts == p.H * p.qr_hs)) && p.qn_hs >= p.Dv &&
                                      p.qr_hs >= p.Dk && p.qn_hs < far && p.qr_hs < far);
}

// Rows of `width` elements that start `stride` apart, in boxes of 64 channels and box_rows rows; what lies outside is zeros.
bool encode_2d(CUtensorMap* map, const void* base, bool bf16, int64_t rows, int width, int64_t stride, int box_rows) {
    const cuuint64_t dims[2] = {cuuint64_t(width), cuuint64_t(rows)}, strides[1] = {cuuint64_t(stride) * 2};
    const cuuint32_t box[2] = {64, cuuint32_t(box_rows)}, one[2] = {1, 1};
    return encoder()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims,
                     strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool key_weight_tc_fits(const KeyWeightParams& w) {
    // cost() of one sequence is at most tiles * (groups + 1), and N of them, which may share rows, are added up. A key's place among
    // the new tokens' (up to 255 behind the last one) and the rows of a query box (up to 127 behind) are counted in 31 bits.
    const MlaParams& p = w.m;
    return p.T * p.H <= 0x7FFFFFFF - 511 && ((p.T * p.H + 31) / 32 + 1) * ((p.max_keys + KW_KEYS - 1) / KW_KEYS + 1) <= (int64_t(1) << 62) / p.N;
}

int64_t key_weight_tc_workspace(const KeyWeightParams& w) {
    const MlaParams& p = w.m;
    int64_t n = round_up(ws_bytes(pairs_of_device()));
    if (!codes_in(p) && q_flat(p)) return n;
    const int64_t rows = p.T * p.H;
    return n + round_up(rows * 4) + round_up(rows * p.Dv * 2) * (two_n(p) ? 2 : 1) + round_up(rows * p.Dk * 2) * (two_r(p) ? 2 : 1);
}

cudaError_t launch_key_weight_tc(const KeyWeightParams& w, int dtype, cudaStream_t s) {
    Tc p = {};
    p.w = w;
    MlaParams& a = p.w.m;
    p.pairs = pairs_of_device();
    const bool codes = codes_in(a), bf = dtype == KVR_BF16;
    if (encoder() == nullptr) return cudaErrorNotSupported;
    // Rows of a group: what a sequence has on average, up to 256.
    const int64_t each = (a.T * a.H + a.N - 1) / a.N;
    p.shift = 5;
    while (p.shift < 8 && int64_t(1) << p.shift < each) ++p.shift;
    p.rows = 1 << p.shift;
    p.slots = int(Q_BYTES) / (p.rows * 64);
    if (p.slots > MAX_SLOTS) p.slots = MAX_SLOTS;
    p.lo_n = two_n(a);
    p.lo_r = two_r(a);
    p.patience = kw_patience(a.T * a.H, a.max_keys);
    const int64_t rows = a.d0 * a.d1, n = a.T * a.H;
    Maps maps = {};
    if (!codes && rows < (int64_t(1) << 31) - CKEYS) {
        int r = CKEYS;
        while (a.table != nullptr && r > 1 && a.d1 % r != 0) r /= 2;
        if (r >= 8 && encode_2d(&maps.latent, a.ckv, bf, rows, a.Dv, a.Dv, r) && encode_2d(&maps.rope, a.kc, bf, rows, a.Dk, a.Dk, r)) p.box_rows = r;
    }
    uint16_t *qn_lo = nullptr, *qr_lo = nullptr;
    if (codes || !q_flat(a)) {
        char* at = static_cast<char*>(a.workspace) + round_up(ws_bytes(p.pairs));
        auto take = [&](int64_t bytes) {
            char* got = at;
            at += round_up(bytes);
            return got;
        };
        float* mul = reinterpret_cast<float*>(take(n * 4));
        uint16_t* qn = reinterpret_cast<uint16_t*>(take(n * a.Dv * 2));
        if (p.lo_n) qn_lo = reinterpret_cast<uint16_t*>(take(n * a.Dv * 2));
        uint16_t* qr = reinterpret_cast<uint16_t*>(take(n * a.Dk * 2));
        if (p.lo_r) qr_lo = reinterpret_cast<uint16_t*>(take(n * a.Dk * 2));
        if (!codes) mul = nullptr;
        const int64_t cap = int64_t(sm_count_current_device()) * 6, need = (n + 7) / 8;
        const dim3 grid(unsigned(need < cap ? need : cap));
        const cudaError_t e = bf ? launch_pdl(key_weight_queries_kernel<BF16>, grid, dim3(256), 0, s, a, qn, qn_lo, qr, qr_lo, mul)
                                 : launch_pdl(key_weight_queries_kernel<F16>, grid, dim3(256), 0, s, a, qn, qn_lo, qr, qr_lo, mul);
        if (e != cudaSuccess) return e;
        p.row_mul = mul;
        a.qn = qn;
        a.qn_hs = a.Dv;
        a.qr = qr;
        a.qr_hs = a.Dk;
    }
    // A part whose cache is codes has halves, the other one q's type.
    const int64_t n_stride = a.T == 1 && a.H == 1 ? a.Dv : a.qn_hs, r_stride = a.T == 1 && a.H == 1 ? a.Dk : a.qr_hs;
    const bool bf_n = bf && a.ckv_kind == OUT16, bf_r = bf && a.k_kind == OUT16;
    if (!encode_2d(&maps.qn, a.qn, bf_n, n, a.Dv, n_stride, p.rows / 2) || !encode_2d(&maps.qr, a.qr, bf_r, n, a.Dk, r_stride, p.rows / 2) ||
        (p.lo_n && !encode_2d(&maps.qn_lo, qn_lo, bf_n, n, a.Dv, a.Dv, p.rows / 2)) ||
        (p.lo_r && !encode_2d(&maps.qr_lo, qr_lo, bf_r, n, a.Dk, a.Dk, p.rows / 2)))
        return cudaErrorInvalidValue;
    const bool tma = p.box_rows > 0;
    const cudaError_t e = launch_pdl(kernel_of(dtype, a.ckv_kind, tma), dim3(unsigned(p.pairs * 2)), dim3(threads_of(tma)), SMEM, s, p, maps);
    // Where no sequence can have two groups, nothing is cut that would have to be joined.
    if (e != cudaSuccess || p.pairs == 1 || n <= p.rows) return e;
    return launch_pdl(key_weight_join_kernel, dim3(unsigned(p.pairs - 1)), dim3(KW_KEYS), 0, s, p);
}

}  // namespace kvr
