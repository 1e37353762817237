// The attention weight of each key on the tensor cores: rows of up to 512 + 64 channels.
//
// For the keys of a sequence and its rows (token, head):
//   S = K Q^T,  w[i] = decay past[i] + sum over the rows r that see key i of 2^(f_r S[i, r] - l_r),
// f = scale log2 e and l_r = lse_r log2 e. The logarithms are given, so that no pass over the keys has to come first.
//
// Keys are the product's first operand: a key's scores then lie in one TMEM lane, and the sum over rows is a sum within a
// thread: no shuffles, no atomics, one number a key and group of rows. What is not a key (a hole, the end of a block)
// only spoils its own lane, which is left out at the end.
//
// Tiling: a CTA pair (cta_group::2, M = 256) has 256 keys a step, 128 in each CTA, and a group of up to 256 rows, half of
// them in each CTA's shared memory, where they stay while the tiles of a block pass. Keys come in boxes of 128 keys x 64
// channels through a ring of 4 (8 where the queries leave room), so that a box is reused for all rows of the group and
// nothing of a tile has to wait for the rest. Scores take turns over two halves of TMEM: the exponentials of a tile run
// beside the products of the next one. The sums of a block's tiles stay in shared memory while the sequence's groups
// pass; with one group (a decode step) they go straight to the weights.
//
// Caches of codes: eight warps decode them into halves (every code is exact there). The queries are divided by the scales
// before and held as the sum of two halves each, 22 bits, as a weight is a float32: one half alone was off by 2e-4 of it.
// The second product of the same keys costs tensor-core time, which such a call has to spare while it decodes.
//
// Work is cut into equal shares by cost over the pairs (key_weight_plan.cuh). A block that the cut goes through leaves its
// sums in the workspace, and a second kernel adds them up in a fixed order.
#include <mutex>

#include "cache_ops.cuh"
#include "key_weight_plan.cuh"
#include "latent_tiles.cuh"

namespace kvr {

namespace {

constexpr int CKEYS = KW_KEYS / 2;   // keys of a CTA
constexpr uint32_t BOX = CKEYS * 128;
constexpr int MAX_STAGES = 8;
constexpr uint32_t TMEM_COLS = 512, COL_D = 256;   // a tile's scores: 256 columns at most
constexpr int LSE_SLOTS = 4;   // groups whose logarithms are in shared memory: those of the three tiles at work, and the next
constexpr uint32_t ACC_BYTES = KW_BLOCK * CKEYS * 4, LSE_BYTES = LSE_SLOTS * 1024;

struct alignas(16) Misc {
    uint64_t k_full[MAX_STAGES], k_empty[MAX_STAGES];
    uint64_t q_full, q_free, d_full[2], d_free[2], lse_full[LSE_SLOTS], drain;
    uint32_t tmem;
    int abort;
    KwPos begin, end;
    double wsum[32];
};

struct Tc {
    KeyWeightParams w;
    const uint16_t* qn_lo;   // lower halves of the queries of codes, or NULL
    const uint16_t* qr_lo;
    const float* row_mul;    // power of two per row that prepared queries lack
    int pairs, rows, stages, box_rows;
};

// Shared memory: queries [boxes][rows / 2], ring, sums, logarithms, barriers.
__host__ __device__ inline uint32_t q_bytes(int rows, bool codes) { return uint32_t(rows) * 64u * (codes ? 18u : 9u); }
__host__ __device__ inline uint32_t smem_of(int rows, bool codes, int stages) {
    return q_bytes(rows, codes) + uint32_t(stages) * BOX + ACC_BYTES + LSE_BYTES + uint32_t(sizeof(Misc));
}
static_assert(256 * 64 * 9 + 4 * BOX + ACC_BYTES + LSE_BYTES + sizeof(Misc) <= 232448, "shared memory of a CTA");
static_assert(128 * 64 * 9 + 8 * BOX + ACC_BYTES + LSE_BYTES + sizeof(Misc) <= 232448, "shared memory of a CTA");

// Workspace: header, the pairs' begins, sums of two blocks a pair.
struct alignas(16) Start {
    KwPos at;
    int L, K, pad[2];
};
__host__ __device__ inline int64_t ws_sums(int pairs) { return 256 + (int64_t(pairs) * int64_t(sizeof(Start)) + 255) / 256 * 256; }
__host__ __device__ inline int64_t ws_bytes(int pairs) { return ws_sums(pairs) + int64_t(pairs) * 2 * KW_BLOCK * KW_KEYS * 4; }
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
    __device__ __forceinline__ KwShape operator()(int n) const {
        const Seq s = load_seq(p.w.m, n);
        return {s.L, s.K, p.w.m.H, p.rows, p.w.m.causal != 0};
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
    double sum = 0;
    int bits = 0;
    for (int n = n0; n < n1; ++n) {
        (void)load_seq(p.w.m, n, &bits);
        sum += shapes(n).cost();
    }
    if (bits != 0 && blockIdx.x == 0 && p.w.m.status != nullptr) atomicOr(p.w.m.status, bits);
    double scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) m->wsum[warp] = scan;
    if (tid == 0) m->begin = m->end = {N, 0, 0, 0};
    __syncthreads();
    double before = 0, total = 0;
    for (int q = 0; q < WARPS; ++q) {
        if (q == warp) before = total;
        total += m->wsum[q];
    }
    // (a thread's sequences begin where its predecessor's end, to the bit: both are the same sum)
    double base = __shfl_up_sync(0xFFFFFFFFu, scan, 1);
    base = before + (lane == 0 ? 0 : base);
    const double upto = before + scan;
    const int active = kw_active(total, p.pairs);
    const double u[2] = {pair >= active ? total : total * pair / active, pair + 1 >= active ? total : total * (pair + 1) / active};
    if ((u[0] >= base && u[0] < upto) || (u[1] >= base && u[1] < upto)) {
        double at[2] = {u[0] - base, u[1] - base};
        bool found[2] = {!(u[0] >= base && u[0] < upto), !(u[1] >= base && u[1] < upto)};
        for (int n = n0; n < n1; ++n) {
            const KwShape s = shapes(n);
            const double c = s.cost();
            for (int h = 0; h < 2; ++h) {
                if (found[h]) continue;
                // (the last one with work takes what rounding leaves over)
                if (c > 0 && (at[h] < c || n + 1 == n1)) {
                    (h ? m->end : m->begin) = s.locate(n, at[h]);
                    found[h] = true;
                } else {
                    at[h] -= c;
                }
            }
        }
        for (int h = 0; h < 2; ++h)
            if (!found[h]) (h ? m->end : m->begin) = {n1, 0, 0, 0};
    }
    if (tid == 0 && pair == 0 && cluster_rank() == 0) *ws_space(p).active = active;
}

// What every role has.
struct Ctx {
    const Tc& p;
    Misc* m;
    uint32_t base, ring, tmem, rank;
    int lane, nb;   // nb: 64-channel boxes of the latent part
    float* acc;
    float* lse;
    volatile int* abort;
    bool ok;

    // As in the attention kernel: a wait that gives up poisons the CTA; the warp that starts TMA copies then stops, the others run
    // their loops to the end without waiting.
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
        if (!mbar_try_wait(bar, parity)) ok = wait_on(bar, parity, abort, 0) && ok;
        __syncwarp();
    }
    __device__ __forceinline__ bool gone() const { return __any_sync(0xFFFFFFFFu, !ok); }
    __device__ __forceinline__ uint32_t stage(int st) const { return ring + uint32_t(st) * BOX; }
    __device__ __forceinline__ uint32_t q_box(int b) const { return base + uint32_t(b) * uint32_t(p.rows) * 64u; }
    // This warp's shared-memory writes are done: tell the MMA warp of the pair.
    __device__ __forceinline__ void arrive(uint64_t* bar) {
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(bar, 0);
    }
    __device__ __forceinline__ Walk walk() const { return Walk(Shapes{p}, m->begin, m->end, int(p.w.m.N)); }
};

constexpr int ROPE_BOX = 8, LO_BOX = 9, ROPE_LO_BOX = 17;   // boxes of the queries

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

// One warp brings the CTA's 16-bit keys through TMA: a box is 128 / R copies of R rows, R what divides the cache's blocks.
__device__ __forceinline__ void tma_warp(Ctx& c, const CUtensorMap* latent, const CUtensorMap* rope) {
    const MlaParams& p = c.p.w.m;
    const int R = c.p.box_rows, copies = CKEYS / R, mask = c.p.stages - 1, log = c.p.stages == 8 ? 3 : 2;
    int j = 0;
    Walk w = c.walk();
    while (w.next_block())
        while (w.next_part()) {
            Look next;
            auto look = [&](int kt) {   // (a lane without a copy, and what lies behind the part, has no key)
                const int key = (w.kb * KW_BLOCK + kt) * KW_KEYS + int(c.rank) * CKEYS + c.lane * R;
                next.begin(p, w.n, c.lane < copies && kt < w.kt1 ? w.s.K : 0, key);
            };
            look(w.kt0);
#pragma unroll 1
            for (int kt = w.kt0; kt < w.kt1; ++kt) {
                const int row = int(next.row(p));
                look(kt + 1);
                const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xFFFFFFFFu, row >= 0))) * uint32_t(R) * 128u;
#pragma unroll 1
                for (int b = 0; b <= c.nb; ++b, ++j) {
                    const int st = j & mask;
                    if (j > mask) c.wait(&c.m->k_empty[st], ((j >> log) & 1) ^ 1);
                    if (c.gone()) return;
                    if (c.lane == 0) mbar_expect_at(&c.m->k_full[st], 0, bytes);
                    __syncwarp();
                    if (row >= 0)
                        tma_box_at(c.stage(st) + uint32_t(c.lane * R) * 128u, b < c.nb ? latent : rope, 0, row, b < c.nb ? b : 0,
                                   &c.m->k_full[st], 0);
                }
            }
        }
}

// The tiles of a share as the loading warps go over them: a thread has rows v >> 2 and 64 + v >> 2 of each tile.
struct Tiles {
    const Ctx& c;
    Walk w;
    int kt, r0;
    bool in = false;
    Look look[2];
    int64_t slot[2];
    __device__ __forceinline__ Tiles(const Ctx& x, int v) : c(x), w(x.walk()), kt(0), r0(v >> 2) {}
    __device__ __forceinline__ void begin(int t) {
        const int key = (w.kb * KW_BLOCK + t) * KW_KEYS + int(c.rank) * CKEYS + r0;
        look[0].begin(c.p.w.m, w.n, w.s.K, key);
        look[1].begin(c.p.w.m, w.n, w.s.K, key + 64);
    }
    __device__ __forceinline__ bool next() {
        if (!in || ++kt >= w.kt1) {
            while (!(in && w.next_part())) {
                if (!w.next_block()) return false;
                in = true;
            }
            kt = w.kt0;
            begin(kt);
        }
        slot[0] = look[0].row(c.p.w.m);
        slot[1] = look[1].row(c.p.w.m);
        if (kt + 1 < w.kt1) begin(kt + 1);   // one tile ahead
        return true;
    }
};

// Eight warps bring 16-bit latent rows that TMA does not take (small blocks, narrow rows, rotary codes): 16-byte copies, three
// boxes in flight. A thread has pieces c4 and c4 + 4 of its rows; odd rows take them the other way round, so that eight
// lanes write to all banks.
__device__ __forceinline__ void copy_warps(Ctx& c, int v) {
    const MlaParams& p = c.p.w.m;
    const int c4 = v & 3, r0 = v >> 2, mask = c.p.stages - 1, log = c.p.stages == 8 ? 3 : 2, nc = p.Dv / 8, nr = p.Dk / 8;
    const bool k8 = p.k_kind != OUT16;
    int j = 0;
    Tiles t(c, v);
    while (t.next()) {
        uint4 codes[2];
        if (k8)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                codes[h] = t.slot[h] >= 0 && c4 < p.Dk / 16 ? ld_ahead_v4(static_cast<const uint8_t*>(p.kc) + t.slot[h] * p.Dk + c4 * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int b = 0; b <= c.nb; ++b, ++j) {
            const int st = j & mask;
            if (j > mask) c.wait(&c.m->k_empty[st], ((j >> log) & 1) ^ 1);
            const uint32_t box = c.stage(st);
            const bool rope = b == c.nb;
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
            if (j >= 3) {
                cp_async_wait<3>();
                c.arrive(&c.m->k_full[(j - 3) & mask]);
            }
        }
    }
    cp_async_wait<0>();
    for (int i = max(0, j - 3); i < j; ++i) c.arrive(&c.m->k_full[i & mask]);
}

// Eight warps decode a cache of codes, half a tile's channels at a time, the next half's loads in flight meanwhile.
template <int CK>
__device__ __forceinline__ void code_warps(Ctx& c, int v) {
    const MlaParams& p = c.p.w.m;
    const int c4 = v & 3, r0 = v >> 2, mask = c.p.stages - 1, log = c.p.stages == 8 ? 3 : 2, nc = p.Dv / 16;
    const bool k8 = p.k_kind != OUT16;
    const int nr = k8 ? p.Dk / 16 : p.Dk / 8;
    int j = 0, unit = 2;   // units of a tile: boxes 0-3, boxes 4-7, the rotary part
    Tiles t(c, v);
    auto advance = [&]() {
        if (++unit == 1 && c.nb <= 4) ++unit;
        if (unit < 3) return true;
        unit = 0;
        return t.next();
    };
    auto load = [&](uint4 (&x)[8]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = t.slot[h];
            if (unit < 2) {
                const uint8_t* src = static_cast<const uint8_t*>(p.ckv) + row * p.Dv + unit * 256 + c4 * 16;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[h * 4 + i] = row >= 0 && unit * 16 + i * 4 + c4 < nc ? ld_ahead_v4(src + i * 64) : make_uint4(0, 0, 0, 0);
            } else {
                const uint8_t* src = static_cast<const uint8_t*>(p.kc) + row * p.Dk * (k8 ? 1 : 2) + c4 * 16;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    x[h * 4 + i] = row >= 0 && i * 4 + c4 < nr ? ld_ahead_v4(src + i * 64) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    auto put = [&](int u, const uint4 (&x)[8]) {
        const int boxes = u == 2 ? 1 : min(4, c.nb - u * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= boxes) break;
            const int st = j & mask;
            if (j > mask) c.wait(&c.m->k_empty[st], ((j >> log) & 1) ^ 1);
            const uint32_t box = c.stage(st);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + 64 * h;
                const uint4 y = x[h * 4 + i];
                if (u < 2) {
                    st_shared_v4(box_at(box, r, 2 * c4), codes_to_halves<CK>(y.x, y.y));
                    st_shared_v4(box_at(box, r, 2 * c4 + 1), codes_to_halves<CK>(y.z, y.w));
                } else if (k8) {
                    st_shared_v4(box_at(box, r, 2 * c4), dec8x8<F16>(p.k_kind, y.x, y.y));
                    st_shared_v4(box_at(box, r, 2 * c4 + 1), dec8x8<F16>(p.k_kind, y.z, y.w));
                } else {
                    st_shared_v4(box_at(box, r, c4), y);
                    st_shared_v4(box_at(box, r, c4 + 4), x[h * 4 + 1]);
                }
            }
            c.arrive(&c.m->k_full[st]);
            ++j;
        }
    };
    uint4 x[8], y[8];
    bool more = advance();
    int ux = unit, uy = 0;
    if (more) load(x);
    while (more) {   // two units a turn: the loads in flight need no copies
        more = advance();
        uy = unit;
        if (more) load(y);
        put(ux, x);
        if (!more) break;
        more = advance();
        ux = unit;
        if (more) load(x);
        put(uy, y);
    }
}

// QW warps bring a group's queries, half of its rows, and the logarithms of all: times log2 e, negative, as they are added;
// -inf (a row that saw nothing) and rows behind the last one as -inf, so that the row adds 2^-inf. With prepared queries each
// row's factor stands beside.
template <bool PREP, int QW>
__device__ __forceinline__ void query_warps(Ctx& c, int v) {
    const MlaParams& p = c.p.w.m;
    const int rows = c.p.rows, half = rows / 2, ch = v & 7, r0 = v >> 3, nc = p.Dv / 8, nr = p.Dk / 8;
    constexpr float LOG2E = 1.4426950408889634f;
    int group = 0;
    Walk w = c.walk();
    while (w.next_block()) {
        const int64_t q0 = p.query_start[w.n];
        const unsigned all = unsigned(w.s.L) * unsigned(p.H);
        while (w.next_part()) {
            if (group > 0) c.wait(&c.m->q_free, (group - 1) & 1);
            const unsigned first = unsigned(w.g) * unsigned(rows);
#pragma unroll 2
            for (int r = r0; r < half; r += 4 * QW) {
                const unsigned row = first + c.rank * half + r;
                const bool live = row < all;
                const int64_t t = live ? q0 + row / unsigned(p.H) : 0, head = live ? row % unsigned(p.H) : 0;
                const uint16_t* qn = static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + head * p.qn_hs;
                const uint16_t* qr = static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + head * p.qr_hs;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const bool in = live && b * 8 + ch < nc;
                    if (b < c.nb) cp_async16(box_at(c.q_box(b), r, ch), in ? qn + (b * 8 + ch) * 8 : qn, in);
                }
                cp_async16(box_at(c.q_box(ROPE_BOX), r, ch), live && ch < nr ? qr + ch * 8 : qr, live && ch < nr);
                if (PREP) {
                    const int64_t at = t * p.H + head;
                    if (c.p.qn_lo != nullptr) {
                        const uint16_t* lo = c.p.qn_lo + at * p.Dv;
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            const bool in = live && b * 8 + ch < nc;
                            if (b < c.nb) cp_async16(box_at(c.q_box(LO_BOX + b), r, ch), in ? lo + (b * 8 + ch) * 8 : lo, in);
                        }
                    }
                    if (c.p.qr_lo != nullptr) {
                        const uint16_t* lo = c.p.qr_lo + at * p.Dk;
                        cp_async16(box_at(c.q_box(ROPE_LO_BOX), r, ch), live && ch < nr ? lo + ch * 8 : lo, live && ch < nr);
                    }
                }
            }
            cp_async_commit();
            float* lse = c.lse + (group % LSE_SLOTS) * 256;
            for (int i = v; i < rows; i += 32 * QW) {
                const bool live = first + i < all;
                const int64_t at = live ? q0 * p.H + first + i : 0;
                const float l = live ? p.lse[at] : -INFINITY, x = l == -INFINITY ? -INFINITY : -l * LOG2E;
                if (PREP) {
                    lse[2 * i] = live ? c.p.row_mul[at] * (p.scale * LOG2E) : 0.f;
                    lse[2 * i + 1] = x;
                } else {
                    lse[i] = x;
                }
            }
            __syncwarp();
            if (c.lane == 0) mbar_arrive(&c.m->lse_full[group % LSE_SLOTS]);
            cp_async_wait<0>();
            c.arrive(&c.m->q_full);
            ++group;
        }
    }
}

// The MMA warp of CTA 0. C8, K8: which operands are halves with a second part.
template <class IT, bool C8>
__device__ __forceinline__ void mma_warp(Ctx& c) {
    const Tc& p = c.p;
    Misc* m = c.m;
    const bool k8 = p.w.m.k_kind != OUT16;
    const uint32_t id_it = tc_idesc(KW_KEYS, p.rows, is_bf16<IT>, false), id_half = tc_idesc(KW_KEYS, p.rows, false, false);
    const uint32_t id_n = C8 ? id_half : id_it, id_r = k8 ? id_half : id_it;
    const int mask = p.stages - 1, log = p.stages == 8 ? 3 : 2;
    const bool leader = elect_one();
    int j = 0, group = 0, used[2] = {0, 0};
    Walk w = c.walk();
    while (w.next_block())
        while (w.next_part()) {
            c.wait(&m->q_full, group & 1);
#pragma unroll 1
            for (int kt = w.kt0; kt < w.kt1; ++kt) {
                const int h = kt & 1;
                const uint32_t d = c.tmem + uint32_t(h) * COL_D;
                if (used[h] > 0) c.wait(&m->d_free[h], (used[h] - 1) & 1);
                ++used[h];
#pragma unroll 1
                for (int b = 0; b <= c.nb; ++b, ++j) {
                    const int st = j & mask;
                    const bool rope = b == c.nb;
                    c.wait(&m->k_full[st], (j >> log) & 1);
                    tc_fence_after();
                    if (leader) {
                        const uint64_t kd = tc_desc(c.stage(st), 16, 1024), qd = tc_desc(c.q_box(rope ? ROPE_BOX : b), 16, 1024);
#pragma unroll
                        for (int s = 0; s < 4; ++s) tc_mma_pair(d, kd + s * 2, qd + s * 2, rope ? id_r : id_n, b > 0 || s > 0);
                        if (rope ? k8 : C8) {
                            const uint64_t lo = tc_desc(c.q_box(rope ? ROPE_LO_BOX : LO_BOX + b), 16, 1024);
#pragma unroll
                            for (int s = 0; s < 4; ++s) tc_mma_pair(d, kd + s * 2, lo + s * 2, rope ? id_r : id_n, true);
                        }
                        tc_commit_pair(&m->k_empty[st]);
                    }
                    __syncwarp();
                }
                if (leader) {
                    tc_commit_pair(&m->d_full[h]);
                    if (kt + 1 == w.kt1) tc_commit_pair(&m->q_free);
                }
                __syncwarp();
            }
            ++group;
        }
    if (!c.ok) {   // let what was issued finish before TMEM goes
        if (leader) {
            tc_commit_pair(&m->drain);
            mbar_wait(&m->drain, 0, nullptr);
        }
        __syncwarp();
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
// The same where causal masking may hide the key from rows: `sees` keys of the token that the column belongs to, as its
// head `head`; the next token sees one more.
template <bool PREP>
__device__ __forceinline__ float2 masked_sum(const float (&s)[32], const float* lse, float f, float2 sum, int key, int H, int& sees, int& head) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float x = PREP ? fmaf(s[i], lse[2 * i], lse[2 * i + 1]) : fmaf(s[i], f, lse[i]);
        if (key < sees) sum.x += exp2_approx(x);
        if (++head == H) {
            head = 0;
            ++sees;
        }
    }
    return sum;
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
    float* acc = c.acc + r;
    int group = 0, used[2] = {0, 0};
    Walk w = c.walk();
    while (w.next_block()) {
        for (int kt = mine; kt < w.tiles; kt += EG) acc[kt * CKEYS] = 0.f;
        int from = KW_BLOCK, upto = 0;   // tiles with sums
        const int key0 = w.kb * (KW_BLOCK * KW_KEYS) + int(c.rank) * CKEYS;
        while (w.next_part()) {
            const float* lse = c.lse + (group % LSE_SLOTS) * 256;
            c.wait(&m->lse_full[group % LSE_SLOTS], (group / LSE_SLOTS) & 1);
            ++group;
            from = min(from, w.kt0);
            upto = max(upto, w.kt1);
            const unsigned first = unsigned(w.g) * unsigned(rows);
            const int t0 = int(first / unsigned(a.H)), h0 = int(first % unsigned(a.H));
            const int sees0 = a.causal ? w.s.K - w.s.L + t0 + 1 : w.s.K;
#pragma unroll 1
            for (int kt = w.kt0; kt < w.kt1; ++kt) {
                const int h = kt & 1;
                if (EG == 2 && h != mine) continue;
                c.wait(&m->d_full[h], used[h] & 1);
                ++used[h];
                tc_fence_after();
                const uint32_t d = lanes + uint32_t(h) * COL_D;
                const int key = key0 + kt * KW_KEYS + r;
                const bool masked = key0 + kt * KW_KEYS + CKEYS > sees0 && a.causal;
                float2 sum = make_float2(0.f, 0.f);
                int sees = sees0, head = h0;
                float x[32], y[32];
                tmem_ld32(d, x);
#pragma unroll 1
                for (int q = 0; q < rows; q += 64) {
                    tmem_wait_ld();
                    if (q + 32 < rows) tmem_ld32(d + q + 32, y);
                    if (masked) sum = masked_sum<PREP>(x, lse + q * (PREP ? 2 : 1), f, sum, key, a.H, sees, head);
                    else sum = column_sum<PREP>(x, lse + q * (PREP ? 2 : 1), f, sum);
                    if (q + 32 >= rows) break;
                    tmem_wait_ld();
                    if (q + 64 < rows) tmem_ld32(d + q + 64, x);
                    if (masked) sum = masked_sum<PREP>(y, lse + (q + 32) * (PREP ? 2 : 1), f, sum, key, a.H, sees, head);
                    else sum = column_sum<PREP>(y, lse + (q + 32) * (PREP ? 2 : 1), f, sum);
                }
                tc_fence_before();
                __syncwarp();
                if (c.lane == 0) mbar_arrive_at(&m->d_free[h], 0);
                acc[kt * CKEYS] += sum.x + sum.y;
            }
        }
        // Out: to the weights where the share has all that adds to them, else to the workspace.
        const bool direct = w.s.groups() == 1 || w.whole(m->begin);
        const bool only = w.s.groups() == 1;   // its tiles alone: others may be another pair's
        const int slot = pair * 2 + (m->begin.n == w.n && m->begin.kb == w.kb ? 0 : 1);
        float* sums = ws_space(p).sums + int64_t(slot) * (KW_BLOCK * KW_KEYS) + int(c.rank) * CKEYS + r;
        const float* past = p.w.past == nullptr ? nullptr : p.w.past + w.n * p.w.past_stride;
        float* weight = p.w.weight + w.n * p.w.weight_stride;
        for (int kt = mine; kt < w.tiles; kt += EG) {
            if (only && (kt < from || kt >= upto)) continue;
            const int key = key0 + kt * KW_KEYS + r;
            float v = acc[kt * CKEYS];
            if (key_row(a, w.n, w.s.K, key) < 0) v = 0.f;   // whatever lay in its place
            if (!direct) {
                sums[kt * KW_KEYS] = v;
            } else if (key < w.s.K) {
                weight[key] = past == nullptr ? v : fmaf(p.w.decay, past[key], v);
            }
        }
    }
}

// TMA: the latent rows come through it. Warps: 0 to 4 EG - 1 sums, then QW queries, 1 MMA, and 1 for TMA or 8 that load and
// decode; at most 16, so that each thread may have 128 registers.
template <bool TMA>
struct Roles {
    static constexpr int EG = TMA ? 2 : 1, QW = TMA ? 4 : 2;
    static constexpr int QUERY = 4 * EG, MMA = QUERY + QW, LOAD = MMA + 1, LOADERS = TMA ? 1 : 8;
    static constexpr int THREADS = (LOAD + LOADERS) * 32;
};

template <class IT, int CK, bool TMA>
__global__ void __launch_bounds__(Roles<TMA>::THREADS, 1) __cluster_dims__(2, 1, 1)
    key_weight_tc_kernel(const __grid_constant__ Tc p, const __grid_constant__ CUtensorMap latent, const __grid_constant__ CUtensorMap rope) {
    using R = Roles<TMA>;
    constexpr bool C8 = CK != OUT16;
    const bool prep = p.row_mul != nullptr;
    extern __shared__ __align__(1024) uint8_t smem_raw[];   // the swizzle repeats every 1024 bytes
    const uint32_t base = smem_u32(smem_raw), qb = q_bytes(p.rows, prep);
    uint8_t* at = smem_raw + qb + uint32_t(p.stages) * BOX;
    float* acc = reinterpret_cast<float*>(at);
    float* lse = reinterpret_cast<float*>(at + ACC_BYTES);
    Misc* m = reinterpret_cast<Misc*>(at + ACC_BYTES + LSE_BYTES);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pair = blockIdx.x >> 1;
    const uint32_t rank = cluster_rank();
    if (base % 1024 != 0) {   // the declaration's alignment was not kept: nothing below would be right
        if (tid == 0 && p.w.m.status != nullptr) atomicOr(p.w.m.status, KVR_DEVERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&m->k_full[s], 2 * R::LOADERS);
            mbar_init(&m->k_empty[s], 1);
        }
        mbar_init(&m->q_full, 2 * R::QW);
        mbar_init(&m->q_free, 1);
        for (int h = 0; h < 2; ++h) {
            mbar_init(&m->d_full[h], 1);
            mbar_init(&m->d_free[h], 8);
        }
        for (int s = 0; s < LSE_SLOTS; ++s) mbar_init(&m->lse_full[s], R::QW);
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
    schedule<R::THREADS>(p, m, pair);
    __syncthreads();
    if (tid == 0 && rank == 0) {
        Seq s = {0, 0, 0};
        if (m->begin.n < p.w.m.N) s = load_seq(p.w.m, m->begin.n);
        ws_space(p).starts[pair] = {m->begin, s.L, s.K, {0, 0}};
    }
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = m->tmem;
    Ctx c{p, m, base, base + qb, tmem, rank, lane, (p.w.m.Dv + 63) / 64, acc, lse, &m->abort, true};
    if (warp < R::QUERY) {
        if (C8 || (!TMA && prep)) sum_warps<true, R::EG>(c, tid, pair);
        else if (!C8) sum_warps<false, R::EG>(c, tid, pair);
    } else if (warp < R::MMA) {
        if (C8 || (!TMA && prep)) query_warps<true, R::QW>(c, tid - R::QUERY * 32);
        else if (!C8) query_warps<false, R::QW>(c, tid - R::QUERY * 32);
    } else if (warp == R::MMA) {
        if (rank == 0) mma_warp<IT, C8>(c);
    } else if constexpr (TMA) {
        tma_warp(c, &latent, &rope);
    } else if constexpr (C8) {
        code_warps<CK>(c, tid - R::LOAD * 32);
    } else {
        copy_warps(c, tid - R::LOAD * 32);
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
// The 16-bit part keeps its type, over the same power. One warp a row.
template <class IT>
__global__ void __launch_bounds__(256) key_weight_queries_kernel(const __grid_constant__ MlaParams p, uint16_t* qn, uint16_t* qn_lo, uint16_t* qr,
                                                                 uint16_t* qr_lo, float* mul) {
    __shared__ float inv[512], invk[64];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int c = threadIdx.x; c < p.Dv; c += 256) inv[c] = qn_lo == nullptr ? 1.f : 1.f / p.ckv_scale[p.ckv_scale_per_ch ? c : 0];
    if (threadIdx.x < p.Dk) invk[threadIdx.x] = qr_lo == nullptr ? 1.f : 1.f / p.k_scale[p.k_scale_per_ch ? threadIdx.x : 0];
    __syncthreads();
    const int64_t rows = p.T * p.H;
    for (int64_t row = int64_t(blockIdx.x) * 8 + warp; row < rows; row += int64_t(gridDim.x) * 8) {
        const int64_t t = row / p.H, head = row - t * p.H;
        float z[3][8], top = 0.f;   // two pieces of the latent part, one of the rotary part
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int ch = (k < 2 ? k * 32 + lane : lane) * 8;
            const bool in = ch < (k < 2 ? p.Dv : p.Dk);
            const uint16_t* q = k < 2 ? static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + head * p.qn_hs
                                      : static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + head * p.qr_hs;
            const uint4 x = in ? ld_stream_v4(q + ch) : make_uint4(0, 0, 0, 0);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
            const float* by = k < 2 ? inv : invk;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                z[k][2 * i] = in ? IT::lo(u[i]) * by[ch + 2 * i] : 0.f;
                z[k][2 * i + 1] = in ? IT::hi(u[i]) * by[ch + 2 * i + 1] : 0.f;
                top = fmaxf(top, fmaxf(fabsf(z[k][2 * i]), fabsf(z[k][2 * i + 1])));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const int e = top > 0.f && top <= 3.0e38f ? min(max(ilogbf(top) - 13, -113), 113) : 0;
        const float g = ldexpf(1.f, -e);
        if (lane == 0) mul[row] = ldexpf(1.f, e);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int ch = (k < 2 ? k * 32 + lane : lane) * 8, width = k < 2 ? p.Dv : p.Dk;
            if (ch >= width) continue;
            uint16_t* hi = (k < 2 ? qn : qr) + row * width + ch;
            uint16_t* lo = k < 2 ? qn_lo : qr_lo;
            uint32_t a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = z[k][2 * i] * g, y = z[k][2 * i + 1] * g;
                if (lo == nullptr) {
                    a[i] = IT::pack(x, y);
                } else {
                    a[i] = F16::pack(x, y);
                    b[i] = F16::pack(x - F16::lo(a[i]), y - F16::hi(a[i]));
                }
            }
            *reinterpret_cast<uint4*>(hi) = make_uint4(a[0], a[1], a[2], a[3]);
            if (lo != nullptr) *reinterpret_cast<uint4*>(lo + row * width + ch) = make_uint4(b[0], b[1], b[2], b[3]);
        }
    }
}

// Adds up the sums of a block that the cut goes through, in the pairs' order: blocks x take the one that the begin of pair
// x + 1 is in, if that is the first inside it. A thread has four keys.
constexpr int JOIN_THREADS = 256;
__global__ void __launch_bounds__(JOIN_THREADS) key_weight_join_kernel(const __grid_constant__ Tc p) {
    const Space ws = ws_space(p);
    const int lane = threadIdx.x & 31, b = blockIdx.x + 1;
    const int i = (blockIdx.y * JOIN_THREADS + threadIdx.x) * 4;   // of the block's keys
    auto start = [&](int q) {
        Start v = {{-1, 0, 0, 0}, 0, 0, {0, 0}};
        if (q < p.pairs) v = ws.starts[q];
        return v;
    };
    pdl_wait();
    pdl_launch_dependents();
    const int active = *ws.active;
    if (b >= active) return;
    const Start here = start(b), before = start(b - 1);
    if (here.at.n >= p.w.m.N || !kw_inside(here.at)) return;
    const KwShape s = {here.L, here.K, p.w.m.H, p.rows, p.w.m.causal != 0};
    const bool same = kw_same_block(before.at, here.at);
    if (s.groups() == 1 || (same && kw_inside(before.at))) return;
    const int key = here.at.kb * (KW_BLOCK * KW_KEYS) + i;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* sums = ws.sums + i;
    auto add = [&](int slot) {
        const float4 v = *reinterpret_cast<const float4*>(sums + int64_t(slot) * (KW_BLOCK * KW_KEYS));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    };
    // The last block of pair b - 1, then the first of each pair that begins inside; none of a pair without work.
    if (!kw_same(before.at, here.at)) add((b - 1) * 2 + (same ? 0 : 1));
    for (int at = b;; at += 31) {
        const Start x = start(at + lane);   // lane i has pair at + i; its end is lane i + 1's begin
        const KwPos y = {__shfl_down_sync(0xFFFFFFFFu, x.at.n, 1), __shfl_down_sync(0xFFFFFFFFu, x.at.kb, 1),
                         __shfl_down_sync(0xFFFFFFFFu, x.at.g, 1), __shfl_down_sync(0xFFFFFFFFu, x.at.kt, 1)};
        const bool in = at + lane < active && kw_same_block(x.at, here.at);
        const uint32_t run = __ballot_sync(0xFFFFFFFFu, in), works = __ballot_sync(0xFFFFFFFFu, in && !(at + lane + 1 < active && kw_same(x.at, y)));
        const int count = min(31, run == 0xFFFFFFFFu ? 32 : __ffs(~run) - 1);
#pragma unroll 4
        for (int q = 0; q < count; ++q)
            if (works >> q & 1) add((at + q) * 2);
        if (count < 31) break;
    }
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
    const int n = here.at.n;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (key + k < here.K) {
            float* to = p.w.weight + n * p.w.weight_stride + key + k;
            *to = p.w.past == nullptr ? v[k] : fmaf(p.w.decay, p.w.past[n * p.w.past_stride + key + k], v[k]);
        }
}
static_assert(KW_BLOCK * KW_KEYS % (JOIN_THREADS * 4) == 0, "whole blocks of threads");

using Kernel = void (*)(Tc, CUtensorMap, CUtensorMap);
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
constexpr int MOST_SMEM = 232448;

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
        cfg.dynamicSmemBytes = MOST_SMEM;
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
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_SMEM) == cudaSuccess;
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

}  // namespace

int64_t key_weight_tc_workspace(const KeyWeightParams& w) {
    const MlaParams& p = w.m;
    int64_t n = round_up(ws_bytes(pairs_of_device()));
    if (p.ckv_kind == OUT16 && p.k_kind == OUT16) return n;
    const int64_t rows = p.T * p.H;
    return n + round_up(rows * 4) + round_up(rows * p.Dv * 2) * (p.ckv_kind != OUT16 ? 2 : 1) + round_up(rows * p.Dk * 2) * (p.k_kind != OUT16 ? 2 : 1);
}

cudaError_t launch_key_weight_tc(const KeyWeightParams& w, int dtype, cudaStream_t s) {
    Tc p = {};
    p.w = w;
    MlaParams& a = p.w.m;
    p.pairs = pairs_of_device();
    const bool codes = a.ckv_kind != OUT16 || a.k_kind != OUT16;
    // Rows of a group: what a sequence has on average, up to 256 (128 where queries are held twice).
    const int64_t each = (a.T * a.H + a.N - 1) / a.N, most = codes ? 128 : 256;
    p.rows = 32;
    while (p.rows < most && p.rows < each) p.rows *= 2;
    p.stages = smem_of(p.rows, codes, 8) <= uint32_t(MOST_SMEM) ? 8 : 4;
    const int64_t rows = a.d0 * a.d1;
    CUtensorMap latent = {}, rope = {};
    if (!codes && a.Dv % 64 == 0 && a.Dk == 64 && rows < (int64_t(1) << 31) - CKEYS) {
        int r = CKEYS;
        while (a.table != nullptr && r > 1 && a.d1 % r != 0) r /= 2;
        const bool bf = dtype == KVR_BF16;
        if (r >= 8 && encoder() != nullptr && encode_rows(&latent, a.ckv, bf, rows, a.Dv, r, 1) && encode_rows(&rope, a.kc, bf, rows, a.Dk, r, 1))
            p.box_rows = r;
    }
    if (codes) {
        char* at = static_cast<char*>(a.workspace) + round_up(ws_bytes(p.pairs));
        const int64_t n = a.T * a.H;
        auto take = [&](int64_t bytes) {
            char* got = at;
            at += round_up(bytes);
            return got;
        };
        float* mul = reinterpret_cast<float*>(take(n * 4));
        uint16_t* qn = reinterpret_cast<uint16_t*>(take(n * a.Dv * 2));
        uint16_t* qn_lo = a.ckv_kind != OUT16 ? reinterpret_cast<uint16_t*>(take(n * a.Dv * 2)) : nullptr;
        uint16_t* qr = reinterpret_cast<uint16_t*>(take(n * a.Dk * 2));
        uint16_t* qr_lo = a.k_kind != OUT16 ? reinterpret_cast<uint16_t*>(take(n * a.Dk * 2)) : nullptr;
        const int64_t cap = int64_t(sm_count_current_device()) * 8, need = (n + 7) / 8;
        const dim3 grid(unsigned(need < cap ? need : cap));
        const cudaError_t e = dtype == KVR_BF16 ? launch_pdl(key_weight_queries_kernel<BF16>, grid, dim3(256), 0, s, a, qn, qn_lo, qr, qr_lo, mul)
                                                : launch_pdl(key_weight_queries_kernel<F16>, grid, dim3(256), 0, s, a, qn, qn_lo, qr, qr_lo, mul);
        if (e != cudaSuccess) return e;
        p.row_mul = mul;
        p.qn_lo = qn_lo;
        p.qr_lo = qr_lo;
        a.qn = qn;
        a.qn_ts = int64_t(a.H) * a.Dv;
        a.qn_hs = a.Dv;
        a.qr = qr;
        a.qr_ts = int64_t(a.H) * a.Dk;
        a.qr_hs = a.Dk;
    }
    const bool tma = p.box_rows > 0;
    const cudaError_t e = launch_pdl(kernel_of(dtype, a.ckv_kind, tma), dim3(unsigned(p.pairs * 2)), dim3(threads_of(tma)),
                                     smem_of(p.rows, codes, p.stages), s, p, latent, rope);
    // Where no sequence can have two groups, nothing is cut that would have to be joined.
    if (e != cudaSuccess || p.pairs == 1 || a.T * a.H <= p.rows) return e;
    return launch_pdl(key_weight_join_kernel, dim3(unsigned(p.pairs - 1), KW_BLOCK * KW_KEYS / (JOIN_THREADS * 4)), dim3(JOIN_THREADS), 0, s, p);
}

}  // namespace kvr
