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
// A key step in a CTA, three steps in flight:
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
#include <mutex>

#include "tcgen05.cuh"

namespace kvr {

namespace {

constexpr int ROWS = 128, CROWS = 64;    // rows of a pair, of a CTA
constexpr int KEYS = 64, CKEYS = 32;     // keys of a step, of a CTA
constexpr int STAGES = 3;
constexpr uint32_t QBOX = CROWS * 128, KBOX = CKEYS * 128;
constexpr uint32_t STAGE_BYTES = 9 * KBOX, PBUF = CROWS * 128;
constexpr uint32_t OFF_Q = 0, OFF_K = 9 * QBOX, OFF_P = OFF_K + STAGES * STAGE_BYTES, OFF_MISC = OFF_P + 2 * PBUF;
constexpr int THREADS = 416;             // 4 softmax, 4 key, 4 swap and query warps, 1 MMA warp
constexpr uint32_t TMEM_COLS = 512, COL_S = 256;   // O: columns 0..255, S: two buffers of 32 + 32
constexpr int64_t ITEM_COST = 128;       // an item's own cost, in keys
constexpr int64_t MIN_KEYS = 128;        // least work of a pair, in keys

struct Bound {
    int n, i, kt, pad;   // sequence, row tile, key tile
};

struct Misc {
    uint64_t k_full[STAGES], v_full[STAGES], empty[STAGES];
    uint64_t s_full[2], p_full[2], pv_done[2], q_full, drain;
    uint32_t tmem;
    int abort;
    Bound begin, end;
    int64_t wsum[16];
    float red[2][128], lred[128];
    float inv_v[512], inv_k[64];
    float lift[2];
};
constexpr uint32_t SMEM_BYTES = OFF_MISC + uint32_t(sizeof(Misc)) + 1024;

// Workspace: header, first bounds of the pairs, (m, l) and O of two parts a pair.
struct Space {
    int32_t* active;
    Bound* bounds;
    float2* ml;
    float* o;
};
__host__ __device__ inline int64_t ws_ml(int pairs) { return 256 + (int64_t(pairs) * 16 + 255) / 256 * 256; }
__host__ __device__ inline int64_t ws_o(int pairs) { return ws_ml(pairs) + int64_t(pairs) * 2 * ROWS * 8; }
__host__ __device__ inline int64_t ws_bytes(int pairs, int Dv) { return ws_o(pairs) + int64_t(pairs) * 2 * ROWS * Dv * 4; }
__device__ __forceinline__ Space ws_space(const MlaParams& p) {
    char* w = static_cast<char*>(p.workspace);
    return {reinterpret_cast<int32_t*>(w), reinterpret_cast<Bound*>(w + 256), reinterpret_cast<float2*>(w + ws_ml(p.pairs)),
            reinterpret_cast<float*>(w + ws_o(p.pairs))};
}

struct Seq {
    int64_t q0;
    int L, K;   // L = 0: nothing to do
};

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
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cost(p, s.L, s.K, mid) <= off) lo = mid;
        else hi = mid - 1;
    }
    const int64_t c0 = cost(p, s.L, s.K, lo), c1 = cost(p, s.L, s.K, lo + 1);
    const int kn = key_tiles(p, s.L, s.K, lo);
    const int kt = int(double(off - c0) / double(c1 - c0) * double(kn));   // monotonic in off: shares neither overlap nor leave gaps
    return {n, lo, min(kt, kn - 1), 0};
}

// The parts of items between two bounds, in order.
struct Walk {
    const MlaParams& p;
    Bound at, end;
    int loaded = -1;
    Seq s;
    // the current part
    int n, i, kt0, kt1;
    bool whole;
    __device__ Walk(const MlaParams& q, const Bound& b, const Bound& e) : p(q), at(b), end(e) {}
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

// This pair's share of the work: every CTA scans all sequences' costs.
__device__ void schedule(const MlaParams& p, Misc* m, int pair) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (int(p.N) + THREADS - 1) / THREADS;
    const int n0 = min(tid * per, int(p.N)), n1 = min(n0 + per, int(p.N));
    int64_t sum = 0;
    int bits = 0;
    for (int n = n0; n < n1; ++n) {
        const Seq s = load_seq(p, n, &bits);
        if (s.L > 0) sum += cost(p, s.L, s.K, row_tiles(p, s.L));
    }
    if (bits != 0 && blockIdx.x == 0 && p.status != nullptr) atomicOr(p.status, bits);
    int64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) m->wsum[warp] = scan;
    if (tid == 0) m->begin = m->end = {int(p.N), 0, 0, 0};
    __syncthreads();
    int64_t base = scan - sum, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += m->wsum[w];
        total += m->wsum[w];
    }
    const int64_t most = total / (p.H * MIN_KEYS);
    const int active = most < 1 ? 1 : (most < p.pairs ? int(most) : p.pairs);
    const int64_t u0 = pair < active ? total * pair / active : total, u1 = pair < active ? total * (pair + 1) / active : total;
    if (sum > 0) {
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const int64_t u = e ? u1 : u0;
            if (u < base || u >= base + sum) continue;
            int64_t b = base;
            for (int n = n0; n < n1; ++n) {
                const Seq s = load_seq(p, n);
                const int64_t c = s.L > 0 ? cost(p, s.L, s.K, row_tiles(p, s.L)) : 0;
                if (u < b + c) {
                    (e ? m->end : m->begin) = locate(p, n, s, u - b);
                    break;
                }
                b += c;
            }
        }
    }
    __syncthreads();
    if (tid == 0 && cluster_rank() == 0) {
        const Space w = ws_space(p);
        w.bounds[pair] = m->begin;
        if (pair == 0) *w.active = active;
    }
}

// Four 8-bit codes to packed 16-bit values (exact in either type).
template <class IT>
__device__ __forceinline__ uint2 dec8x4(int kind, uint32_t u) {
    uint32_t h[2];
    if (kind == OUT_I8) {   // 1024 + (code + 128) as a half, less 1152
        u ^= 0x80808080u;
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t x = __byte_perm(u, 0x64646464u, k ? 0x4342 : 0x4140);
            __half2 r = __hsub2(*reinterpret_cast<__half2*>(&x), off);
            h[k] = *reinterpret_cast<uint32_t*>(&r);
        }
    } else if (kind == OUT_E5M2) {   // the upper byte of a half
        h[0] = __byte_perm(u, 0, 0x1404);
        h[1] = __byte_perm(u, 0, 0x3424);
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(h[0]), "=r"(h[1])
            : "r"(u));
    }
    if constexpr (IT::is_bf16) {
        return make_uint2(BF16::pack(F16::lo(h[0]), F16::hi(h[0])), BF16::pack(F16::lo(h[1]), F16::hi(h[1])));
    } else {
        return make_uint2(h[0], h[1]);
    }
}
template <class IT>
__device__ __forceinline__ uint4 dec8x8(int kind, uint32_t a, uint32_t b) {
    const uint2 x = dec8x4<IT>(kind, a), y = dec8x4<IT>(kind, b);
    return make_uint4(x.x, x.y, y.x, y.y);
}

// Cache row of a key, or -1 where there is none to read.
__device__ __forceinline__ int64_t key_slot(const MlaParams& p, int n, int K, int key) {
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

__device__ __forceinline__ uint32_t box_at(uint32_t box, int row, int chunk) {
    return box + uint32_t(row) * 128u + (uint32_t(chunk ^ (row & 7)) << 4);
}

template <class IT, bool C8>
__global__ void __launch_bounds__(THREADS, 1) __cluster_dims__(2, 1, 1) mla_tc_kernel(const __grid_constant__ MlaParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    Misc* m = reinterpret_cast<Misc*>(smem_raw + (base - smem_u32(smem_raw)) + OFF_MISC);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;
    const int na = p.Dv > 256 ? 2 : 1, nb = (p.Dv + 63) / 64;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&m->k_full[s], 8);
            mbar_init(&m->v_full[s], 8);
            mbar_init(&m->empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m->s_full[s], 1);
            mbar_init(&m->p_full[s], 8);
            mbar_init(&m->pv_done[s], 1);
        }
        mbar_init(&m->q_full, 8);
        mbar_init(&m->drain, 1);
        m->abort = 0;
        fence_mbar_init();
    }
    if (warp == 12) tmem_alloc_pair(&m->tmem, TMEM_COLS);
    pdl_wait();
    pdl_launch_dependents();
    schedule(p, m, pair);
    // 1 / scale of each channel, and per part the power of two that the query is divided by (below).
    if (C8 || p.k_kind != OUT16) {
        for (int c = tid; c < 512; c += THREADS)
            m->inv_v[c] = p.ckv_kind == OUT16 || c >= p.Dv ? 1.f : 1.f / p.ckv_scale[p.ckv_scale_per_ch ? c : 0];
        if (tid < 64) m->inv_k[tid] = p.k_kind == OUT16 || tid >= p.Dk ? 1.f : 1.f / p.k_scale[p.k_scale_per_ch ? tid : 0];
        __syncthreads();
        if (warp < 2) {
            float v = 0.f;
            for (int c = lane; c < (warp ? p.Dk : p.Dv); c += 32) v = fmaxf(v, fabsf(warp ? m->inv_k[c] : m->inv_v[c]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            if (lane == 0) m->lift[warp] = exp2f(ceilf(log2f(v)));
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = m->tmem;
    volatile int* abort = &m->abort;
    bool ok = true;
    // A wait that gives up (one second) poisons the CTA: the others give up at their first look, and every role
    // runs its loops to the end without waiting, so that no barrier is left with threads missing.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!mbar_wait_cluster(bar, parity, abort)) {
            *abort = 1;
            ok = false;
        }
    };
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        wait(bar, parity);
        __syncwarp();
    };

    if (warp < 4) {
        // ------------------------------------------------------------------
        // Softmax and output: thread (row r, half h of the keys and channels).
        // ------------------------------------------------------------------
        const int r = tid & 63, h = tid >> 6;
        const uint32_t lanes = tmem + (uint32_t(warp) << 21);
        // Score = fn * (latent product) + fr * (rotary product), in powers of two.
        const float l2 = p.scale * 1.4426950408889634f;
        float fn = l2, fr = l2;
        const bool split = C8 || p.k_kind != OUT16;
        if (split) {
            fn = l2 * (p.ckv_scale_per_ch ? m->lift[0] : m->inv_v[0]);
            fr = l2 * (p.k_scale_per_ch ? m->lift[1] : m->inv_k[0]);
        }
        int j = 0, part = 0;
        Walk w(p, m->begin, m->end);
        while (w.next()) {
            const unsigned row = unsigned(w.i) * ROWS + rank * CROWS + r;
            const bool live = row < unsigned(w.s.L) * unsigned(p.H);
            const int t = int(row / unsigned(p.H)), head = int(row % unsigned(p.H));
            const int vis = live ? seen(p, w.s.L, w.s.K, t) : 0;
            int wmin = live ? vis : 0x7FFFFFFF;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) wmin = min(wmin, __shfl_xor_sync(0xFFFFFFFFu, wmin, o));
            float mx = -INFINITY, sum = 0.f;
            for (int kt = w.kt0; kt < w.kt1; ++kt, ++j) {
                const int key0 = kt * KEYS + h * CKEYS;
                // Keys that exist: bit i for key0 + i.
                const uint32_t held = __ballot_sync(0xFFFFFFFFu, key_slot(p, w.n, w.s.K, key0 + lane) >= 0);
                wait_warp(&m->s_full[j & 1], (j >> 1) & 1);
                tc_fence_after();
                float s[32];
                tmem_ld32(lanes + COL_S + uint32_t(j & 1) * 64, s);
                if (split) {
                    float s2[32];
                    tmem_ld32(lanes + COL_S + uint32_t(j & 1) * 64 + 32, s2);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = fmaf(s2[i], fr, s[i] * fn);
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] *= fn;
                }
                if (held != 0xFFFFFFFFu || key0 + CKEYS > wmin) {
                    const int left = vis - key0;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i >= left || !(held >> i & 1)) s[i] = -INFINITY;
                }
                float top = s[0];
#pragma unroll
                for (int i = 1; i < 32; ++i) top = fmaxf(top, s[i]);
                m->red[j & 1][tid] = top;
                asm volatile("bar.sync 1, 128;" ::: "memory");
                top = fmaxf(fmaxf(top, m->red[j & 1][tid ^ 64]), mx);
                // The sum is rescaled only when the maximum grows by more than 2^8: weights then stay below 2^8,
                // and the 16-bit rounding of a weight is relative.
                const bool grow = top > mx + 8.f;
                const float f = grow ? exp2f(mx - top) : 1.f;
                if (grow) {
                    mx = top;
                    sum *= f;
                }
                if (__any_sync(0xFFFFFFFFu, grow) && kt > w.kt0) {
                    wait_warp(&m->pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1);
                    tc_fence_after();
                    for (int c = 0; c < na * 128; c += 32) {
                        float o[32];
                        tmem_ld32(lanes + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= f;
                        tmem_st32(lanes + c, o);
                    }
                    tmem_wait_st();
                }
                const float ref = mx == -INFINITY ? 0.f : mx;
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float a = exp2f(s[2 * i] - ref), b = exp2f(s[2 * i + 1] - ref);
                    sum += a + b;
                    pk[i] = IT::pack(a, b);
                }
                if (j >= 2) wait_warp(&m->pv_done[j & 1], ((j - 2) >> 1) & 1);
                const uint32_t pb = base + OFF_P + uint32_t(j & 1) * PBUF;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_shared_v4(box_at(pb, r, h * 4 + q), make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]));
                fence_async_proxy();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(&m->p_full[j & 1], 0);
            }
            // Output of the part.
            wait_warp(&m->pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1);
            tc_fence_after();
            m->lred[tid] = sum;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const float l = m->lred[tid & 63] + m->lred[(tid & 63) + 64];
            const bool none = l == 0.f;
            const float inv = w.whole ? (none ? 0.f : 1.f / l) : 1.f;
            uint16_t* out = nullptr;
            float* po = nullptr;
            if (w.whole) {
                out = static_cast<uint16_t*>(p.out) + (w.s.q0 + t) * p.o_ts + int64_t(head) * p.o_hs;
                if (live && h == 0 && p.lse != nullptr)
                    p.lse[(w.s.q0 + t) * p.H + head] = none ? -INFINITY : (mx + log2f(l)) * 0.6931471805599453f;
            } else {
                const Space ws = ws_space(p);
                const int64_t at = (int64_t(pair) * 2 + (part ? 1 : 0)) * ROWS + rank * CROWS + r;
                po = ws.o + at * p.Dv;
                if (live && h == 0) ws.ml[at] = make_float2(mx, l);
            }
            for (int c = 0; c < na * 128; c += 32) {
                float o[32];
                tmem_ld32(lanes + c, o);
                tmem_wait_ld();
                const int ch = (c >> 7) * 256 + h * 128 + (c & 127);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    o[i] = none ? 0.f : o[i] * inv;
                    if (C8) o[i] *= m->inv_v[ch + i];
                }
                if (!live) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (ch + 8 * q >= p.Dv) break;
                    if (w.whole) {
                        *reinterpret_cast<uint4*>(out + ch + 8 * q) =
                            make_uint4(IT::pack(o[8 * q], o[8 * q + 1]), IT::pack(o[8 * q + 2], o[8 * q + 3]),
                                       IT::pack(o[8 * q + 4], o[8 * q + 5]), IT::pack(o[8 * q + 6], o[8 * q + 7]));
                    } else {
                        *reinterpret_cast<float4*>(po + ch + 8 * q) = make_float4(o[8 * q], o[8 * q + 1], o[8 * q + 2], o[8 * q + 3]);
                        *reinterpret_cast<float4*>(po + ch + 8 * q + 4) =
                            make_float4(o[8 * q + 4], o[8 * q + 5], o[8 * q + 6], o[8 * q + 7]);
                    }
                }
            }
            tc_fence_before();
            ++part;
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------------
        // Keys: thread (key tk, quarter c4 of each 64-byte group).
        // ------------------------------------------------------------------
        const int tk = (tid - 128) >> 2, c4 = tid & 3;
        int j = 0, pend = -1;
        const int nc = p.Dv / 8, nr = p.Dk / 8;
        Walk w(p, m->begin, m->end);
        while (w.next()) {
            for (int kt = w.kt0; kt < w.kt1; ++kt, ++j) {
                const int st = j % STAGES;
                const uint32_t stage = base + OFF_K + st * STAGE_BYTES;
                const int64_t slot = key_slot(p, w.n, w.s.K, kt * KEYS + int(rank) * CKEYS + tk);
                const bool have = slot >= 0;
                const int64_t row = have ? slot : 0;
                uint4 x[8], xr = make_uint4(0, 0, 0, 0);
                if constexpr (C8) {
                    const uint8_t* src = static_cast<const uint8_t*>(p.ckv) + row * p.Dv;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int q = c4 + 4 * i;   // 16 codes
                        x[i] = have && q * 2 < nc ? ld_stream_v4(src + q * 16) : make_uint4(0, 0, 0, 0);
                    }
                }
                if (p.k_kind != OUT16 && have && c4 * 2 < nr) xr = ld_stream_v4(static_cast<const uint8_t*>(p.kc) + row * p.Dk + c4 * 16);
                if (j >= STAGES) {
                    const uint32_t ph = ((j / STAGES) & 1) ^ 1;
                    if (pend >= 0 && !__all_sync(0xFFFFFFFFu, mbar_try_wait_cluster(&m->empty[st], ph))) {
                        cp_async_wait<0>();
                        fence_async_proxy();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_at(&m->k_full[pend], 0);
                        pend = -1;
                    }
                    wait(&m->empty[st], ph);
                    __syncwarp();
                }
                if constexpr (C8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int q = 2 * (c4 + 4 * i);
                        if (q >= nb * 8) continue;
                        const uint32_t box = stage + uint32_t(q >> 3) * KBOX;
                        st_shared_v4(box_at(box, tk, q & 7), dec8x8<IT>(p.ckv_kind, x[i].x, x[i].y));
                        st_shared_v4(box_at(box, tk, (q & 7) + 1), dec8x8<IT>(p.ckv_kind, x[i].z, x[i].w));
                    }
                } else {
                    const uint16_t* src = static_cast<const uint16_t*>(p.ckv) + row * p.Dv;
                    for (int q = c4; q < nb * 8; q += 4) {
                        const bool in = have && q < nc;
                        cp_async16(box_at(stage + uint32_t(q >> 3) * KBOX, tk, q & 7), in ? src + q * 8 : src, in);
                    }
                }
                if (p.k_kind != OUT16) {
                    st_shared_v4(box_at(stage + 8 * KBOX, tk, 2 * c4), dec8x8<IT>(p.k_kind, xr.x, xr.y));
                    st_shared_v4(box_at(stage + 8 * KBOX, tk, 2 * c4 + 1), dec8x8<IT>(p.k_kind, xr.z, xr.w));
                } else {
                    const uint16_t* src = static_cast<const uint16_t*>(p.kc) + row * p.Dk;
                    for (int q = c4; q < 8; q += 4) {
                        const bool in = have && q < nr;
                        cp_async16(box_at(stage + 8 * KBOX, tk, q), in ? src + q * 8 : src, in);
                    }
                }
                cp_async_commit();
                if (pend >= 0) {
                    cp_async_wait<1>();
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_at(&m->k_full[pend], 0);
                }
                pend = st;
            }
        }
        cp_async_wait<0>();
        fence_async_proxy();
        __syncwarp();
        if (pend >= 0 && lane == 0) mbar_arrive_at(&m->k_full[pend], 0);
    } else if (warp < 12) {
        // ------------------------------------------------------------------
        // Queries of a part, then for each step the other CTA's keys.
        // ------------------------------------------------------------------
        const int v = tid - 256, tk = v >> 2, c4 = v & 3;
        int j = 0, pend = -1;
        const int nc = p.Dv / 8, nr = p.Dk / 8;
        Walk w(p, m->begin, m->end);
        while (w.next()) {
            // The last product with the old queries is done: the loop below has waited for its S.
            if (pend >= 0) {
                cp_async_wait<0>();
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(&m->v_full[pend], 0);
                pend = -1;
            }
            const int c = v & 7;
#pragma unroll 1
            for (int it = 0; it < 4; ++it) {
                const int r = it * 16 + (v >> 3);
                const unsigned row = unsigned(w.i) * ROWS + rank * CROWS + r;
                const bool live = row < unsigned(w.s.L) * unsigned(p.H);
                const int64_t t = w.s.q0 + row / unsigned(p.H), head = row % unsigned(p.H);
                const uint16_t* qn = static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + head * p.qn_hs;
                const uint16_t* qr = static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + head * p.qr_hs;
                uint4 x[9];
#pragma unroll
                for (int b = 0; b < 9; ++b) {
                    const int q = b < 8 ? b * 8 + c : c;
                    x[b] = live && q < (b < 8 ? nc : nr) ? ld_stream_v4((b < 8 ? qn : qr) + q * 8) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int b = 0; b < 9; ++b) {
                    // A scale per channel goes into the query, rounded once; over the part's largest 1 / scale
                    // (as a power of two, put back into the score), so that float16 neither overflows nor loses bits.
                    if (b < 8 ? C8 && p.ckv_scale_per_ch : p.k_scale_per_ch && p.k_kind != OUT16) {
                        const float* f = b < 8 ? m->inv_v + b * 64 + c * 8 : m->inv_k + c * 8;
                        const float g = 1.f / m->lift[b < 8 ? 0 : 1];
                        uint32_t* u = reinterpret_cast<uint32_t*>(&x[b]);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            u[k] = IT::pack(IT::lo(u[k]) * (f[2 * k] * g), IT::hi(u[k]) * (f[2 * k + 1] * g));
                    }
                    st_shared_v4(box_at(base + OFF_Q + b * QBOX, r, c), x[b]);
                }
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(&m->q_full, 0);
            for (int kt = w.kt0; kt < w.kt1; ++kt, ++j) {
                const int st = j % STAGES;
                const uint32_t stage = base + OFF_K + st * STAGE_BYTES;
                const int64_t slot = key_slot(p, w.n, w.s.K, kt * KEYS + int(rank ^ 1) * CKEYS + tk);
                const bool have = slot >= 0;
                const int64_t row = have ? slot : 0;
                uint4 x[4];
                if constexpr (C8) {
                    const uint8_t* src = static_cast<const uint8_t*>(p.ckv) + row * p.Dv;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int cb = (i >> 1) * 4 + int(rank) * 2 + (i & 1), q = cb * 4 + c4;
                        x[i] = have && q * 2 < nc ? ld_stream_v4(src + q * 16) : make_uint4(0, 0, 0, 0);
                    }
                }
                if (pend >= 0 && !__all_sync(0xFFFFFFFFu, mbar_try_wait_cluster(&m->s_full[j & 1], (j >> 1) & 1))) {
                    cp_async_wait<0>();
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_at(&m->v_full[pend], 0);
                    pend = -1;
                }
                wait(&m->s_full[j & 1], (j >> 1) & 1);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int cb = (i >> 1) * 4 + int(rank) * 2 + (i & 1), db = (i >> 1) * 4 + int(rank ^ 1) * 2 + (i & 1);
                    if (cb * 8 >= nc) continue;
                    const uint32_t box = stage + uint32_t(db) * KBOX;
                    if constexpr (C8) {
                        st_shared_v4(box_at(box, tk, 2 * c4), dec8x8<IT>(p.ckv_kind, x[i].x, x[i].y));
                        st_shared_v4(box_at(box, tk, 2 * c4 + 1), dec8x8<IT>(p.ckv_kind, x[i].z, x[i].w));
                    } else {
                        const uint16_t* src = static_cast<const uint16_t*>(p.ckv) + row * p.Dv;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int q = cb * 8 + c4 + 4 * k;
                            const bool in = have && q < nc;
                            cp_async16(box_at(box, tk, c4 + 4 * k), in ? src + q * 8 : src, in);
                        }
                    }
                }
                cp_async_commit();
                if (pend >= 0) {
                    cp_async_wait<1>();
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_at(&m->v_full[pend], 0);
                }
                pend = st;
            }
        }
        cp_async_wait<0>();
        fence_async_proxy();
        __syncwarp();
        if (pend >= 0 && lane == 0) mbar_arrive_at(&m->v_full[pend], 0);
    } else if (rank == 0 && lane == 0) {
        // ------------------------------------------------------------------
        // MMA: S of a step is issued before O of the one before, which waits for its softmax.
        // ------------------------------------------------------------------
        constexpr uint32_t id_s = tc_idesc(ROWS, KEYS, IT::is_bf16, false), id_o = tc_idesc(ROWS, 256, IT::is_bf16, true);
        const bool split = C8 || p.k_kind != OUT16;
        int j = 0, parts = 0;
        bool prev = false, prev_first = false;
        auto issue_o = [&](int i, bool first) {
            wait(&m->p_full[i & 1], (i >> 1) & 1);
            wait(&m->v_full[i % STAGES], (i / STAGES) & 1);
            tc_fence_after();
            const uint64_t pd = tc_desc(base + OFF_P + uint32_t(i & 1) * PBUF, 16, 1024);
            const uint64_t vd = tc_desc(base + OFF_K + (i % STAGES) * STAGE_BYTES, KBOX, 1024);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                if (a >= na) break;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    tc_mma_pair(tmem + a * 128, pd + s * 2, vd + ((a * 4 + (s >> 1) * 2) * KBOX + (s & 1) * 2048) / 16, id_o,
                                !(first && s == 0));
            }
            tc_commit_pair(&m->pv_done[i & 1]);
            tc_commit_pair(&m->empty[i % STAGES]);
        };
        Walk w(p, m->begin, m->end);
        while (w.next()) {
            if (prev) issue_o(j - 1, prev_first);
            prev = false;
            wait(&m->q_full, parts & 1);
            ++parts;
            for (int kt = w.kt0; kt < w.kt1; ++kt, ++j) {
                const int st = j % STAGES;
                wait(&m->k_full[st], (j / STAGES) & 1);
                tc_fence_after();
                const uint64_t qd = tc_desc(base + OFF_Q, 16, 1024), kd = tc_desc(base + OFF_K + st * STAGE_BYTES, 16, 1024);
                const uint32_t d = tmem + COL_S + uint32_t(j & 1) * 64;
                for (int b = 0; b < nb; ++b)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        tc_mma_pair(d, qd + (b * QBOX) / 16 + s * 2, kd + (b * KBOX) / 16 + s * 2, id_s, b > 0 || s > 0);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    tc_mma_pair(d + (split ? 32 : 0), qd + (8 * QBOX) / 16 + s * 2, kd + (8 * KBOX) / 16 + s * 2, id_s, !split || s > 0);
                tc_commit_pair(&m->s_full[j & 1]);
                if (prev) issue_o(j - 1, prev_first);
                prev = true;
                prev_first = kt == w.kt0;
            }
        }
        if (prev) issue_o(j - 1, prev_first);
        if (!ok) {   // let what was issued finish before TMEM goes
            tc_commit_pair(&m->drain);
            mbar_wait(&m->drain, 0, nullptr);
        }
    }
    if (!ok && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 12) tmem_free_pair(tmem, TMEM_COLS);
}

// Joins the parts of the items that were cut: block x takes the item at the
// first bound inside it, if bound x + 1 is that one; 16 rows a block, 4 a warp.
template <class IT>
__global__ void __launch_bounds__(128) mla_join_kernel(const __grid_constant__ MlaParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const Space ws = ws_space(p);
    const int active = *ws.active, b = blockIdx.x + 1;
    if (b >= active) return;
    const Bound at = ws.bounds[b], before = ws.bounds[b - 1];
    const bool same = before.n == at.n && before.i == at.i;
    if (at.n >= p.N || at.kt == 0 || (same && before.kt > 0)) return;
    const Seq s = load_seq(p, at.n);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Parts: the last of pair b - 1, then the first of each pair whose bound is inside the item.
    int last = b;
    while (last + 1 < active && ws.bounds[last + 1].n == at.n && ws.bounds[last + 1].i == at.i && ws.bounds[last + 1].kt > 0) ++last;
    for (int k = 0; k < 4; ++k) {
        const int r = blockIdx.y * 16 + warp * 4 + k;
        const unsigned row = unsigned(at.i) * ROWS + r;
        if (row >= unsigned(s.L) * unsigned(p.H)) break;
        float mx = -INFINITY;
        for (int q = b - 1; q <= last; ++q) {
            if (q < last && ws.bounds[q].n == ws.bounds[q + 1].n && ws.bounds[q].i == ws.bounds[q + 1].i && ws.bounds[q].kt == ws.bounds[q + 1].kt) continue;
            mx = fmaxf(mx, ws.ml[(int64_t(q) * 2 + (q == b - 1 && !same ? 1 : 0)) * ROWS + r].x);
        }
        float l = 0.f;
        float4 o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = b - 1; q <= last; ++q) {
            if (q < last && ws.bounds[q].n == ws.bounds[q + 1].n && ws.bounds[q].i == ws.bounds[q + 1].i && ws.bounds[q].kt == ws.bounds[q + 1].kt) continue;
            const int64_t slot = (int64_t(q) * 2 + (q == b - 1 && !same ? 1 : 0)) * ROWS + r;
            const float2 ml = ws.ml[slot];
            if (ml.y == 0.f) continue;
            const float f = exp2f(ml.x - mx);
            l += ml.y * f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int ch = (c * 32 + lane) * 4;
                if (ch >= p.Dv) break;
                const float4 x = *reinterpret_cast<const float4*>(ws.o + slot * p.Dv + ch);
                o[c].x += x.x * f, o[c].y += x.y * f, o[c].z += x.z * f, o[c].w += x.w * f;
            }
        }
        const int64_t t = s.q0 + row / unsigned(p.H), head = row % unsigned(p.H);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* out = static_cast<uint16_t*>(p.out) + t * p.o_ts + head * p.o_hs;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int ch = (c * 32 + lane) * 4;
            if (ch >= p.Dv) break;
            *reinterpret_cast<uint2*>(out + ch) = make_uint2(IT::pack(o[c].x * inv, o[c].y * inv), IT::pack(o[c].z * inv, o[c].w * inv));
        }
        if (lane == 0 && p.lse != nullptr) p.lse[t * p.H + head] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.6931471805599453f;
    }
}

}  // namespace

int mla_tc_pairs() {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return 1;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == 0) {
        // Pairs that fit on the GPU at once (a GPC with an odd number of SMs leaves one over).
        int n = 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(sm_count_current_device()));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = SMEM_BYTES;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        bool good = true;
        for (auto f : {mla_tc_kernel<BF16, false>, mla_tc_kernel<BF16, true>, mla_tc_kernel<F16, false>, mla_tc_kernel<F16, true>})
            good = good && cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) == cudaSuccess;
        good = good && cudaOccupancyMaxActiveClusters(&n, mla_tc_kernel<BF16, false>, &cfg) == cudaSuccess && n > 0;
        if (!good) {
            (void)cudaGetLastError();
            return 1;
        }
        cache[dev] = n;
    }
    return cache[dev];
}

int64_t mla_tc_workspace(int Dv) { return ws_bytes(mla_tc_pairs(), Dv); }

template <class IT>
static cudaError_t launch_mla_tc_t(const MlaParams& p, cudaStream_t s) {
    const dim3 g(unsigned(p.pairs * 2)), b(THREADS);
    cudaError_t e = p.ckv_kind == OUT16 ? launch_pdl(mla_tc_kernel<IT, false>, g, b, SMEM_BYTES, s, p)
                                        : launch_pdl(mla_tc_kernel<IT, true>, g, b, SMEM_BYTES, s, p);
    if (e != cudaSuccess || p.pairs == 1) return e;
    return launch_pdl(mla_join_kernel<IT>, dim3(unsigned(p.pairs - 1), ROWS / 16), dim3(128), 0, s, p);
}

cudaError_t launch_mla_tc(MlaParams p, int dtype, cudaStream_t s) {
    p.pairs = mla_tc_pairs();
    return dtype == KVR_BF16 ? launch_mla_tc_t<BF16>(p, s) : launch_mla_tc_t<F16>(p, s);
}

}  // namespace kvr
