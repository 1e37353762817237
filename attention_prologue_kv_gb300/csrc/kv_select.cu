// Which keys of a sequence to keep: the `keep` of largest rank, in order of their positions.
//
// A weight's rank is its bits, made to order as unsigned numbers (NaN above every number). Keys that stay anyway, the first
// `sink` and the last `recent`, stand above all and are left out of the search. The rank t that divides the others is found
// between the least and the greatest one by counting: their range is cut into at most 1024 bins, the ranks of each counted,
// the bin walked down to that holds the wanted one, and so on inside it, until all of a bin is wanted or a bin is one rank.
// Of the keys equal to t the earliest fill up: with G(i), E(i) the keys before i of rank above t and equal to t, key i stays
// if it is above t, or equal and E(i) is below what is missing, and its place is G(i) + min(E(i), missing). Counts are whole
// numbers: the order in which they are added changes nothing.
//
// A cluster of CTAs has one sequence, each a run of its keys in registers, so that weights are read once (beyond 16384 keys a
// CTA their ranks are in shared memory, beyond 49152 they are read anew, from L2). The CTAs read one another's counts: a barrier
// of the cluster for the range, one a round of counting (two or three: bits of floats spread weights by their logarithm) and one
// for the keys before a CTA's own.
//
// Latency is what it costs. Measured, with the same weights in each call and with others from DRAM: 32768 of one sequence's 131000
// keys 16.8 us and 17.2 to 19.6 (3.6 to load and rank, 3 for the range, 3 a round, 3.5 to write), 2048 of 4095 keys of 64 sequences
// 5.9 and 7.1 to 8.2, 500 of 1000 keys of 256 sequences 7.3 and 8.1.
#include <mutex>

#include "cache_ops.cuh"
#include "select_plan.cuh"
#include "tcgen05.cuh"

namespace kvr {

namespace {

// Bins: one a thread. With 2048, which all CTAs read of one another too, 131000 keys took 19.8 us instead of 15.9.
constexpr int NT = SEL_THREADS, WARPS = NT / 32, BINS = NT;
constexpr int MAX_CTAS = 16;   // beyond 8, where the device is asked, for what 8 have no registers for

__device__ __forceinline__ uint32_t rank_of(float w) {
    if (w != w) return 0xFFFFFFFEu;
    const uint32_t b = __float_as_uint(w + 0.f);   // -0 becomes 0
    return b >> 31 ? ~b : b | 0x80000000u;
}
constexpr uint32_t STAYS = 0xFFFFFFFFu, NONE = 0u;   // (no number's rank)

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
// What is at this place in CTA `rank` of the cluster.
__device__ __forceinline__ int peer_load(const int* at, uint32_t rank) {
    int v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.b32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(smem_u32(at)), "r"(rank)
                 : "memory");
    return v;
}
__device__ __forceinline__ int2 peer_load(const int2* at, uint32_t rank) {
    int2 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\tld.shared::cluster.v2.b32 {%0, %1}, [a];\n\t}"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(smem_u32(at)), "r"(rank)
                 : "memory");
    return v;
}

struct Shared {
    int hist[2][BINS];   // of a round; the next one's meanwhile
    int2 range, total;        // this CTA's least and greatest rank; its keys above and equal
    int2 part[WARPS];
    int sums[WARPS];
    int found[3];             // the bin, what is wanted of it, what it has
};

// VPT: keys of a thread in registers; SHARED: as many as there are, their ranks in shared memory; AGAIN: read whenever they are
// looked at. Key j of a lane is the warp's first + 32 j + lane.
constexpr int SHARED = SEL_SHARED, AGAIN = SEL_AGAIN;
template <int VPT>
__global__ void __launch_bounds__(NT) kv_select_kernel(const __grid_constant__ SelectParams p) {
    __shared__ Shared m;
    extern __shared__ uint32_t held[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const int n = int(blockIdx.x / size);
    auto sync = [&]() {
        if (size > 1) cluster_sync_all();
        else __syncthreads();
    };
    m.hist[0][tid] = 0;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t length = p.key_length[n];
    const bool good = length >= 0 && length <= p.weight_len;
    if (!good && rank == 0 && tid == 0 && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_KEY_LENGTH);
    const int K = good ? int(length) : 0;
    const bool all = K <= p.keep;
    // This CTA's keys are [first, first + mine), this warp's [at, end).
    const int share = (K + int(size) - 1) / int(size), first = min(K, int(rank) * share), mine = min(share, K - first);
    const int run = VPT > 0 ? 32 * VPT : ((mine + WARPS - 1) / WARPS + 31) / 32 * 32;
    const int at = first + min(mine, warp * run), end = min(first + mine, at + run);
    const float* weight = p.weight + n * p.weight_stride;
    const int last = K - p.recent;
    auto rank_at = [&](int i, float w) { return i >= end ? NONE : (all || i < p.sink || i >= last ? STAYS : rank_of(w)); };
    float value[VPT > 0 ? VPT : 1];
    uint32_t ranks[VPT > 0 ? VPT : 1];
    if (VPT > 0) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = at + 32 * j + lane;
            value[j] = i < end ? weight[i] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) ranks[j] = rank_at(at + 32 * j + lane, value[j]);
    } else if (VPT == SHARED) {
#pragma unroll 8
        for (int i = at + lane; i < end; i += 32) held[i - first] = rank_at(i, weight[i]);
    }
    // For each of this lane's keys, warp after warp the same number of times.
    auto each = [&](auto&& f) {
        if constexpr (VPT > 0) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) f(at + 32 * j + lane, ranks[j], value[j]);
        } else if constexpr (VPT == SHARED) {
#pragma unroll 4
            for (int i = at + lane; i < at + run; i += 32) f(i, i < end ? held[i - first] : NONE, 0.f);
        } else {
#pragma unroll 4
            for (int i = at + lane; i < at + run; i += 32) {
                const float w = i < end ? weight[i] : 0.f;
                f(i, rank_at(i, w), w);
            }
        }
    };
    uint32_t t = NONE;
    int missing = 0;
    if (!all) {   // (the same in all CTAs of the cluster)
        uint32_t lo = STAYS, hi = NONE;
        each([&](int, uint32_t r, float) {
            if (r != NONE && r != STAYS) {
                lo = min(lo, r);
                hi = max(hi, r);
            }
        });
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        if (lane == 0) m.part[warp] = make_int2(int(lo), int(hi));
        __syncthreads();
        if (warp == 0) {
            const int2 v = m.part[lane];
            lo = __reduce_min_sync(0xFFFFFFFFu, uint32_t(v.x));
            hi = __reduce_max_sync(0xFFFFFFFFu, uint32_t(v.y));
            if (lane == 0) m.range = make_int2(int(lo), int(hi));
        }
        sync();
        lo = STAYS;
        hi = NONE;
        for (uint32_t q = 0; q < size; ++q) {
            const int2 v = peer_load(&m.range, q);
            lo = min(lo, uint32_t(v.x));
            hi = max(hi, uint32_t(v.y));
        }
        int want = p.keep - p.sink - p.recent;   // of the others: less than there are
        t = STAYS - 1;                           // where none is wanted
#pragma unroll 1
        for (int round = 0; want > 0 && round < 4; ++round) {   // (32 bits, 10 a round)
            const uint32_t range = hi - lo;
            const int bits = 32 - __clz(range), shift = bits > 10 ? bits - 10 : 0;
            int* hist = m.hist[round & 1];
            each([&](int, uint32_t r, float) {
                if (r >= lo && r <= hi) atomicAdd(&hist[(r - lo) >> shift], 1);
            });
            sync();
            // (everyone has read the round before's counts)
            m.hist[(round & 1) ^ 1][tid] = 0;
            if (VPT == AGAIN && tid == 0) {   // what stands if no bin is found, in all CTAs alike: weights may change between two readings
                m.found[0] = 0;
                m.found[1] = m.found[2] = want;
            }
            // Thread i has the i-th bin from the top.
            int sum = 0;
#pragma unroll
            for (uint32_t q = 0; q < MAX_CTAS; ++q)
                if (q < size) sum += peer_load(&m.hist[round & 1][BINS - 1 - tid], q);
            int scan = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
                if (lane >= o) scan += v;
            }
            if (lane == 31) m.sums[warp] = scan;
            __syncthreads();
            int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? m.sums[lane] : 0) + scan - sum;
            if (before < want && want <= before + sum) {
                m.found[0] = BINS - 1 - tid;
                m.found[1] = want - before;
                m.found[2] = sum;
            }
            __syncthreads();
            lo += uint32_t(m.found[0]) << shift;
            hi = lo + min(hi - lo, (1u << shift) - 1);   // (lo + 2^shift may not fit)
            want = m.found[1];
            if (want == m.found[2]) {   // all of it
                t = lo - 1;
                break;
            }
            if (shift == 0) {
                t = lo;
                missing = want;
                break;
            }
        }
    }
    // Keys above and equal in each warp's run.
    int above = 0, equal = 0;
    each([&](int, uint32_t r, float) {
        above += r > t;
        equal += r == t && r != NONE;
    });
    above = __reduce_add_sync(0xFFFFFFFFu, above);
    equal = __reduce_add_sync(0xFFFFFFFFu, equal);
    if (lane == 0) m.part[warp] = make_int2(above, equal);
    __syncthreads();
    const int2 of = m.part[lane];
    int G = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? of.x : 0), E = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? of.y : 0);
    if (warp == WARPS - 1 && lane == 0) m.total = make_int2(G + above, E + equal);
    if (size > 1) {
        cluster_sync_all();
        for (uint32_t q = 0; q < rank; ++q) {
            const int2 v = peer_load(&m.total, q);
            G += v.x;
            E += v.y;
        }
        cluster_arrive();   // a CTA stays until the others have its counts
    }
    int64_t* kept = p.kept + int64_t(n) * p.keep;
    float* carried = p.kept_weight == nullptr ? nullptr : p.kept_weight + n * p.kept_weight_stride;
    const uint32_t below = (1u << lane) - 1;
    each([&](int i, uint32_t r, float w) {
        const uint32_t up = __ballot_sync(0xFFFFFFFFu, r > t), same = __ballot_sync(0xFFFFFFFFu, r == t && r != NONE);
        const int e = E + __popc(same & below);
        const int to = G + __popc(up & below) + min(e, missing);
        if ((r > t || (same >> lane & 1 && e < missing)) && (VPT != AGAIN || to < p.keep)) {
            kept[to] = i;
            if (carried != nullptr) carried[to] = VPT == SHARED ? weight[i] : w;
        }
        G += __popc(up);
        E += __popc(same);
    });
    const int count = all ? K : p.keep;
    const int64_t step = int64_t(size) * NT, begin = count + int64_t(rank) * NT + tid;
    for (int64_t i = begin; i < p.keep; i += step) kept[i] = -1;
    if (carried != nullptr)
        for (int64_t i = begin; i < p.kept_weight_len; i += step) carried[i] = 0.f;
    if (rank == 0 && tid == 0) p.kept_length[n] = count;
    if (size > 1) cluster_wait();
}

using Kernel = void (*)(SelectParams);
Kernel kernel_of(int form) {
    switch (form) {
        case 1: return kv_select_kernel<1>;
        case 2: return kv_select_kernel<2>;
        case 4: return kv_select_kernel<4>;
        case 8: return kv_select_kernel<8>;
        case 16: return kv_select_kernel<16>;
        case SHARED: return kv_select_kernel<SHARED>;
        default: return kv_select_kernel<AGAIN>;
    }
}

// Whether a cluster of 16 CTAs, each with all that one can have of an SM, fits anywhere on the current device; asked once per
// device.
bool wide_clusters() {
    static std::mutex mu;
    static int known[64] = {0};   // 1: they do, 2: they do not
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return false;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
        const void* kernel = reinterpret_cast<const void*>(kernel_of(SHARED));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(MAX_CTAS);
        cfg.blockDim = dim3(NT);
        cfg.dynamicSmemBytes = SEL_ROOM * sizeof(uint32_t);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = MAX_CTAS;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(cfg.dynamicSmemBytes)) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            return false;
        }
        known[dev] = n > 0 ? 1 : 2;
    }
    return known[dev] == 1;
}

}  // namespace

cudaError_t launch_select(SelectParams p, cudaStream_t s) {
    const bool wide = p.weight_len > int64_t(8) * NT * 16 && wide_clusters();
    const SelectForm f = select_form(p.weight_len, p.N, sm_count_current_device(), wide ? MAX_CTAS : 8);
    const int ctas = f.ctas;
    Kernel kernel = kernel_of(f.form);
    const size_t smem = f.form == SHARED ? size_t(f.each) * sizeof(uint32_t) : 0;
    if (smem + sizeof(Shared) > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, int(SEL_ROOM * sizeof(uint32_t)));
        if (e != cudaSuccess) return e;
    }
    if (ctas > 8) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.N) * unsigned(ctas));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace kvr
