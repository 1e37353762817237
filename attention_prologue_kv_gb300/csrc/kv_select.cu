// Which keys of a sequence to keep: the `keep` of largest rank, in order of their positions.
//
// A weight's rank is its bits, made to order as unsigned numbers (NaN above every number, protected keys above all). The
// keep-th largest rank t is found digit by digit from the top (11, 11 and 10 bits): count the ranks of each digit among
// those that agree so far, walk down to the digit that holds the wanted one. Of the keys equal to t the earliest fill up:
// with G(i), E(i) the keys before i of rank above t and equal to t, key i is kept if it is above t, or equal and E(i) is
// below what is missing, and its place is G(i) + min(E(i), missing). Counts are whole numbers: the order in which they are
// added changes nothing.
//
// A cluster of CTAs has one sequence, a run of its keys in each CTA's shared memory, so that weights are read once (a
// share beyond that is read again, from L2). The CTAs read one another's counts: a barrier of the cluster a digit, and one
// for the keys before a CTA's own.
#include "cache_ops.cuh"
#include "tcgen05.cuh"

namespace kvr {

namespace {

constexpr int NT = 512, WARPS = NT / 32, BINS = 2048;
constexpr int MAX_CTAS = 8;
constexpr int ROOM = 49152;   // weights a CTA's shared memory takes at most

__device__ __forceinline__ uint32_t rank_of(float w) {
    if (w != w) return 0xFFFFFFFEu;
    const uint32_t b = __float_as_uint(w + 0.f);   // -0 becomes 0
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
// A word at this place in CTA `rank` of the cluster.
__device__ __forceinline__ int peer_load(const int* at, uint32_t rank) {
    int v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.b32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(smem_u32(at)), "r"(rank)
                 : "memory");
    return v;
}

struct Shared {
    int hist[2][BINS];    // of a digit; the next one's meanwhile
    int warp_sum[WARPS];
    int found[2];         // the digit, and what is wanted of it
    int above[WARPS], equal[WARPS];
    int total[2];         // this CTA's keys above and equal
};

__global__ void __launch_bounds__(NT) kv_select_kernel(const __grid_constant__ SelectParams p) {
    extern __shared__ float held[];
    __shared__ Shared m;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const int n = int(blockIdx.x / size);
    for (int i = tid; i < BINS; i += NT) m.hist[0][i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t length = p.key_length[n];
    const bool good = length >= 0 && length <= p.weight_len;
    if (!good && rank == 0 && tid == 0 && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_KEY_LENGTH);
    const int K = good ? int(length) : 0;
    const float* weight = p.weight + n * p.weight_stride;
    // This CTA's keys: [first, first + mine).
    const int share = (K + int(size) - 1) / int(size), first = min(K, int(rank) * share), mine = min(share, K - first);
    const int cached = min(mine, p.share);
    const bool all = K <= p.keep;
    for (int i = tid; i < cached; i += NT) held[i] = weight[first + i];
    auto value = [&](int i) { return i < cached ? held[i] : weight[first + i]; };
    const int last = K - p.recent;   // (only where K > keep >= recent)
    auto rank_at = [&](int i) {
        const int at = first + i;
        return at < p.sink || at >= last ? 0xFFFFFFFFu : rank_of(value(i));
    };
    __syncthreads();
    uint32_t t = 0;
    int missing = 0;
    if (!all) {   // (the same in all CTAs of the cluster)
        int want = p.keep;
        uint32_t prefix = 0;
#pragma unroll 1
        for (int digit = 0; digit < 3; ++digit) {
            const int shift = digit == 0 ? 21 : (digit == 1 ? 10 : 0), bits = digit == 2 ? 10 : 11, bins = 1 << bits;
            int* hist = m.hist[digit & 1];
#pragma unroll 4
            for (int i = tid; i < mine; i += NT) {
                const uint32_t r = rank_at(i);
                if (digit == 0 || r >> (shift + bits) == prefix) atomicAdd(&hist[r >> shift & (bins - 1)], 1);
            }
            for (int i = tid; i < BINS; i += NT) m.hist[(digit & 1) ^ 1][i] = 0;
            cluster_sync_all();
            // Thread i has the bins 4 i .. 4 i + 3 counted from the top.
            int c[4], sum = 0;
            const int top = bins - 1 - 4 * tid;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                c[k] = 0;
                if (top - k >= 0)
                    for (uint32_t q = 0; q < size; ++q) c[k] += peer_load(&hist[top - k], q);
                sum += c[k];
            }
            int scan = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
                if (lane >= o) scan += v;
            }
            if (lane == 31) m.warp_sum[warp] = scan;
            __syncthreads();
            int before = scan - sum;
            for (int q = 0; q < warp; ++q) before += m.warp_sum[q];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (before < want && want <= before + c[k]) {
                    m.found[0] = top - k;
                    m.found[1] = want - before;
                }
                before += c[k];
            }
            __syncthreads();
            prefix = prefix << bits | uint32_t(m.found[0]);
            want = m.found[1];
            // (the next digit's counts go to the other array, which the CTAs have cleared behind the barrier above)
            cluster_sync_all();
        }
        t = prefix;
        missing = want;
    }
    // Keys above and equal in each warp's run.
    const int run = ((mine + WARPS - 1) / WARPS + 31) / 32 * 32, r0 = min(mine, warp * run), r1 = min(mine, r0 + run);
    int above = 0, equal = 0;
    for (int i = r0; i < r1; i += 32) {
        const uint32_t r = i + lane < r1 ? (all ? 1u : rank_at(i + lane)) : 0u;
        above += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < r1 && r > t));
        equal += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < r1 && r == t));
    }
    if (lane == 0) {
        m.above[warp] = above;
        m.equal[warp] = equal;
    }
    __syncthreads();
    if (tid == 0) {
        int a = 0, e = 0;
        for (int q = 0; q < WARPS; ++q) {
            a += m.above[q];
            e += m.equal[q];
        }
        m.total[0] = a;
        m.total[1] = e;
    }
    cluster_sync_all();
    int G = 0, E = 0;
    for (uint32_t q = 0; q < rank; ++q) {
        G += peer_load(&m.total[0], q);
        E += peer_load(&m.total[1], q);
    }
    for (int q = 0; q < warp; ++q) {
        G += m.above[q];
        E += m.equal[q];
    }
    cluster_arrive();   // a CTA stays until the others have its counts
    int64_t* kept = p.kept + int64_t(n) * p.keep;
    float* carried = p.kept_weight == nullptr ? nullptr : p.kept_weight + n * p.kept_weight_stride;
    const uint32_t below = (1u << lane) - 1;
    for (int i = r0; i < r1; i += 32) {
        const bool in = i + lane < r1;
        const uint32_t r = in ? (all ? 1u : rank_at(i + lane)) : 0u;
        const uint32_t up = __ballot_sync(0xFFFFFFFFu, in && r > t), same = __ballot_sync(0xFFFFFFFFu, in && r == t);
        const int e = E + __popc(same & below);
        if (in && (r > t || (r == t && e < missing))) {
            const int at = G + __popc(up & below) + min(e, missing);
            kept[at] = first + i + lane;
            if (carried != nullptr) carried[at] = value(i + lane);
        }
        G += __popc(up);
        E += __popc(same);
    }
    const int count = all ? K : p.keep;
    const int64_t step = int64_t(size) * NT, begin = count + int64_t(rank) * NT + tid;
    for (int64_t i = begin; i < p.keep; i += step) kept[i] = -1;
    if (carried != nullptr)
        for (int64_t i = begin; i < p.kept_weight_len; i += step) carried[i] = 0.f;
    if (rank == 0 && tid == 0) p.kept_length[n] = count;
    cluster_wait();
}

}  // namespace

cudaError_t launch_select(SelectParams p, cudaStream_t s) {
    int ctas = 1;
    while (ctas < MAX_CTAS && p.weight_len > int64_t(ctas) * 2048 && int64_t(p.N) * ctas * 2 <= 2 * sm_count_current_device()) ctas *= 2;
    while (ctas < MAX_CTAS && p.weight_len > int64_t(ctas) * ROOM) ctas *= 2;
    const int64_t share = (p.weight_len + ctas - 1) / ctas;
    p.share = int(share < ROOM ? share : ROOM);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.N) * unsigned(ctas));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = size_t(p.share) * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cfg.dynamicSmemBytes + sizeof(Shared) > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kv_select_kernel),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, ROOM * int(sizeof(float)));
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kv_select_kernel, p);
}

}  // namespace kvr
