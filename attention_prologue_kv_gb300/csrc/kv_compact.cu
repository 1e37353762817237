// Kept rows of a sequence moved together, in place, in both caches.
//
// Row i goes from place kept[i] to place start + i, kept ascending and kept[i] >= start + i. In place, a row that is
// written may still be wanted: place start + i is read by some i' <= i. So a chunk of consecutive rows is read by all
// before any of it is written; later chunks read only places behind those that earlier ones write (kept[i] > start + i' for
// i' < i), so that the next chunk's reads may run ahead.
//
// Columns do not depend on one another: a row of both caches is cut into slices of 128 bytes, and each slice of each sequence is a
// CTA's (or, where these are few, a cluster's, which reads a chunk and waits for one another). Few rows go whole to one
// CTA. A row's two addresses are worked out by one thread and shared.
// Measured: 64 sequences of about 4050 keys to 2024 rows of 1152 bytes 49.5 us (6.05 TB/s read and written, 89% of the copy rate);
// 256 accepted branches of 1-7 rows 4.2 us, a launch and the chain place, block table, row.
#include "cache_ops.cuh"
#include "tcgen05.cuh"

namespace kvr {

namespace {

constexpr int NT = 256, UN = 8;   // threads of a CTA, units of a thread a chunk
constexpr int MAX_CTAS = 8;

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}

template <class U>
__device__ __forceinline__ U load_unit(const uint8_t* at) {
    return __ldcg(reinterpret_cast<const U*>(at));
}
// Have the loaded values here before what follows: a barrier alone does not say that a load is done with its address.
__device__ __forceinline__ uint32_t fold(uint4 v) { return v.x ^ v.y ^ v.z ^ v.w; }
__device__ __forceinline__ uint32_t fold(uint8_t v) { return v; }

struct Move {
    int64_t of, to;   // cache rows; to = -1: the row stays
};

// Rows of a CTA a chunk, `su` units of each: at most one a thread.
__host__ __device__ inline int chunk_rows(int su) { return NT * UN / su < NT ? NT * UN / su : NT; }

// SU: units of a slice, 0: p.su.
template <class U, int SU>
__global__ void __launch_bounds__(NT) kv_compact_kernel(const __grid_constant__ CompactParams p) {
    __shared__ Move moves[3][NT];
    const int tid = threadIdx.x;
    const int size = int(cluster_size()), rank = int(cluster_rank());
    const int su = SU > 0 ? SU : p.su, slice = int(blockIdx.x) / size, col0 = slice * su, cols = min(su, p.cu + p.ku - col0);
    const int rows = chunk_rows(su);
    const unsigned d1 = unsigned(p.d1 < 0x7FFFFFFF ? p.d1 : 0x7FFFFFFF);   // keys are below that
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int64_t count = p.kept_length[n], start = p.start == nullptr ? 0 : p.start[n];
        if (count < 0 || count > p.M || start < 0 || start > p.max_keys - count) {   // (the same in all threads)
            if (tid == 0 && slice == 0 && rank == 0 && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_KEY_LENGTH);
            continue;
        }
        const int64_t* kept = p.kept + n * p.M;
        const int64_t* table = p.table == nullptr ? nullptr : p.table + n * p.max_blocks;
        auto row_of = [&](int64_t key) -> int64_t {
            if (table == nullptr) return n * p.d1 + key;
            const unsigned b = unsigned(key) / d1;
            const int64_t e = table[b];
            return e < 0 || e >= p.d0 ? -1 : e * p.d1 + (unsigned(key) - b * d1);
        };
        // This CTA's rows of a chunk, from row `at` on.
        auto look = [&](int64_t at, Move* m) {
            Move v = {-1, -1};
            const int64_t i = at + tid;
            if (tid < rows && i < count) {
                const int64_t key = kept[i], before = i > 0 ? kept[i - 1] : -1, place = start + i;
                bool good = key > before && key >= place && key < p.max_keys;
                if (good && key != place) {
                    v = {row_of(key), row_of(place)};
                    good = v.of >= 0 && v.to >= 0;
                }
                if (!good) {
                    v.to = -1;
                    if (p.status != nullptr) atomicOr(p.status, KVR_DEVERR_INDEX);
                }
            }
            m[tid] = v;
        };
        auto address = [&](int64_t row, int col) {
            return col < p.cu ? p.ckv + (row * p.cu + col) * int64_t(sizeof(U)) : p.kc + (row * p.ku + (col - p.cu)) * int64_t(sizeof(U));
        };
        auto load = [&](const Move* m, U (&v)[UN]) {
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                const int u = tid + k * NT, r = u / su, c = u - r * su;
                v[k] = U{};
                if (r < rows && c < cols && m[r].to >= 0) v[k] = load_unit<U>(address(m[r].of, col0 + c));
            }
        };
        auto store = [&](const Move* m, const U (&v)[UN]) {
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                const int u = tid + k * NT, r = u / su, c = u - r * su;
                if (r < rows && c < cols && m[r].to >= 0) *reinterpret_cast<U*>(address(m[r].to, col0 + c)) = v[k];
            }
        };
        const int64_t step = int64_t(rows) * size, mine = int64_t(rank) * rows;
        U now[UN], next[UN];
        look(mine, moves[0]);
        __syncthreads();
        load(moves[0], now);
        int at = 0;
        for (int64_t c = 0; c < count; c += step) {
            const int then = at == 2 ? 0 : at + 1;
            const bool more = c + step < count;
            if (more) look(c + step + mine, moves[then]);
            uint32_t x = 0;
#pragma unroll
            for (int k = 0; k < UN; ++k) x ^= fold(now[k]);
            asm volatile("{\n\t.reg .pred q;\n\tsetp.eq.u32 q, %0, 0x9E3779B9;\n\t@q nanosleep.u32 0;\n\t}" ::"r"(x) : "memory");
            if (size > 1) cluster_sync_all();
            else __syncthreads();
            if (more) load(moves[then], next);
            store(moves[at], now);
#pragma unroll
            for (int k = 0; k < UN; ++k) now[k] = next[k];
            at = then;
        }
        __syncthreads();   // `moves` is written anew for the next sequence
    }
}

}  // namespace

cudaError_t launch_compact(CompactParams p, bool vec, cudaStream_t s) {
    const int units = p.cu + p.ku, sms = sm_count_current_device();
    const bool whole = p.M <= NT && p.M * units <= NT * UN;   // few rows: one chunk
    p.su = whole ? units : (units < 8 ? units : 8);
    p.slices = (units + p.su - 1) / p.su;
    const int64_t seqs = p.N < 65535 ? p.N : 65535, rows = chunk_rows(p.su);
    int ctas = 1;
    while (ctas < MAX_CTAS && p.M > rows * ctas && seqs * p.slices * ctas * 2 <= 2 * sms) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.slices) * unsigned(ctas), unsigned(seqs));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (p.su == 8) return vec ? cudaLaunchKernelEx(&cfg, kv_compact_kernel<uint4, 8>, p) : cudaLaunchKernelEx(&cfg, kv_compact_kernel<uint8_t, 8>, p);
    return vec ? cudaLaunchKernelEx(&cfg, kv_compact_kernel<uint4, 0>, p) : cudaLaunchKernelEx(&cfg, kv_compact_kernel<uint8_t, 0>, p);
}

}  // namespace kvr
