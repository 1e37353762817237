// Ancestors and positions of drafted tokens.
//
// anc(j) = {j} + anc(parent(j)), anc(-1) = {}; position = start + |anc(j)| - 1.
// One CTA a sequence, its parents in shared memory, one thread a token: it walks up to the context and
// sets a bit a step. A parent comes before its token, so that the walk goes down through the words: a word is written once,
// from a register. What it costs is a launch and two dependent loads; a step of the walk is one
// load from shared memory. Measured: one sequence of 26 tokens 2.8 us, 256 of 9-127 tokens 2.9 to 3.3. What a token
// costs is its depth, so that chains, which drafts do not have at such lengths, are quadratic: 64 tokens 5.9 us, 512 129, 4096 7100.
#include "cache_ops.cuh"

namespace kvr {

constexpr int TREE_THREADS = 128;

__global__ void __launch_bounds__(TREE_THREADS) draft_tree_kernel(const __grid_constant__ TreeParams p) {
    extern __shared__ int up[];   // parents of the sequence's tokens
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
        const int64_t a = p.query_start[n], b = p.query_start[n + 1];
        if (a < 0 || b < a || b > p.T || b - a > int64_t(p.words) * 64) {
            if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_QUERY);
            continue;   // (the same for all threads)
        }
        const int L = int(b - a);
        for (int j = threadIdx.x; j < L; j += TREE_THREADS) {
            const int64_t x = p.parent[a + j];
            const bool good = x >= -1 && x < j;
            if (!good && p.status != nullptr) atomicOr(p.status, KVR_DEVERR_INDEX);
            up[j] = good ? int(x) : -1;
        }
        __syncthreads();
        const int64_t first = p.positions != nullptr ? p.position_start[n] : 0;
        for (int j = threadIdx.x; j < L; j += TREE_THREADS) {
            int64_t* mask = p.mask + (a + j) * p.words;
            int word = p.words - 1, at = j, depth = -1;
            uint64_t bits = 0;
            while (at >= 0) {
                for (; word > at >> 6; --word) {
                    mask[word] = int64_t(bits);
                    bits = 0;
                }
                bits |= uint64_t(1) << (at & 63);
                ++depth;
                at = up[at];
            }
            for (; word >= 0; --word) {
                mask[word] = int64_t(bits);
                bits = 0;
            }
            if (p.positions != nullptr) p.positions[a + j] = first + depth;
        }
        __syncthreads();
    }
}

cudaError_t launch_tree(const TreeParams& p, cudaStream_t s) {
    const int64_t cap = int64_t(sm_count_current_device()) * 16;
    const int64_t longest = p.T < int64_t(p.words) * 64 ? p.T : int64_t(p.words) * 64;
    return launch_pdl(draft_tree_kernel, dim3(unsigned(p.N < cap ? p.N : cap)), dim3(TREE_THREADS), size_t(longest) * sizeof(int), s, p);
}

}  // namespace kvr
