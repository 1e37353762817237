// What the operators of an attention step share: their arguments as the kernels take them, launches, small device helpers.
#pragma once

#include <cuda_fp8.h>

#include "kvr_internal.cuh"

namespace kvr {

template <class IT>
constexpr bool is_bf16 = false;
template <>
inline constexpr bool is_bf16<BF16> = true;

// One 8-bit code of a runtime kind to float (exact).
__device__ __forceinline__ float dec8(int kind, uint8_t c) {
    if (kind == OUT_I8) return float(int8_t(c));
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, kind == OUT_E4M3 ? __NV_E4M3 : __NV_E5M2);
    return __half2float(__half(h));
}

// 32 bytes to global memory, 32-byte aligned: a whole sector from one thread.
__device__ __forceinline__ void st_global_v8(void* dst, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The same back.
__device__ __forceinline__ void ld_global_v8(const float* src, float* v) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(src)
                 : "memory");
}

struct RopeParams {
    const void* q;
    void* out;
    const int64_t* positions;
    void* cos;           // table outputs, or NULL
    void* sin;
    int64_t T, H;
    int64_t q_ts, q_hs, o_ts, o_hs;   // token and head strides in elements
    int D;               // row width
    int tokens;          // tokens a CTA takes at a time
    uint64_t step[128];  // turns of pair i per position, in units of 2^-64 turn
    uint8_t axis[128];   // axis of pair i
};

struct ReadParams {
    const void* ckv;
    const void* kc;
    const float* ckv_scale;
    const float* k_scale;
    const int64_t* index;
    void* out;
    int32_t* status;
    int64_t T, S, d0, d1, nblk, out_stride;
    int Dv, Dk, mode;
    int ckv_kind, k_kind;
    int ckv_scale_per_ch, k_scale_per_ch;
    int small;           // T, S, d1 and the cache's rows fit 31 bits
    int out_wide;        // the output's rows lie on 32-byte boundaries
};

struct MlaParams {
    const void* qn;
    const void* qr;
    void* out;
    float* lse;
    const void* ckv;
    const void* kc;
    const float* ckv_scale;
    const float* k_scale;
    const int64_t* query_start;
    const int64_t* key_length;
    const int64_t* table;       // NULL: Norm mode
    int32_t* status;
    void* workspace;
    int64_t T, N, d0, d1, max_blocks, max_keys;
    int64_t qn_ts, qn_hs, qr_ts, qr_hs, o_ts, o_hs;
    int H, Dv, Dk;
    int causal;
    int ckv_kind, k_kind;
    int ckv_scale_per_ch, k_scale_per_ch;
    float scale;                // softmax scale
    int pairs;                  // tensor-core kernel: CTA pairs of the grid
    int q_flat;                 // its query rows are evenly spaced over heads and tokens
    int out_wide;               // its output rows lie on 32-byte boundaries
    const float* row_mul;       // power of two per row that its prepared queries lack, or NULL
    int runs, groups;           // its blocks hold whole halves of a step, whole groups of 8 keys
    int box_rows;               // its TMA boxes' rows (0: none)
    const int64_t* tree;        // [T, words] words of the new tokens that each token sees, or NULL
    int64_t words;
    int64_t max_new;            // new tokens of a sequence: T, or what the words have bits for
};

// Which of the 32 keys from key0 on a token sees by its words: all before the new ones, the first of which is key `first`.
__device__ __forceinline__ uint32_t tree_bits(const int64_t* words, int64_t count, int first, int key0) {
    const int off = key0 - first;   // bit of key0
    if (off <= -32) return 0xFFFFFFFFu;
    const int w = off >> 6, s = off & 63;   // (off < 0: the word -1 that comes before is all ones)
    const uint64_t a = w < 0 ? ~uint64_t(0) : (w < count ? uint64_t(words[w]) : 0);
    if (s <= 32) return uint32_t(a >> s);
    return uint32_t(a >> s) | uint32_t((w + 1 < count ? uint64_t(words[w + 1]) : 0) << (64 - s));
}

cudaError_t launch_rope(const RopeParams& p, int dtype, bool half_pairs, bool vec, cudaStream_t s);
cudaError_t launch_read(const ReadParams& p, int out_dtype, bool vec, cudaStream_t s);
cudaError_t launch_mla_generic(const MlaParams& p, int dtype, cudaStream_t s);
cudaError_t launch_mla_tc(MlaParams p, int dtype, cudaStream_t s);
bool mla_tc_fits(const MlaParams& p);                       // whether its work can be counted in 64 bits
int64_t mla_tc_workspace(const MlaParams& p, int dtype);   // bytes on the current device

}  // namespace kvr
