// What the tensor-core kernels over the latent cache share: sequences, cache rows of keys, swizzled tiles, codes as halves,
// waits, tensor maps.
#pragma once

#include "tcgen05.cuh"

namespace kvr {

struct Seq {
    int64_t q0;
    int L, K;   // L = 0: nothing to do
};

__device__ __forceinline__ Seq load_seq(const MlaParams& p, int n, int* bits = nullptr) {
    const int64_t a = p.query_start[n], b = p.query_start[n + 1], K = p.key_length[n];
    if (a < 0 || b < a || b > p.T || b - a > p.max_new) {
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

__device__ __forceinline__ uint32_t box_at(uint32_t box, int row, int chunk) {
    return box + uint32_t(row) * 128u + (uint32_t(chunk ^ (row & 7)) << 4);
}


// The rest of a wait, out of line: the roles' loops have to stay in the instruction cache. `more`: seconds beyond the first.
static __device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, int more) {
    while (*abort == 0) {
        if (mbar_wait(bar, parity, abort)) return true;
        if (--more < 0) *abort = 1;
    }
    return false;
}

// The driver's tensor-map encoder, found through the runtime (no link to libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encoder() {
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
inline bool encode_rows(CUtensorMap* map, const void* base, bool bf16, int64_t rows, int width, int box_rows, int boxes) {
    const cuuint64_t dims[3] = {64, cuuint64_t(rows), cuuint64_t(width) / 64}, strides[2] = {cuuint64_t(width) * 2, 128};
    const cuuint32_t box[3] = {64, cuuint32_t(box_rows), cuuint32_t(boxes)}, one[3] = {1, 1, 1};
    return encoder()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
                     dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kvr
