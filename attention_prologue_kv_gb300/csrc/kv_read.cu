// Reading cache rows back: the inverse of the prologue's scatter.
//
// Operation: out[t] = [ckv_cache[slot(t)] / ckv_scale | k_cache[slot(t)] / k_scale]
// with the slots of "aclnnKvRmsNormRopeCache" ("Restrictions on index").
//
// A stream, bound by HBM: one warp per row, each lane moves 8-channel chunks
// (a 16-byte or 8-byte load, a 16-byte store).
#include "kvr_internal.cuh"

namespace kvr {

constexpr int READ_THREADS = 128;

// Cache row of token t, or -1.
__device__ __forceinline__ int64_t read_row(const ReadParams& p, int64_t t) {
    const int64_t b = t / p.S, s = t - b * p.S;
    if (p.mode == KVR_CACHE_PA_BLK_BSND) {
        const int64_t q = s / p.d1, r = s - q * p.d1;
        const int64_t e = p.index[b * p.nblk + q];
        if (e == -1) return -1;
        if (e < 0 || e >= p.d0 * p.d1 || e % p.d1 + r >= p.d1) {
            if (p.status != nullptr) atomicOr(p.status, KVR_DEVERR_INDEX);
            return -1;
        }
        return e + r;
    }
    const int64_t e = p.index[t];
    if (e == -1) return -1;
    const int64_t range = p.mode == KVR_CACHE_NORM ? p.d1 : p.d0 * p.d1;
    if (e < 0 || e >= range) {
        if (p.status != nullptr) atomicOr(p.status, KVR_DEVERR_INDEX);
        return -1;
    }
    return p.mode == KVR_CACHE_NORM ? b * p.d1 + e : e;
}

// Eight values of a row, from channel c0 on.
template <class OT>
__device__ __forceinline__ uint4 read_chunk(const void* cache, int kind, int64_t at, const float* scale, bool per_ch, int c0) {
    if (kind == OUT16) return ld_stream_v4(static_cast<const uint16_t*>(cache) + at);
    const uint2 w = ld_stream_v2(static_cast<const uint8_t*>(cache) + at);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = dec8(kind, uint8_t((j < 4 ? w.x : w.y) >> (8 * (j & 3)))) * __frcp_rn(scale[per_ch ? c0 + j : 0]);
    return make_uint4(OT::pack(v[0], v[1]), OT::pack(v[2], v[3]), OT::pack(v[4], v[5]), OT::pack(v[6], v[7]));
}

template <class OT>
__global__ void __launch_bounds__(READ_THREADS) read_vec_kernel(const __grid_constant__ ReadParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (READ_THREADS / 32);
    const int nv = p.Dv / 8, n = nv + p.Dk / 8;
    for (int64_t t = int64_t(blockIdx.x) * (READ_THREADS / 32) + (threadIdx.x >> 5); t < p.T; t += warps) {
        int64_t row = 0;
        if (lane == 0) row = read_row(p, t);
        row = __shfl_sync(0xFFFFFFFFu, row, 0);
        if (row < 0) continue;
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + t * p.out_stride);
        for (int q = lane; q < n; q += 32)
            o[q] = q < nv ? read_chunk<OT>(p.ckv, p.ckv_kind, row * p.Dv + q * 8, p.ckv_scale, p.ckv_scale_per_ch, q * 8)
                          : read_chunk<OT>(p.kc, p.k_kind, row * p.Dk + (q - nv) * 8, p.k_scale, p.k_scale_per_ch, (q - nv) * 8);
    }
}

// Any width and alignment, element by element.
template <class OT>
__device__ __forceinline__ uint16_t read_one(const void* cache, int kind, int64_t at, const float* scale, bool per_ch, int c) {
    if (kind == OUT16) return static_cast<const uint16_t*>(cache)[at];
    return OT::one_out(dec8(kind, static_cast<const uint8_t*>(cache)[at]) * __frcp_rn(scale[per_ch ? c : 0]));
}

template <class OT>
__global__ void __launch_bounds__(READ_THREADS) read_generic_kernel(const __grid_constant__ ReadParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (READ_THREADS / 32);
    for (int64_t t = int64_t(blockIdx.x) * (READ_THREADS / 32) + (threadIdx.x >> 5); t < p.T; t += warps) {
        int64_t row = 0;
        if (lane == 0) row = read_row(p, t);
        row = __shfl_sync(0xFFFFFFFFu, row, 0);
        if (row < 0) continue;
        uint16_t* o = static_cast<uint16_t*>(p.out) + t * p.out_stride;
        for (int c = lane; c < p.Dv; c += 32) o[c] = read_one<OT>(p.ckv, p.ckv_kind, row * p.Dv + c, p.ckv_scale, p.ckv_scale_per_ch, c);
        for (int c = lane; c < p.Dk; c += 32) o[p.Dv + c] = read_one<OT>(p.kc, p.k_kind, row * p.Dk + c, p.k_scale, p.k_scale_per_ch, c);
    }
}

cudaError_t launch_read(const ReadParams& p, int out_dtype, bool vec, cudaStream_t s) {
    const int per = READ_THREADS / 32;
    const int64_t cap = int64_t(sm_count_current_device()) * 16;
    int64_t grid = (p.T + per - 1) / per;
    if (grid > cap) grid = cap;
    const dim3 g{unsigned(grid)}, b{unsigned(READ_THREADS)};
    if (out_dtype == KVR_BF16)
        return vec ? launch_pdl(read_vec_kernel<BF16>, g, b, 0, s, p) : launch_pdl(read_generic_kernel<BF16>, g, b, 0, s, p);
    return vec ? launch_pdl(read_vec_kernel<F16>, g, b, 0, s, p) : launch_pdl(read_generic_kernel<F16>, g, b, 0, s, p);
}

}  // namespace kvr
