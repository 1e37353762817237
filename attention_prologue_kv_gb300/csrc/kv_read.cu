// Reading cache rows back: the inverse of the prologue's scatter.
//
// Operation: out[t] = [ckv_cache[slot(t)] / ckv_scale | k_cache[slot(t)] / k_scale]
// with the slots of "aclnnKvRmsNormRopeCache" ("Restrictions on index").
//
// A stream, bound by HBM. Rows of 512 + 64 channels: a warp takes four rows at
// a time, their loads in flight together: a lane has 16 channels of each latent
// row and an eighth of one rotary row.
// Other widths on 16-byte boundaries: one warp per row, chunks of 8 channels.
// Measured: 32768 rows of E4M3 codes 13.2 us (4.5 TB/s, 66% of the copy rate; index, row and store follow one another in
// a warp), 19647 rows of int8 codes 7.9 us, 256 bf16 rows 2.9 us, a launch.
// 32768 bf16 rows 14.6 us (5.2 TB/s); 32768 rows of 256 + 64 channels 13.0 us, as codes 16.8 us, where codes are decoded
// one by one; of 500 + 60 channels as codes, element by element, 44 us.
#include "attention_step.cuh"

namespace kvr {

constexpr int READ_THREADS = 128;

// Cache row of token t, or -1. I: 32-bit arithmetic where everything fits, as 64-bit divisions take about 100 instructions.
template <class I>
__device__ __forceinline__ int64_t read_row_t(const ReadParams& p, int64_t token) {
    const I t = I(token), S = I(p.S), d1 = I(p.d1), rows = I(p.d0) * d1;
    const I b = t / S, s = t - b * S;
    const bool blocks = p.mode == KVR_CACHE_PA_BLK_BSND, norm = p.mode == KVR_CACHE_NORM;
    const I q = blocks ? s / d1 : 0, r = blocks ? s - q * d1 : 0;
    const int64_t e = p.index[blocks ? int64_t(b) * p.nblk + q : token];
    if (e == -1) return -1;
    if (e < 0 || e >= int64_t(norm ? d1 : rows) || (blocks && I(e) % d1 + r >= d1)) {
        if (p.status != nullptr) atomicOr(p.status, KVR_DEVERR_INDEX);
        return -1;
    }
    return norm ? int64_t(b) * p.d1 + e : e + int64_t(r);
}
__device__ __forceinline__ int64_t read_row(const ReadParams& p, int64_t t) {
    return p.small ? read_row_t<uint32_t>(p, t) : read_row_t<uint64_t>(p, t);
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

// Four codes of kind K, times four factors, to two packed values.
template <class OT, int K>
__device__ __forceinline__ uint2 codes4(uint32_t u, const float4& f) {
    float v[4];
    if constexpr (K == OUT_I8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = float(int8_t(u >> (8 * k)));
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(uint16_t(u >> (16 * k)), K == OUT_E4M3 ? __NV_E4M3 : __NV_E5M2);
            v[2 * k] = __half2float(__ushort_as_half(h.x));
            v[2 * k + 1] = __half2float(__ushort_as_half(h.y));
        }
    }
    return make_uint2(OT::pack(v[0] * f.x, v[1] * f.y), OT::pack(v[2] * f.z, v[3] * f.w));
}

constexpr int READ_ROWS = 4;   // rows of a warp at a time
constexpr int READ_ROWS_THREADS = 256;
template <class OT, int K>
__global__ void __launch_bounds__(READ_ROWS_THREADS, K == OUT16 ? 3 : 4) read_rows_kernel(const __grid_constant__ ReadParams p) {
    constexpr int Dv = 512, Dk = 64;
    // 1 / scale, once a CTA (read by every warp of the grid from global memory it took as long as the rows), four
    // channels of lane l's 16 at [i][l]: registers for it would leave a quarter of the warps.
    __shared__ float4 inv_s[4][32];
    __shared__ float4 invk_s[2][8];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, eighth = lane & 7, sub = lane >> 3;
    const int64_t step = int64_t(gridDim.x) * (READ_ROWS_THREADS / 32) * READ_ROWS;
    int64_t t = (int64_t(blockIdx.x) * (READ_ROWS_THREADS / 32) + (threadIdx.x >> 5)) * READ_ROWS;
    int64_t mine = -1;
    if (lane < READ_ROWS && t + lane < p.T) mine = read_row(p, t + lane);
    if (K != OUT16 || p.k_kind != OUT16) {
        if constexpr (K != OUT16)
            for (int c = threadIdx.x; c < Dv; c += READ_ROWS_THREADS)
                reinterpret_cast<float*>(&inv_s[c >> 2 & 3][c >> 4])[c & 3] = __frcp_rn(p.ckv_scale[p.ckv_scale_per_ch ? c : 0]);
        if (p.k_kind != OUT16 && threadIdx.x < Dk)
            reinterpret_cast<float*>(&invk_s[threadIdx.x >> 2 & 1][threadIdx.x >> 3])[threadIdx.x & 3] =
                __frcp_rn(p.k_scale[p.k_scale_per_ch ? threadIdx.x : 0]);
        __syncthreads();
    }
#pragma unroll 1
    for (; t < p.T; t += step) {
        constexpr int NW = K == OUT16 ? 2 : 1;
        uint4 x[READ_ROWS][NW], y = make_uint4(0, 0, 0, 0);
        uint32_t live = 0;
#pragma unroll
        for (int k = 0; k < READ_ROWS; ++k) {
            const int64_t row = __shfl_sync(0xFFFFFFFFu, mine, k);
            if (row < 0) continue;
            live |= 1u << k;
            if constexpr (K == OUT16) {   // 8 channels of each half of the row
                const uint16_t* src = static_cast<const uint16_t*>(p.ckv) + row * Dv + lane * 8;
                x[k][0] = ld_stream_v4(src);
                x[k][1] = ld_stream_v4(src + 256);
            } else {
                x[k][0] = ld_stream_v4(static_cast<const uint8_t*>(p.ckv) + row * Dv + lane * 16);
            }
        }
        const int64_t krow = __shfl_sync(0xFFFFFFFFu, mine, sub);
        if (krow >= 0) {
            if (p.k_kind == OUT16) {
                y = ld_stream_v4(static_cast<const uint16_t*>(p.kc) + krow * Dk + eighth * 8);
            } else {
                const uint2 w = ld_stream_v2(static_cast<const uint8_t*>(p.kc) + krow * Dk + eighth * 8);
                y.x = w.x;
                y.y = w.y;
            }
        }
        // The next rows' index entries, while these rows come.
        const int64_t after = t + step + lane;
        mine = lane < READ_ROWS && after < p.T ? read_row(p, after) : -1;
        uint16_t* out = static_cast<uint16_t*>(p.out) + t * p.out_stride;
        if constexpr (K == OUT16) {
#pragma unroll
            for (int k = 0; k < READ_ROWS; ++k)
                if (live >> k & 1) {
                    *reinterpret_cast<uint4*>(out + k * p.out_stride + lane * 8) = x[k][0];
                    *reinterpret_cast<uint4*>(out + k * p.out_stride + 256 + lane * 8) = x[k][1];
                }
        } else {
#pragma unroll
            for (int k = 0; k < READ_ROWS; ++k)
                if (live >> k & 1) {
                    uint16_t* o = out + k * p.out_stride + lane * 16;
                    const uint32_t w[4] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w};
                    uint32_t u[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 z = codes4<OT, K>(w[i], inv_s[i][lane]);
                        u[2 * i] = z.x;
                        u[2 * i + 1] = z.y;
                    }
                    if (p.out_wide) {
                        st_global_v8(o, u);
                    } else {
                        *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
                        *reinterpret_cast<uint4*>(o + 8) = make_uint4(u[4], u[5], u[6], u[7]);
                    }
                }
        }
        if (krow >= 0) {
            if (p.k_kind != OUT16) {
                uint2 a, b;
                const float4 f = invk_s[0][eighth], g = invk_s[1][eighth];
                if (p.k_kind == OUT_I8) a = codes4<OT, OUT_I8>(y.x, f), b = codes4<OT, OUT_I8>(y.y, g);
                else if (p.k_kind == OUT_E4M3) a = codes4<OT, OUT_E4M3>(y.x, f), b = codes4<OT, OUT_E4M3>(y.y, g);
                else a = codes4<OT, OUT_E5M2>(y.x, f), b = codes4<OT, OUT_E5M2>(y.y, g);
                y = make_uint4(a.x, a.y, b.x, b.y);
            }
            *reinterpret_cast<uint4*>(out + sub * p.out_stride + Dv + eighth * 8) = y;
        }
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

template <class OT>
static cudaError_t launch_read_t(const ReadParams& p, bool vec, cudaStream_t s) {
    // 16 codes a load need rows on 16-byte boundaries; 8-byte ones take the narrower chunks.
    const bool rows = vec && p.Dv == 512 && p.Dk == 64 && reinterpret_cast<uintptr_t>(p.ckv) % 16 == 0;
    const int threads = rows ? READ_ROWS_THREADS : READ_THREADS;
    const int64_t per = threads / 32 * (rows ? READ_ROWS : 1);
    const int64_t cap = int64_t(sm_count_current_device()) * (rows ? 4 : 16);
    int64_t grid = (p.T + per - 1) / per;
    if (grid > cap) grid = cap;
    const dim3 g{unsigned(grid)}, b{unsigned(threads)};
    if (rows) switch (p.ckv_kind) {
            case OUT_I8: return launch_pdl(read_rows_kernel<OT, OUT_I8>, g, b, 0, s, p);
            case OUT_E4M3: return launch_pdl(read_rows_kernel<OT, OUT_E4M3>, g, b, 0, s, p);
            case OUT_E5M2: return launch_pdl(read_rows_kernel<OT, OUT_E5M2>, g, b, 0, s, p);
            default: return launch_pdl(read_rows_kernel<OT, OUT16>, g, b, 0, s, p);
        }
    return vec ? launch_pdl(read_vec_kernel<OT>, g, b, 0, s, p) : launch_pdl(read_generic_kernel<OT>, g, b, 0, s, p);
}

cudaError_t launch_read(const ReadParams& p, int out_dtype, bool vec, cudaStream_t s) {
    return out_dtype == KVR_BF16 ? launch_read_t<BF16>(p, vec, s) : launch_read_t<F16>(p, vec, s);
}

}  // namespace kvr
