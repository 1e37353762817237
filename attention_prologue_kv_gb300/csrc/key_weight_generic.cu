// The attention weight of each key, for rows that the tensor-core kernel does not take.
//
//   w[i] = decay * past[i] + sum over the rows r that see key i of e^(scale <q_r, key_i> - lse_r)
//
// One warp per key: the key's channels stay in registers (lane l has channels l, l + 32, ...), the sequence's rows come one
// after the other. 64 rows are summed on their own before they join the key's sum. This is the plain kernel, bound by the
// loads and the warp sum of each (row, key). Measured: one token of 16 heads over 1000 keys 17 us (the tensor-core kernel 7),
// 256 sequences of one token, 128 heads, 1-4095 keys 39.8 ms (110 us).
#include "cache_ops.cuh"

namespace kvr {

constexpr int KW_GEN_THREADS = 128, KW_GEN_BLOCK = 64;

template <class IT>
__device__ __forceinline__ float kw_value(const void* cache, int kind, int64_t at) {
    if (kind == OUT16) return IT::one(static_cast<const uint16_t*>(cache)[at]);
    return dec8(kind, static_cast<const uint8_t*>(cache)[at]);
}

// NV, NK: channels of a lane, Dv <= 32 NV and Dk <= 32 NK.
template <class IT, int NV, int NK>
__global__ void __launch_bounds__(KW_GEN_THREADS) key_weight_generic_kernel(const __grid_constant__ KeyWeightParams w) {
    const MlaParams& p = w.m;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (KW_GEN_THREADS / 32);
    const int64_t w0 = int64_t(blockIdx.x) * (KW_GEN_THREADS / 32) + (threadIdx.x >> 5);
    if (w0 == 0)   // the sequences that are left out
        for (int64_t n = lane; n < p.N; n += 32) {
            const int64_t a = p.query_start[n], b = p.query_start[n + 1], K = p.key_length[n];
            int bits = 0;
            if (a < 0 || b < a || b > p.T) bits = KVR_DEVERR_QUERY;
            else if (a < b && (K < 0 || K > p.max_keys)) bits = KVR_DEVERR_KEY_LENGTH;
            if (bits && p.status != nullptr) atomicOr(p.status, bits);
        }
    for (int64_t n = 0; n < p.N; ++n) {
        const int64_t q0 = p.query_start[n], q1 = p.query_start[n + 1], K = p.key_length[n];
        if (q0 < 0 || q1 <= q0 || q1 > p.T || K < 0 || K > p.max_keys) continue;
        for (int64_t i = w0; i < K; i += warps) {
            int64_t slot = n * p.d1 + i;
            bool held = true;
            if (p.table != nullptr) {
                const int64_t q = i / p.d1, e = p.table[n * p.max_blocks + q];
                held = e >= 0 && e < p.d0;
                if (!held && e != -1 && p.status != nullptr && lane == 0) atomicOr(p.status, KVR_DEVERR_INDEX);
                slot = e * p.d1 + (i - q * p.d1);
            }
            float sum = 0.f, part = 0.f;
            if (held) {
                float v[NV], u[NK];
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = lane + 32 * j;
                    v[j] = c < p.Dv ? kw_value<IT>(p.ckv, p.ckv_kind, slot * p.Dv + c) : 0.f;
                    if (p.ckv_kind != OUT16 && c < p.Dv) v[j] /= p.ckv_scale[p.ckv_scale_per_ch ? c : 0];
                }
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    const int c = lane + 32 * j;
                    u[j] = c < p.Dk ? kw_value<IT>(p.kc, p.k_kind, slot * p.Dk + c) : 0.f;
                    if (p.k_kind != OUT16 && c < p.Dk) u[j] /= p.k_scale[p.k_scale_per_ch ? c : 0];
                }
                // With causal masking the first token that sees key i is the one with K - L + j + 1 > i.
                int64_t t0 = q0;
                if (p.causal) t0 = max(q0, q1 - (K - i));
                int count = 0;
                for (int64_t t = t0; t < q1; ++t)
                    for (int64_t h = 0; h < p.H; ++h) {
                        const uint16_t* qn = static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + h * p.qn_hs;
                        const uint16_t* qr = static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + h * p.qr_hs;
                        float s = 0.f;
#pragma unroll
                        for (int j = 0; j < NV; ++j)
                            if (lane + 32 * j < p.Dv) s = fmaf(IT::one(qn[lane + 32 * j]), v[j], s);
#pragma unroll
                        for (int j = 0; j < NK; ++j)
                            if (lane + 32 * j < p.Dk) s = fmaf(IT::one(qr[lane + 32 * j]), u[j], s);
                        s = warp_sum(s) * p.scale;
                        const float l = p.lse[t * p.H + h];
                        part += l == -INFINITY ? 0.f : expf(s - l);
                        if (++count % KW_GEN_BLOCK == 0) {
                            sum += part;
                            part = 0.f;
                        }
                    }
                sum += part;
            }
            if (lane == 0) {
                if (w.past != nullptr) sum = fmaf(w.decay, w.past[n * w.past_stride + i], sum);
                w.weight[n * w.weight_stride + i] = sum;
            }
        }
    }
}

template <class IT>
static cudaError_t launch_t(const KeyWeightParams& p, cudaStream_t s) {
    const dim3 g(unsigned(sm_count_current_device() * 8)), b(KW_GEN_THREADS);
    if (p.m.Dk <= 64) {
        if (p.m.Dv <= 128) return launch_pdl(key_weight_generic_kernel<IT, 4, 2>, g, b, 0, s, p);
        if (p.m.Dv <= 512) return launch_pdl(key_weight_generic_kernel<IT, 16, 2>, g, b, 0, s, p);
    }
    return launch_pdl(key_weight_generic_kernel<IT, 32, 8>, g, b, 0, s, p);
}

cudaError_t launch_key_weight_generic(const KeyWeightParams& p, int dtype, cudaStream_t s) {
    return dtype == KVR_BF16 ? launch_t<BF16>(p, s) : launch_t<F16>(p, s);
}

}  // namespace kvr
