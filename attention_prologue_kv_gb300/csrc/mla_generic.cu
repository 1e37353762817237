// Latent attention for rows the tensor-core kernel does not take (widths that
// are no multiple of 8 or beyond 512 + 64, rows off 16-byte boundaries).
//
// One warp per (token, head): the query's channels and the output sum stay in
// registers (lane l has channels l, l + 32, ...), keys come one after the
// other, with the running maximum m and sum l of the softmax:
//   s = scale * <q, key>,  m' = max(m, s),  o = o e^(m - m') + e^(s - m') c.
// 64 keys are summed on their own (lb, ob) before they join l and o: added one by one beside a key of large weight, many
// small ones would all round to the same side (131072 equal ones 23.4 octaves below it: off by a third).
// Every key row is read once per head, from L1 or L2: this is the plain kernel,
// bound by the loads and the warp sum of each key. Measured: one token of 16 heads over 1000 keys of 512 + 64 channels
// 1417 us (the tensor-core kernel 14.9).
#include "attention_step.cuh"

namespace kvr {

constexpr int MLA_GEN_THREADS = 128, MLA_GEN_BLOCK = 64;

template <class IT>
__device__ __forceinline__ float mla_value(const void* cache, int kind, int64_t at) {
    if (kind == OUT16) return IT::one(static_cast<const uint16_t*>(cache)[at]);
    return dec8(kind, static_cast<const uint8_t*>(cache)[at]);
}

// NV, NK: channels of a lane, Dv <= 32 NV and Dk <= 32 NK.
template <class IT, int NV, int NK>
__global__ void __launch_bounds__(MLA_GEN_THREADS) mla_generic_kernel(const __grid_constant__ MlaParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (MLA_GEN_THREADS / 32);
    const int64_t w0 = int64_t(blockIdx.x) * (MLA_GEN_THREADS / 32) + (threadIdx.x >> 5);
    if (w0 == 0)   // the sequences that are left out
        for (int64_t n = lane; n < p.N; n += 32) {
            const int64_t a = p.query_start[n], b = p.query_start[n + 1], K = p.key_length[n];
            int bits = 0;
            if (a < 0 || b < a || b > p.T) bits = KVR_DEVERR_QUERY;
            else if (a < b && (K < 0 || K > p.max_keys)) bits = KVR_DEVERR_KEY_LENGTH;
            if (bits && p.status != nullptr) atomicOr(p.status, bits);
        }
    // Sequences in the outer loop: a query_start that decreases at one sequence
    // leaves the others' ranges as they are.
    for (int64_t n = 0; n < p.N; ++n) {
        const int64_t q0 = p.query_start[n], q1 = p.query_start[n + 1], K = p.key_length[n];
        if (q0 < 0 || q1 <= q0 || q1 > p.T || K < 0 || K > p.max_keys) continue;
        const int64_t rows = (q1 - q0) * p.H;
        for (int64_t r = w0; r < rows; r += warps) {
            const int64_t t = q0 + r / p.H, h = r % p.H;
            int64_t seen = p.causal ? K - (q1 - 1 - t) : K;
            const uint16_t* qn = static_cast<const uint16_t*>(p.qn) + t * p.qn_ts + h * p.qn_hs;
            const uint16_t* qr = static_cast<const uint16_t*>(p.qr) + t * p.qr_ts + h * p.qr_hs;
            float a[NV], b[NK], o[NV], ob[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + 32 * j;
                o[j] = ob[j] = 0.f;
                a[j] = c < p.Dv ? IT::one(qn[c]) : 0.f;
                if (p.ckv_kind != OUT16 && c < p.Dv) a[j] /= p.ckv_scale[p.ckv_scale_per_ch ? c : 0];
            }
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int c = lane + 32 * j;
                b[j] = c < p.Dk ? IT::one(qr[c]) : 0.f;
                if (p.k_kind != OUT16 && c < p.Dk) b[j] /= p.k_scale[p.k_scale_per_ch ? c : 0];
            }
            float m = -INFINITY, l = 0.f, lb = 0.f;
            int held = 0;   // keys in lb and ob
            auto join = [&]() {
                l += lb;
                lb = 0.f;
                held = 0;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    o[j] += ob[j];
                    ob[j] = 0.f;
                }
            };
            for (int64_t i = 0; i < seen; ++i) {
                int64_t slot = n * p.d1 + i;
                if (p.table != nullptr) {
                    const int64_t q = i / p.d1, e = p.table[n * p.max_blocks + q];
                    if (e < 0 || e >= p.d0) {
                        if (e != -1 && p.status != nullptr && lane == 0) atomicOr(p.status, KVR_DEVERR_INDEX);
                        i = (q + 1) * p.d1 - 1;
                        continue;
                    }
                    slot = e * p.d1 + (i - q * p.d1);
                }
                float v[NV], s = 0.f;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = lane + 32 * j;
                    v[j] = c < p.Dv ? mla_value<IT>(p.ckv, p.ckv_kind, slot * p.Dv + c) : 0.f;
                    s = fmaf(a[j], v[j], s);
                }
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    const int c = lane + 32 * j;
                    if (c < p.Dk) s = fmaf(b[j], mla_value<IT>(p.kc, p.k_kind, slot * p.Dk + c), s);
                }
                s = warp_sum(s) * p.scale;
                const float mn = fmaxf(m, s);   // a NaN score leaves m, and makes the weight NaN
                const float e = s == -INFINITY ? 0.f : expf(s - mn);
                if (m != mn) {   // (the same in all lanes)
                    const float f = expf(m - mn);
                    m = mn;
                    l *= f;
                    lb *= f;
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        o[j] *= f;
                        ob[j] *= f;
                    }
                }
                lb += e;
#pragma unroll
                for (int j = 0; j < NV; ++j) ob[j] = fmaf(e, v[j], ob[j]);
                if (++held == MLA_GEN_BLOCK) join();
            }
            join();
            uint16_t* out = static_cast<uint16_t*>(p.out) + t * p.o_ts + h * p.o_hs;
            const float inv = l == 0.f ? 0.f : 1.f / l;   // no key: zeros
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + 32 * j;
                if (c >= p.Dv) continue;
                float y = o[j] * inv;
                if (p.ckv_kind != OUT16) y /= p.ckv_scale[p.ckv_scale_per_ch ? c : 0];
                out[c] = IT::one_out(l == 0.f ? 0.f : y);
            }
            if (p.lse != nullptr && lane == 0) p.lse[t * p.H + h] = l == 0.f ? -INFINITY : m + logf(l);
        }
    }
}

template <class IT>
static cudaError_t launch_mla_generic_t(const MlaParams& p, cudaStream_t s) {
    const dim3 g(unsigned(sm_count_current_device() * 4)), b(MLA_GEN_THREADS);
    if (p.Dk <= 64) {
        if (p.Dv <= 128) return launch_pdl(mla_generic_kernel<IT, 4, 2>, g, b, 0, s, p);
        if (p.Dv <= 512) return launch_pdl(mla_generic_kernel<IT, 16, 2>, g, b, 0, s, p);
    }
    return launch_pdl(mla_generic_kernel<IT, 32, 8>, g, b, 0, s, p);
}

cudaError_t launch_mla_generic(const MlaParams& p, int dtype, cudaStream_t s) {
    return dtype == KVR_BF16 ? launch_mla_generic_t<BF16>(p, s) : launch_mla_generic_t<F16>(p, s);
}

}  // namespace kvr
