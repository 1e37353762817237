// RoPE of the query's rotary part with positions of several axes.
//
// Operation: "aclnnMlaPrologV3WeightNz" (hiascend.com), "Formula", query path
// (q^R = ROPE(...)), by "aclnnKvRmsNormRopeCache", "Formulas (1)
// interleaveRope": with the pair (a, b) of lane i turned by t,
//   y[i] = a cos t - b sin t,  y[i + D/2] = b cos t + a sin t,
//   t = position[axis(i)] * base^(-2i/D).
//
// The angle: t / 2 pi is position * step[i] with step[i] = base^(-2i/D) / 2 pi
// in units of 2^-64 turn. The product modulo 2^64 drops whole turns exactly,
// so far positions lose nothing; read as a signed integer it is the rest in
// [-1/2, 1/2) turn, and sincospif takes it from there.
//
// A stream, bound by HBM: each thread keeps one 8-channel chunk of a token's
// row (4 angles in registers) and walks a block of heads with it: 16-byte
// loads, two 8-byte stores a row.
#include "kvr_internal.cuh"

namespace kvr {

constexpr int ROPE_THREADS = 128;

__device__ __forceinline__ void turn(const RopeParams& p, int64_t t, int i, float& c, float& s) {
    const uint64_t r = uint64_t(p.positions[int64_t(p.axis[i]) * p.T + t]) * p.step[i];
    sincospif(__ll2float_rn(int64_t(r)) * 0x1p-63f, &s, &c);   // r * 2^-64 turns = r * 2^-63 half turns
}

// V pairs (2V channels) a thread: 4 for rows on 16-byte boundaries, 1 otherwise.
template <class IT, bool HALF, int V>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int half = p.D / 2, nc = half / V;
    const int64_t stride = int64_t(gridDim.x) * ROPE_THREADS;
    for (int64_t it = int64_t(blockIdx.x) * ROPE_THREADS + threadIdx.x; it < p.items; it += stride) {
        const int64_t row = it / nc;
        const int i0 = int(it - row * nc) * V;
        const int64_t t = row / p.nhb;
        const int64_t h0 = (row - t * p.nhb) * p.hb;
        const int64_t h1 = h0 + p.hb < p.H ? h0 + p.hb : p.H;
        float c[V], s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) turn(p, t, i0 + j, c[j], s[j]);
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + t * p.q_ts;
        uint16_t* o = static_cast<uint16_t*>(p.out) + t * p.o_ts + i0;
        if constexpr (V == 4) {
            if (p.cos != nullptr && h0 == 0) {
                const uint2 cc = make_uint2(IT::pack(c[0], c[1]), IT::pack(c[2], c[3]));
                const uint2 ss = make_uint2(IT::pack(s[0], s[1]), IT::pack(s[2], s[3]));
                uint16_t* pc = static_cast<uint16_t*>(p.cos) + t * p.D + i0;
                uint16_t* ps = static_cast<uint16_t*>(p.sin) + t * p.D + i0;
                *reinterpret_cast<uint2*>(pc) = cc;
                *reinterpret_cast<uint2*>(pc + half) = cc;
                *reinterpret_cast<uint2*>(ps) = ss;
                *reinterpret_cast<uint2*>(ps + half) = ss;
            }
#pragma unroll 4
            for (int64_t h = h0; h < h1; ++h) {
                float a[4], b[4];
                if constexpr (HALF) {
                    const uint2 x = ld_stream_v2(q + h * p.q_hs + i0), y = ld_stream_v2(q + h * p.q_hs + half + i0);
                    a[0] = IT::lo(x.x), a[1] = IT::hi(x.x), a[2] = IT::lo(x.y), a[3] = IT::hi(x.y);
                    b[0] = IT::lo(y.x), b[1] = IT::hi(y.x), b[2] = IT::lo(y.y), b[3] = IT::hi(y.y);
                } else {
                    const uint4 x = ld_stream_v4(q + h * p.q_hs + 2 * i0);
                    a[0] = IT::lo(x.x), b[0] = IT::hi(x.x), a[1] = IT::lo(x.y), b[1] = IT::hi(x.y);
                    a[2] = IT::lo(x.z), b[2] = IT::hi(x.z), a[3] = IT::lo(x.w), b[3] = IT::hi(x.w);
                }
                float u[4], v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[j] = a[j] * c[j] - b[j] * s[j];
                    v[j] = b[j] * c[j] + a[j] * s[j];
                }
                *reinterpret_cast<uint2*>(o + h * p.o_hs) = make_uint2(IT::pack(u[0], u[1]), IT::pack(u[2], u[3]));
                *reinterpret_cast<uint2*>(o + h * p.o_hs + half) = make_uint2(IT::pack(v[0], v[1]), IT::pack(v[2], v[3]));
            }
        } else {
            if (p.cos != nullptr && h0 == 0) {
                uint16_t* pc = static_cast<uint16_t*>(p.cos) + t * p.D + i0;
                uint16_t* ps = static_cast<uint16_t*>(p.sin) + t * p.D + i0;
                pc[0] = pc[half] = IT::one_out(c[0]);
                ps[0] = ps[half] = IT::one_out(s[0]);
            }
            for (int64_t h = h0; h < h1; ++h) {
                const uint16_t* x = q + h * p.q_hs;
                const float a = IT::one(x[HALF ? i0 : 2 * i0]), b = IT::one(x[HALF ? i0 + half : 2 * i0 + 1]);
                o[h * p.o_hs] = IT::one_out(a * c[0] - b * s[0]);
                o[h * p.o_hs + half] = IT::one_out(b * c[0] + a * s[0]);
            }
        }
    }
}

template <class IT, bool HALF, int V>
static cudaError_t launch_rope_t(RopeParams p, cudaStream_t s) {
    p.hb = 8;
    p.nhb = p.H > 0 ? int((p.H + p.hb - 1) / p.hb) : 1;   // without heads: the tables alone
    p.items = p.T * p.nhb * (p.D / 2 / V);
    const int64_t cap = int64_t(sm_count_current_device()) * 16;
    int64_t grid = (p.items + ROPE_THREADS - 1) / ROPE_THREADS;
    if (grid > cap) grid = cap;
    return launch_pdl(rope_kernel<IT, HALF, V>, dim3(unsigned(grid)), dim3(ROPE_THREADS), 0, s, p);
}

cudaError_t launch_rope(const RopeParams& p, int dtype, bool half_pairs, bool vec, cudaStream_t s) {
    if (dtype == KVR_BF16) {
        if (vec) return half_pairs ? launch_rope_t<BF16, true, 4>(p, s) : launch_rope_t<BF16, false, 4>(p, s);
        return half_pairs ? launch_rope_t<BF16, true, 1>(p, s) : launch_rope_t<BF16, false, 1>(p, s);
    }
    if (vec) return half_pairs ? launch_rope_t<F16, true, 4>(p, s) : launch_rope_t<F16, false, 4>(p, s);
    return half_pairs ? launch_rope_t<F16, true, 1>(p, s) : launch_rope_t<F16, false, 1>(p, s);
}

}  // namespace kvr
