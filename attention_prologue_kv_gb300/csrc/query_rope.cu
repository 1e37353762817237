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
// A stream, bound by HBM. A CTA takes a few tokens at a time: one thread a
// (token, pair) turns the angle into shared memory, then the threads take the
// tokens' rows in order, 8 channels each: 16-byte loads, two 8-byte stores. The
// first rows are loaded before the angles are waited for. Measured: 8191 tokens x 128 heads x 64 channels, three
// axes, 50 us (5.4 TB/s, 80% of the copy rate); 256 tokens x 128 heads 4.3 us, of which the bytes take 1.25: a chain of
// position, angle, rows. 8192 tokens x 128 heads x 64 channels, one axis: 48 us, half pairs (8-byte loads) 64 us; of 62
// channels, pair by pair, 162 us.
#include "attention_step.cuh"

namespace kvr {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_BATCH = 4;      // rows of a thread in flight
constexpr int ROPE_TOKENS = 8;     // most tokens of a CTA at a time

__device__ __forceinline__ float2 turn(const RopeParams& p, int64_t t, int i) {
    const uint64_t r = uint64_t(p.positions[int64_t(p.axis[i]) * p.T + t]) * p.step[i];
    float2 cs;
    sincospif(__ll2float_rn(int64_t(r)) * 0x1p-63f, &cs.y, &cs.x);   // r * 2^-64 turns = r * 2^-63 half turns
    return cs;
}

// Where a thread is in the rows (token, head) of a batch of tokens.
struct RopeRow {
    int t;
    int64_t h;
    __device__ __forceinline__ void next(int dt, int64_t dh, int64_t H) {
        t += dt;
        h += dh;
        if (h >= H) {
            h -= H;
            ++t;
        }
    }
};

// V pairs (2V channels) a thread: 4 for rows on 16-byte boundaries, 1 otherwise.
template <class IT, bool HALF, int V>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs[ROPE_TOKENS][128];
    const int half = p.D / 2, nc = half / V, tid = threadIdx.x;
    const int slots = ROPE_THREADS / nc;               // rows at a time
    const int chunk = tid % nc, i0 = chunk * V;
    const bool works = tid < slots * nc;
    const int dt = int(p.H > 0 ? slots / p.H : 0);
    const int64_t dh = p.H > 0 ? slots % p.H : 0;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t0 = int64_t(blockIdx.x) * p.tokens; t0 < p.T; t0 += int64_t(gridDim.x) * p.tokens) {
        const int n = int(p.T - t0 < p.tokens ? p.T - t0 : p.tokens);
        RopeRow at = {n, 0};
        if (works && p.H > 0) at = {int((tid / nc) / p.H), (tid / nc) % p.H};
        uint32_t x[ROPE_BATCH][V];   // V = 4: a row's 16 bytes (HALF: 8 and 8); V = 1: its two values
        auto load = [&](RopeRow r) {
#pragma unroll
            for (int k = 0; k < ROPE_BATCH; ++k) {
                if (r.t < n) {
                    const uint16_t* q = static_cast<const uint16_t*>(p.q) + (t0 + r.t) * p.q_ts + r.h * p.q_hs;
                    if constexpr (V == 4 && HALF) {
                        const uint2 a = ld_stream_v2(q + i0), b = ld_stream_v2(q + half + i0);
                        x[k][0] = a.x, x[k][1] = a.y, x[k][2] = b.x, x[k][3] = b.y;
                    } else if constexpr (V == 4) {
                        const uint4 a = ld_stream_v4(q + 2 * i0);
                        x[k][0] = a.x, x[k][1] = a.y, x[k][2] = a.z, x[k][3] = a.w;
                    } else {
                        x[k][0] = uint32_t(q[HALF ? i0 : 2 * i0]) | uint32_t(q[HALF ? i0 + half : 2 * i0 + 1]) << 16;
                    }
                }
                r.next(dt, dh, p.H);
            }
        };
        load(at);
        for (int e = tid; e < n * half; e += ROPE_THREADS) {
            const int t = e / half, i = e - t * half;
            const float2 v = turn(p, t0 + t, i);
            cs[t][i] = v;
            if (p.cos != nullptr) {
                uint16_t* pc = static_cast<uint16_t*>(p.cos) + (t0 + t) * p.D + i;
                uint16_t* ps = static_cast<uint16_t*>(p.sin) + (t0 + t) * p.D + i;
                pc[0] = pc[half] = IT::one_out(v.x);
                ps[0] = ps[half] = IT::one_out(v.y);
            }
        }
        __syncthreads();
        while (at.t < n) {
#pragma unroll
            for (int k = 0; k < ROPE_BATCH; ++k) {
                if (at.t < n) {
                    uint16_t* o = static_cast<uint16_t*>(p.out) + (t0 + at.t) * p.o_ts + at.h * p.o_hs + i0;
                    if constexpr (V == 4) {
                        float u[4], v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 c = cs[at.t][i0 + j];
                            const float a = HALF ? ((j & 1) ? IT::hi(x[k][j >> 1]) : IT::lo(x[k][j >> 1])) : IT::lo(x[k][j]);
                            const float b = HALF ? ((j & 1) ? IT::hi(x[k][2 + (j >> 1)]) : IT::lo(x[k][2 + (j >> 1)])) : IT::hi(x[k][j]);
                            u[j] = a * c.x - b * c.y;
                            v[j] = b * c.x + a * c.y;
                        }
                        *reinterpret_cast<uint2*>(o) = make_uint2(IT::pack(u[0], u[1]), IT::pack(u[2], u[3]));
                        *reinterpret_cast<uint2*>(o + half) = make_uint2(IT::pack(v[0], v[1]), IT::pack(v[2], v[3]));
                    } else {
                        const float2 c = cs[at.t][i0];
                        const float a = IT::lo(x[k][0]), b = IT::hi(x[k][0]);
                        o[0] = IT::one_out(a * c.x - b * c.y);
                        o[half] = IT::one_out(b * c.x + a * c.y);
                    }
                }
                at.next(dt, dh, p.H);
            }
            load(at);
        }
        __syncthreads();   // the angles are read
    }
}

template <class IT, bool HALF, int V>
static cudaError_t launch_rope_t(RopeParams p, cudaStream_t s) {
    // Tokens a CTA takes at a time: 8 make one (token, pair) a thread at 64 channels; fewer where that would leave SMs
    // without two CTAs each.
    const int64_t sms = sm_count_current_device();
    const int64_t t = p.T / (sms * 2);
    p.tokens = int(t < 1 ? 1 : (t < ROPE_TOKENS ? t : ROPE_TOKENS));
    const int64_t need = (p.T + p.tokens - 1) / p.tokens, cap = sms * 8;
    return launch_pdl(rope_kernel<IT, HALF, V>, dim3(unsigned(need < cap ? need : cap)), dim3(ROPE_THREADS), 0, s, p);
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
