// The router of the mixture-of-experts layer, in one launch with the
// quantisation of the tokens' activations (which does not depend on it):
//
//   l[t, e] = sum_h X[t, h] R[e, h]         64-bit sums of exact products
//   p       = softmax over the experts; each token takes its top_k experts
//             (ties to the lower index); weight p, or p / (sum of the chosen p)
//
// The scores are summed in 64 bits because a rounding there can change which
// expert a token takes, a whole expert's output and not a rounding's worth.
// The work is small (T * E * H multiply-adds); what bounds the kernel is the
// chain of its steps: 16 tokens, 64 experts of 2048, have their scores at
// 3.5 us, the choices at 6 and the list at 8 us (one token of 8 experts of
// 4096: 3.5, 4.6, 5.3 us).  A block takes 4 experts x kTT tokens; the last block of
// a token group (a ticket) picks the experts of those tokens, a warp per
// token, and the last group lists the chosen experts in ascending order.
#pragma once

#include "fp8_quant_sm100.cuh"

namespace i8mm {

struct RouteParams {
    const uint16_t* X;       // T x H
    const uint16_t* R;       // E x H
    int T, H, E, top_k, renorm;
    int log_blocks;          // blocks of scores; the rest quantise X
    double* logits;          // T x E
    int32_t* ids;            // T x top_k
    float* wts;              // T x top_k
    int32_t* active;         // count, then chosen experts
    unsigned long long* masks;  // for each of those the tokens that chose it, a bit each
    unsigned* tickets;       // one per token group and one more, zero between calls
    uint8_t* xq;             // T x H codes, scales [b * T + t]
    float* xs;
};

constexpr int kRouteThreads = 256;
constexpr int kRouteExperts = 4;     // experts of a score block
constexpr int kMaxExperts = 256;

// Order-preserving integer of a score: larger score, larger key; -0 as +0; a
// NaN below every number, so that the choice is always top_k distinct experts.
__device__ __forceinline__ unsigned long long score_key(double l) {
    if (l != l) return 0ull;
    const long long b = __double_as_longlong(l + 0.0);
    return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

template <int kTT, typename T>
__global__ void __launch_bounds__(kRouteThreads)
    k_moe_route(const RouteParams p) {
    __shared__ double red[kRouteThreads / 32][kRouteExperts * kTT];
    __shared__ unsigned chose[kMaxExperts][2];  // the tokens that chose an expert, a bit each
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x >= p.log_blocks) {
        const int KB = (p.H + 127) / 128;
        const long long b = (int)blockIdx.x - p.log_blocks, nb = (int)gridDim.x - p.log_blocks;
        quant_fp8_blocks<T>(p.X, (long long)p.T * KB, p.H, KB, p.xq, p.xs, 1, p.T, (b * kRouteThreads + tid) >> 3,
                            nb * (kRouteThreads / 8));
        return;
    }
    const int eb = (p.E + kRouteExperts - 1) / kRouteExperts;
    const int tg = (int)blockIdx.x / eb, e0 = ((int)blockIdx.x % eb) * kRouteExperts, t0 = tg * kTT;

    double acc[kRouteExperts][kTT];
#pragma unroll
    for (int i = 0; i < kRouteExperts; ++i)
#pragma unroll
        for (int j = 0; j < kTT; ++j) acc[i][j] = 0.0;
    for (int c = tid; c < p.H / 8; c += kRouteThreads) {
        uint4 r[kRouteExperts], x[kTT];
#pragma unroll
        for (int i = 0; i < kRouteExperts; ++i)
            r[i] = e0 + i < p.E ? __ldg(reinterpret_cast<const uint4*>(p.R + (size_t)(e0 + i) * p.H) + c)
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kTT; ++j)
            x[j] = t0 + j < p.T ? __ldg(reinterpret_cast<const uint4*>(p.X + (size_t)(t0 + j) * p.H) + c)
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            double xa[kTT], xb[kTT];
#pragma unroll
            for (int j = 0; j < kTT; ++j) {
                const float2 f = T::to_float2(reinterpret_cast<const uint32_t*>(&x[j])[w]);
                xa[j] = f.x;
                xb[j] = f.y;
            }
#pragma unroll
            for (int i = 0; i < kRouteExperts; ++i) {
                const float2 f = T::to_float2(reinterpret_cast<const uint32_t*>(&r[i])[w]);
                const double ra = f.x, rb = f.y;
#pragma unroll
                for (int j = 0; j < kTT; ++j) acc[i][j] = fma(rb, xb[j], fma(ra, xa[j], acc[i][j]));
            }
        }
    }
    // Sums over the warp: at each step a lane gives half of its values to its
    // partner and keeps the other half (16 exchanges for 16 values, not 80).
    constexpr int kV = kRouteExperts * kTT;
    double v[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = acc[i / kTT][i % kTT];
    int which = 0, d = 16;  // this lane's value in the end
#pragma unroll
    for (int n = kV / 2; n >= 1; n >>= 1, d >>= 1) {
        const bool up = lane & d;
        which += up ? n : 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const double give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
        }
    }
#pragma unroll
    for (; d >= 1; d >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
    if ((lane & (32 / kV - 1)) == 0) red[warp][which] = v[0];
    __syncthreads();
    if (tid < kRouteExperts * kTT) {
        const int e = e0 + tid / kTT, t = t0 + tid % kTT;
        double a = 0.0;
#pragma unroll
        for (int w = 0; w < kRouteThreads / 32; ++w) a += red[w][tid];
        if (e < p.E && t < p.T) __stcg(p.logits + (size_t)t * p.E + e, a);
    }
    __syncthreads();
    if (tid == 0) {
        const bool last = ticket_take(&p.tickets[tg]) == (unsigned)(eb - 1);
        if (last) p.tickets[tg] = 0;
        s_last = last;
    }
    for (int e = tid; e < kMaxExperts; e += kRouteThreads) chose[e][0] = chose[e][1] = 0;
    __syncthreads();
    if (!s_last) return;

    // the experts of token t0 + warp
    if (warp < kTT && t0 + warp < p.T) {
        const int t = t0 + warp;
        constexpr int kPer = kMaxExperts / 32;
        double l[kPer];
        unsigned long long key[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < p.E ? __ldcg(p.logits + (size_t)t * p.E + e) : 0.0;
            key[i] = score_key(l[i]);
        }
        unsigned gone = 0;  // this lane's experts already chosen (or past E)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i >= p.E) gone |= 1u << i;
        double top = 0.0;       // the largest score
        float mine = 0.0f;      // lane j: e^(l - top) of choice j
        int mine_id = 0;
        for (int j = 0; j < p.top_k; ++j) {
            unsigned long long best = 0;
            int at = kMaxExperts;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i)  // downwards: an equal key at a lower index wins
                if (!((gone >> i) & 1u) && key[i] >= best) {
                    best = key[i];
                    at = lane + 32 * i;
                }
            const unsigned hi = __reduce_max_sync(0xffffffffu, at < kMaxExperts ? (unsigned)(best >> 32) : 0u);
            const bool in_hi = at < kMaxExperts && (unsigned)(best >> 32) == hi;
            const unsigned lo = __reduce_max_sync(0xffffffffu, in_hi ? (unsigned)best : 0u);
            const int e = (int)__reduce_min_sync(
                0xffffffffu, in_hi && (unsigned)best == lo ? (unsigned)at : (unsigned)kMaxExperts);
            double le = 0.0;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i == e) {
                    gone |= 1u << i;
                    le = l[i];
                }
            le = __shfl_sync(0xffffffffu, le, e & 31);
            if (j == 0) top = le;
            if (lane == j) {
                mine = expf((float)(le - top));
                mine_id = e;
            }
        }
        float sum = 0.0f;
        if (p.renorm) {
            sum = lane < p.top_k ? mine : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < p.E) sum += expf((float)(l[i] - top));
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane < p.top_k) {
            __stcg(p.ids + (size_t)t * p.top_k + lane, mine_id);
            __stcg(p.wts + (size_t)t * p.top_k + lane, __fdiv_rn(mine, sum));
            atomicOr(&chose[mine_id][t >> 5], 1u << (t & 31));  // all there is to list if these are the only tokens
        }
    }
    const int groups = (p.T + kTT - 1) / kTT;
    __syncthreads();
    if (groups > 1) {
        if (tid == 0) {
            const bool last = ticket_take(&p.tickets[groups]) == (unsigned)(groups - 1);
            if (last) p.tickets[groups] = 0;
            s_last = last;
        }
        __syncthreads();
        if (!s_last) return;
        for (int i = tid; i < p.T * p.top_k; i += kRouteThreads) {
            const int t = i / p.top_k;
            atomicOr(&chose[__ldcg(p.ids + i)][t >> 5], 1u << (t & 31));
        }
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        for (int e = lane; e < kMaxExperts; e += 32) {
            const unsigned lo = chose[e][0], hi = chose[e][1];
            const unsigned m = __ballot_sync(0xffffffffu, (lo | hi) != 0);
            if (lo | hi) {
                const int at = n + __popc(m & ((1u << lane) - 1u));
                p.active[1 + at] = e;
                p.masks[at] = (unsigned long long)hi << 32 | lo;
            }
            n += __popc(m);
        }
        if (lane == 0) p.active[0] = n;
    }
}

}  // namespace i8mm
