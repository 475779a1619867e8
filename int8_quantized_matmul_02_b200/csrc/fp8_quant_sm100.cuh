// Block-scaled e4m3 codes of activations (one scale per row and block of 128
// consecutive k) and of weights (one scale per 128 x 128 block); the rule is
// in fp8_common.cuh.
//
// Activations: bound by HBM, 2 bytes read and 1 written per value, if the
// instructions per value are few.  A block of 128 16-bit values is held by 8
// lanes in registers, 8 values of either half of the block each (so that both
// loads of a warp are whole lines); its maximum takes packed 16-bit
// instructions and three shuffles, its scale no division, and where the next
// block lies is found by additions.  kQuantBlocks blocks are in flight per
// group of 8 lanes.  4096 x 12288: 25.8 us a launch, 5.9 TB/s (0.90 of a plain
// copy); calls back to back 26.5 us in runs of 20 ms (0.88), 27.6 us in runs of
// seconds (0.84, at 1.77 GHz under the power cap).  With divisions for a block's
// scale and position and 16 lanes a block it was 40.7 us, bound by issue.
#pragma once

#include "fp8_common.cuh"

namespace i8mm {

constexpr int kQuantBlocks = 2;    // blocks of 128 in flight per group of 8 lanes
constexpr int kQuantThreads = 256;

// Group `gr` of `ngr` groups of 8 lanes takes blocks gr, gr + ngr, ... of the
// M x KB blocks (row-major; ngr a multiple of 4).  scale(m, b) goes to
// scales[m * sm + b * sb].
template <typename T>
__device__ __forceinline__ void quant_fp8_blocks(const uint16_t* __restrict__ X, long long nblocks, int K, int KB,
                                                 uint8_t* __restrict__ codes, float* __restrict__ scales, long long sm,
                                                 long long sb, long long gr, long long ngr) {
    const int sub = threadIdx.x & 7;
    const long long dm = ngr / KB;
    const int dk = (int)(ngr - dm * KB);
    long long m = gr / KB, b = gr;
    int kb = (int)(gr - m * KB);
    // every group of a warp runs the same number of rounds: the shuffles below
    // stay inside a group but name the whole warp
    for (long long w0 = gr - ((threadIdx.x >> 3) & 3); w0 < nblocks; w0 += ngr * kQuantBlocks) {
        uint4 x[kQuantBlocks][2];
        long long at[kQuantBlocks], sat[kQuantBlocks];
        bool in[kQuantBlocks][2];
#pragma unroll
        for (int i = 0; i < kQuantBlocks; ++i) {
            const int k = kb * 128 + sub * 8;
            at[i] = m * K + k;
            sat[i] = m * sm + kb * sb;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                in[i][h] = b < nblocks && k + 64 * h < K;  // K % 16 == 0: all 8 values or none
                x[i][h] = make_uint4(0, 0, 0, 0);
                if (in[i][h]) x[i][h] = __ldg(reinterpret_cast<const uint4*>(X + at[i] + 64 * h));
            }
            b += ngr;
            m += dm;
            kb += dk;
            if (kb >= KB) {
                kb -= KB;
                ++m;
            }
        }
#pragma unroll
        for (int i = 0; i < kQuantBlocks; ++i) {
            float a = T::pair_max(fp8_amax8<T>(fp8_amax8<T>(T::as_pair(0u), x[i][0]), x[i][1]));
#pragma unroll
            for (int d = 4; d >= 1; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
            const float s = fp8_block_scale16(a), inv = __frcp_rn(s);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (in[i][h]) *reinterpret_cast<uint2*>(codes + at[i] + 64 * h) = fp8_codes8<T>(x[i][h], inv);
            if (sub == 0 && in[i][0]) scales[sat[i]] = s;
        }
    }
}

// grid-stride over the blocks; launched with PDL (it waits before it reads).
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    k_quant_fp8(const uint16_t* __restrict__ X, long long nblocks, int K, int KB, uint8_t* __restrict__ codes,
                float* __restrict__ scales, long long sm, long long sb) {
    pdl_wait();
    pdl_launch_dependents();
    const long long gr = ((long long)blockIdx.x * kQuantThreads + threadIdx.x) >> 3;
    quant_fp8_blocks<T>(X, nblocks, K, KB, codes, scales, sm, sb, gr, (long long)gridDim.x * (kQuantThreads / 8));
}

// One 128 x 128 block of a weight per thread block: W is K x N (row-major, 16
// bits), the codes N x K, scales[n_block * KB + k_block].  Once, at load.
template <typename T>
__global__ void __launch_bounds__(256)
    k_quant_weight_fp8(const uint16_t* __restrict__ W, int K, int N, uint8_t* __restrict__ codes,
                       float* __restrict__ scales) {
    __shared__ uint16_t tile[128][130];  // [k][n]
    __shared__ float red[8];
    const int k0 = blockIdx.y * 128, n0 = blockIdx.x * 128;
    const int nk = min(128, K - k0), nn = min(128, N - n0);
    float a = 0.0f;
    for (int i = threadIdx.x; i < 128 * 64; i += 256) {
        const int k = i >> 6, n = (i & 63) * 2;
        uint32_t w = 0;
        if (k < nk && n < nn) w = *reinterpret_cast<const uint32_t*>(W + (size_t)(k0 + k) * N + n0 + n);  // N even
        tile[k][n] = (uint16_t)w;
        tile[k][n + 1] = (uint16_t)(w >> 16);
        a = fmaxf(a, T::pair_max(T::abs_max(T::as_pair(0u), w)));
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, red[i]);
    const float s = fp8_block_scale(a), inv = __frcp_rn(s);
    if (threadIdx.x == 0) scales[(size_t)blockIdx.x * gridDim.y + blockIdx.y] = s;
    for (int i = threadIdx.x; i < 128 * 32; i += 256) {
        const int n = i >> 5, k = (i & 31) * 4;
        if (n < nn && k < nk) {
            const uint32_t q = e4m3x4(__fmul_rn(T::to_float(tile[k][n]), inv), __fmul_rn(T::to_float(tile[k + 1][n]), inv),
                                      __fmul_rn(T::to_float(tile[k + 2][n]), inv),
                                      __fmul_rn(T::to_float(tile[k + 3][n]), inv));
            *reinterpret_cast<uint32_t*>(codes + (size_t)(n0 + n) * K + k0 + k) = q;
        }
    }
}

}  // namespace i8mm
