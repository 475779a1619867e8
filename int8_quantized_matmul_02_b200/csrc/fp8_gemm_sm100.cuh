// Block-scaled e4m3 GEMM on SM pairs (cta_group::2):
//
//   acc_b[m, n] = sum_{k in block b} xq[m, k] * wq[n, k]      tcgen05 kind::f8f6f4, fp32 in TMEM
//   v[m, n]     = sum_b acc_b[m, n] * (xs[m, b] * ws[n / 128, b])   fp32, ascending b
//   Y[m, n]     = 16-bit(v[m, n])
//
// The scales change every 128 k and are not powers of two, so a block's sum
// has to leave the tensor cores before the next block is added: every 128 k
// the accumulator is read back and added to running sums in registers, two
// columns per instruction.  Two TMEM accumulators alternate, so that this runs
// beside the next block's MMAs.
//
// What bounds it is the way round that one accumulator takes: MMAs (565
// cycles a block), completion seen by the epilogue (~450), reading it back and
// adding (~300), release seen by the issuing thread (~220), issue (~150).
// With two accumulators a block takes half of that, ~850 cycles, against the
// MMAs' 565; TMEM (512 columns) holds no third.  4096 x 12288 x 49152 takes
// 2.31 ms (2.14 PFLOP/s, 0.65 of twice the measured bf16 rate) and 2048 x 8192
// x 28672 0.465 ms in runs of 20 ms; in runs of seconds the power cap holds the
// clock at 1.43 and 1.51 GHz, and they take 2.68 to 2.79 and 0.54 to 0.55 ms.
// (Other boxes: 2.26 to 2.40 and 0.457 to 0.482 in short runs.)  Measured and not kept,
// for the first (2.22 ms then and there): the two column halves as separate
// accumulators of 128 columns (2.48 ms: MMAs of N = 128 run at a lower rate);
// 16 epilogue warps of 64 columns (2.41 ms: more threads to see the
// completion and to release); the scale products made by two other warps
// (2.58 ms: the scale is read after the completion instead of before).
// The 256 x 256 pair tile is the largest whose sums fit the registers: 128
// sums and two loads of 32 columns per thread, with the register file split by
// setmaxnreg.
//   warp 0      TMA producer (both CTAs; completion on the even CTA's barrier);
//   warp 1      TMEM allocation (512 columns) and, in the even CTA, MMA issue;
//   warps 2-3   idle (they complete the group of four that gives up registers);
//   warps 4-11  epilogue: TMEM lane quadrant w % 4, column half (w - 4) / 4.
// The scales of the next four blocks are copied to shared memory ahead of use
// (cp.async, one group per block); half of a tile's columns lie in one block
// of 128 channels, so a thread needs one xs and one ws per block.
#pragma once

#include "fp8_common.cuh"
#include "gemm_sm100.cuh"

namespace i8mm {

struct Fp8GemmParams {
    int M, N, KB;                  // KB = ceil(K / 128)
    int num_m_blocks, num_n_blocks, num_tiles, group_m;
    const float* xs;               // KB x xs_pitch: xs[b * xs_pitch + m]; the pitch is a multiple of 256
    long long xs_pitch;
    const float* ws;               // ceil(N / 128) x KB
    int* status;
    uint64_t wait_limit_ns;
    uint32_t test_flags;           // bit 0: never signal the first accumulator (timeout test)
};

constexpr int kF8BM = 256;
constexpr int kF8Stages = 5;
constexpr int kF8EpiWarps = 8;
constexpr int kF8Threads = 128 + 32 * kF8EpiWarps;
constexpr int kF8EpiRegs = 232, kF8CtlRegs = 40;  // registers per thread after the split
constexpr int kF8LaunchRegs = 168;                // and before it
static_assert(kF8EpiWarps * kF8EpiRegs + 4 * kF8CtlRegs <= (kF8EpiWarps + 4) * kF8LaunchRegs, "register split");
constexpr int kF8Ahead = 4;        // blocks whose scales are fetched ahead
constexpr int kF8Slots = 2 * kF8Ahead;
constexpr int kF8ScaleBytes = kF8Slots * (32 + 4) * 4;  // per epilogue warp
constexpr int kF8EpiBufBytes = 32 * 64;           // 32 rows x 32 16-bit columns

__host__ __device__ constexpr int f8_stage_bytes(int bn) { return 128 * 128 + (bn / 2) * 128; }
__host__ __device__ constexpr int f8_smem_bytes(int bn) {
    return 1024 + kF8Stages * f8_stage_bytes(bn) + kF8EpiWarps * (kF8EpiBufBytes + kF8ScaleBytes) + 256;
}
static_assert(f8_smem_bytes(256) <= 232448, "shared memory of one SM");

// Waits for this thread's TMEM loads; the registers are operands so that no
// use of them can be moved before the wait.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// Running sums are kept as pairs in 64-bit registers: an fma.rn.f32x2 on
// separate 32-bit sums costs moves into and out of register pairs (measured:
// 357 instructions per warp and block against the FMAs' 64).
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f32x2_parts(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ void fma_f32x2(uint64_t& acc, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

// v[0..15] (32 sums) += acc[0..31] * s.
__device__ __forceinline__ void fma32(uint64_t* v, const uint32_t (&r)[32], uint64_t s2) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
        fma_f32x2(v[i], f32x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), s2);
}

// 32 fp32 values of one row to 16 bits, into the row's 64-byte line of a
// staging buffer with the 64-byte swizzle.
template <typename T>
__device__ __forceinline__ void stage_row32_t(uint8_t* buf, int row, const uint64_t* v) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = f32x2_parts(v[4 * c + i]);
            h[i] = T::pack(f.x, f.y);
        }
        *reinterpret_cast<uint4*>(buf + row * 64 + ((c ^ ((row >> 1) & 3)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

template <int kBN, typename TOut>
__global__ void __launch_bounds__(kF8Threads, 1)
    k_gemm_fp8_2sm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_y, const Fp8GemmParams p) {
    constexpr int kStageBytes = f8_stage_bytes(kBN);
    constexpr int kCols = kBN / 2;  // columns per epilogue thread
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = smem;
    uint8_t* epi = smem + kF8Stages * kStageBytes;
    float* sscale = reinterpret_cast<float*>(epi + kF8EpiWarps * kF8EpiBufBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(epi + kF8EpiWarps * (kF8EpiBufBytes + kF8ScaleBytes));
    uint64_t* full = bars;                    // [stages] even CTA: both CTAs' bytes
    uint64_t* empty = bars + kF8Stages;       // [stages] each CTA: its stage is free
    uint64_t* tfull = bars + 2 * kF8Stages;   // [2] each CTA: a block's sums are ready
    uint64_t* tempty = tfull + 2;             // [2] even CTA: both epilogues have read the accumulator
    uint64_t* drain = tfull + 4;              // [1]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0 = the CTA that issues the MMAs
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};
    const auto coords = [&](int tile, int& mb, int& nb) {
        const int group_size = p.group_m * p.num_n_blocks;
        const int g = tile / group_size;
        const int first_m = g * p.group_m;
        const int gm = min(p.group_m, p.num_m_blocks - first_m);
        const int local = tile - g * group_size;
        mb = first_m + local % gm;
        nb = local / gm;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kF8Stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * kF8EpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_a);
        prefetch_tmap(&tm_b);
        prefetch_tmap(&tm_y);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers and TMEM are ready
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    pdl_wait();  // the codes and scales of X come from the kernel before
    pdl_launch_dependents();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8CtlRegs));
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (both CTAs)
            if (elect_one()) {
                const uint64_t pol_a = policy_evict_last();
                const uint64_t pol_b = policy_evict_first();
                int stage = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int tile = cid; tile < p.num_tiles && ok; tile += ncl) {
                    int mb, nb;
                    coords(tile, mb, nb);
                    const int row_a = mb * kF8BM + (int)rank * 128;
                    const int row_b = nb * kBN + (int)rank * (kBN / 2);
                    for (int kb = 0; kb < p.KB; ++kb) {
                        if (!wait_fast(&empty[stage], phase ^ 1, wctx)) {
                            ok = false;
                            break;
                        }
                        uint8_t* sa = ring + stage * kStageBytes;
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
                        const uint32_t fbar = map_to_rank(&full[stage], 0);
                        tma_load_2d_pair(sa, &tm_a, fbar, kb * 128, row_a, pol_a);
                        tma_load_2d_pair(sa + 128 * 128, &tm_b, fbar, kb * 128, row_b, pol_b);
                        if (++stage == kF8Stages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer (even CTA)
            if (rank == 0 && elect_one()) {
                const uint32_t idesc = idesc_e4m3_f32(kF8BM, kBN);
                int stage = 0;
                uint32_t phase = 0;
                bool issued = false;
                const uint32_t blocks = (uint32_t)((p.num_tiles - cid + ncl - 1) / ncl) * (uint32_t)p.KB;
                // a look at a barrier takes ~170 cycles while the tensor core reads
                // shared memory, so the next stage's is taken during this block's issue
                bool loaded = false;
                for (uint32_t q = 0; q < blocks; ++q) {
                    const uint32_t acc = q & 1;
                    if (!wait_fast(&tempty[acc], ((q >> 1) & 1) ^ 1, wctx)) break;
                    if (!loaded && !wait_fast(&full[stage], phase, wctx)) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ring + stage * kStageBytes);
                    mma_e4m3_k128_2sm(tmem_base + acc * 256, sdesc_k128sw(sa), sdesc_k128sw(sa + 128 * 128), idesc);
                    issued = true;
                    if (!((p.test_flags & 1u) && q == 0)) tc_commit_pair(&tfull[acc]);
                    tc_commit_pair(&empty[stage]);
                    if (++stage == kF8Stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    loaded = mbar_try_wait(&full[stage], phase);
                }
                if (issued) {  // every pair MMA has retired before TMEM is freed
                    tc_commit_pair(drain);
                    wait_drain_inline(drain, 0, kDrainLimitNs);
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue (warps 4..11, both CTAs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8EpiRegs));
        const int ew = warp - 4;
        const int quad = warp & 3, half = ew >> 2;
        uint8_t* buf = epi + ew * kF8EpiBufBytes;
        float* slots = sscale + ew * (kF8ScaleBytes / 4);  // [slots] of 32 xs and one ws (padded to 36)
        const uint32_t tempty0 = map_to_rank(&tempty[0], 0), tempty1 = map_to_rank(&tempty[1], 0);
        const uint32_t tcol = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * kCols);
        uint32_t fetched = 0;  // scale groups so far
        uint32_t q = 0;        // blocks so far: accumulator q & 1
        bool ok = true;
        // the stream of scales: tile, block and source of the next fetch
        int ft = cid - ncl, fk = p.KB;
        const float *fx = nullptr, *fw = nullptr;
        int fw_bytes = 0;
        // the next block's scales to the next slot (an empty group past the last tile)
        const auto fetch = [&]() {
            if (fk == p.KB) {
                ft += ncl;
                fk = 0;
                if (ft < p.num_tiles) {
                    int mb, nb;
                    coords(ft, mb, nb);
                    const int nblk = (nb * kBN + half * kCols) >> 7;
                    fx = p.xs + mb * kF8BM + (int)rank * 128 + quad * 32 + lane;  // rows past M: in the pitch, unused
                    fw_bytes = nblk * 128 < p.N ? 4 : 0;
                    fw = p.ws + (fw_bytes ? (size_t)nblk * p.KB : 0);
                }
            }
            if (ft < p.num_tiles) {
                float* s = slots + (fetched & (kF8Slots - 1)) * 36;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(s + lane)), "l"(fx) : "memory");
                if (lane == 0)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(s + 32)), "l"(fw),
                                 "r"(fw_bytes)
                                 : "memory");
                fx += p.xs_pitch;
                ++fw;
                ++fk;
            }
            ++fetched;
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < kF8Ahead; ++i) fetch();
        for (int tile = cid; tile < p.num_tiles && ok; tile += ncl) {
            uint64_t v[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) v[i] = 0;
            for (int kb = 0; kb < p.KB; ++kb, ++q) {
                fetch();
                asm volatile("cp.async.wait_group %0;" ::"n"(kF8Ahead) : "memory");
                __syncwarp();
                const float* sl = slots + (q & (kF8Slots - 1)) * 36;
                const float s1 = __fmul_rn(sl[lane], sl[32]);
                const uint64_t s = f32x2(s1, s1);
                if (!__all_sync(0xffffffffu, wait_fast(&tfull[q & 1], (q >> 1) & 1, wctx))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t t = tcol + ((q & 1) << 8);
                const auto release = [&]() {  // the accumulator is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                         (q & 1) ? tempty1 : tempty0)
                                     : "memory");
                };
                // one load of 32 columns in flight beside the FMAs of the 32 before
                uint32_t ra[32], rb[32];
                tmem_ld32(t, ra);
                tmem_wait_ld32(ra);
#pragma unroll
                for (int c = 0; c < kCols; c += 64) {
                    tmem_ld32(t + c + 32, rb);
                    fma32(v + c / 2, ra, s);
                    tmem_wait_ld32(rb);
                    if (c + 64 < kCols) {
                        tmem_ld32(t + c + 64, ra);
                        fma32(v + c / 2 + 16, rb, s);
                        tmem_wait_ld32(ra);
                    } else {
                        release();
                        fma32(v + c / 2 + 16, rb, s);
                    }
                }
            }
            if (!ok) break;
            int mb, nb;
            coords(tile, mb, nb);
            const int row0 = mb * kF8BM + (int)rank * 128 + quad * 32;
            const int colw = nb * kBN + half * kCols;
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
                if (lane == 0) bulk_wait_read<0>();  // the buffer's last store has read it
                __syncwarp();
                stage_row32_t<TOut>(buf, lane, v + c / 2);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (colw + c < p.N && row0 < p.M) tma_store_2d(&tm_y, buf, colw + c, row0);
                    bulk_commit();
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // no copy into shared memory outlives the loop
        if (lane == 0) bulk_wait_all<0>();
        __syncwarp();
    }

    if (threadIdx.x == 0 && *abort_flag) settle_inline();  // copies issued before the abort land first
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // the even CTA's MMAs no longer read this CTA's shared memory or TMEM
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace i8mm
