// Block-scaled e4m3 GEMM on SM pairs (cta_group::2):
//
//   acc_b[m, n] = sum_{k in block b} xq[m, k] * wq[n, k]      tcgen05 kind::f8f6f4, fp32 in TMEM
//   v[m, n]     = sum_b acc_b[m, n] * (xs[m, b] * ws[n / 128, b])   fp32, ascending b
//   Y[m, n]     = 16-bit(v[m, n])
//
// The scales change every 128 k and are not powers of two, so a block's sum
// has to leave the tensor cores before the next block is added: every 128 k
// the accumulator is read back and added to running sums in registers.  Two
// TMEM accumulators alternate, so that this runs beside the next block's MMAs.
// What it costs per block and SM: a 128 x kBN tile is 128 * kBN FMAs against
// 128 * kBN * 128 MACs, and a column of TMEM words per lane quadrant and FMA.
// The 256 x 256 pair tile (a row of 128 columns per epilogue thread) is the
// largest whose sums fit the registers: 128 sums and 32 columns being added
// per thread.  It also halves the operand bytes that a pair stages per MAC
// against 256 x 128.
//   warp 0      TMA producer (both CTAs; completion on the even CTA's barrier);
//   warp 1      TMEM allocation (512 columns) and, in the even CTA, MMA issue;
//   warps 2-9   epilogue: TMEM lane quadrant w % 4, column half (w - 2) / 4.
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
    const float* xs;               // KB x xs_pitch: xs[b * xs_pitch + m]
    long long xs_pitch;
    const float* ws;               // ceil(N / 128) x KB
    int* status;
    uint64_t wait_limit_ns;
    uint32_t test_flags;           // bit 0: never signal the first accumulator (timeout test)
};

constexpr int kF8BM = 256;
constexpr int kF8Stages = 5;
constexpr int kF8EpiWarps = 8;
constexpr int kF8Threads = 64 + 32 * kF8EpiWarps;
constexpr int kF8Ahead = 4;        // blocks whose scales are fetched ahead
constexpr int kF8Slots = 2 * kF8Ahead;
constexpr int kF8ScaleBytes = kF8Slots * (32 + 4) * 4;  // per epilogue warp

__host__ __device__ constexpr int f8_stage_bytes(int bn) { return 128 * 128 + (bn / 2) * 128; }
__host__ __device__ constexpr int f8_smem_bytes(int bn) {
    return 1024 + kF8Stages * f8_stage_bytes(bn) + kF8EpiWarps * (kGemmEpiBufBytes + kF8ScaleBytes) + 256;
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

// v[0..31] += acc[0..31] * s, two lanes per instruction.
__device__ __forceinline__ void fma32(float* v, const uint32_t (&r)[32], float s) {
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        asm("{\n\t.reg .b64 x, y, z;\n\t"
            "mov.b64 x, {%2, %3};\n\t"
            "mov.b64 y, {%4, %4};\n\t"
            "mov.b64 z, {%0, %1};\n\t"
            "fma.rn.f32x2 z, x, y, z;\n\t"
            "mov.b64 {%0, %1}, z;\n\t}"
            : "+f"(v[i]), "+f"(v[i + 1])
            : "f"(__uint_as_float(r[i])), "f"(__uint_as_float(r[i + 1])), "f"(s));
}

// 32 fp32 values of one row to 16 bits, into half of the row's 128-byte line
// of a staging buffer with the 128-byte swizzle.
template <typename T>
__device__ __forceinline__ void stage_row32_t(uint8_t* buf, int row, int half32, const float* v) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 w;
        w.x = T::pack(v[8 * c + 0], v[8 * c + 1]);
        w.y = T::pack(v[8 * c + 2], v[8 * c + 3]);
        w.z = T::pack(v[8 * c + 4], v[8 * c + 5]);
        w.w = T::pack(v[8 * c + 6], v[8 * c + 7]);
        const int chunk = half32 * 4 + c;
        *reinterpret_cast<uint4*>(buf + row * 128 + ((chunk ^ (row & 7)) << 4)) = w;
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
    float* sscale = reinterpret_cast<float*>(epi + kF8EpiWarps * kGemmEpiBufBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(epi + kF8EpiWarps * (kGemmEpiBufBytes + kF8ScaleBytes));
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

    if (warp < 2) {
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
                        if (!wait_bounded_cluster(&empty[stage], phase ^ 1, wctx)) {
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
        } else {
            // ------------------------------------------------ MMA issuer (even CTA)
            if (rank == 0 && elect_one()) {
                const uint32_t idesc = idesc_e4m3_f32(kF8BM, kBN);
                int stage = 0, acc = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool ok = true, issued = false;
                for (int tile = cid; tile < p.num_tiles && ok; tile += ncl) {
                    for (int kb = 0; kb < p.KB; ++kb) {
                        if (!wait_bounded_cluster(&tempty[acc], acc_phase ^ 1, wctx) ||
                            !wait_bounded(&full[stage], phase, wctx)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(ring + stage * kStageBytes);
                        mma_e4m3_k128_2sm(tmem_base + (uint32_t)(acc * 256), sdesc_k128sw(sa),
                                          sdesc_k128sw(sa + 128 * 128), idesc);
                        issued = true;
                        tc_commit_pair(&empty[stage]);
                        if (!((p.test_flags & 1u) && tile == cid && kb == 0)) tc_commit_pair(&tfull[acc]);
                        if (++stage == kF8Stages) {
                            stage = 0;
                            phase ^= 1;
                        }
                        acc ^= 1;
                        acc_phase ^= (acc == 0);
                    }
                }
                if (issued) {  // every pair MMA has retired before TMEM is freed
                    tc_commit_pair(drain);
                    wait_drain(drain, 0, kDrainLimitNs);
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2..9, both CTAs)
        const int ew = warp - 2;
        const int quad = warp & 3, half = ew >> 2;
        uint8_t* buf = epi + ew * kGemmEpiBufBytes;
        float* slots = sscale + ew * (kF8ScaleBytes / 4);  // [slots] of 32 xs and one ws (padded to 36)
        const uint32_t tempty0 = map_to_rank(&tempty[0], 0), tempty1 = map_to_rank(&tempty[1], 0);
        int acc = 0;
        uint32_t acc_phase = 0;
        uint32_t fetched = 0, used = 0;  // running counts of scale groups
        bool ok = true;
        // scales of the kb-th block from a tile's start to the next slot (an
        // empty group past the last tile)
        const auto fetch = [&](int tile, int kb) {
            while (kb >= p.KB && tile < p.num_tiles) {  // on into this pair's next tiles
                kb -= p.KB;
                tile += ncl;
            }
            if (tile < p.num_tiles) {
                int mb, nb;
                coords(tile, mb, nb);
                const int row = mb * kF8BM + (int)rank * 128 + quad * 32 + lane;
                const int nblk = (nb * kBN + half * kCols) >> 7;
                float* s = slots + (fetched & (kF8Slots - 1)) * 36;
                const bool row_in = row < p.M, blk_in = nblk * 128 < p.N;
                const float* src = p.xs + (row_in ? (size_t)kb * p.xs_pitch + row : 0);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(s + lane)), "l"(src),
                             "r"(row_in ? 4 : 0)
                             : "memory");
                if (lane == 0) {
                    const float* sw = p.ws + (blk_in ? (size_t)nblk * p.KB + kb : 0);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(s + 32)), "l"(sw),
                                 "r"(blk_in ? 4 : 0)
                                 : "memory");
                }
            }
            ++fetched;
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < kF8Ahead; ++i) fetch(cid, i);
        for (int tile = cid; tile < p.num_tiles && ok; tile += ncl) {
            int mb, nb;
            coords(tile, mb, nb);
            const int row0 = mb * kF8BM + (int)rank * 128 + quad * 32;
            const int colw = nb * kBN + half * kCols;
            float v[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] = 0.0f;
            for (int kb = 0; kb < p.KB; ++kb) {
                fetch(tile, kb + kF8Ahead);
                asm volatile("cp.async.wait_group %0;" ::"n"(kF8Ahead) : "memory");
                __syncwarp();
                const float* s = slots + (used & (kF8Slots - 1)) * 36;
                const float sc = __fmul_rn(s[lane], s[32]);
                ++used;
                if (!__all_sync(0xffffffffu, wait_bounded_inline<true>(&tfull[acc], acc_phase, wctx))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t t = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * 256 + half * kCols);
                uint32_t r[32];
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    tmem_ld32(t + c, r);
                    tmem_wait_ld32(r);
                    if (c + 32 == kCols) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)  // the accumulator is free
                            asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                             acc ? tempty1 : tempty0)
                                         : "memory");
                    }
                    fma32(v + c, r, sc);
                }
                acc ^= 1;
                acc_phase ^= (acc == 0);
            }
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < kCols; c += 64) {
                if (lane == 0) bulk_wait_read<0>();  // the buffer's last store has read it
                __syncwarp();
                stage_row32_t<TOut>(buf, lane, 0, v + c);
                stage_row32_t<TOut>(buf, lane, 1, v + c + 32);
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

    if (threadIdx.x == 0 && *abort_flag) settle_after_abort();  // copies issued before the abort land first
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // the even CTA's MMAs no longer read this CTA's shared memory or TMEM
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace i8mm
