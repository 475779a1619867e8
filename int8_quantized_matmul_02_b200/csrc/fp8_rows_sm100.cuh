// Block-scaled e4m3 products for few rows: the weights are streamed once and
// HBM is the bound, so what matters is that every SM streams, and streams the
// same share.
//
//   out[m, n] = sum_b (xs[m, b] * ws[n / 128, b]) * sum_{k in block b} xq[m, k] * wq[n, k]
//
// Swapped operands: a 128-channel x 128-k box of the weight (16 KB, one 128 x
// 128 scale block) is the A operand of tcgen05.mma (M = 128), the rows of X
// are B (N = kNT >= rows).  A unit of work is one box (two in the gated
// layer) with the rows' 128 k; its sums go to one of four TMEM accumulators,
// and the epilogue thread of channel n (TMEM lane n) adds them, scaled, to one
// running fp32 sum per row in registers.
//
// The units, ordered by output tile and then k, are cut into equal consecutive
// shares, one per CTA (one CTA per SM), whatever the shape: a CTA's share may
// start and end inside a tile.  A tile that several CTAs share is finished by
// the last of them to arrive (a ticket per tile): every one stores its fp32
// sums, and the last adds them in the order of k, so the result does not
// depend on who came last.  No CTA waits for another.
//
// Three products are made of this:
//   kRows    Y = X W;
//   kGateUp  per chosen expert h = silu(X Wg) * (X Wu), two boxes per unit, h
//            in codes: a tile's 128 channels are one block of 128 of the next
//            product, so its scale is a maximum over the tile;
//   kDown    Y = sum over experts of weight * (h Wd): the experts' products
//            are one product over the concatenated k of the chosen experts,
//            with the routing weight in the scale, so the weighted sum of a
//            token's experts happens in the same running sums.
// In the gated layer every token takes a column of B for every expert; tokens
// that did not choose an expert have zero codes there.
//
//   warp 0     TMA producer of the weight boxes (and of B unless kFuse);
//   warp 1     TMEM allocation and MMA issue;
//   warps 2-5  every fourth unit each: the unit's scale products into shared
//              memory, and with kFuse the rows' codes (the rows' 16-bit values
//              are read, quantised and written to the swizzled B operand);
//   warps 6-   epilogue, TMEM lane quadrant w % 4: four warps, or eight with
//              half of the rows each where a thread would have to hold more
//              than 64 sums (128 of them spilled: 85 us for 100 x 11008 x 4096).
#pragma once

#include "fp8_common.cuh"
#include "fp8_gemm_sm100.cuh"

namespace i8mm {

enum { kRows = 0, kGateUp = 1, kDown = 2 };

struct Fp8RowsParams {
    int M;                 // rows of X (tokens)
    int N;                 // output channels
    int K;
    int KB;                // ceil(K / 128)
    int NB;                // ceil(N / 128)
    int MB;                // kRows: ceil(M / kNT) row blocks; else 1
    const uint16_t* X;     // kFuse: M x K
    const float* xs;       // else: scale of row m, block b at [b * xs_pitch + m]; kDown: [(a * KB + b) * xs_pitch + m]
    long long xs_pitch;
    const float* ws;       // NB x KB (kGateUp, kDown: per expert)
    const float* ws2;      // kGateUp: the up weight's
    const int32_t* active; // kGateUp, kDown: count, then the chosen experts in ascending order
    const int32_t* ids;    // M x top_k chosen experts and their weights
    const float* wts;
    int top_k;
    void* Y;               // kRows, kDown: M x N, 16 bits
    uint8_t* hq;           // kGateUp: codes [a][M][N], scales [(a * NB + nb) * M + m]
    float* hs;
    float* parts;          // two slots of kA x kNT x 128 floats per CTA
    unsigned* tickets;     // one per tile, zero between calls
    int* status;
    uint64_t wait_limit_ns;
    uint32_t test_flags;   // bit 0: block 0 never signals its first accumulator (timeout test)
};

constexpr int kFRBufs = 4;       // TMEM accumulators in rotation
constexpr int kFRSideWarps = 4;
constexpr int kFRMinUnits = 4;   // a share smaller than this costs more in joining than it saves
constexpr int kFRMaxCtas = 160;  // shares (a fixed bound, so that the workspace depends on the shape only)

template <int kMode>
__host__ __device__ constexpr int fr_a() { return kMode == kGateUp ? 2 : 1; }
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_epi_warps() { return fr_a<kMode>() * kNT > 64 ? 8 : 4; }
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_threads() { return 32 * (2 + kFRSideWarps + fr_epi_warps<kMode, kNT>()); }
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_stage_bytes() { return fr_a<kMode>() * 16384 + kNT * 128; }
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_h_bytes() { return kMode == kGateUp ? kNT * 132 * 4 : 0; }
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_stages() {
    int s = 12;
    while (1024 + s * (fr_stage_bytes<kMode, kNT>() + fr_a<kMode>() * kNT * 4 + 16) +
               kFRBufs * (fr_a<kMode>() * kNT * 4 + 16) + fr_h_bytes<kMode, kNT>() + 256 > 232448)
        --s;
    return s;
}
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_smem_bytes() {
    constexpr int s = fr_stages<kMode, kNT>();
    return 1024 + s * fr_stage_bytes<kMode, kNT>() + (s + kFRBufs) * fr_a<kMode>() * kNT * 4 +
           fr_h_bytes<kMode, kNT>() + (2 * s + 2 * kFRBufs + 1) * 8 + 64;
}

// Shares for `units` units in `tiles` tiles on at most `ctas` CTAs.
__host__ __device__ __forceinline__ int fr_shares(long long units, long long tiles, int ctas) {
    const long long want = units / kFRMinUnits > tiles ? units / kFRMinUnits : tiles;
    return (int)(want < ctas ? want : ctas);
}

template <int kMode, int kNT, bool kFuse, typename T>
__global__ void __launch_bounds__(fr_threads<kMode, kNT>(), 1)
    k_fp8_rows(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_w2,
               const __grid_constant__ CUtensorMap tm_x, const Fp8RowsParams p) {
    constexpr int kA = fr_a<kMode>();
    constexpr int kStageBytes = fr_stage_bytes<kMode, kNT>();
    constexpr int kStages = fr_stages<kMode, kNT>();
    constexpr int kSlots = kStages + kFRBufs;
    constexpr int kCols = kA * kNT;  // columns of an accumulator
    constexpr int kEpi = fr_epi_warps<kMode, kNT>(), kEpiThreads = 32 * kEpi;
    constexpr int kRowsT = kNT / (kEpi / 4);  // rows per epilogue thread
    constexpr int kSums = kA * kRowsT;        // running sums per epilogue thread
    constexpr uint32_t kTmemCols = kFRBufs * kCols < 32 ? 32 : kFRBufs * kCols;
    static_assert(kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM columns");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = smem;
    // scale products of the units in flight.  A slot is rewritten kSlots units
    // later; its writer has seen the MMAs of kStages units earlier done, and
    // those were issued after the epilogue had read the slot's last content
    // (an accumulator is released only once its scales have been read).
    float* slots = reinterpret_cast<float*>(ring + kStages * kStageBytes);
    float* hbuf = slots + kSlots * kCols;  // kGateUp: [kNT][132]
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(hbuf) + fr_h_bytes<kMode, kNT>());
    uint64_t* full = bars;
    uint64_t* empty = bars + kStages;
    uint64_t* tfull = bars + 2 * kStages;
    uint64_t* tempty = tfull + kFRBufs;
    uint64_t* drain = tempty + kFRBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* last_flag = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 2);  // the producer's expected bytes and the side warp
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kFRBufs; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], kEpi);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_w);
        if (kMode == kGateUp) prefetch_tmap(&tm_w2);
        if (!kFuse) prefetch_tmap(&tm_x);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // nothing is read before the work ahead on the stream is done, weights
    // included: a kernel there may have written them
    pdl_wait();
    pdl_launch_dependents();

    const int n_active = kMode == kRows ? 1 : p.active[0];
    const int kbt = kMode == kDown ? p.KB * n_active : p.KB;  // units per tile
    const long long tiles = kMode == kRows ? (long long)p.NB * p.MB
                            : kMode == kGateUp ? (long long)p.NB * n_active : (long long)p.NB;
    const long long units = tiles * kbt;
    const int C = fr_shares(units, tiles, (int)gridDim.x);
    const int c = (int)blockIdx.x;
    const long long u0 = c < C ? c * units / C : 0, u1 = c < C ? (c + 1) * units / C : 0;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (elect_one()) {
            const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
            int stage = 0;
            uint32_t phase = 0;
            int tile = (int)(u0 / kbt), kb = (int)(u0 - (long long)tile * kbt);
            for (long long u = u0; u < u1; ++u) {
                if (!wait_fast(&empty[stage], phase ^ 1, wctx)) break;
                uint8_t* sa = ring + stage * kStageBytes;
                uint8_t* sb = sa + kA * 16384;
                mbar_arrive_expect_tx(&full[stage], kFuse ? kA * 16384 : kStageBytes);
                if (kMode == kRows) {
                    tma_load_2d(sa, &tm_w, &full[stage], kb * 128, (tile / p.MB) * 128, pol_w);
                    if (!kFuse) tma_load_2d(sb, &tm_x, &full[stage], kb * 128, (tile % p.MB) * kNT, pol_x);
                } else if (kMode == kGateUp) {
                    const int e = p.active[1 + tile / p.NB], nb = tile % p.NB;
                    tma_load_3d(sa, &tm_w, &full[stage], kb * 128, nb * 128, e, pol_w);
                    tma_load_3d(sa + 16384, &tm_w2, &full[stage], kb * 128, nb * 128, e, pol_w);
                    tma_load_2d(sb, &tm_x, &full[stage], kb * 128, 0, pol_x);
                } else {
                    const int a = kb / p.KB, ib = kb - a * p.KB;
                    tma_load_3d(sa, &tm_w, &full[stage], ib * 128, tile * 128, p.active[1 + a], pol_w);
                    tma_load_3d(sb, &tm_x, &full[stage], ib * 128, 0, a, pol_x);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++kb == kbt) {
                    kb = 0;
                    ++tile;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (elect_one()) {
            const uint32_t idesc = idesc_e4m3_f32(128, kNT);
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool issued = false;
            for (long long u = u0; u < u1; ++u) {
                if (!wait_fast(&tempty[buf], buf_phase ^ 1, wctx) || !wait_fast(&full[stage], phase, wctx))
                    break;
                tc_fence_after();
                const uint32_t sa = smem_u32(ring + stage * kStageBytes);
                const uint64_t db = sdesc_k128sw(sa + kA * 16384);
                const uint32_t d = tmem_base + (uint32_t)(buf * kCols);
#pragma unroll
                for (int i = 0; i < kA; ++i)
                    mma_e4m3_k128(d + (uint32_t)(i * kNT), sdesc_k128sw(sa + i * 16384), db, idesc);
                issued = true;
                tc_commit(&empty[stage]);
                if (!((p.test_flags & 1u) && c == 0 && u == u0)) tc_commit(&tfull[buf]);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++buf == kFRBufs) {
                    buf = 0;
                    buf_phase ^= 1;
                }
            }
            if (issued) {  // every MMA has retired before TMEM is freed
                tc_commit(drain);
                wait_drain(drain, 0, kDrainLimitNs);
            }
        }
    } else if (warp >= 2 + kFRSideWarps) {
        // ------------------------------------------------ epilogue
        const int quad = warp & 3, ch = quad * 32 + lane;
        const int et = (int)threadIdx.x - 32 * (2 + kFRSideWarps);  // 0 .. kEpiThreads - 1
        const int r0 = (et >> 7) * kRowsT;                           // this thread's first row
        int buf = 0, slot = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        long long u = u0;
        while (u < u1) {
            const int tile = (int)(u / kbt);
            const long long t0 = (long long)tile * kbt, t1 = t0 + kbt;
            const long long end = u1 < t1 ? u1 : t1;
            const bool whole = u == t0 && end == t1, starts = u == t0;
            uint64_t v2[kSums / 2];  // pairs of rows
#pragma unroll
            for (int i = 0; i < kSums / 2; ++i) v2[i] = 0;
            for (; u < end; ++u) {
                // after a wait that ran out the loops go on without waiting, so
                // that every barrier and ticket below is still met
                if (ok) ok = __all_sync(0xffffffffu, wait_fast(&tfull[buf], buf_phase, wctx));
                tc_fence_after();
                const float* s = slots + slot * kCols + r0;
                const uint32_t t = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * kCols + r0);
#pragma unroll
                for (int a = 0; a < kA; ++a) {
                    if constexpr (kRowsT == 16) {
                        uint32_t r[16];
                        tmem_ld16(t + a * kNT, r);
                        asm volatile("tcgen05.wait::ld.sync.aligned;"
                                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                                       "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                                       "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
                        const ulonglong2* sa = reinterpret_cast<const ulonglong2*>(s + a * kNT);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const ulonglong2 f = sa[i];
                            fma_f32x2(v2[a * 8 + 2 * i], f32x2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), f.x);
                            fma_f32x2(v2[a * 8 + 2 * i + 1],
                                      f32x2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])), f.y);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < kRowsT; c += 32) {
                            uint32_t r[32];
                            tmem_ld32(t + (uint32_t)(a * kNT + c), r);
                            tmem_wait_ld32(r);
                            const ulonglong2* sa = reinterpret_cast<const ulonglong2*>(s + a * kNT + c);
                            uint64_t* vv = v2 + (a * kRowsT + c) / 2;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const ulonglong2 f = sa[i];
                                fma_f32x2(vv[2 * i], f32x2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), f.x);
                                fma_f32x2(vv[2 * i + 1],
                                          f32x2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])), f.y);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[buf]);
                if (++buf == kFRBufs) {
                    buf = 0;
                    buf_phase ^= 1;
                }
                if (++slot == kSlots) slot = 0;
            }

            bool finish = true;
            if (!whole) {
                // this CTA's sums of the tile; slot 0 for a tile that began in an
                // earlier share, slot 1 for one that begins here and goes on
                const int rows = (kMode == kRows ? min(kNT, p.M - (tile % p.MB) * kNT) : p.M) - r0;
                float2* part = reinterpret_cast<float2*>(p.parts + (size_t)(2 * c + (starts ? 1 : 0)) * (kCols * 128)) +
                               (size_t)(r0 / 2) * 128 + ch;  // rows in pairs: [kA][kNT / 2][128] of two
#pragma unroll
                for (int i = 0; i < kSums / 2; ++i) {
                    const int a = i / (kRowsT / 2), j = i % (kRowsT / 2);
                    if (2 * j < rows) __stcg(part + (size_t)(a * (kNT / 2) + j) * 128, f32x2_parts(v2[i]));
                }
                __threadfence();
                named_bar_sync(1, kEpiThreads);
                // the CTA that owns unit x is floor(((x + 1) C - 1) / units)
                const int cf = (int)(((t0 + 1) * C - 1) / units), cl = (int)((t1 * C - 1) / units);
                if (et == 0) {
                    const unsigned old = atomicAdd(&p.tickets[tile], 1u);
                    const bool last = old == (unsigned)(cl - cf);
                    if (last) p.tickets[tile] = 0;  // ready for the next call
                    *last_flag = last;
                }
                named_bar_sync(1, kEpiThreads);
                finish = *last_flag != 0;
                if (finish) {
                    __threadfence();
#pragma unroll
                    for (int i = 0; i < kSums / 2; ++i) v2[i] = 0;
                    for (int o = cf; o <= cl; ++o) {
                        // the first owner's share of the tile starts it, unless it starts mid-tile
                        const bool o_starts = o * units / C <= t0;
                        const float2* from =
                            reinterpret_cast<const float2*>(p.parts + (size_t)(2 * o + (o_starts ? 1 : 0)) * (kCols * 128)) +
                            (size_t)(r0 / 2) * 128 + ch;
#pragma unroll
                        for (int i = 0; i < kSums / 2; ++i) {
                            const int a = i / (kRowsT / 2), j = i % (kRowsT / 2);
                            if (2 * j < rows) {
                                const float2 x = __ldcg(from + (size_t)(a * (kNT / 2) + j) * 128), y = f32x2_parts(v2[i]);
                                v2[i] = f32x2(__fadd_rn(y.x, x.x), __fadd_rn(y.y, x.y));
                            }
                        }
                    }
                }
            }
            if (!finish) continue;
            if constexpr (kMode == kGateUp) {
                const int a = tile / p.NB, nb = tile % p.NB, e = p.active[1 + a];
#pragma unroll
                for (int i = 0; i < kRowsT / 2; ++i) {
                    const float2 g = f32x2_parts(v2[i]), up = f32x2_parts(v2[kRowsT / 2 + i]);
                    hbuf[(r0 + 2 * i) * 132 + ch] = __fmul_rn(__fdiv_rn(g.x, __fadd_rn(1.0f, expf(-g.x))), up.x);
                    hbuf[(r0 + 2 * i + 1) * 132 + ch] = __fmul_rn(__fdiv_rn(g.y, __fadd_rn(1.0f, expf(-g.y))), up.y);
                }
                named_bar_sync(1, kEpiThreads);
#pragma unroll 1
                for (int it = et; it < kNT * 8; it += kEpiThreads) {
                    const int m = it >> 3, col = (it & 7) * 16;
                    float f[16], amax = 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 h = *reinterpret_cast<const float4*>(hbuf + m * 132 + col + i);
                        f[i] = h.x, f[i + 1] = h.y, f[i + 2] = h.z, f[i + 3] = h.w;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
                    for (int d = 4; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                    if (m < p.M) {
                        bool chosen = false;
                        for (int j = 0; j < p.top_k; ++j) chosen |= p.ids[m * p.top_k + j] == e;
                        const float s = fp8_block_scale(amax), inv = __frcp_rn(s);
                        uint4 q = make_uint4(0, 0, 0, 0);
                        if (chosen) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                w[i] = e4m3x4(__fmul_rn(f[4 * i], inv), __fmul_rn(f[4 * i + 1], inv),
                                              __fmul_rn(f[4 * i + 2], inv), __fmul_rn(f[4 * i + 3], inv));
                            q = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        if (nb * 128 + col < p.N)  // N % 16 == 0
                            *reinterpret_cast<uint4*>(p.hq + ((size_t)a * p.M + m) * p.N + nb * 128 + col) = q;
                        if (col == 0) p.hs[((size_t)a * p.NB + nb) * p.M + m] = chosen ? s : 0.0f;
                    }
                }
                named_bar_sync(1, kEpiThreads);  // hbuf has been read
            } else {
                const int nb = kMode == kRows ? tile / p.MB : tile, m0 = (kMode == kRows ? (tile % p.MB) * kNT : 0) + r0;
                const int n = nb * 128 + ch;
                if (n < p.N) {
                    uint16_t* y = reinterpret_cast<uint16_t*>(p.Y) + (size_t)m0 * p.N + n;
#pragma unroll
                    for (int i = 0; i < kRowsT / 2; ++i) {
                        const float2 f = f32x2_parts(v2[i]);
                        if (m0 + 2 * i < p.M) y[(size_t)(2 * i) * p.N] = T::from_float(f.x);
                        if (m0 + 2 * i + 1 < p.M) y[(size_t)(2 * i + 1) * p.N] = T::from_float(f.y);
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------ scales, and codes with kFuse
        const int sw = warp - 2;
        for (long long u = u0 + sw; u < u1; u += kFRSideWarps) {
            const long long i = u - u0;
            const int stage = (int)(i % kStages), slot = (int)(i % kSlots);
            const uint32_t phase = (uint32_t)(i / kStages) & 1u;
            const int tile = (int)(u / kbt), kb = (int)(u - (long long)tile * kbt);
            float* s = slots + slot * kCols;
            bool ok;
            if constexpr (kFuse) {
                // 8 lanes per row, 16 values each; 4 rows per step
                static_assert(!kFuse || kMode == kRows, "fused codes: plain product only");
                const int chunk = lane & 7, rsub = lane >> 3;
                const int k = kb * 128 + chunk * 16;
                uint4 x[kNT / 4][2];
#pragma unroll
                for (int r = 0; r < kNT / 4; ++r) {
                    const int m = r * 4 + rsub;
                    x[r][0] = x[r][1] = make_uint4(0, 0, 0, 0);
                    if (m < p.M && k < p.K) {  // K % 16 == 0: all 16 values or none
                        const uint4* src = reinterpret_cast<const uint4*>(p.X + (size_t)m * p.K + k);
                        x[r][0] = __ldg(src);
                        x[r][1] = __ldg(src + 1);
                    }
                }
                const float w = __ldg(p.ws + (size_t)tile * p.KB + kb);
                ok = __all_sync(0xffffffffu, wait_fast(&empty[stage], phase ^ 1, wctx));
                if (!ok) break;
                uint8_t* sb = ring + stage * kStageBytes + kA * 16384;
#pragma unroll
                for (int r = 0; r < kNT / 4; ++r) {
                    const int m = r * 4 + rsub;
                    float a = T::pair_max(fp8_amax8<T>(fp8_amax8<T>(T::as_pair(0u), x[r][0]), x[r][1]));
#pragma unroll
                    for (int d = 4; d >= 1; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
                    const float sc = fp8_block_scale(a), inv = __frcp_rn(sc);
                    const uint2 lo = fp8_codes8<T>(x[r][0], inv), hi = fp8_codes8<T>(x[r][1], inv);
                    *reinterpret_cast<uint4*>(sb + m * 128 + ((chunk ^ (m & 7)) << 4)) =
                        make_uint4(lo.x, lo.y, hi.x, hi.y);
                    if (chunk == 0) s[m] = __fmul_rn(sc, w);
                }
                fence_proxy_async_smem();
            } else {
                float f[(kNT + 31) / 32], g[(kNT + 31) / 32];
#pragma unroll
                for (int j = 0; j < (kNT + 31) / 32; ++j) {
                    const int m = lane + 32 * j;
                    f[j] = g[j] = 0.0f;
                    if (kMode == kRows) {
                        const int row = (tile % p.MB) * kNT + m;
                        if (m < kNT && row < p.M)
                            f[j] = __fmul_rn(p.xs[kb * p.xs_pitch + row], __ldg(p.ws + (size_t)(tile / p.MB) * p.KB + kb));
                    } else if (kMode == kGateUp) {
                        const int e = p.active[1 + tile / p.NB], nb = tile % p.NB;
                        if (m < p.M) {
                            const float xs = p.xs[kb * p.xs_pitch + m];
                            const size_t o = ((size_t)e * p.NB + nb) * p.KB + kb;
                            f[j] = __fmul_rn(xs, __ldg(p.ws + o));
                            g[j] = __fmul_rn(xs, __ldg(p.ws2 + o));
                        }
                    } else {
                        const int a = kb / p.KB, ib = kb - a * p.KB, e = p.active[1 + a];
                        if (m < p.M) {
                            float w = 0.0f;  // the token's weight for this expert
                            for (int q = 0; q < p.top_k; ++q)
                                if (p.ids[m * p.top_k + q] == e) w = p.wts[m * p.top_k + q];
                            f[j] = __fmul_rn(__fmul_rn(p.xs[((long long)a * p.KB + ib) * p.xs_pitch + m],
                                                       __ldg(p.ws + ((size_t)e * p.NB + tile) * p.KB + ib)), w);
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, wait_fast(&empty[stage], phase ^ 1, wctx));
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < (kNT + 31) / 32; ++j) {
                    const int m = lane + 32 * j;
                    if (m < kNT) {
                        s[m] = f[j];
                        if (kA == 2) s[kNT + m] = g[j];
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[stage]);
        }
    }

    if (threadIdx.x == 0 && *abort_flag) settle_after_abort();  // copies issued before the abort land first
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace i8mm
