// Block-scaled e4m3 products for few rows: the weights are streamed once and
// HBM is the bound, so what matters is that every SM streams, and streams the
// same share.
//
//   out[m, n] = sum_b (xs[m, b] * ws[n / 128, b]) * sum_{k in block b} xq[m, k] * wq[n, k]
//
// A unit of work is one 128-channel x 128-k box of the weight (16 KB, one
// scale block; two boxes in the gated layer) with the rows' 128 k.  A unit's
// sums go to one of the TMEM accumulators in rotation, and the epilogue adds
// them, scaled, to running fp32 sums in registers.  Which operand the box is
// depends on the number of rows:
//   kNT <= 32 rows: the box is A of tcgen05.mma (M = 128 channels), the rows B
//     (N = kNT).  An epilogue thread owns a channel and reads every row's scale
//     from shared memory, 16 bytes a time.  The other way round the tensor core
//     multiplies 128 rows for the sake of a few, and that is power: a single
//     token through 12288 x 49152 took 97 us cold, but 117 us in a long run, at
//     1.05 GHz under the power cap.
//   kNT >= 64: the rows are A (M = 128, of which only kNT are staged: what is
//     read past them makes accumulator rows that nobody reads), the box B
//     (N = 128).  An epilogue thread owns a row and reads one scale.  (The
//     scales of 64 or 128 rows, read by every thread, slowed the tensor core's
//     own reads of shared memory to 2400 cycles a unit, against 260.)
//
// Where there are fewer tiles than SMs a block takes a tile, or a cluster's
// blocks take equal pieces of one; the caller decides (`cut`).  Otherwise the
// units, ordered by output tile and then k, are cut into equal consecutive
// shares, one per CTA (one CTA per SM): a CTA's share may start and end inside
// a tile.  Of a tile that several CTAs share every one stores its fp32 sums; at
// the end of its share, so that the stream is never held up, each takes a
// ticket for its first and last tile, and the last one to come adds the stored
// sums in the order of k: the result does not depend on who that is, and no
// CTA waits for another.
//
// That join takes 2 us for 8 rows and 9 for 128 (one block reads all the
// others' sums).  The blocks of a cluster leave their sums in shared memory and
// each finish a part of the rows, reading from one another: 1 to 2 us.
//
// Three products are made of this:
//   kRows    Y = X W;
//   kGateUp  per chosen expert h = silu(X Wg) * (X Wu), two boxes per unit, h
//            in codes: a tile's 128 channels are one block of 128 of the next
//            product, so its scale is a maximum over the tile;
//   kDown    Y = sum over experts of weight * (h Wd): the experts' products
//            are one product over the concatenated k of the chosen experts,
//            with the routing weight in the scale of h, so the weighted sum of
//            a token's experts happens in the same running sums.
// In the gated layer every token is a row for every expert.  Of tokens that did
// not choose an expert kGateUp stores zero codes, and kDown leaves out what the
// accumulators hold for them there (kFRNotChosen): an infinity or a NaN in an
// expert's weights reaches the tokens that chose it and no other.
//
// Warps: the epilogue is warps 0-3 (a TMEM lane quadrant of channels each) for
// kNT <= 32; above, with rows in kQ quadrants, the warps w with w % 4 < kQ
// (w < 16), one for each quadrant and quarter of the channels.  Of the others
//   the first   is the TMA producer of the weight boxes (and of the rows
//               unless kFuse);
//   the second  allocates TMEM and issues the MMAs;
//   the rest    (two to six) take the units in turn: the unit's scale products
//               into shared memory, and with kFuse the rows' codes (the rows'
//               16-bit values are read, quantised and written to the swizzled
//               operand).  In kGateUp two do that, and the others finish
//               whole tiles (the epilogue, which sits on one or two schedulers,
//               would hold up the stream for 8 us a tile with it).
// At the end all but the first two join the shared tiles, a warp per row.
//
// Measured (calls back to back, weights from HBM): 1 x 12288 x 49152 95 us, 6.36
// TB/s, which is what HBM gives (98 us in runs of seconds, at 1.73 GHz under the
// power cap); 8 x 4096 x 11008 12.2 us, of which 9 are the stream of 86 blocks
// (56 to 60 GB/s each) and the rest the start and the first boxes' latency; 16 x
// 256 x 384 3.8 us on the GPU, all start; 100 x 11008 x 4096 19.5 us and 333 x
// 4112 x 5136 21 us with the quantiser before.  In the first of these no unit of
// the GPU is the bound (shared memory's banks 11 % of their peak for reads and
// 11 % for writes, L2 20 %, HBM 27 %, tensor pipe 13 %, issue 43 %); in the
// second a unit of 128 rows takes ~670 cycles on its way round, 520 of them in
// the epilogue, and the issuing thread waits 270 for a free accumulator.  The
// gate/up kernel streams at 6.2 to 7 TB/s.
#pragma once

#include "fp8_common.cuh"
#include "fp8_gemm_sm100.cuh"

namespace i8mm {

enum { kRows = 0, kGateUp = 1, kDown = 2 };

constexpr int kFRMinUnits = 4;   // a share smaller than this costs more in joining than it saves
constexpr int kFRPrefetch = 10;  // boxes of the next product fetched into L2 per block (24 MB in all)
// In place of the scale of a row that did not choose the expert: the bits of -0.
// No scale of h is that (it is 2^-126 at least, times a weight that is not
// negative), and kDown adds +0 to its scale products, which turns a -0 into +0
// and leaves every other number as it is, whatever a caller's weight scales are.
constexpr uint32_t kFRNotChosen = 0x80000000u;
__device__ __forceinline__ bool fr_not_chosen(float s) { return __float_as_uint(s) == kFRNotChosen; }
constexpr int kFRMaxCtas = 160;  // shares (a fixed bound, so that the workspace depends on the shape only)

// How `tiles` tiles of kbt units are shared out on at most `ctas` CTAs: `cut`
// pieces a tile if the caller says so, and where that keeps at least 4 of 5
// CTAs busy (one SM's stream, 56 GB/s of a matrix that is not in L2, times 118
// is still all that HBM gives).  Otherwise equal runs of units, of `per` units
// each, the first `more` of them one unit more.  A share smaller than
// kFRMinUnits costs more in joining than it saves.
// (Units are 16 KB of weight each, so their number is far below 2^31.)
struct FrShares {
    int kbt, count, cut, per, more;
    FrShares() = default;
    __host__ __device__ __forceinline__ FrShares(int tiles, int kbt_, int ctas, int cut_ = 0) : kbt(kbt_), cut(cut_) {
        const int units = tiles * kbt;
        if (cut) {
            count = cut * tiles;
            per = more = 0;
            return;
        }
        int most = units / kFRMinUnits > tiles ? units / kFRMinUnits : tiles;
        if (most > ctas) most = ctas;
        const int c = tiles <= most ? most / tiles : 0;
        if (c > 0 && 5 * c * tiles >= 4 * most) cut = c;
        count = cut ? cut * tiles : most;
        per = units / count;
        more = units % count;
    }
    // Where share c begins, and its number of units (none for c >= count).  Divisions are few here:
    // the stream waits for them, and each is 50 ns.
    __device__ __forceinline__ void locate(int c, int& tile, int& kb, int& n) const {
        if (c >= count) {
            tile = kb = n = 0;
        } else if (cut == 1) {
            tile = c;
            kb = 0;
            n = kbt;
        } else if (cut) {
            tile = c / cut;
            const int piece = c - tile * cut;
            kb = piece * kbt / cut;
            n = (piece + 1) * kbt / cut - kb;
        } else {
            const int u = start(c);
            tile = u / kbt;
            kb = u - tile * kbt;
            n = per + (c < more ? 1 : 0);
        }
    }
    __device__ __forceinline__ int start(int share) const {
        if (cut) {
            const int t = share / cut;
            return t * kbt + (share - t * cut) * kbt / cut;
        }
        return share * per + min(share, more);
    }
    __device__ __forceinline__ int owner(int unit) const {
        if (cut) {
            const int t = unit / kbt;
            return t * cut + ((unit - t * kbt + 1) * cut - 1) / kbt;
        }
        const int big = more * (per + 1);
        return unit < big ? unit / (per + 1) : more + (unit - big) / per;
    }
};

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
    int max_active;        // the count is at most this
    const unsigned long long* masks;  // for each chosen expert its tokens, a bit each
    const int32_t* ids;    // kGateUp: M x top_k chosen experts and their weights
    const float* wts;
    int top_k;
    void* Y;               // kRows, kDown: M x N, 16 bits
    uint8_t* hq;           // kGateUp: codes [a][M][N], scales times routing weights [(a * NB + nb) * M + m]
    float* hs;
    FrShares shares;       // kRows
    int cut;               // blocks of a cluster that share each tile (1: a tile per block); 0: FrShares' own choice
    int next_grid, next_cut;  // kGateUp: grid and cut of the down product
    float* parts;          // per CTA two slots (kGateUp: four) of part_rows x kA x 128 floats
    int part_rows;         // rows of a tile: min(M, kNT)
    unsigned* tickets;     // one per tile, zero between calls
    int* status;
    uint64_t wait_limit_ns;
    uint32_t test_flags;   // bit 0: block 0 never signals its first unit (timeout test)
};

// 12 warps where the epilogue is 4 (168 registers a thread), 16 where it is 8
// (128), 20 where it is 16 (96)
template <int kNT>
__host__ __device__ constexpr int fr_threads() { return kNT == 128 ? 640 : kNT == 64 ? 512 : 384; }
template <int kMode>
__host__ __device__ constexpr int fr_a() { return kMode == kGateUp ? 2 : 1; }
template <int kNT>
__host__ __device__ constexpr int fr_cols() { return kNT <= 32 ? kNT : 128; }  // accumulator columns of a box
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_bufs() { return kNT <= 32 ? 4 : 512 / (128 * fr_a<kMode>()); }  // accumulators
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_stage_bytes() { return fr_a<kMode>() * 16384 + kNT * 128; }
// !kBoxA: a 32-row x 64-byte staging buffer per epilogue warp (rows 80 bytes apart)
constexpr int kFRStageRow = 80;
constexpr int kFRSumRow = 132;  // floats from row to row of a tile's sums in shared memory
template <int kNT>
__host__ __device__ constexpr int fr_out_bytes() { return kNT <= 32 ? 0 : 4 * (kNT / 32) * 32 * kFRStageRow; }
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_fixed_bytes() { return 1024 + fr_out_bytes<kNT>() + (fr_bufs<kMode, kNT>() + 1) * 8 + 64; }
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_bytes(int stages) {
    return fr_fixed_bytes<kMode, kNT>() + stages * (fr_stage_bytes<kMode, kNT>() + 16) +
           (stages + fr_bufs<kMode, kNT>()) * fr_a<kMode>() * kNT * 4;
}
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_stages() {
    int s = 12;
    while (fr_bytes<kMode, kNT>(s) > 232448) --s;
    return s;
}
template <int kMode, int kNT>
__host__ __device__ constexpr int fr_smem_bytes() { return fr_bytes<kMode, kNT>(fr_stages<kMode, kNT>()); }

// silu(g) * u
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fmul_rn(__fdiv_rn(g, __fadd_rn(1.0f, expf(-g))), u);
}

// tmem_wait_ld32 / 16 with a look (that does not wait) at a barrier taken before
// the wait: the answers arrive together.
__device__ __forceinline__ bool tmem_wait_ld_look(uint32_t (&r)[32], uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%33], %34;\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "selp.u32 %32, 1, 0, p;\n\t}\n"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool tmem_wait_ld_look(uint32_t (&r)[16], uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%17], %18;\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "selp.u32 %16, 1, 0, p;\n\t}\n"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// v[0 .. 2 kQuads - 1] (4 kQuads sums) += r * s, a scale for each; with kSkip a
// sum whose scale is kFRNotChosen stays as it is, whatever r holds (r counts as 0).
template <int kQuads, bool kSkip>
__device__ __forceinline__ void fma_scaled(uint64_t* v, const uint32_t* r, const ulonglong2* s) {
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
        const ulonglong2 f = s[i];
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(r[4 * i + j]);
        if constexpr (kSkip) {
            const float2 lo = f32x2_parts(f.x), hi = f32x2_parts(f.y);
            x[0] = fr_not_chosen(lo.x) ? 0.0f : x[0];
            x[1] = fr_not_chosen(lo.y) ? 0.0f : x[1];
            x[2] = fr_not_chosen(hi.x) ? 0.0f : x[2];
            x[3] = fr_not_chosen(hi.y) ? 0.0f : x[3];
        }
        fma_f32x2(v[2 * i], f32x2(x[0], x[1]), f.x);
        fma_f32x2(v[2 * i + 1], f32x2(x[2], x[3]), f.y);
    }
}

// 16 bytes of the shared memory of CTA `rank` of the cluster, at this CTA's address `addr`.
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}\n"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// 64 bytes of each of 32 rows (a lane's w is its row's) to dst + row * stride,
// through a staging buffer: written as they are, 16 bytes of 32 rows at a time,
// they take 32 transactions a store (4500 cycles for a tile of 128 rows).
// Rows from `rows` on, rows not in `mask` and 16-byte pieces from `pieces` on
// are left out.
__device__ __forceinline__ void store_rows64(uint8_t* stage, int lane, const uint32_t (&w)[16], uint8_t* dst, size_t stride,
                                             int rows, int pieces, uint32_t mask) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(stage + lane * kFRStageRow + q * 16) =
            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    __syncwarp();
    const int piece = lane & 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = j * 8 + (lane >> 2);
        const uint4 x = *reinterpret_cast<const uint4*>(stage + r * kFRStageRow + piece * 16);
        if (r < rows && ((mask >> r) & 1u) && piece < pieces) __stcg(reinterpret_cast<uint4*>(dst + r * stride + piece * 16), x);
    }
    __syncwarp();
}

// Nothing that follows is moved before the computation of v, nor that after it.
__device__ __forceinline__ void pin16(uint64_t (&v)[16]) {
    asm volatile("" : "+l"(v[0]), "+l"(v[1]), "+l"(v[2]), "+l"(v[3]), "+l"(v[4]), "+l"(v[5]), "+l"(v[6]), "+l"(v[7]),
                 "+l"(v[8]), "+l"(v[9]), "+l"(v[10]), "+l"(v[11]), "+l"(v[12]), "+l"(v[13]), "+l"(v[14]),
                 "+l"(v[15])::"memory");
}

template <int kMode, int kNT, bool kFuse, typename T>
__global__ void __launch_bounds__(fr_threads<kNT>(), 1)
    k_fp8_rows(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_w2,
               const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_next,
               const __grid_constant__ Fp8RowsParams p) {
    constexpr int kA = fr_a<kMode>();
    constexpr int kStageBytes = fr_stage_bytes<kMode, kNT>();
    constexpr int kStages = fr_stages<kMode, kNT>();
    constexpr int kBufs = fr_bufs<kMode, kNT>();
    constexpr int kSlots = kStages + kBufs;
    constexpr bool kBoxA = kNT <= 32;              // the box is the A operand
    constexpr int kCols = fr_cols<kNT>();
    constexpr uint32_t kTmemCols = kBufs * kA * kCols;
    constexpr int kQ = kNT / 32;                   // !kBoxA: TMEM lane quadrants with rows
    constexpr int kEpiWarps = kBoxA ? 4 : 4 * kQ, kEpiThreads = 32 * kEpiWarps;
    constexpr int kSpare = fr_threads<kNT>() / 32 - kEpiWarps - 2;  // warps that make scales (and codes):
    // all of those left over if there are codes to make; a scale needs fewer
    constexpr int kSide = kFuse ? kSpare : kMode == kGateUp || kSpare < 4 ? 2 : 4;
    constexpr int kFin = kMode == kGateUp ? kSpare - kSide : 0;  // warps that finish whole tiles
    constexpr bool kEarly = kMode == kDown || (kMode == kRows && !kFuse);
    constexpr int kSlotsCta = kMode == kGateUp ? 4 : 2;          // stored sums: shared tiles, whole tiles in turn
    constexpr int kJoinWarps = fr_threads<kNT>() / 32 - 2;       // (an even number)
    static_assert(kNT == 16 || kNT == 32 || kNT == 64 || kNT == 128, "rows");
    static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM columns");
    // a stage's MMAs may complete again only after the epilogue has seen their last completion
    static_assert(kStages > kBufs, "stages");
    // a side warp waits for the stage's last completion by parity, so it must not be two rounds
    // ahead: its previous unit, kSide earlier, has seen that unit's stage done one round earlier
    static_assert(kSide <= kStages, "side warps");
    static_assert(kNT * kFRSumRow * 4 <= kStages * kStageBytes, "a tile's sums fit the ring");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* xring = smem;                         // [stages][kNT rows]; reads of M = 128 rows run on into wring
    uint8_t* wring = smem + kStages * kNT * 128;   // [stages][kA boxes]
    // scale products of the units in flight.  A slot is rewritten kSlots units
    // later; its writer has seen the MMAs of kStages units earlier done, and
    // those were issued after the epilogue had read the slot's last content
    // (an accumulator is released only once its scales have been read).
    float* slots = reinterpret_cast<float*>(smem + kStages * kStageBytes);  // [slots][kA][kNT]
    uint8_t* outs = reinterpret_cast<uint8_t*>(slots + kSlots * kA * kNT);  // [epilogue warps][32 rows][80]
    uint64_t* bars = reinterpret_cast<uint64_t*>(outs + fr_out_bytes<kNT>());
    uint64_t* full = bars;                         // [stages] boxes, rows and scales are there
    uint64_t* done = bars + kStages;               // [stages] the stage's MMAs are complete
    uint64_t* tempty = bars + 2 * kStages;         // [bufs] the epilogue has read the accumulator
    uint64_t* drain = tempty + kBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* last_flag = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool epilogue = kBoxA ? warp < 4 : warp < 16 && (warp & 3) < kQ;
    // the others, counted: 0 producer, 1 MMA issuer, 2 and on side warps
    const int role = epilogue ? -1 : kBoxA ? warp - 4 : warp >= 16 ? warp - 16 : (warp >> 2) * (4 - kQ) + (warp & 3) - kQ;
    WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 2);  // the producer's expected bytes and the side warp
            mbar_init(&done[s], 1);
        }
        for (int b = 0; b < kBufs; ++b) mbar_init(&tempty[b], kEpiWarps);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_w);
        if (kMode == kGateUp) prefetch_tmap(&tm_w2);
        if (!kFuse) prefetch_tmap(&tm_x);
    }
    if (role == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // nothing is read before the work ahead on the stream is done, weights
    // included: a kernel there may have written them.  Behind a kernel of the
    // same call (kEarly: the quantiser, or the gate/up kernel) it starts on its
    // weights while that one finishes: that kernel lets this one start only
    // after its own wait, when all before it was done, and writes neither
    // weights nor routing.  (100 x 11008 x 4096: 18.9
    // us, 19.7 without.)
    if (!kEarly) {
        pdl_wait();
        pdl_launch_dependents();
    }

    // the chosen experts: their count and the first 31 with one load per warp
    const int act = kMode == kRows ? 0 : (lane < p.max_active + 1 ? __ldcg(p.active + lane) : 0);
    const int n_active = kMode == kRows ? 1 : __shfl_sync(0xffffffffu, act, 0);
    const int kbt = kMode == kDown ? p.KB * n_active : p.KB;  // units per tile
    const int tiles = kMode == kRows ? p.NB * p.MB : kMode == kGateUp ? p.NB * n_active : p.NB;
    const int c = (int)blockIdx.x;
    const FrShares own = kMode == kRows ? FrShares() : FrShares(tiles, kbt, (int)gridDim.x, p.cut);
    const FrShares& sh = kMode == kRows ? p.shares : own;
    const bool clustered = kMode != kGateUp && p.cut > 1;
    int first_tile, first_kb, nu;  // where this CTA's share begins, and its units
    sh.locate(c, first_tile, first_kb, nu);
    const auto by_rows = [&](int tile) { return p.MB == 1 ? tile : tile / p.MB; };  // kRows: a tile's block of channels
    const auto row0_of = [&](int tile) { return kMode == kRows && p.MB > 1 ? tile % p.MB * kNT : 0; };
    const size_t slot_floats = (size_t)p.part_rows * kA * 128;

    // the a-th chosen expert (by a whole warp)
    const auto expert = [&](int a) {
        const int e = __shfl_sync(0xffffffffu, act, (1 + a) & 31);
        return a < 31 ? e : __ldcg(p.active + 1 + a);
    };

    // Rows row0, row0 + step, ... of a tile from its stored sums: added over
    // the owners cf .. cl (in the order of k), then the output.  By one warp,
    // 4 channels per lane.
    const auto finish_rows = [&](int t, int row0, int step, int cf, int cl, const auto& part_of) {
        constexpr int kR = 4, kO = kA == 2 ? 1 : 4;  // kR rows' loads of kO owners in flight together
        const int m0 = row0_of(t), rows = min(kNT, p.M - m0);
        const int nb = kMode == kRows ? by_rows(t) : kMode == kGateUp ? t % p.NB : t;
        const int n = nb * 128 + 4 * lane;
        // kGateUp: rows that did not choose the expert have no sums; their codes are zero
        const unsigned long long mask = kMode == kGateUp ? __ldcg(p.masks + t / p.NB) : ~0ull;
        const int e = kMode == kGateUp ? expert(t / p.NB) : 0;
#pragma unroll 1
        for (int r0 = row0; r0 < rows; r0 += step * kR) {
            float4 sum[kR][kA];
            bool have[kR];
            float wt[kR];  // kGateUp: the row's weight for the expert, in the lane of that choice
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const int row = r0 + r * step;
                have[r] = row < rows && (kMode != kGateUp || ((mask >> row) & 1u));
                wt[r] = -1.0f;
                if (kMode == kGateUp && have[r] && lane < p.top_k && __ldcg(p.ids + row * p.top_k + lane) == e)
                    wt[r] = __ldcg(p.wts + row * p.top_k + lane);
#pragma unroll
                for (int a = 0; a < kA; ++a) sum[r][a] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll 1
            for (int o0 = cf; o0 <= cl; o0 += kO) {
                float4 x[kO][kR][kA];
#pragma unroll
                for (int o = 0; o < kO; ++o) {
                    const float4* from = reinterpret_cast<const float4*>(part_of(min(o0 + o, cl))) + lane;
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        const int row = r0 + r * step;
#pragma unroll
                        for (int a = 0; a < kA; ++a)
                            x[o][r][a] = o0 + o <= cl && have[r] ? __ldcg(from + (row * kA + a) * 32)
                                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
#pragma unroll
                for (int o = 0; o < kO; ++o)
#pragma unroll
                    for (int r = 0; r < kR; ++r)
#pragma unroll
                        for (int a = 0; a < kA; ++a) {
                            sum[r][a].x = __fadd_rn(sum[r][a].x, x[o][r][a].x);
                            sum[r][a].y = __fadd_rn(sum[r][a].y, x[o][r][a].y);
                            sum[r][a].z = __fadd_rn(sum[r][a].z, x[o][r][a].z);
                            sum[r][a].w = __fadd_rn(sum[r][a].w, x[o][r][a].w);
                        }
            }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const int row = r0 + r * step;
                if (row >= rows) continue;  // the same for the whole warp
                if constexpr (kMode == kGateUp) {
                    const int a = t / p.NB;
                    const bool chosen = have[r];
                    const float4 g = sum[r][0], up = sum[r][kA - 1];
                    float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (chosen)
                        h = make_float4(silu_mul(g.x, up.x), silu_mul(g.y, up.y), silu_mul(g.z, up.z), silu_mul(g.w, up.w));
                    float amax = fmaxf(fmaxf(fabsf(h.x), fabsf(h.y)), fmaxf(fabsf(h.z), fabsf(h.w)));
                    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
                    const float s = fp8_block_scale(amax), inv = __frcp_rn(s);
                    const uint32_t q =
                        e4m3x4(__fmul_rn(h.x, inv), __fmul_rn(h.y, inv), __fmul_rn(h.z, inv), __fmul_rn(h.w, inv));
                    if (n < p.N) *reinterpret_cast<uint32_t*>(p.hq + ((size_t)a * p.M + row) * p.N + n) = q;
                    // the scale that the down product adds the row with: the routing weight in it
                    const unsigned by = __ballot_sync(0xffffffffu, !(wt[r] < 0.0f));
                    const float w = __shfl_sync(0xffffffffu, wt[r], by ? __ffs(by) - 1 : 0);
                    if (lane == 0) p.hs[((size_t)a * p.NB + nb) * p.M + row] = chosen ? __fmul_rn(s, w) : __uint_as_float(kFRNotChosen);
                } else if (n < p.N) {  // N % 16 == 0
                    const float4 x = sum[r][0];
                    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.Y) + (size_t)(m0 + row) * p.N + n) =
                        make_uint2(T::pack(x.x, x.y), T::pack(x.z, x.w));
                }
            }
        }
    };

    if (role == 0) {
        // ------------------------------------------------ TMA producer
        const int first_a = kMode == kGateUp ? first_tile / p.NB : kMode == kDown ? first_kb / p.KB : 0;
        const int first_e = __shfl_sync(0xffffffffu, act, (1 + first_a) & 31);
        if (elect_one()) {
            const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
            int stage = 0;
            uint32_t phase = 0;
            // where the boxes are: k, channel, and expert or row of X; kept up to date with
            // additions (a division per unit would set the pace of the stream)
            int kb = first_kb;
            int nb = kMode == kRows ? by_rows(first_tile) : kMode == kGateUp ? first_tile - first_a * p.NB : first_tile;
            const int mb0 = kMode == kRows ? first_tile - nb * p.MB : 0;
            int mb = mb0;
            int a = first_a, ib = kMode == kDown ? first_kb - first_a * p.KB : 0, e = first_a < 31 ? first_e : __ldcg(p.active + 1 + first_a);
            // kEarly: the rows of the units whose boxes went ahead of the wait
            const auto early_rows = [&](int n) {
                pdl_wait();
                pdl_launch_dependents();
                int da = kMode == kDown ? first_a : mb0, dk = kMode == kDown ? first_kb - first_a * p.KB : first_kb;
                for (int j = 0; j < n; ++j) {
                    if (kMode == kDown)
                        tma_load_3d(xring + j * (kNT * 128), &tm_x, &full[j], dk * 128, 0, da, pol_x);
                    else
                        tma_load_2d(xring + j * (kNT * 128), &tm_x, &full[j], dk * 128, da * kNT, pol_x);
                    if (++dk == p.KB) {
                        dk = 0;
                        if (++da == (kMode == kDown ? n_active : p.MB)) da = 0;
                    }
                }
            };
            for (int i = 0; i < nu; ++i) {
                if (kEarly && i == kStages) early_rows(kStages);
                if (i >= kStages && !wait_fast(&done[stage], phase ^ 1, wctx)) break;
                uint8_t* sw = wring + stage * (kA * 16384);
                uint8_t* sx = xring + stage * (kNT * 128);
                mbar_arrive_expect_tx(&full[stage], kFuse ? kA * 16384 : kStageBytes);
                if (kMode == kRows) {
                    tma_load_2d(sw, &tm_w, &full[stage], kb * 128, nb * 128, pol_w);
                    if (!kFuse && i >= kStages) tma_load_2d(sx, &tm_x, &full[stage], kb * 128, mb * kNT, pol_x);
                } else if (kMode == kGateUp) {
                    tma_load_3d(sw, &tm_w, &full[stage], kb * 128, nb * 128, e, pol_w);
                    tma_load_3d(sw + 16384, &tm_w2, &full[stage], kb * 128, nb * 128, e, pol_w);
                    tma_load_2d(sx, &tm_x, &full[stage], kb * 128, 0, pol_x);
                } else {
                    tma_load_3d(sw, &tm_w, &full[stage], ib * 128, nb * 128, e, pol_w);
                    if (i >= kStages) tma_load_3d(sx, &tm_x, &full[stage], ib * 128, 0, a, pol_x);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (kMode == kDown && ++ib == p.KB) {
                    ib = 0;
                    if (++a == n_active) a = 0;
                    if (i + 1 < nu) e = __ldcg(p.active + 1 + a);
                }
                if (++kb == kbt) {
                    kb = 0;
                    if (kMode == kRows) {
                        if (++mb == p.MB) {
                            mb = 0;
                            ++nb;
                        }
                    } else if (++nb == p.NB && kMode == kGateUp) {
                        nb = 0;
                        ++a;
                        if (i + 1 < nu) e = __ldcg(p.active + 1 + a);
                    }
                }
            }
            if (kEarly && nu <= kStages) early_rows(nu);
            if (kMode == kGateUp) {
                // the down product's first boxes of this block's share, into L2 while the
                // last tiles are joined and the next kernel starts
                const int kbd = p.NB * n_active;
                const FrShares sd(p.KB, kbd, p.next_grid, p.next_cut);
                if (c < sd.count) {
                    const int end = min(sd.start(c + 1), sd.start(c) + kFRPrefetch);
                    for (int u = sd.start(c); u < end; ++u) {
                        const int t = u / kbd, k = u - t * kbd, a = k / p.NB;
                        tma_prefetch_3d(&tm_next, (k - a * p.NB) * 128, t * 128, __ldcg(p.active + 1 + a));
                    }
                }
            }
        }
    } else if (role == 1) {
        // ------------------------------------------------ MMA issuer
        if (elect_one()) {
            const uint32_t idesc = idesc_e4m3_f32(128, kCols);
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool issued = false;
            uint32_t seen = 0;
            for (int i = 0; i < nu; ++i) {
                if (!(seen & 1u) && !wait_fast(&full[stage], phase, wctx)) break;
                if (!(seen & 2u) && !wait_fast(&tempty[buf], buf_phase ^ 1, wctx)) break;
                tc_fence_after();
                const uint64_t dx = sdesc_k128sw(smem_u32(xring + stage * (kNT * 128)));
                const uint64_t dw = sdesc_k128sw(smem_u32(wring + stage * (kA * 16384)));
                const uint32_t d = tmem_base + (uint32_t)(buf * kA * kCols);
                uint64_t* const dn = &done[stage];
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++buf == kBufs) {
                    buf = 0;
                    buf_phase ^= 1;
                }
                seen = mma_unit<kA, kCols, kBoxA>(d, kBoxA ? dw : dx, kBoxA ? dx : dw, idesc, dn,
                                                  !((p.test_flags & 1u) && c == 0 && i == 0), &full[stage], phase,
                                                  &tempty[buf], buf_phase ^ 1);
                issued = true;
            }
            if (issued) {  // every MMA has retired before TMEM is freed
                tc_commit(drain);
                wait_drain(drain, 0, kDrainLimitNs);
            }
        }
    } else if (epilogue) {
        // ------------------------------------------------ epilogue
        if (kEarly) pdl_wait();  // Y, parts and tickets are other kernels' too until then
        const int quad = warp & 3;
        const int row = quad * 32 + lane, c0 = (warp >> 2) * 32;  // !kBoxA: a row, channels c0 .. c0 + 31 of the tile
        const int ch = quad * 32 + lane;                          // kBoxA: a channel, all rows
        uint8_t* const out = outs + ((warp >> 2) * kQ + quad) * (32 * kFRStageRow);
        constexpr int kPairs = kBoxA ? kNT / 2 : 16;              // sums, in pairs of channels (kBoxA: of rows)
        int buf = 0, slot = 0, stage = 0;
        uint32_t phase = 0;
        bool ok = true, seen = false;  // the next unit's MMAs are known to be complete
        int whole_tiles = 0;
        int tile = first_tile, kb = first_kb;
        for (int left = nu; left > 0; ++tile, kb = 0) {
            const int seg = min(kbt - kb, left);  // this share's units of the tile
            const bool starts = kb == 0, whole = seg == kbt;
            // kGateUp: the tokens that chose the tile's expert; the others' sums are not stored
            // (the word with this warp's rows)
            const uint32_t mask =
                kMode == kGateUp ? __ldcg(reinterpret_cast<const uint32_t*>(p.masks + tile / p.NB) + (kBoxA ? 0 : quad))
                                 : ~0u;
            uint64_t v[kA][kPairs];
#pragma unroll
            for (int a = 0; a < kA; ++a)
#pragma unroll
                for (int i = 0; i < kPairs; ++i) v[a][i] = 0;
            for (int i = 0; i < seg; ++i) {
                // after a wait that ran out the loops go on without waiting, so
                // that every barrier and ticket below is still met
                if (ok && !__all_sync(0xffffffffu, seen))
                    ok = __all_sync(0xffffffffu, wait_fast(&done[stage], phase, wctx));
                tc_fence_after();
                // (a look past the share's last unit is at a barrier of this block all the
                // same, and its answer is not used)
                const int next = stage + 1 == kStages ? 0 : stage + 1;
                const uint32_t next_phase = stage + 1 == kStages ? phase ^ 1 : phase;
                const uint32_t t = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * kA * kCols + (kBoxA ? 0 : c0));
#pragma unroll
                for (int a = 0; a < kA; ++a) {
                    if constexpr (!kBoxA) {
                        const float s1 = slots[(slot * kA + a) * kNT + row];
                        uint32_t r[32];
                        tmem_ld32(t + (uint32_t)(a * kCols), r);
                        seen = tmem_wait_ld_look(r, &done[next], next_phase);
                        if (kMode != kDown || !fr_not_chosen(s1)) fma32(v[a], r, f32x2(s1, s1));
                        if (kA == 2) pin16(v[a]);  // these FMAs first: the next load's registers are these
                    } else {
                        const ulonglong2* s2 = reinterpret_cast<const ulonglong2*>(slots + (slot * kA + a) * kNT);
                        if constexpr (kNT == 32) {
                            uint32_t r[32];
                            tmem_ld32(t + (uint32_t)(a * kCols), r);
                            seen = tmem_wait_ld_look(r, &done[next], next_phase);
                            fma_scaled<8, kMode == kDown>(v[a], r, s2);
                            if (kA == 2) pin16(v[a]);
                        } else {
                            uint32_t r[16];
                            tmem_ld16(t + (uint32_t)(a * kCols), r);
                            seen = tmem_wait_ld_look(r, &done[next], next_phase);
                            fma_scaled<4, kMode == kDown>(v[a], r, s2);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[buf]);
                if (++buf == kBufs) buf = 0;
                if (++slot == kSlots) slot = 0;
                stage = next;
                phase = next_phase;
            }
            left -= seg;

            const int m0 = row0_of(tile);
            if (!whole || kMode == kGateUp || clustered) {
                // this CTA's sums of the tile, [rows][kA][128 channels]; slot 0 for a tile that
                // began in an earlier share, slot 1 for one that begins here and goes on,
                // slots 2 and 3 for whole ones
                const int ps = !whole ? (starts ? 1 : 0) : 2 + (whole_tiles & 1);
                if (kMode == kGateUp && whole && whole_tiles >= 2) named_bar_sync(4 + (whole_tiles & 1), kEpiThreads + 32 * kFin);
                float* const part = p.parts + (size_t)(kSlotsCta * c + ps) * slot_floats;
                if (clustered) {
                    // every box and row of this share has been read: the ring holds the sums now
                    float* mine = reinterpret_cast<float*>(smem);
                    if constexpr (kBoxA) {
#pragma unroll
                        for (int i = 0; i < kPairs; ++i) {
                            const float2 x = f32x2_parts(v[0][i]);
                            mine[(2 * i) * kFRSumRow + ch] = x.x;
                            mine[(2 * i + 1) * kFRSumRow + ch] = x.y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 x = f32x2_parts(v[0][2 * i]), y = f32x2_parts(v[0][2 * i + 1]);
                            *reinterpret_cast<float4*>(mine + row * kFRSumRow + c0 + 4 * i) = make_float4(x.x, x.y, y.x, y.y);
                        }
                    }
                    continue;
                }
                if constexpr (kBoxA) {
#pragma unroll
                    for (int a = 0; a < kA; ++a)
#pragma unroll
                        for (int i = 0; i < kPairs; ++i) {
                            const float2 x = f32x2_parts(v[a][i]);
                            if (2 * i < p.part_rows && ((mask >> (2 * i)) & 1u)) __stcg(part + (2 * i * kA + a) * 128 + ch, x.x);
                            if (2 * i + 1 < p.part_rows && ((mask >> (2 * i + 1)) & 1u)) __stcg(part + ((2 * i + 1) * kA + a) * 128 + ch, x.y);
                        }
                } else {
#pragma unroll
                    for (int a = 0; a < kA; ++a)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 x = f32x2_parts(v[a][8 * q + i]);
                                w[2 * i] = __float_as_uint(x.x);
                                w[2 * i + 1] = __float_as_uint(x.y);
                            }
                            store_rows64(out, lane, w,
                                         reinterpret_cast<uint8_t*>(part + (size_t)(quad * 32) * (kA * 128) + a * 128 + c0 + 16 * q),
                                         kA * 128 * 4, p.M - m0 - quad * 32, 4, mask);
                        }
                }
                if (kMode == kGateUp && whole) {
                    named_bar_arrive(2 + (whole_tiles & 1), kEpiThreads + 32 * kFin);
                    ++whole_tiles;
                }
                continue;
            }
            const int n = (kMode == kRows ? by_rows(tile) : tile) * 128 + (kBoxA ? ch : c0);
            if constexpr (kBoxA) {
                if (n < p.N) {
                    uint16_t* y = reinterpret_cast<uint16_t*>(p.Y) + n;  // (kNT rows hold all: m0 is 0)
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        const float2 f = f32x2_parts(v[0][i]);
                        if (2 * i < p.M) y[(size_t)(2 * i) * p.N] = T::from_float(f.x);
                        if (2 * i + 1 < p.M) y[(size_t)(2 * i + 1) * p.N] = T::from_float(f.y);
                    }
                }
            } else {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = f32x2_parts(v[0][i]);
                    w[i] = T::pack(f.x, f.y);
                }
                // N % 16 == 0: a 16-byte piece is in or out
                store_rows64(out, lane, w,
                             reinterpret_cast<uint8_t*>(reinterpret_cast<uint16_t*>(p.Y) + (size_t)(m0 + quad * 32) * p.N + n),
                             (size_t)p.N * 2, p.M - m0 - quad * 32, (p.N - n) >> 3, ~0u);
            }
        }
    } else if (kFin > 0 && role >= 2 + kSide) {
        // ------------------------------------------------ whole tiles of the gated layer
        int tile = first_tile, kb = first_kb, n = 0;
        for (int left = nu; left > 0; ++tile, kb = 0) {
            const int seg = min(kbt - kb, left);
            left -= seg;
            if (seg != kbt) continue;
            named_bar_sync(2 + (n & 1), kEpiThreads + 32 * kFin);  // its sums are stored
            const float* part = p.parts + (size_t)(kSlotsCta * c + 2 + (n & 1)) * slot_floats;
            finish_rows(tile, role - 2 - kSide, kFin > 0 ? kFin : 1, 0, 0, [&](int) { return part; });
            // the slot may be filled again (by the tile after the next, if that one is whole)
            if (left >= 2 * kbt) named_bar_arrive(4 + (n & 1), kEpiThreads + 32 * kFin);
            ++n;
        }
    } else {
        // ------------------------------------------------ scales, and codes with kFuse
        const int sidx = role - 2;
        int kb = first_kb + sidx;
        int nb = kMode == kRows ? by_rows(first_tile) : kMode == kGateUp ? first_tile % p.NB : first_tile;
        int mb = kMode == kRows ? first_tile - nb * p.MB : 0, a = kMode == kGateUp ? first_tile / p.NB : 0;
        const auto settle = [&]() {  // kb counts on from a tile's start: to the tile that it is in
            while (kb >= kbt) {
                kb -= kbt;
                if (kMode == kRows) {
                    if (++mb == p.MB) {
                        mb = 0;
                        ++nb;
                    }
                } else if (++nb == p.NB && kMode == kGateUp) {
                    nb = 0;
                    ++a;
                }
            }
        };
        settle();
        if (kEarly) pdl_wait();
        if constexpr (!kFuse) {
            // Scales of the rows and of the boxes, kDeep of this warp's units ahead in registers.
            // (Two ahead for the experts' products, whose loads wait for an expert's number: 16
            // tokens of 8 of 64 experts, 2048 x 1408, 91.8 -> 90.5 us; more is no faster, and
            // 0.2 us slower for kRows, where one is enough.)
            constexpr int kDeep = kMode == kRows ? 1 : 2, kPer = (kNT + 31) / 32;  // rows per lane
            float ax[kDeep][kPer], aw[kDeep][kA];
            const auto load = [&](int d) {  // those of the unit at kb, and kb on to this warp's next one
                const float* xs = p.xs + kb * p.xs_pitch + mb * kNT;
                size_t o = (size_t)nb * p.KB + kb;
                if (kMode == kGateUp) o += (size_t)expert(a) * p.NB * p.KB;
                if (kMode == kDown) {
                    const int c = kb / p.KB;
                    o = ((size_t)expert(c) * p.NB + nb) * p.KB + (kb - c * p.KB);
                }
                aw[d][0] = __ldg(p.ws + o);
                if (kA == 2) aw[d][kA - 1] = __ldg(p.ws2 + o);
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int m = lane + 32 * j;
                    ax[d][j] = mb * kNT + m < p.M ? xs[m] : 0.0f;
                }
                kb += kSide;
                settle();
            };
            const int end = sidx < kSide ? nu : 0;
#pragma unroll
            for (int d = 0; d < kDeep; ++d)
                if (sidx + d * kSide < end) load(d);
            bool ok = true;
            for (int i0 = sidx; i0 < end && ok; i0 += kDeep * kSide) {
#pragma unroll
                for (int d = 0; d < kDeep; ++d) {
                    const int i = i0 + d * kSide, stage = i % kStages, slot = i % kSlots;
                    if (i >= end || !ok) continue;
                    float* s = slots + slot * (kA * kNT);
                    float f[kA][kPer];
#pragma unroll
                    for (int b = 0; b < kA; ++b)
#pragma unroll
                        for (int j = 0; j < kPer; ++j) {
                            f[b][j] = __fmul_rn(ax[d][j], aw[d][b]);
                            if (kMode == kDown)  // the mark stays, and no product is the mark
                                f[b][j] = fr_not_chosen(ax[d][j]) ? ax[d][j] : __fadd_rn(f[b][j], 0.0f);
                        }
                    if (i + kDeep * kSide < end) load(d);
                    ok = __all_sync(0xffffffffu, wait_fast(&done[stage], ((uint32_t)(i / kStages) & 1u) ^ 1u, wctx));
                    if (!ok) continue;
#pragma unroll
                    for (int b = 0; b < kA; ++b)
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            if (kNT >= 32 || lane < kNT) s[b * kNT + lane + 32 * j] = f[b][j];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[stage]);
                }
            }
        }
        for (int i = kFuse ? sidx : nu; i < nu; i += kSide) {
            const int stage = i % kStages, slot = i % kSlots;
            const uint32_t phase = (uint32_t)(i / kStages) & 1u;
            float* s = slots + slot * (kA * kNT);
            if constexpr (kFuse) {
                static_assert(kMode == kRows && kBoxA, "fused codes: the plain product of at most 16 rows");
                // 8 lanes per row, 16 values each; 4 rows per step
                const int chunk = lane & 7, rsub = lane >> 3;
                const int k = kb * 128 + chunk * 16;
                const int steps = (p.M + 3) >> 2;
                uint4 x[kNT / 4][2];
#pragma unroll
                for (int r = 0; r < kNT / 4; ++r) {
                    if (r < steps) {
                        const int m = r * 4 + rsub;
                        x[r][0] = x[r][1] = make_uint4(0, 0, 0, 0);
                        if (m < p.M && k < p.K) {  // K % 16 == 0: all 16 values or none
                            const uint4* src = reinterpret_cast<const uint4*>(p.X + (size_t)m * p.K + k);
                            x[r][0] = __ldg(src);
                            x[r][1] = __ldg(src + 1);
                        }
                    }
                }
                const float w = __ldg(p.ws + (size_t)nb * p.KB + kb);
                if (!__all_sync(0xffffffffu, wait_fast(&done[stage], phase ^ 1, wctx))) break;
                uint8_t* sx = xring + stage * (kNT * 128);
#pragma unroll
                for (int r = 0; r < kNT / 4; ++r) {
                    if (r < steps) {
                        const int m = r * 4 + rsub;
                        float a = T::pair_max(fp8_amax8<T>(fp8_amax8<T>(T::as_pair(0u), x[r][0]), x[r][1]));
#pragma unroll
                        for (int d = 4; d >= 1; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
                        const float sc = fp8_block_scale16(a), inv = __frcp_rn(sc);
                        const uint2 lo = fp8_codes8<T>(x[r][0], inv), hi = fp8_codes8<T>(x[r][1], inv);
                        *reinterpret_cast<uint4*>(sx + m * 128 + ((chunk ^ (m & 7)) << 4)) =
                            make_uint4(lo.x, lo.y, hi.x, hi.y);
                        if (chunk == 0) s[m] = __fmul_rn(sc, w);
                    }
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[stage]);
            kb += kSide;
            settle();
        }
    }

    // The tiles that this share holds only a part of come last, after it has
    // been streamed: the sums are stored by now, and nothing waits for this.
    if (clustered) {
        __syncwarp();
        cluster_sync_all();  // everyone's sums are in shared memory
        const int t = first_tile, m0 = row0_of(t), rows = min(kNT, p.M - m0);
        const int n = (kMode == kRows ? by_rows(t) : t) * 128 + 4 * lane;
        constexpr int kWarps = fr_threads<kNT>() / 32;
        const uint32_t at = smem_u32(smem) + (uint32_t)lane * 16;
#pragma unroll 1
        for (int row = (int)cluster_ctarank() * kWarps + warp; row < rows; row += p.cut * kWarps) {
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int o = 0; o < p.cut; ++o) {  // in the order of k
                const float4 x = ld_cluster_v4(at + (uint32_t)row * (kFRSumRow * 4), (uint32_t)o);
                sum.x = __fadd_rn(sum.x, x.x);
                sum.y = __fadd_rn(sum.y, x.y);
                sum.z = __fadd_rn(sum.z, x.z);
                sum.w = __fadd_rn(sum.w, x.w);
            }
            if (n < p.N)  // N % 16 == 0
                *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.Y) + (size_t)(m0 + row) * p.N + n) =
                    make_uint2(T::pack(sum.x, sum.y), T::pack(sum.z, sum.w));
        }
        cluster_sync_all();  // nobody leaves while its sums are read
    }
    int head_tile = -1, tail_tile = -1;
    if (nu > 0 && sh.cut != 1) {
        const int end_kb = first_kb + nu;  // the share's end, in units from its first tile's start
        if (first_kb > 0) head_tile = first_tile;
        if (end_kb % kbt != 0 && (first_kb == 0 || end_kb > kbt)) tail_tile = first_tile + end_kb / kbt;
    }
    if (!clustered && role != 0 && role != 1 && (head_tile >= 0 || tail_tile >= 0)) {
        named_bar_sync(1, 32 * kJoinWarps);
        if (warp == 0) {  // lane 0: the head's ticket, lane 1: the tail's
            const int t = lane == 0 ? head_tile : lane == 1 ? tail_tile : -1;
            bool last = false;
            if (t >= 0) {
                const int others = sh.owner((t + 1) * kbt - 1) - sh.owner(t * kbt);
                last = ticket_take(&p.tickets[t]) == (unsigned)others;
                if (last) p.tickets[t] = 0;  // ready for the next call
            }
            const unsigned f = __ballot_sync(0xffffffffu, last);
            if (lane == 0) *last_flag = (int)f;
        }
        named_bar_sync(1, 32 * kJoinWarps);
        const int f = *last_flag;
        const int jw = !epilogue ? kEpiWarps + role - 2 : kBoxA ? warp : (warp >> 2) * kQ + (warp & 3);  // 0 .. kJoinWarps - 1
        if (f) {
            // one tile: a row per warp; two: half of the warps each
            const bool both = f == 3;
            const int t = f == 1 || (both && (jw & 1) == 0) ? head_tile : tail_tile;
            finish_rows(t, both ? jw >> 1 : jw, both ? kJoinWarps / 2 : kJoinWarps, sh.owner(t * kbt),
                        sh.owner((t + 1) * kbt - 1), [&](int o) {
                            return p.parts + (size_t)(kSlotsCta * o + (sh.start(o) <= t * kbt ? 1 : 0)) * slot_floats;
                        });
        }
    }

    if (threadIdx.x == 0 && *abort_flag) settle_after_abort();  // copies issued before the abort land first
    tc_fence_before();
    __syncthreads();
    if (role == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace i8mm
