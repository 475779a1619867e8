// What the block-scaled e4m3 kernels share: the rule of the codes, the 16-bit
// types they take and return, and the tcgen05 / TMA forms that only they use.
//
// The rule, for a block of values with absolute maximum a (all steps in fp32):
//   s = max(RN(a / 448), 2^-126),  code = e4m3(RN(x * RN(1 / s))),  value = code * s.
// 448 is the largest e4m3 value, so a's element gets the largest code.  The
// floor keeps 1 / s finite: a block of zeros (or of values so small that their
// scale would not be a normal number) gets finite codes, and zeros stay zeros.
// The conversion rounds half to even and saturates (RN(a * RN(1 / s)) may
// exceed 448 by a rounding).  A NaN gets the NaN code; an infinity makes s
// infinite.  Either way the row's products are NaN, and only that row's.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "sm100_ptx.cuh"

namespace i8mm {

constexpr float kE4m3Max = 448.0f;
constexpr float kFp8ScaleFloor = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ float fp8_block_scale(float amax) {
    return fmaxf(__fdiv_rn(amax, kE4m3Max), kFp8ScaleFloor);
}

// The same for a maximum of 16-bit values, without the division: q = a * c with
// c = RN(1 / 448), then one correction by the exact remainder (Markstein's
// division with a fused multiply-add).  Equal to RN(a / 448) for every fp16
// and bf16 value that reaches the floor (tested for each of them).
__device__ __forceinline__ float fp8_block_scale16(float amax) {
    constexpr float c = 1.0f / kE4m3Max;
    const float q = __fmul_rn(amax, c);
    const float s = __fmaf_rn(__fmaf_rn(-kE4m3Max, q, amax), c, q);
    return amax > 3.4e38f ? amax : fmaxf(s, kFp8ScaleFloor);  // an infinite maximum stays infinite
}

// Two codes in 16 bits: lo in bits 0-7, hi in bits 8-15.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// The two 16-bit types.  A 32-bit word holds two values; amax2 is the larger
// magnitude of the word's two values and `a`'s (a NaN operand is ignored).
struct F16 {
    using pair = __half2;
    static __device__ __forceinline__ pair as_pair(uint32_t w) { return *reinterpret_cast<pair*>(&w); }
    static __device__ __forceinline__ pair abs_max(pair a, uint32_t w) { return __hmax2(a, __habs2(as_pair(w))); }
    static __device__ __forceinline__ float2 to_float2(uint32_t w) { return __half22float2(as_pair(w)); }
    static __device__ __forceinline__ float to_float(uint16_t h) { return __half2float(__ushort_as_half(h)); }
    static __device__ __forceinline__ uint16_t from_float(float f) { return __half_as_ushort(__float2half_rn(f)); }
    static __device__ __forceinline__ float pair_max(pair a) {
        const float2 f = __half22float2(a);
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const pair h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
struct BF16 {
    using pair = __nv_bfloat162;
    static __device__ __forceinline__ pair as_pair(uint32_t w) { return *reinterpret_cast<pair*>(&w); }
    static __device__ __forceinline__ pair abs_max(pair a, uint32_t w) { return __hmax2(a, __habs2(as_pair(w))); }
    static __device__ __forceinline__ float2 to_float2(uint32_t w) { return __bfloat1622float2(as_pair(w)); }
    static __device__ __forceinline__ float to_float(uint16_t h) { return __bfloat162float(__ushort_as_bfloat16(h)); }
    static __device__ __forceinline__ uint16_t from_float(float f) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    }
    static __device__ __forceinline__ float pair_max(pair a) {
        const float2 f = __bfloat1622float2(a);
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const pair h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// Codes of the 8 values in four words, scaled by inv.
template <typename T>
__device__ __forceinline__ uint2 fp8_codes8(uint4 x, float inv) {
    const float2 a = T::to_float2(x.x), b = T::to_float2(x.y), c = T::to_float2(x.z), d = T::to_float2(x.w);
    uint2 r;
    r.x = e4m3x4(__fmul_rn(a.x, inv), __fmul_rn(a.y, inv), __fmul_rn(b.x, inv), __fmul_rn(b.y, inv));
    r.y = e4m3x4(__fmul_rn(c.x, inv), __fmul_rn(c.y, inv), __fmul_rn(d.x, inv), __fmul_rn(d.y, inv));
    return r;
}

template <typename T>
__device__ __forceinline__ typename T::pair fp8_amax8(typename T::pair m, uint4 x) {
    return T::abs_max(T::abs_max(T::abs_max(T::abs_max(m, x.x), x.y), x.z), x.w);
}

// wait_bounded for the waits that the pace of a kernel hangs on: no call (the
// caller may hold most of its registers live), and no look at the timer until
// the wait has polled for a while (a timer read between polls delays the
// moment at which a completed phase is seen).  CTA-scope acquire also for
// barriers that the pair's other CTA or the tensor core arrives on: what they
// order is TMEM and the async proxy, through tcgen05 fences, and no ordinary
// memory of the other CTA is read after them.
__device__ __forceinline__ bool wait_fast(uint64_t* bar, uint32_t parity, const WaitCtx& c) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*c.abort_flag) return false;
        if (globaltimer_ns() - t0 > c.limit_ns) {
            raise_abort(c);
            return false;
        }
    }
}

// wait_drain and settle_after_abort without a call (a kernel that splits its
// registers with setmaxnreg makes none).
__device__ __forceinline__ void wait_drain_inline(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit_ns) return;
}
__device__ __forceinline__ void settle_inline() {
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (globaltimer_ns() - t0 < 200ull * 1000) {
    }
}

// ---------------------------------------------------------------- tcgen05 / TMA forms

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B (format 0 in bits
// 7-9 and 10-12), fp32 D, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A unit of the weight-streaming kernel in one block: a look at the two
// barriers that the next unit needs, this unit's MMAs, and a commit to `done`
// unless !commit.  kA boxes of one operand (16 KB apart: the A operand if
// kBoxA, else B) against the other, kCols accumulator columns each.  Returns
// the looks' answers (bit 0 `full`, bit 1 `empty`): a look takes ~170 cycles
// while the tensor core reads shared memory, and only inside one block can its
// answer be picked up after the MMAs.
#define I8MM_MMA4(D, A, B)                                                                \
    "add.s64 a1, " A ", 2;\n\tadd.s64 a2, " A ", 4;\n\tadd.s64 a3, " A ", 6;\n\t"         \
    "add.s64 b1, " B ", 2;\n\tadd.s64 b2, " B ", 4;\n\tadd.s64 b3, " B ", 6;\n\t"         \
    "tcgen05.mma.cta_group::1.kind::f8f6f4 [" D "], " A ", " B ", %5, {%6, %6, %6, %6}, p;\n\t" \
    "tcgen05.mma.cta_group::1.kind::f8f6f4 [" D "], a1, b1, %5, {%6, %6, %6, %6}, q;\n\t"       \
    "tcgen05.mma.cta_group::1.kind::f8f6f4 [" D "], a2, b2, %5, {%6, %6, %6, %6}, q;\n\t"       \
    "tcgen05.mma.cta_group::1.kind::f8f6f4 [" D "], a3, b3, %5, {%6, %6, %6, %6}, q;\n\t"
template <int kA, int kCols, bool kBoxA>
__device__ __forceinline__ uint32_t mma_unit(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint64_t* done, bool commit, uint64_t* full, uint32_t pf, uint64_t* empty,
                                             uint32_t pe) {
    const uint32_t z = 0, one = 1;
    uint32_t ra, rb;
    if constexpr (kA == 1) {
        asm volatile(
            "{\n\t.reg .pred p, q, r, s, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 r, [%10], %11;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 s, [%12], %13;\n\t"
            "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\tsetp.ne.b32 t, %9, 0;\n\t"
            I8MM_MMA4("%2", "%3", "%4")
            "@t tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%8];\n\t"
            "selp.u32 %0, 1, 0, r;\n\tselp.u32 %1, 2, 0, s;\n\t}\n"
            : "=r"(ra), "=r"(rb)
            : "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(z), "r"(one), "r"(smem_u32(done)),
              "r"((uint32_t)commit), "r"(smem_u32(full)), "r"(pf), "r"(smem_u32(empty)), "r"(pe)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p, q, r, s, t;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t.reg .b32 d;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 r, [%10], %11;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 s, [%12], %13;\n\t"
            "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\tsetp.ne.b32 t, %9, 0;\n\t"
            I8MM_MMA4("%2", "%3", "%4")
            "add.u32 d, %2, %14;\n\tadd.s64 a0, %3, %15;\n\tadd.s64 b0, %4, %16;\n\t"
            I8MM_MMA4("d", "a0", "b0")
            "@t tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%8];\n\t"
            "selp.u32 %0, 1, 0, r;\n\tselp.u32 %1, 2, 0, s;\n\t}\n"
            : "=r"(ra), "=r"(rb)
            : "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(z), "r"(one), "r"(smem_u32(done)),
              "r"((uint32_t)commit), "r"(smem_u32(full)), "r"(pf), "r"(smem_u32(empty)), "r"(pe), "n"(kCols),
              "n"(kBoxA ? 1024 : 0), "n"(kBoxA ? 0 : 1024)
            : "memory");
    }
    return ra | rb;
}
#undef I8MM_MMA4

// One 128-byte K block on an SM pair (issued by the even CTA's elected thread):
// D[tmem] = A[smem] * B[smem]^T, four e4m3 MMAs of K = 32 (32 bytes = +2 in the
// descriptors' address field apart), the first one overwriting D.
__device__ __forceinline__ void mma_e4m3_k128_2sm(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
    const uint32_t z = 0, one = 1;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, {%4, %4, %4, %4, %4, %4, %4, %4}, p;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a1, b1, %3, {%4, %4, %4, %4, %4, %4, %4, %4}, q;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a2, b2, %3, {%4, %4, %4, %4, %4, %4, %4, %4}, q;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a3, b3, %3, {%4, %4, %4, %4, %4, %4, %4, %4}, q;\n\t}\n" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(z), "r"(one)
        : "memory");
}

// Ask for one box of a 3-D tensor in L2.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* m, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// One more at *p; what this thread's block wrote before the last barrier is
// visible (at GPU scope) to whoever sees this addition, and what others
// published this way is visible to this thread and, after a barrier, its block.
__device__ __forceinline__ unsigned ticket_take(unsigned* p) {
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}

// 3-D tiled load of one box (x times the element size a multiple of 16).
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

}  // namespace i8mm
