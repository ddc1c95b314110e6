// Pieces of the tensor-core attention kernels (prompt and drafted-token
// attention): tiles of 128 query rows against tiles of 128 keys, the scores and
// the output accumulators in TMEM, one softmax thread per row.
//
// TMEM (512 columns, 128 lanes = the tile's rows): two score slots of 128 fp32
// columns at 0 and 128, the output accumulators from column 256 on.  A slot is
// two halves of 64 keys with barriers of their own, so that the products and the
// next scores of one half are under way during the softmax of the other.  A
// row's weights are written back as 16-bit pairs over the first 32 columns of
// their half, which the second product reads as its A operand.
//
// A wait on an mbarrier names a phase by its parity, so the barrier may be at
// that phase or one past it when the wait begins, not further: every wait below
// says why it is not.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <cstdint>

#include "tq_tc.cuh"

namespace tq {
namespace fm {

constexpr int kTile = 128;                     // rows of a query tile, keys of a key tile
constexpr uint32_t kSlotCols = 128;            // TMEM columns of a score slot
constexpr uint32_t kHalfCols = 64;             // of them, the scores of half a key tile
constexpr uint32_t kOutCol = 256;              // first column of the output accumulators
constexpr uint64_t kWaitNs = 1000000000ull;    // bound of every wait

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t * r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15"
        "}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr) : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t * r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
        "%27,%28,%29,%30,%31"
        "}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr) : "memory");
}

// The same without the wait: r holds the columns after tmem_wait32(r).
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t * r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
        "%27,%28,%29,%30,%31"
        "}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr) : "memory");
}
// Waits for all loads of this thread; r is an operand, so that no use of it can
// move in front of the wait.
__device__ __forceinline__ void tmem_wait32(uint32_t * r) {
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
        :: "memory");
}

// 16 32-bit values into consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t * r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
        "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16"
        "};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Bounded wait for a phase of an mbarrier.  The waiting thread sleeps: polling
// instead answers some 150 cycles earlier, but takes issue slots from the
// softmax (8192-token prompt 0.556 ms against 0.504 ms).
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
    if (tc::mbar_try(bar, parity)) return true;
    const uint64_t t0 = tc::global_ns();
#pragma unroll 1
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (tc::mbar_try_sleep(bar, parity, 20000u)) return true;
        if (tc::global_ns() - t0 > kWaitNs) return false;
    }
    return false;
}

// The same for a converged warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity));
}

// Position in a ring of N buffers: the buffer and the parity of its use.
template <int N>
struct Ring {
    uint32_t at = 0, parity = 0;
    __device__ __forceinline__ void step() {
        if (++at == N) {
            at = 0;
            parity ^= 1u;
        }
    }
};

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The issuing warps run converged, with one lane elected inside each
// instruction: operands that are the same in all lanes then live in uniform
// registers, which the MMAs read.  From a branch that one lane takes, every
// operand is moved there first, MMA by MMA.
__device__ __forceinline__ uint32_t elected() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(e));
    return e;
}

// D[tmem] (+)= A[smem] B[smem] by the elected lane, 16-bit A and B, fp32 D.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead));
}

// The same with A in TMEM, two values per 32-bit column (16 of the contracted
// index in 8 columns).
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
        :: "r"(tmem_d), "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead));
}

// An arrival on `bar` when the MMAs that the elected lane issued are done.
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
        :: "r"(bar), "r"(lead) : "memory");
}

// The same value; keeps the compiler from holding sums of it in registers
// across a loop.
__device__ __forceinline__ uint64_t opaque(uint64_t x) {
    asm volatile("" : "+l"(x));
    return x;
}

// Descriptor of a value tile as the second product's B operand: rows of 64
// columns (128 bytes, 128-byte swizzle) per key, so the contracted index (the
// key) is the strided one.  `slice` = bytes from one 64-column slice to the
// next, 1024 bytes from one group of 8 keys to the next.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t slice) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((slice >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Instruction descriptor of kind::f16: fp32 D of 128 x n, A and B both fp16 or
// both bf16, B with the contracted index strided when `mn` is set.
__host__ __device__ constexpr uint32_t idesc(bool bf16, int n, bool mn) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTile >> 4) << 24);
}

// 2^x with the hardware approximation (relative error below 2^-22; -inf -> 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in one 64-bit register pair, multiplied or added at once.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The largest of three (a NaN is passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Running softmax of one row, in base 2: weights are 2^(s mul - ref + kShift).
// `ref` is raised only when a row's maximum passes it by more than kLazy, so
// that the accumulator is rescaled a few times a row instead of once a tile;
// the factor 2^kLazy that a weight may exceed 1 by cancels in the quotient.
// fp16 weights are kept 2^kShift larger (at most 2^15): what falls under the
// type's normal range is then below 2^-21 of the row's largest weight.
constexpr float kLazy = 8.0f;
template <bool BF16>
constexpr float kShift = BF16 ? 0.0f : 7.0f;

struct RowState {
    float ref;     // -inf until a key was seen
    float sum;
};

// Maximum of 32 scores.
__device__ __forceinline__ float top32(const uint32_t * r) {
    float m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = max3(__uint_as_float(r[i]), __uint_as_float(r[i + 2]), __uint_as_float(r[i + 4]));
#pragma unroll
    for (int c = 6; c < 30; c += 4)
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = max3(m[i], __uint_as_float(r[c + i]), __uint_as_float(r[c + 2 + i]));
    return fmaxf(max3(m[0], m[1], __uint_as_float(r[30])), __uint_as_float(r[31]));
}

// Weights of 32 scores into the 16 columns at p_tm, and onto the sum.  (All
// exponentials on the special-function unit: a polynomial on the FMA units for
// one pair in eight, four or three cost 4, 6 and 8 % of the 8192-token prompt's
// time, for the instructions, although that unit is half busy.)
template <bool BF16>
__device__ __forceinline__ void weights32(const uint32_t * r, uint64_t mul, uint64_t bias, uint32_t p_tm, uint64_t * sum) {
    uint32_t w[16];
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const uint64_t x = fma2(pair(r[c], r[c + 1]), mul, bias);
        const float a = ex2(__uint_as_float((uint32_t)x)), b = ex2(__uint_as_float((uint32_t)(x >> 32)));
        sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pair(a, b));
        w[c >> 1] = pack2<BF16>(a, b);
    }
    tmem_st16(p_tm, w);
}

template <bool MASKED>
__device__ __forceinline__ void drop32(uint32_t * r, uint32_t allowed) {
    if constexpr (MASKED) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (!((allowed >> c) & 1u)) r[c] = 0xFF800000u;
    }
}

// Multiplies cols columns of this thread's accumulator by f.
__device__ __forceinline__ void rescale(uint32_t o_tm, int cols, float f) {
    tc::fence_after_sync();
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
        uint32_t o[16];
        tmem_ld16(o_tm + (uint32_t)c, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st16(o_tm + (uint32_t)c, o);
    }
}

// Half a tile of scores (64 keys): reads the 64 columns at `s_tm` (lane
// included), drops those whose bit in `allowed` is clear (MASKED), updates the
// row's state, has the accumulator multiplied where needed -- scale_acc(f) waits
// for the products so far and multiplies the row by f -- and writes the weights over the first 32 of the columns.  All 32 lanes of the warp call it
// together.
template <bool BF16, bool MASKED, typename ScaleAcc>
__device__ __forceinline__ bool softmax_half(uint32_t s_tm, bool first, float mul, const uint32_t * allowed, RowState & st,
                                             ScaleAcc scale_acc) {
    uint32_t r0[32], r1[32];
    tmem_ld32_start(s_tm, r0);
    tmem_ld32_start(s_tm + 32u, r1);
    tmem_wait32(r0);
    tmem_wait32(r1);
    drop32<MASKED>(r0, MASKED ? allowed[0] : 0u);
    drop32<MASKED>(r1, MASKED ? allowed[1] : 0u);
    const float top = fmaxf(top32(r0), top32(r1)) * mul;
    bool ok = true;
    const bool raise = top > st.ref + kLazy;          // (ref = -inf: any finite score)
    if (first) {
        st.ref = top;
    } else if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
        const float f = raise ? ex2(st.ref - top) : 1.0f;
        if (raise) st.ref = top;
        st.sum *= f;
        ok = scale_acc(f);
    }
    const float bias = kShift<BF16> - (st.ref == -CUDART_INF_F ? 0.0f : st.ref);
    const uint64_t m2 = pair(mul, mul), b2 = pair(bias, bias);
    uint64_t sum[2] = {0ull, 0ull};
    weights32<BF16>(r0, m2, b2, s_tm, sum);
    weights32<BF16>(r1, m2, b2, s_tm + 16u, sum);
    const uint64_t s2 = add2(sum[0], sum[1]);
    st.sum += __uint_as_float((uint32_t)s2) + __uint_as_float((uint32_t)(s2 >> 32));
    tmem_wait_st();
    tc::fence_before_sync();
    return ok;
}

}  // namespace fm
}  // namespace tq
