// Device pieces shared by the attention kernels of the 8-bit paged cache: operand and
// instruction descriptors, tensor-memory loads, the two-term split of queries, values widened to fp16.
#pragma once

#include <cuda_bf16.h>

#include "host_util.h"
#include "kv8_list.cuh"
#include "tc_common.cuh"

namespace sv {

// kind::f8f6f4, D fp32, A e4m3 or e5m2 (the second query term), B e4m3, both K-major, M = 128, N = n.
__device__ __forceinline__ uint32_t kv8_idesc(int n, int e5m2) {
    return (1u << 4) | ((uint32_t)e5m2 << 7) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void kv8_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// K-major rows of D bytes (keys, queries): 128-byte swizzle for D = 128, 64-byte for D = 64;
// groups of eight rows follow each other.
template <int D> __device__ __forceinline__ uint64_t kv8_desc_rows(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(8 * D >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)(D == 128 ? 2 : 4) << 61);
}

// Values widened to fp16, K-major over the keys without swizzle: core matrices of 8 dimensions x 8 keys,
// 128 bytes apart along the dimensions, D * 16 bytes apart along the keys.
template <int D> __device__ __forceinline__ uint64_t kv8_desc_v16(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(D * 16 >> 4) << 16) | ((uint64_t)(128 >> 4) << 32) |
           ((uint64_t)1 << 46);
}

// Bounded wait for the phase with the given parity: false when `cycles` SM clocks (about 2 s) ran out.
constexpr long long WAIT_CYCLES = 4000000000ll;
__device__ __forceinline__ bool kv8_wait(uint64_t& bar, uint32_t parity, long long cycles = WAIT_CYCLES) {
    const uint32_t b = smem_u32(&bar);
    if (mbar_try_wait(b, parity)) return true;
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(b, parity))
        if (clock64() - t0 > cycles) return false;
    return true;
}
// A wait of this block gave up.
__device__ __forceinline__ void kv8_report(int* err) {
    if (err) atomicExch(err, SPEC_E_TIMEOUT);
}

// The same for a converged warp, one answer for all lanes; false too when another role of the
// block gave up.  What a wait does when its phase is not complete at once stays out of the loops:
// the roles of a block compete for the instruction caches.
static __device__ __noinline__ int kv8_wait_more(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
    bool ok = true;
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > WAIT_CYCLES) {
            ok = false;
            break;
        }
    return __all_sync(FULL, ok && !*abort_flag);
}
__device__ __forceinline__ bool kv8_wait_warp(uint64_t& bar, uint32_t parity, const volatile int& abort_flag) {
    if (__builtin_expect(__all_sync(FULL, mbar_try_wait(smem_u32(&bar), parity & 1)) != 0, 1)) return true;
    return kv8_wait_more(smem_u32(&bar), parity & 1, &abort_flag) != 0;
}

// 16 columns of this warp's lane quarter.
__device__ __forceinline__ void kv8_tmem_st16(uint32_t taddr, const float (&v)[16]) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
           "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr) : "memory");
}
__device__ __forceinline__ void kv8_tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// kind::f16, D fp32, A (tensor memory) and B fp16, M = 128, N = n.
__device__ __forceinline__ uint32_t kv8_idesc_f16(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void kv8_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// The same; lanes of D whose bit is set in `off` are not written.
__device__ __forceinline__ void kv8_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, const uint32_t (&off)[4], uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]) : "memory");
}

__device__ __forceinline__ void kv8_tmem_ld16(uint32_t taddr, float (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                   "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(taddr));
}

__device__ __forceinline__ void kv8_tmem_ld32(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void kv8_tmem_st32(uint32_t taddr, const float* v) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
           "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
           "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
           "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr) : "memory");
}
__device__ __forceinline__ void kv8_tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two probabilities in fp16 (never infinite: past its range only by the rounding of enormous scores).
__device__ __forceinline__ uint32_t kv8_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 at once.
__device__ __forceinline__ float2 kv8_fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 kv8_mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 kv8_add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// One lane of a converged warp.
__device__ __forceinline__ bool kv8_elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// The SFU's approximations (a few ulp); kv8_exp2(-inf) = 0.
__device__ __forceinline__ float kv8_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float kv8_lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// What raw scores of a page are multiplied by, never below the smallest normal number: masked scores are
// -inf, and -inf times an underflowed factor (a zero query's 2^-118 and a zero page's 2^-64) would be NaN.
// Finite raw scores are below 2^24: where this factor replaces a smaller one, the score is below 2^-102 anyway.
__device__ __forceinline__ float kv8_factor(float key_scale, float row) { return fmaxf(fabsf(key_scale) * row, 1.1754944e-38f); }

// Barrier of the row kernel's 256 softmax threads, true if any of them passes pred != 0.
__device__ __forceinline__ int kv8_rows_any(int pred) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 256, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(pred) : "memory");
    return r;
}

// The same for the row kernel's 128 query threads.
__device__ __forceinline__ int kv8_query_any(int pred) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(pred) : "memory");
    return r;
}

// Eight bf16 as floats, their largest exponent field, and the exponent e for which a row's
// largest lies in [2^7, 2^8) x 2^e, from the largest field (2^-e stays a normal number).
__device__ __forceinline__ void kv8_unpack8(uint4 w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t kv8_top_exponent(uint4 w) {
    constexpr uint32_t M = 0x7fff7fffu;          // magnitudes order as unsigned numbers
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & M, w.y & M), __vmaxu2(w.z & M, w.w & M));
    return max(m & 0xffffu, m >> 16) >> 7;
}
__device__ __forceinline__ int kv8_exponent_of(uint32_t top) { return max((int)top - 127 - 7, -118); }

// Four numbers (at most 448) as hi in e4m3 + lo in e5m2.  The remainder is taken in half precision (11
// bits, 7 more than hi), where it is exact.  Of a number of 8 bits it is at most 8 of its last units, which 3
// bits hold, and e5m2 ends at 2^-16, 2^7 below e4m3: a second term in e4m3 lost bits of elements from
// 2^-9 of the row's largest on, which decide the scores of queries with an outlier channel.
__device__ __forceinline__ void kv8_split4(float2 a, float2 b, uint32_t& hi, uint32_t& lo) {
    asm("{\n\t.reg .b32 h, g;\n\t.reg .b16 x, y, u, v;\n\t"
        "cvt.rn.f16x2.f32 h, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 x, h;\n\t"
        "cvt.rn.f16x2.e4m3x2 g, x;\n\t"
        "sub.rn.f16x2 h, h, g;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 u, h;\n\t"
        "cvt.rn.f16x2.f32 h, %5, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 y, h;\n\t"
        "cvt.rn.f16x2.e4m3x2 g, y;\n\t"
        "sub.rn.f16x2 h, h, g;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 v, h;\n\t"
        "mov.b32 %0, {x, y};\n\tmov.b32 %1, {u, v};\n\t}"
        : "=r"(hi), "=r"(lo) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}

// x 2^-e as hi + lo (NaN or infinite x: NaN).  x has 8 bits, so that half precision holds x 2^-e < 2^8
// as it is, but for bits below 2^-24.  Exact from 2^-6 on (2^-13 of 2^7), off by 2^-14 at most below.
__device__ __forceinline__ void kv8_split8(float (&x)[8], int e, uint2& hi, uint2& lo) {
    const float f = __uint_as_float((uint32_t)(127 - e) << 23);
    if (e == kv8_exponent_of(255))          // the exponent of infinities and NaN
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(x[i]) == INFINITY) x[i] = __uint_as_float(0x7fffffffu);
    kv8_split4(make_float2(x[0] * f, x[1] * f), make_float2(x[2] * f, x[3] * f), hi.x, lo.x);
    kv8_split4(make_float2(x[4] * f, x[5] * f), make_float2(x[6] * f, x[7] * f), hi.y, lo.y);
}

// The first `keep` of 16 bytes (none below 1), zeros behind them.
__device__ __forceinline__ void kv8_keep(uint4& w, int keep) {
    uint32_t* u = &w.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = keep - 4 * i;
        u[i] &= k >= 4 ? 0xffffffffu : (k <= 0 ? 0u : (1u << (8 * k)) - 1);
    }
}

// Four e4m3 codes as two pairs of fp16.
__device__ __forceinline__ void kv8_widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

// The 16 codes of a dimension in a page as fp16, into the two core matrices that hold its first and last eight keys.
template <int D> __device__ __forceinline__ void kv8_widen16(uint4 w, uint8_t* dst) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) kv8_widen4(u[e], h[2 * e], h[2 * e + 1]);
    *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(dst + D * 16) = make_uint4(h[4], h[5], h[6], h[7]);
}

// The two attention kernels, and the join of the groups that their runs share.  The second of a
// call (after) overlaps the first: it writes nothing that the first reads or writes, and the first
// lets it start only when the kernels before the call are done.  It is done itself only
// when the first is, so that the join waits for both.
__device__ __forceinline__ void kv8_begin(bool after) {
    // (the second reads what the kernels before the call wrote without a wait of its own: no line of
    // them may be left in this SM's L1 from before)
    if (after) __threadfence();
    else pdl_wait();
    pdl_launch_dependents();
}
__device__ __forceinline__ void kv8_finish(bool after) {
    if (after) pdl_wait();
}
// part_o [2 * KV8_RUNS][rows of a group][D], part_ml [2 * KV8_RUNS][rows of a group]: slot 2 c + 1 is
// the group that run c begins and does not end, slot 2 c the one that began before it.
cudaError_t kv8_rows_attention(const Kv8Attn& a, int D, const Kv8Parts& parts, bool after, cudaStream_t st);
cudaError_t kv8_blocks_attention(const Kv8Attn& a, int D, const Kv8Parts& parts, bool after, cudaStream_t st);

}  // namespace sv
