// Causal attention over the 8-bit paged cache for sequences of more than 128 query rows per kv
// head (prompt chunks).  Bound by the tensor cores' 1,024 clocks for the products of 128 rows and
// 128 keys, against 256 bytes of cache per key, and, as measured, by the row threads: 2,048 rows of
// 8,192 keys take 240 us (52% of the bf16 rate), the tensor pipe 44% and the issue slots 49%
// busy; a tile of 256 rows takes 3,800 clocks, of which a thread's 128 keys are 3,100.
//
// A group is 2 x floor(128 / G) tokens of one sequence and kv head: two blocks of up to 128
// rows (token-major, G query heads each), the M of the products, that share the key and value
// tiles.  Per tile of 128 keys and block:
//  * S = Q K^T (tcgen05 kind::f8f6f4): the cache's key codes as they are, q = hi + lo in
//    e4m3 and e5m2 (exact for bf16, see the rows kernel), accumulated in tensor memory;
//  * one thread per row, 64 keys at a time: p = 2^(s log2(e) - ref + 7), summed in fp32, and P =
//    p x value scale in fp16 (11 bits; at most 2^15) over the scores.  The row's reference
//    moves only when its maximum of s log2(e) + log2(value scale) passes it by 2^8 (then the
//    output in tensor memory is rescaled, which after the first tiles is rare);
//  * O += P V (kind::f16, P from tensor memory), the value codes widened to fp16 (exact) once
//    per tile by four warps: two e4m3 terms of P would cost its threads twice the conversions.
// The halves of a tile have score columns of their own, so that one half's scores are computed
// while the threads work on the other's (2,048 rows of 8,192 keys, with 128 columns as one,
// whose scores wait for the product that reads the probabilities in their place: 297 us
// against 274).
// While one block's row threads work, the tensor cores run the other block's products.
// Warps: 0-3 and 4-7 the rows of the two blocks, 8-11 widen values, 12 copies, 13 and 15
// issue the MMAs of the two blocks, 14 page scales.  A block takes a run of the blocks list (kv8_list.cuh).
#include <cuda_bf16.h>
#include <cmath>

#include "kv8_mma.cuh"

namespace sv {

constexpr int KB_THREADS = 512;
constexpr int KB_META = 8;              // tiles whose page factors are kept
constexpr int KB_NK = 3;                // key tiles in shared memory
constexpr int KB_NV = 2;                // value tiles, as codes and as fp16

template <int D> struct KbCfg {
    static constexpr uint32_t TILE = KV8_TILE * D;
    static constexpr uint32_t QBYTES = 2 * 128 * D;          // one block: hi rows, lo rows
    static constexpr size_t SMEM = 1024 + 2 * (size_t)QBYTES + KB_NK * TILE + KB_NV * TILE + KB_NV * 2 * TILE;
};

template <int D>
__global__ void __launch_bounds__(KB_THREADS, 1)
kv8_blocks_kernel(const __grid_constant__ Kv8Attn a, float* part_o, float2* part_ml, Kv8Run* runs, bool after) {
    using C = KbCfg<D>;
    extern __shared__ uint8_t kb_smem[];
    __shared__ __align__(8) uint64_t k_full[KB_NK], k_empty[KB_NK], c_full[KB_NV], c_empty[KB_NV], v_full[KB_NV], v_empty[KB_NV];
    __shared__ __align__(8) uint64_t q_full[2], s_full[2][2], p_full[2][2], o_rest[2], o_done[2], turn[2], m_full[KB_META], m_empty[KB_META], done_bar[2];
    __shared__ uint32_t tmem_sh;
    __shared__ volatile int abort_flag;
    __shared__ long long scan[36];
    __shared__ __align__(16) float4 meta[KB_META][8];   // per page: key scale (-1: none), log2 of the value scale, value scale

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // barriers, a lane to each slot, before anything is waited for
    if (warp == 15) {
        if (lane < KB_NK) {
            mbar_init(smem_u32(&k_full[lane]), 1);
            mbar_init(smem_u32(&k_empty[lane]), 2);
        }
        if (lane < KB_NV) {
            mbar_init(smem_u32(&c_full[lane]), 1);
            mbar_init(smem_u32(&c_empty[lane]), 4);
            mbar_init(smem_u32(&v_full[lane]), 4);
            mbar_init(smem_u32(&v_empty[lane]), 2);
        }
        if (lane < 2) {
            mbar_init(smem_u32(&q_full[lane]), 4);
            mbar_init(smem_u32(&s_full[lane][0]), 1);
            mbar_init(smem_u32(&s_full[lane][1]), 1);
            mbar_init(smem_u32(&p_full[lane][0]), 4);
            mbar_init(smem_u32(&p_full[lane][1]), 4);
            mbar_init(smem_u32(&o_rest[lane]), 1);
            mbar_init(smem_u32(&o_done[lane]), 1);
            mbar_init(smem_u32(&turn[lane]), 1);
            mbar_init(smem_u32(&done_bar[lane]), 1);
        }
        if (lane < KB_META) {
            mbar_init(smem_u32(&m_full[lane]), 1);
            mbar_init(smem_u32(&m_empty[lane]), 12);
        }
        if (lane == 0) abort_flag = 0;
        fence_barrier_init();
    }
    kv8_begin(after);
    const int G = a.hq / a.hkv, half = 128 / G;
    if (threadIdx.x == 0) {
        runs[blockIdx.x].first = KV8_NONE;
        runs[blockIdx.x].open = 0;
    }
    int fb;
    long long fbase;
    const long long total = kv8_find(
        a.B, scan,
        [&](int b) { return kb_units(a, b); },
        [&](long long t) { return kv8_run_begin(t, blockIdx.x); }, fb, fbase);
    KbWalk walk;
    walk.start(a, kv8_run_begin(total, blockIdx.x), kv8_run_begin(total, blockIdx.x + 1), fb, fbase);
    if (walk.left <= 0) {        // no run for this block
        kv8_finish(after);
        return;
    }
    const uint32_t base = (smem_u32(kb_smem) + 1023u) & ~1023u;
    uint8_t* gbase = kb_smem + (base - smem_u32(kb_smem));
    const uint32_t kring = base + 2 * C::QBYTES, cring = kring + KB_NK * C::TILE, vring = cring + KB_NV * C::TILE;
    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&tmem_sh)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    Kv8Seg s;
    bool ok = true;
    // a bounded wait, the same answer for the whole warp
    auto wait = [&](uint64_t& bar, uint32_t parity) { return kv8_wait_warp(bar, parity, abort_flag); };
    auto blocks_of = [&](const Kv8Seg& s) { return (2 * s.rb + 1) * half < s.n ? 2 : 1; };

    if (warp >= 12) {
        if (warp == 12) {
            // ---- copies: lane p < 8 the tile's p-th key page, lane 8 + p its values ----
            const uint64_t pol = policy_evict_last();
            uint32_t i = 0, kd = 0, vd = 0;          // tiles begun; keys and values issued
#pragma unroll 1
            while (ok && walk.next(a, s)) {
                const int* row = a.block_table + (size_t)s.slot * a.max_pages;
                const int npages = min((s.len + 15) >> 4, s.t1 * 8);
                auto window = [&](int t) {
                    const int p = t * 8 + lane;
                    const int id = p < npages ? row[p] : -1;
                    return id >= 0 && id < a.num_pages ? id : -1;
                };
                int ids = window(s.t0), ahead = window(s.t0 + 4);
#pragma unroll 1
                for (int t = s.t0; t < s.t1; ++t, ++i) {
                    const int w = (t - s.t0) & 3;
                    if (w == 0 && t > s.t0) {
                        ids = ahead;
                        ahead = window(t + 4);
                    }
                    const int page = __shfl_sync(FULL, ids, w * 8 + (lane & 7));
                    const uint32_t bytes = __popc(__ballot_sync(FULL, lane < 8 && page >= 0)) * 16 * D;
                    const uint8_t* src = a.pool + ((size_t)page * a.hkv + s.h) * 2 * (16 * D);
                    const int ks = (int)(i % KB_NK), vs = (int)(i % KB_NV);
                    if (i >= KB_NK) ok = wait(k_empty[ks], i / KB_NK - 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(smem_u32(&k_full[ks]), bytes);
                    __syncwarp();
                    if (lane < 8 && page >= 0)
                        bulk_g2s(kring + ks * C::TILE + lane * 16 * D, src, 16 * D, smem_u32(&k_full[ks]), pol);
                    kd = i + 1;
                    if (i >= KB_NV) ok = wait(c_empty[vs], i / KB_NV - 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(smem_u32(&c_full[vs]), bytes);
                    __syncwarp();
                    if (lane < 8 && page >= 0)
                        bulk_g2s(cring + vs * C::TILE + lane * 16 * D, src + 16 * D, 16 * D, smem_u32(&c_full[vs]), pol);
                    vd = i + 1;
                }
            }
            if (!ok) abort_flag = 1;
            if (lane == 0) {          // no copy may still be landing when the block leaves
#pragma unroll 1
                for (uint32_t j = kd > KB_NK ? kd - KB_NK : 0; j < kd; ++j)
                    if (!kv8_wait(k_full[j % KB_NK], (j / KB_NK) & 1)) abort_flag = 1;
#pragma unroll 1
                for (uint32_t j = vd > KB_NV ? vd - KB_NV : 0; j < vd; ++j)
                    if (!kv8_wait(c_full[j % KB_NV], (j / KB_NV) & 1)) abort_flag = 1;
            }
        } else if (warp == 13 || warp == 15) {
            // ---- MMA issuers, one per block of rows.  They take turns, so that the waits of one hide behind
            // the MMAs of the other without their MMAs alternating between two accumulators.  Per half
            // tile P V, then the scores of the same half of the next tile, which overwrite the
            // probabilities read by it: MMAs of one thread run in order.  The whole warp walks, so
            // that the descriptors stay uniform; one lane issues.  A slot of keys or values is free
            // after both issuers ----
            const uint32_t id_s = kv8_idesc(64, 0), id_lo = kv8_idesc(64, 1), id_o = kv8_idesc_f16(D);
            const int blk = warp == 13 ? 0 : 1;
            uint32_t i = 0, seg = 0, done = 0;       // tiles of the run; groups and tiles of this block
            uint32_t turns = 0;                      // this issuer's turns
#pragma unroll 1
            while (ok && walk.next(a, s)) {
                const int nb = blocks_of(s), nt = s.t1 - s.t0;
                if (blk >= nb) {
                    // a group of one block: this issuer passes its tiles on, one phase after the other
#pragma unroll 1
                    for (int t = 0; ok && t < nt; ++t, ++i) {
                        ok = wait(k_full[i % KB_NK], i / KB_NK);
                        if (ok && lane == 0) mbar_arrive(smem_u32(&k_empty[i % KB_NK]));
                        ok = ok && wait(v_full[i % KB_NV], i / KB_NV);
                        if (ok && lane == 0) mbar_arrive(smem_u32(&v_empty[i % KB_NV]));
                    }
                    continue;
                }
                auto scores = [&](uint32_t j, int u) {       // by the elected lane
                    const uint64_t kd = kv8_desc_rows<D>(kring + (j % KB_NK) * C::TILE + u * 64 * D), qd = kv8_desc_rows<D>(base + blk * C::QBYTES);
#pragma unroll
                    for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            kv8_mma(tmem + blk * 128 + u * 64, qd + (lo * 128 * D >> 4) + k * 2, kd + k * 2, lo ? id_lo : id_s, lo | k);
                    mma_commit(smem_u32(&s_full[blk][u]));
                    if (u) mma_commit(smem_u32(&k_empty[j % KB_NK]));
                };
                ok = wait(q_full[blk], seg) && wait(k_full[i % KB_NK], i / KB_NK);
                if (!ok) break;
                if (kv8_elect()) {
                    scores(i, 0);
                    scores(i, 1);
                }
                __syncwarp();
#pragma unroll 1
                for (int t = 0; ok && t < nt; ++t, ++i, ++done) {
                    const bool next = t + 1 < nt;
                    ok = wait(v_full[i % KB_NV], i / KB_NV) && (!next || wait(k_full[(i + 1) % KB_NK], (i + 1) / KB_NK));
#pragma unroll 1
                    for (int u = 0; u < 2; ++u) {
                        ok = ok && wait(p_full[blk][u], done);
                        // the first block begins the run; from then on each turn of one follows the other's
                        if (nb == 2) {
                            if (blk || turns) ok = ok && wait(turn[blk], turns - (blk ^ 1));
                            ++turns;
                        }
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = kv8_desc_v16<D>(vring + (i % KB_NV) * 2 * C::TILE) + u * 4 * (2 * D * 16 >> 4);
                        if (kv8_elect()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                kv8_mma_f16_ts(tmem + 256 + blk * 128, tmem + blk * 128 + u * 64 + k * 8,
                                               vd + k * (2 * D * 16 >> 4), id_o, (t | u | k) ? 1u : 0u);
                            mma_commit(smem_u32(&o_rest[blk]));
                            if (u) mma_commit(smem_u32(&v_empty[i % KB_NV]));
                            if (u && !next) mma_commit(smem_u32(&o_done[blk]));
                            if (next) scores(i + 1, u);
                            if (nb == 2) mbar_arrive(smem_u32(&turn[blk ^ 1]));
                        }
                        __syncwarp();
                    }
                }
                ++seg;
            }
            if (!ok) abort_flag = 1;
            if (kv8_elect()) mma_commit(smem_u32(&done_bar[blk]));     // nothing may still write tensor memory when it is freed
            __syncwarp();
            if (!kv8_wait(done_bar[blk], 0)) abort_flag = 1;
        } else if (warp == 14) {
            // ---- factors of the tiles' pages ----
            uint32_t i = 0;
#pragma unroll 1
            while (ok && walk.next(a, s)) {
                const int* row = a.block_table + (size_t)s.slot * a.max_pages;
                const int npages = (s.len + 15) >> 4;
#pragma unroll 1
                for (int t = s.t0; t < s.t1; ++t, ++i) {
                    float4 m = make_float4(-1.0f, 0.0f, 1.0f, 0.0f);
                    const int p = t * 8 + lane;
                    const int page = lane < 8 && p < npages ? row[p] : -1;
                    if (page >= 0 && page < a.num_pages) {
                        const float2 sc = *reinterpret_cast<const float2*>(a.scales + ((size_t)page * a.hkv + s.h) * 2);
                        m = make_float4(sc.x, kv8_lg2(sc.y), sc.y, 0.0f);
                    }
                    if (i >= KB_META) ok = wait(m_empty[i % KB_META], i / KB_META - 1);
                    if (!ok) break;
                    if (lane < 8) meta[i % KB_META][lane] = m;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&m_full[i % KB_META]));
                }
            }
            if (!ok) abort_flag = 1;
        }
    } else if (warp >= 8) {
        // ---- values: codes to fp16, zeros where there is no key ----
        const int tid = threadIdx.x - 256, d = tid % D;
        constexpr int STEP = 128 / D;                // D = 64: each half of the threads takes every other page
        uint32_t i = 0;
#pragma unroll 1
        while (ok && walk.next(a, s)) {
#pragma unroll 1
            for (int t = s.t0; ok && t < s.t1; ++t, ++i) {
                const int sl = (int)(i % KB_NV), ms = (int)(i % KB_META);
                ok = wait(m_full[ms], i / KB_META) && wait(c_full[sl], i / KB_NV);
                if (ok && i >= KB_NV) ok = wait(v_empty[sl], i / KB_NV - 1);
                if (!ok) break;
                const uint8_t* src = gbase + (cring - base) + sl * C::TILE + d * 16;
                uint8_t* dst = gbase + (vring - base) + sl * 2 * C::TILE + d * 16;
#pragma unroll 2
                for (int p = tid / D; p < 8; p += STEP) {
                    uint4 w = *reinterpret_cast<const uint4*>(src + p * 16 * D);
                    const int keys = s.len - (t * 8 + p) * 16;
                    if (keys < 16 || meta[ms][p].x < 0.0f) kv8_keep(w, meta[ms][p].x < 0.0f ? 0 : keys);
                    kv8_widen16<D>(w, dst + (2 * p) * D * 16);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&v_full[sl]));
                    mbar_arrive(smem_u32(&c_empty[sl]));
                    mbar_arrive(smem_u32(&m_empty[ms]));
                }
            }
        }
        if (!ok) abort_flag = 1;
    } else {
        // ---- rows: thread = row of its block ----
        const int blk = warp >> 2, q4 = warp & 3, j = q4 * 32 + lane;
        constexpr int LR = D / 8;                    // lanes of a row's 16-byte pieces
        const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t ts = tl + blk * 128, to = tl + 256 + blk * 128;
        // positive, so that maxima can be taken of raw scores: a negative scale goes into q
        const float sl2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.1754944e-38f);
        uint32_t i = 0, done = 0, seg = 0;           // tiles of the run; tiles and groups of this block
        bool begun = false;
#pragma unroll 1
        while (ok && walk.next(a, s)) {
            if (threadIdx.x == 0) kv8_note(runs[blockIdx.x], s, begun);
            if (blk >= blocks_of(s)) {
                // a group of one block: the other's threads only pass its tiles on
#pragma unroll 1
                for (int t = s.t0; ok && t < s.t1; ++t, ++i) {
                    ok = wait(m_full[i % KB_META], i / KB_META);
                    if (ok && lane == 0) mbar_arrive(smem_u32(&m_empty[i % KB_META]));
                }
                if (!ok) break;
                continue;
            }
            const int tok0 = (2 * s.rb + blk) * half, tok = tok0 + j / G, head = s.h * G + j % G;
            const bool mine = j < half * G && tok < s.n;
            const int lim = mine ? s.len - s.n + tok : -1;       // the last key this row sees
            const int safe = s.len - s.n + tok0;                 // the last key that every row of the block sees
            // the row's query as hi + lo terms; the block's scores before are done
            float qs;
            {
                // D / 8 lanes to a row, so that a warp reads whole rows (5 us; a thread with a row to itself, and
                // the sectors of 32 rows a load, 7)
                const unsigned rows = __ballot_sync(FULL, mine);
                const unsigned long long qp = reinterpret_cast<unsigned long long>(static_cast<const __nv_bfloat16*>(a.q) +
                                                                                   (long long)(s.row0 + tok) * a.q_stride + (size_t)head * D);
                uint8_t* qb = gbase + blk * C::QBYTES;
                const uint32_t sign = a.scale < 0.0f ? 0x80808080u : 0u;
                int e = 0;
                auto piece = [&](int k) {
                    const int row = k * (32 / LR) + lane / LR;
                    const unsigned long long from = __shfl_sync(FULL, qp, row);
                    return rows >> row & 1 ? reinterpret_cast<const uint4*>(from)[lane % LR] : make_uint4(0, 0, 0, 0);
                };
                uint4 v[4], next[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) next[u] = piece(u);
#pragma unroll 1
                for (int k = 0; k < LR; k += 4) {        // four rows of a lane at a time, their steps side by side
                    uint32_t top[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        v[u] = next[u];
                        top[u] = kv8_top_exponent(v[u]);
                    }
                    if (k + 4 < LR)
#pragma unroll
                        for (int u = 0; u < 4; ++u) next[u] = piece(k + 4 + u);
#pragma unroll
                    for (int o = LR / 2; o > 0; o >>= 1)
#pragma unroll
                        for (int u = 0; u < 4; ++u) top[u] = max(top[u], __shfl_xor_sync(FULL, top[u], o));
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int er = kv8_exponent_of(top[u]), mine_e = __shfl_sync(FULL, er, lane % (32 / LR) * LR);
                        if (lane / (32 / LR) == k + u) e = mine_e;
                        float x[8];
                        uint2 hi, lo;
                        kv8_unpack8(v[u], x);
                        kv8_split8(x, er, hi, lo);
                        hi.x ^= sign; hi.y ^= sign; lo.x ^= sign; lo.y ^= sign;
                        const uint32_t off = kv8_key_off<D>(q4 * 32 + (k + u) * (32 / LR) + lane / LR, lane % LR * 8);
                        *reinterpret_cast<uint2*>(qb + off) = hi;
                        *reinterpret_cast<uint2*>(qb + 128 * D + off) = lo;
                    }
                }
                qs = __uint_as_float((uint32_t)(e + 127) << 23) * sl2;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&q_full[blk]));
            }
            float ref = -INFINITY, l = 0.0f;
#pragma unroll 1
            for (int t = s.t0; ok && t < s.t1; ++t, ++i, ++done) {
                const int ms = (int)(i % KB_META);
                ok = wait(m_full[ms], i / KB_META);
                const int rel = lim - t * KV8_TILE;              // last column that this row sees
                const bool masked = (t + 1) * KV8_TILE - 1 > safe || __any_sync(FULL, meta[ms][lane & 7].x < 0.0f);
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    ok = ok && wait(s_full[blk][u], done);
                    if (!ok) break;
                    tc_fence_after();
                    const float4* pm = meta[ms] + 4 * u;         // the half's four pages
                    float x[64];
                    kv8_tmem_ld32(ts + u * 64, x);
                    kv8_tmem_ld32(ts + u * 64 + 32, x + 32);
                    kv8_tmem_wait();
#pragma unroll
                    for (int e = 0; e < 64; ++e) asm volatile("" : "+f"(x[e]));
                    if (masked) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const int last = pm[p].x < 0.0f ? -1 : rel - u * 64;
#pragma unroll
                            for (int e = p * 16; e < p * 16 + 16; ++e)
                                if (e > last) x[e] = -INFINITY;
                        }
                    }
                    float mx = -INFINITY;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        float m = -INFINITY;
#pragma unroll
                        for (int e = p * 16; e < p * 16 + 16; e += 2) m = fmaxf(fmaxf(m, x[e]), x[e + 1]);
                        mx = fmaxf(mx, fmaf(m, kv8_factor(pm[p].x, qs), pm[p].y));
                    }
                    if (__any_sync(FULL, mx > ref + 8.0f)) {
                        const bool move = mx > ref + 8.0f;
                        // in two halves: with value scales far apart the factor can be below the smallest
                        // float where the sum times it is not
                        const float ah = move ? kv8_exp2(0.5f * (ref - mx)) : 1.0f, al = ah * ah;
                        if (move) ref = mx;
                        l = l * ah * ah;
                        if (t > s.t0 || u) {
                            // the output at rest: after the product of the half tile before (the one before
                            // that was complete with these scores)
                            ok = wait(o_rest[blk], done * 2 + u - 1);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                float o[16];
                                kv8_tmem_ld16(to + c, o);
                                kv8_tmem_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    asm volatile("" : "+f"(o[e]));
                                    o[e] *= al;
                                }
                                kv8_tmem_st16(to + c, o);
                            }
                        }
                    }
                    const float sub = 7.0f - (ref == -INFINITY ? 0.0f : ref);
                    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float h[16];
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const float vs = pm[2 * c + p].z, sc = kv8_factor(pm[2 * c + p].x, qs);
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const int k = c * 32 + p * 16 + e;
                                const float2 z = kv8_fma2(make_float2(x[k], x[k + 1]), make_float2(sc, sc), make_float2(sub, sub));
                                const float2 y = make_float2(kv8_exp2(z.x), kv8_exp2(z.y));
                                sum = kv8_add2(sum, y);
                                const float2 w = kv8_mul2(y, make_float2(vs, vs));
                                h[p * 8 + e / 2] = __uint_as_float(kv8_half2(w.x, w.y));
                            }
                        }
                        kv8_tmem_st16(ts + u * 64 + c * 16, h);
                    }
                    l += sum.x + sum.y;
                    kv8_tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&p_full[blk][u]));
                        if (u) mbar_arrive(smem_u32(&m_empty[ms]));
                    }
                }
            }
            if (!ok) break;
            // the group's (or this run's part's) output
            // (a barrier of its own: by now o_rest can be any of two phases ahead of what these threads know)
            ok = wait(o_done[blk], seg);
            if (!ok) break;
            ++seg;
            tc_fence_after();
            const bool whole = s.t0 == 0 && s.t1 == s.tiles;
            const size_t part = (size_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * KB_ROWS + blk * 128 + j;
            const bool none = ref == -INFINITY && l == 0.0f;
            const float il = none ? 0.0f : 1.0f / l;
            // through this warp's rows of the query buffer (its scores are done), so that the warp writes
            // whole rows: bf16 at once, fp32 partials in two halves
            const unsigned rows = __ballot_sync(FULL, mine);
            const unsigned long long dst =
                whole ? reinterpret_cast<unsigned long long>(static_cast<__nv_bfloat16*>(a.out) + (long long)(s.row0 + tok) * a.o_stride + (size_t)head * D)
                      : reinterpret_cast<unsigned long long>(part_o + part * D);
            auto stage = [&](int row, int c) {           // 16 bytes c of a row's 2 D
                const int x = row * 2 * D + ((c ^ (row & 7)) << 4);
                return reinterpret_cast<uint4*>(gbase + blk * C::QBYTES + q4 * 32 * D + (x < 32 * D ? x : x + 96 * D));
            };
#pragma unroll 1
            for (int part_at = 0; part_at < (whole ? 1 : 2); ++part_at) {
#pragma unroll 1
                for (int c = 0; c < (whole ? D : D / 2); c += 16) {
                    float o[16];
                    kv8_tmem_ld16(to + part_at * (D / 2) + c, o);
                    kv8_tmem_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) asm volatile("" : "+f"(o[e]));
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            __nv_bfloat162 y[4];
#pragma unroll
                            for (int f = 0; f < 4; ++f)
                                y[f] = none ? __floats2bfloat162_rn(0.0f, 0.0f)
                                            : __floats2bfloat162_rn(o[e * 8 + 2 * f] * il, o[e * 8 + 2 * f + 1] * il);
                            *stage(lane, c / 8 + e) = *reinterpret_cast<uint4*>(y);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4*>(stage(lane, c / 4 + e)) = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
                __syncwarp();
#pragma unroll 2
                for (int k = 0; k < LR; ++k) {
                    const int row = k * (32 / LR) + lane / LR;
                    const unsigned long long to_row = __shfl_sync(FULL, dst, row) + part_at * 2 * D;
                    if (rows >> row & 1) reinterpret_cast<uint4*>(to_row)[lane % LR] = *stage(row, lane % LR);
                }
                __syncwarp();
            }
            if (mine) {
                if (!whole) part_ml[part] = make_float2(ref - 7.0f, l);
                else if (a.lse) a.lse[(size_t)(s.row0 + tok) * a.hq + head] = none ? -INFINITY : 0.6931471805599453f * (ref - 7.0f + log2f(l));
            }
            tc_fence_before();
        }
        if (!ok) {
            // a bounded wait gave up: the remaining rows of this block become NaN
            abort_flag = 1;
            do {
                if (threadIdx.x == 0) kv8_note(runs[blockIdx.x], s, begun);
                const int tok = (2 * s.rb + blk) * half + j / G, head = s.h * G + j % G;
                if (blk < blocks_of(s) && j < half * G && tok < s.n) {
                    if (s.t0 == 0 && s.t1 == s.tiles) {
#pragma unroll 1
                        for (int d = 0; d < D; ++d)
                            static_cast<__nv_bfloat16*>(a.out)[(long long)(s.row0 + tok) * a.o_stride + (size_t)head * D + d] =
                                __float2bfloat16_rn(__uint_as_float(0x7fc00000u));
                        if (a.lse) a.lse[(size_t)(s.row0 + tok) * a.hq + head] = __uint_as_float(0x7fc00000u);
                    } else
                        part_ml[(size_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * KB_ROWS + blk * 128 + j] =
                            make_float2(__uint_as_float(0x7fc00000u), 1.0f);
                }
            } while (walk.next(a, s));
        }
    }
    kv8_finish(after);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && abort_flag) kv8_report(a.err);
    if (warp == 13) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512u) : "memory");
}

template <int D> static cudaError_t blocks_launch(const Kv8Attn& a, const Kv8Parts& parts, bool after, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(kv8_blocks_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)KbCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    return kv8_launch(kv8_blocks_kernel<D>, dim3(KV8_RUNS), KB_THREADS, KbCfg<D>::SMEM, st, a, parts.o, parts.ml, parts.runs, after);
}

cudaError_t kv8_blocks_attention(const Kv8Attn& a, int D, const Kv8Parts& parts, bool after, cudaStream_t st) {
    return D == 128 ? blocks_launch<128>(a, parts, after, st) : blocks_launch<64>(a, parts, after, st);
}

}  // namespace sv
