// Causal attention over the 8-bit paged cache for sequences of up to 128 query rows per kv head
// (n new tokens x G query heads: decoding, verify passes, short chunks).  Bound by the cache's
// bytes: every key and value code is read once, by bulk copies that land as operands.
//
// A block takes a run of the rows list (kv8_list.cuh).  The 128 lanes of an accumulator hold the
// group's rows in 4, 2 or 1 copies (up to 32, 64, 128 rows), and copy k of a row takes only
// every k-th part of a tile's 128 keys: all lanes work however few rows there are, one
// thread has one row, and nothing is reduced over lanes until the end.  Per tile:
//  * S = Q K^T (tcgen05 kind::f8f6f4).  K are the cache's codes; q = (hi + lo) 2^e per row, hi in
//    e4m3 and lo in e5m2, which hold a bf16's 8 bits exactly (elements below 2^-13 of the row's
//    largest are off by up to 2^-21 of it);
//  * with x = s log2(e): p = 2^(x - ref + 12), the sum adds p, P = p x value scale in fp16 (11 bits
//    down to 2^-26 of the row's largest, then in steps of 2^-36 of it).  ref follows the largest x +
//    log2(value scale) when that passes it by 3 (P <= 2^15), which after the first tiles is rare; then
//    the row's output is rescaled.  In an 8-bit format the probabilities of a long context's many small
//    keys do not survive beside a large one: two e4m3 terms end at 2^-15 of it, and with 90% of the sum on
//    one key of 16k the other 10% came out up to half too small (short of them the sum, which is fp32, is not);
//  * O += P V (kind::f16): P lies over the scores in tensor memory, each 32 keys' over their own
//    scores; a product of 16 keys leaves the lanes of the other copies alone; V are the codes widened to
//    fp16 (exact) by the warps that prepare the queries.
// Two groups of four warps take alternate tiles with outputs of their own; at the end of a
// run's part of a group the copies and both outputs are added through shared memory.
// What it replaced (32 verify passes of up to 16k keys): the running maximum of every tile over
// lanes that held keys, 580 us; a vote per tile instead, 212 us, bound by the latency of some 4,600 warp
// instructions a tile.  Now 143 us for those (70% of the copy rate, the tensor
// pipe 51% and the issue slots 37% busy), 62 us for 5 rows of 128k keys, 74 us for 48 decodes of D = 64; with two-term e4m3 probabilities, whose products
// need no widened values, 135, 59 and 76.
// Warps: 0-3 and 4-7 softmax, 8 copies keys, 9 copies values and writes the pages' factors, 10 and
// 11 issue the MMAs of the two groups, 12-15 widen values and prepare the queries of the next group of rows.
#include <cuda_bf16.h>
#include <algorithm>
#include <cmath>

#include "kv8_mma.cuh"

namespace sv {

constexpr int KR_THREADS = 512;
constexpr int KR_WIDEN = 128;           // threads that widen values
constexpr int KR_WIN = 4;               // tiles of a window: a lane of the copy warps to each page
constexpr float KR_LEAD = 12.0f;        // exponent of P at the reference
constexpr float KR_MOVE = 3.0f;         // how far a maximum passes the reference before it moves

// Tensor memory columns of a group: scores (and probabilities), output.
constexpr uint32_t KR_S = 0, KR_O = 256;

template <int D> struct KrCfg {
    static constexpr uint32_t TILE = KV8_TILE * D;           // bytes of a tile's keys (values)
    static constexpr uint32_t QBYTES = 32768;                // hi rows, lo rows; 32 outputs of 256 lanes
    static constexpr int NK = D == 128 ? 3 : 5;              // ring slots of keys,
    static constexpr int NC = D == 128 ? 2 : 5;              // of values as codes
    static constexpr int NV = D == 128 ? 2 : 4;              // and as fp16 (even: an issuer waits for every phase of its slots)
    static constexpr size_t SMEM = 1024 + 2 * QBYTES + (size_t)(NK + NC + 2 * NV) * TILE;
};

// Lanes of one copy of a group of R rows.
__device__ __forceinline__ int kr_span(int R) { return R <= 32 ? 32 : (R <= 64 ? 64 : 128); }

// A row without a key: zeros.
__device__ __forceinline__ void kr_zero_row(const Kv8Attn& a, int row, int D, int tid, int T) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + (long long)row * a.o_stride;
#pragma unroll 1
    for (int i = tid; i < a.hq * D / 8; i += T) reinterpret_cast<uint4*>(o)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
#pragma unroll 1
        for (int i = tid; i < a.hq; i += T) a.lse[(size_t)row * a.hq + i] = -INFINITY;
}

template <int D>
__global__ void __launch_bounds__(KR_THREADS, 1)
kv8_rows_kernel(const __grid_constant__ Kv8Attn a, float* part_o, float2* part_ml, Kv8Run* runs, bool after) {
    using C = KrCfg<D>;
    extern __shared__ uint8_t kr_smem[];
    __shared__ __align__(8) uint64_t k_full[C::NK], k_empty[C::NK], c_full[C::NC], c_empty[C::NC], v_full[C::NV], v_empty[C::NV];
    __shared__ __align__(8) uint64_t q_full[2], q_free[2], s_full[2], p_full[2], o_done[2], m_full[2], m_empty[2], turn[2], done_bar[2];
    __shared__ uint32_t tmem_sh;
    __shared__ volatile int abort_flag;
    __shared__ long long scan[36];
    __shared__ __align__(16) float4 meta[2][KR_WIN * 8]; // per page of two windows: key scale (-1: none), log2 of the value scale, value scale
    __shared__ float qs[2][128];                         // row scale x softmax scale x log2(e)
    __shared__ uint8_t q_top[128];                       // the query warps' largest exponent fields
    __shared__ float2 ml[2][128];                        // per group and lane: reference, sum

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // barriers, a lane to each slot, before anything is waited for
    if (warp == 11) {
        if (lane < C::NK) {
            mbar_init(smem_u32(&k_full[lane]), 1);
            mbar_init(smem_u32(&k_empty[lane]), 1);
        }
        if (lane < C::NC) {
            mbar_init(smem_u32(&c_full[lane]), 1);
            mbar_init(smem_u32(&c_empty[lane]), KR_WIDEN / 32);
        }
        if (lane < C::NV) {
            mbar_init(smem_u32(&v_full[lane]), KR_WIDEN / 32);
            mbar_init(smem_u32(&v_empty[lane]), 1);
        }
        if (lane < 2) {
            mbar_init(smem_u32(&q_full[lane]), 4);
            mbar_init(smem_u32(&q_free[lane]), 8);
            mbar_init(smem_u32(&s_full[lane]), 1);
            mbar_init(smem_u32(&p_full[lane]), 4);
            mbar_init(smem_u32(&o_done[lane]), 1);
            mbar_init(smem_u32(&m_full[lane]), 1);
            mbar_init(smem_u32(&m_empty[lane]), 8);
            mbar_init(smem_u32(&turn[lane]), 1);
            mbar_init(smem_u32(&done_bar[lane]), 1);
        }
        if (lane == 0) abort_flag = 0;
        fence_barrier_init();
    }
    kv8_begin(after);
    const int G = a.hq / a.hkv;
    if (threadIdx.x == 0) {
        runs[blockIdx.x].first = KV8_NONE;
        runs[blockIdx.x].open = 0;
    }
    int fb;
    long long fbase;
    const long long total = kv8_find(
        a.B, scan,
        [&](int b) { return kr_units<D>(a, b); },
        [&](long long t) { return kv8_run_begin(t, blockIdx.x); }, fb, fbase);
    // rows without a key: those before the first and behind the last sequence, and the first n - len
    // of a sequence of len < n positions; spread over the blocks
    {
        const int first = min(max(kv8_row_begin(a, 0), 0), a.n_rows), last = min(max(kv8_row_begin(a, a.B), first), a.n_rows);
#pragma unroll 1
        for (int r = blockIdx.x; r < a.n_rows - (last - first); r += gridDim.x)
            kr_zero_row(a, r < first ? r : r - first + last, D, threadIdx.x, KR_THREADS);
#pragma unroll 1
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            int slot, row0, n, len;
            kv8_sequence(a, b, slot, row0, n, len);
#pragma unroll 1
            for (int r = 0; r < min(n, n - len); ++r) kr_zero_row(a, row0 + r, D, threadIdx.x, KR_THREADS);
        }
    }
    KrWalk<D> walk;
    walk.start(a, kv8_run_begin(total, blockIdx.x), kv8_run_begin(total, blockIdx.x + 1), fb, fbase);
    if (walk.left <= 0) {        // no run for this block
        kv8_finish(after);
        return;
    }
    const uint32_t base = (smem_u32(kr_smem) + 1023u) & ~1023u;
    uint8_t* gbase = kr_smem + (base - smem_u32(kr_smem));
    const uint32_t kring = base + 2 * C::QBYTES, cring = kring + C::NK * C::TILE, vring = cring + C::NC * C::TILE;
    if (warp == 10) {
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

    if (warp >= 12) {
        // ---- values: codes to fp16, zeros behind the last key; in between the queries of the next group.
        // A group's queries come before its values, the next one's as soon as their buffer is free: when
        // the softmax is done with the group two before, whose values are all behind us.  A warp
        // whose wait gave up goes on voting, so that all four leave together ----
        const int tid = threadIdx.x - 384;
        constexpr int NL = 8 * D / KR_WIDEN;         // 16-byte pieces of a thread
        KrWalk<D> qw = walk;
        Kv8Seg qseg;
        bool qmore = qw.next(a, qseg);
        uint32_t seg = 0, at = 0, i = 0;             // groups prepared, the group and the tile that are widened
        // queries as hi + lo terms: 128 / span threads to a row, each with its share of the dimensions,
        // which it writes to every copy
        auto prepare = [&]() {
            const int R = qseg.n * G, span = kr_span(R), r = tid & (span - 1), t = r / G;
            const int cnt = D / 8 * span / 128, c0 = tid / span * cnt;          // chunks of eight dimensions: 2, 4, 8 or 16
            const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (long long)(qseg.row0 + t) * a.q_stride +
                                                             (size_t)(qseg.h * G + r - t * G) * D) + c0;
            uint32_t top = 0;
#pragma unroll 4
            for (int c = 0; c < cnt; ++c) top = max(top, kv8_top_exponent(r < R ? qp[c] : make_uint4(0, 0, 0, 0)));
            q_top[tid] = (uint8_t)top;
            kv8_query_any(0);
#pragma unroll 1
            for (int k = r; k < 128; k += span) top = max(top, (uint32_t)q_top[k]);
            const int e = kv8_exponent_of(top);
            // the factor is positive, so that maxima can be taken of raw scores: a negative scale goes into q
            qs[seg & 1][tid] = __uint_as_float((uint32_t)(e + 127) << 23) * fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.1754944e-38f);
            uint8_t* qb = gbase + (seg & 1) * C::QBYTES;
            const uint32_t sign = a.scale < 0.0f ? 0x80808080u : 0u;
#pragma unroll 1
            for (int c = 0; c < cnt; ++c) {          // (rolled: this code is always cold)
                float x[8];
                uint2 hi, lo;
                kv8_unpack8(r < R ? qp[c] : make_uint4(0, 0, 0, 0), x);
                kv8_split8(x, e, hi, lo);
                hi.x ^= sign; hi.y ^= sign; lo.x ^= sign; lo.y ^= sign;
#pragma unroll 1
                for (int j = r; j < 128; j += span) {
                    const uint32_t off = kv8_key_off<D>(j, (c0 + c) * 8);
                    *reinterpret_cast<uint2*>(qb + off) = hi;
                    *reinterpret_cast<uint2*>(qb + 128 * D + off) = lo;
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&q_full[seg & 1]));
            ++seg;
            qmore = qw.next(a, qseg);
        };
#pragma unroll 1
        while (walk.next(a, s)) {
            bool now = seg == at;                    // this group's queries are not there yet
#pragma unroll 1
            for (int t = s.t0; t <= s.t1; ++t) {
                if (now || (qmore && seg == at + 1 && t > s.t0)) {
                    // (a vote also says that q_top is read)
                    bool free_ = true;
                    if (seg >= 2) {
                        if (now) ok = ok && wait(q_free[seg & 1], (seg >> 1) - 1);
                        else free_ = mbar_test(smem_u32(&q_free[seg & 1]), ((seg >> 1) - 1) & 1);
                    }
                    const bool no = kv8_query_any(!ok || !free_) != 0;
                    if (!no) prepare();
                    else if (now) {
                        ok = false;
                        break;
                    }
                    now = false;
                }
                if (t == s.t1) break;
                const int cs = (int)(i % C::NC), vs = (int)(i % C::NV);
                ok = ok && wait(c_full[cs], i / C::NC);
                // all pieces at once, and the codes' slot given back before they are converted: one warp a scheduler has
                // nothing but its own latency to hide (two pages at a time, the slot at the end: 166 us for 152)
                uint4 w[NL];
                if (ok) {
                    const uint4* src = reinterpret_cast<const uint4*>(gbase + (cring - base) + cs * C::TILE) + tid;
#pragma unroll
                    for (int k = 0; k < NL; ++k) w[k] = src[k * KR_WIDEN];
                    // these loads before the copy that the slot is given back to: without the fence it landed while
                    // they were still on their way, and some dimensions of a tile had another tile's values
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&c_empty[cs]));
                    if (i >= C::NV) ok = wait(v_empty[vs], i / C::NV - 1);
                }
                if (!ok) abort_flag = 1;
                else {
                    const int left = s.len - t * KV8_TILE;
                    if (left < KV8_TILE)                     // codes behind the last key: anything, and 0 x NaN is NaN
#pragma unroll
                        for (int k = 0; k < NL; ++k) kv8_keep(w[k], left - (k * KR_WIDEN + tid) / D * 16);
                    uint8_t* dst = gbase + (vring - base) + vs * 2 * C::TILE;
#pragma unroll
                    for (int k = 0; k < NL; ++k) kv8_widen16<D>(w[k], dst + ((k * KR_WIDEN + tid) / D * 2 * D + (k * KR_WIDEN + tid) % D) * 16);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&v_full[vs]));
                }
                ++i;
            }
            if (now) break;
            ++at;
        }
        if (!ok) abort_flag = 1;
    } else if (warp == 8 || warp == 9) {
        // ---- copies, keys (8) and values (9): a lane holds a page of a window of four tiles and copies it
        // when its tile comes.  Eight copies of a warp take it some 600 clocks, so that little else may
        // be done tile by tile: the pages' factors go out a window at a time ----
        const bool vals = warp == 9;
        uint64_t* full = vals ? c_full : k_full;
        uint64_t* empty = vals ? c_empty : k_empty;
        const uint32_t ring = vals ? cring : kring, NS = vals ? C::NC : C::NK;
        const uint64_t pol = policy_evict_first();
        const uint32_t mine = (uint32_t)(lane & 7) * 16 * D;          // this lane's page in a tile
        uint32_t i = 0, win = 0;                 // tiles and windows of the run
#pragma unroll 1
        while (ok && walk.next(a, s)) {
            const int* row = a.block_table + (size_t)s.slot * a.max_pages;
            const int npages = min((s.len + 15) >> 4, s.t1 * 8);
            auto window = [&](int t) {           // page ids of tiles t .. t + 3
                const int p = t * 8 + lane;
                const int id = p < npages ? row[p] : -1;
                return id >= 0 && id < a.num_pages ? id : -1;
            };
            // (the value warp's) scales of the lane's page
            auto factors = [&](int id) {
                return vals && id >= 0 ? *reinterpret_cast<const float2*>(a.scales + ((size_t)id * a.hkv + s.h) * 2) : make_float2(-1.0f, 1.0f);
            };
            int id = window(s.t0), ahead = window(s.t0 + KR_WIN);
            float2 sc = factors(id), sc_ahead = make_float2(-1.0f, 1.0f);
            const uint8_t* src = nullptr;
            unsigned have = 0;
#pragma unroll 1
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int w = (t - s.t0) & (KR_WIN - 1);
                if (w == 0) {
                    if (t > s.t0) {
                        id = ahead;
                        sc = sc_ahead;
                        ahead = window(t + KR_WIN);
                    }
                    have = __ballot_sync(FULL, id >= 0);
                    src = a.pool + (((size_t)id * a.hkv + s.h) * 2 + (vals ? 1 : 0)) * (16 * D);
                    if (vals) {
                        if (win >= 2) ok = wait(m_empty[win & 1], (win >> 1) - 1);
                        if (!ok) break;
                        meta[win & 1][lane] = make_float4(sc.x, kv8_lg2(sc.y), sc.y, 0.0f);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&m_full[win & 1]));
                        ++win;
                    }
                }
                if (w == 2) sc_ahead = factors(ahead);
                const unsigned pages = have >> (w * 8) & 0xffu;
                const int sl = (int)(i % NS);
                if (i >= NS) ok = wait(empty[sl], i / NS - 1);
                if (!ok) break;
                const uint32_t fb = smem_u32(&full[sl]);
                if (vals && pages != 0xffu) {
                    // values of missing pages are multiplied by P = 0 and must be finite
#pragma unroll 1
                    for (int p = 0; p < 8; ++p)
                        if (!(pages >> p & 1))
#pragma unroll 1
                            for (int e = lane; e < D; e += 32)
                                *reinterpret_cast<uint4*>(gbase + (ring - base) + sl * C::TILE + (p * D + e) * 16) = make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive_expect_tx(fb, __popc(pages) * 16 * D);
                __syncwarp();
                if (lane >> 3 == w && id >= 0) bulk_g2s(ring + sl * C::TILE + mine, src, 16 * D, fb, pol);
            }
        }
        if (!ok) abort_flag = 1;
        // no copy may still be landing when the block leaves
        if (lane == 0)
#pragma unroll 1
            for (uint32_t j = i > NS ? i - NS : 0; j < i; ++j)
                if (!kv8_wait(full[j % NS], (j / NS) & 1)) abort_flag = 1;
    } else if (warp == 10 || warp == 11) {
        // ---- MMA issuers, one per group of softmax warps (tile i belongs to group i % 2).  They take
        // turns, tile by tile, so that the waits of one hide behind the MMAs of the other without
        // their MMAs alternating between two accumulators (unordered issuers took 2,700 clocks a
        // tile, a single one 1,850, of which the MMAs are 1,024).  A tile's scores follow the
        // product of tile i - 2, whose probabilities they overwrite: MMAs of one thread run in
        // order.  The whole warp walks, so that the descriptors stay uniform; one lane issues.  Keys
        // and values are waited for ahead of the probabilities.  A product of 16 keys writes only
        // the lanes of the copy that has them (what the others hold there is their scores) ----
        const uint32_t id_s = kv8_idesc(128, 0), id_lo = kv8_idesc(128, 1), id_o = kv8_idesc_f16(D);
        const int g = warp == 10 ? 0 : 1;
        KrWalk<D> pw = walk;
        Kv8Seg ps;
        uint32_t i = 0, seg = 0;             // this group's next tile to score, its group of rows
        int t = 0;
        bool more = walk.next(a, s), pmore = pw.next(a, ps);
        if (more) t = s.t0;
        auto step = [&](int n) {             // n tiles on
#pragma unroll 1
            for (; more && n > 0; --n) {
                ++i;
                if (++t == s.t1) {
                    ++seg;
                    more = walk.next(a, s);
                    t = s.t0;
                }
            }
        };
        auto scores = [&]() {                // by the elected lane
            const uint64_t kd = kv8_desc_rows<D>(kring + (i % C::NK) * C::TILE), qd = kv8_desc_rows<D>(base + (seg & 1) * C::QBYTES);
#pragma unroll
            for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    kv8_mma(tmem + KR_S + g * 128, qd + (lo * 128 * D >> 4) + k * 2, kd + k * 2, lo ? id_lo : id_s, lo | k);
            mma_commit(smem_u32(&k_empty[i % C::NK]));
            mma_commit(smem_u32(&s_full[g]));
        };
        step(g);
        if (more) {
            ok = wait(q_full[seg & 1], seg >> 1) && wait(k_full[i], 0);
            if (ok && kv8_elect()) scores();
            __syncwarp();
            step(2);
        }
        uint32_t j = 0;
#pragma unroll 1
        while (ok && pmore) {
#pragma unroll 1
            for (int pt = ps.t0; pt < ps.t1; ++pt, ++j) {
                if ((int)(j & 1) != g) continue;
                const int sl = (int)(j % C::NV);
                // the queries of a group two after the product's need that group's end: not waited for
                // before its last product
                const bool with = more && (t - s.t0 >= 2 || __all_sync(FULL, mbar_test(smem_u32(&q_full[seg & 1]), (seg >> 1) & 1)));
                // (the turn ahead of the keys: a slot whose tiles go to both issuers can be waited for only when its
                // phase before is complete, and the other issuer has waited for that one before it passes the turn)
                ok = wait(v_full[sl], j / C::NV) && (j == 0 || wait(turn[g], g ? j >> 1 : (j >> 1) - 1)) &&
                     (!more || wait(k_full[i % C::NK], i / C::NK)) && wait(p_full[g], j >> 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = kv8_desc_v16<D>(vring + sl * 2 * C::TILE);
                const uint32_t keep = pt - ps.t0 >= 2 ? 1u : 0u;      // not its group's first tile
                const int span = kr_span(ps.n * G);
                if (kv8_elect()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // lanes not written: all but the span that has keys 16 k ..
                        uint32_t off[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) off[q] = q * 32 / span == k * 16 / span ? 0u : 0xffffffffu;
                        kv8_mma_f16_ts(tmem + KR_O + g * 128, tmem + KR_S + g * 128 + k / 2 * 32 + (k & 1) * 8, vd + k * (2 * D * 16 >> 4), id_o, off,
                                       k * 16 & (span - 1) ? 1u : keep);
                    }
                    mma_commit(smem_u32(&v_empty[sl]));
                    if (pt + 2 >= ps.t1) mma_commit(smem_u32(&o_done[g]));
                    if (with) scores();
                    mbar_arrive(smem_u32(&turn[g ^ 1]));
                }
                __syncwarp();
                if (more && !with) {
                    ok = wait(q_full[seg & 1], seg >> 1);
                    if (!ok) break;
                    if (kv8_elect()) scores();
                    __syncwarp();
                }
                step(2);
            }
            pmore = ok && pw.next(a, ps);
        }
        if (!ok) abort_flag = 1;
        if (kv8_elect()) mma_commit(smem_u32(&done_bar[g]));     // nothing may still write tensor memory when it is freed
        __syncwarp();
        if (!kv8_wait(done_bar[g], 0)) abort_flag = 1;
    } else {
        // ---- softmax: thread = lane of its group's accumulators ----
        const int grp = warp >> 2, j = (warp & 3) * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = tl + KR_S + grp * 128, to = tl + KR_O + grp * 128;
        uint32_t i = 0, seg = 0, parts = 0, win = 0; // tiles and groups of the run; groups that this one had tiles of; windows
        bool begun = false;
#pragma unroll 1
        while (ok && walk.next(a, s)) {
            if (threadIdx.x == 0) kv8_note(runs[blockIdx.x], s, begun);
            const int R = s.n * G, span = kr_span(R), r = j & (span - 1);
            const int nchk = span >> 5, c0 = (j / span) * nchk;         // chunks of 32 keys of a tile, the first of this copy
            const int lim = r < R ? s.len - s.n + r / G : -1;           // the last key this row sees
            float ref = -INFINITY, l = 0.0f, rq = 0.0f;
            bool any = false;                                           // this group had a tile
#pragma unroll 1
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int w = (t - s.t0) & (KR_WIN - 1);
                if (w == 0) {
                    ok = wait(m_full[win & 1], win >> 1);
                    if (!ok) break;
                }
                const bool last_of = w == KR_WIN - 1 || t + 1 == s.t1;       // of its window
                if ((int)(i & 1) != grp) {
                    if (last_of && lane == 0) mbar_arrive(smem_u32(&m_empty[win & 1]));
                    win += last_of;
                    continue;
                }
                const float4* tm = meta[win & 1] + w * 8;
                ok = wait(s_full[grp], i >> 1);
                if (!ok) break;
                tc_fence_after();
                rq = qs[seg & 1][j];
                const bool masked = (t + 1) * KV8_TILE > s.len - s.n + 1 || __any_sync(FULL, tm[lane & 7].x < 0.0f);
                float x[32];
                float mx = -INFINITY;
                // the raw scores of chunk c; -inf where there is no key
                auto load = [&](int c) {
                    kv8_tmem_ld32(ts + c * 32, x);
                    kv8_tmem_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) asm volatile("" : "+f"(x[e]));
                    if (masked) {
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const int last = tm[2 * c + p].x < 0.0f ? -1 : lim - t * KV8_TILE - c * 32;
#pragma unroll
                            for (int e = p * 16; e < p * 16 + 16; ++e)
                                if (e > last) x[e] = -INFINITY;
                        }
                    }
                };
#pragma unroll 1
                for (int u = 0; u < nchk; ++u) {
                    load(c0 + u);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        float m = -INFINITY;
#pragma unroll
                        for (int e = p * 16; e < p * 16 + 16; e += 2) m = fmaxf(fmaxf(m, x[e]), x[e + 1]);
                        const float4 pm = tm[2 * (c0 + u) + p];
                        mx = fmaxf(mx, fmaf(m, kv8_factor(pm.x, rq), pm.y));
                    }
                }
                if (__any_sync(FULL, mx > ref + KR_MOVE)) {
                    const bool move = mx > ref + KR_MOVE;
                    // in two halves: with value scales far apart the factor can be below the smallest
                    // float where the sum times it is not
                    const float ah = move ? kv8_exp2(0.5f * (ref - mx)) : 1.0f, al = ah * ah;
                    if (move) ref = mx;
                    l = l * ah * ah;
                    // the scores' commit came after the product of this group's tile before: the output
                    // is at rest
                    if (any) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            kv8_tmem_ld32(to + c, o);
                            kv8_tmem_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                asm volatile("" : "+f"(o[e]));
                                o[e] *= al;
                            }
                            kv8_tmem_st32(to + c, o);
                        }
                    }
                }
                const float sub = KR_LEAD - (ref == -INFINITY ? 0.0f : ref);
                float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
                for (int u = nchk - 1; u >= 0; --u) {
                    const int c = c0 + u;
                    if (u < nchk - 1) load(c);           // the last chunk is still here
                    float h[16];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float4 pm = tm[2 * c + p];
                        const float vs = pm.z, sc = kv8_factor(pm.x, rq);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 y = kv8_fma2(make_float2(x[p * 16 + e], x[p * 16 + e + 1]), make_float2(sc, sc), make_float2(sub, sub));
                            const float2 z = make_float2(kv8_exp2(y.x), kv8_exp2(y.y));
                            sum = kv8_add2(sum, z);
                            const float2 w = kv8_mul2(z, make_float2(vs, vs));
                            h[p * 8 + e / 2] = __uint_as_float(kv8_half2(w.x, w.y));
                        }
                    }
                    kv8_tmem_st16(ts + c * 32, h);
                }
                l += sum.x + sum.y;
                kv8_tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&p_full[grp]));
                    if (last_of) mbar_arrive(smem_u32(&m_empty[win & 1]));
                }
                win += last_of;
                any = true;
            }
            if (ok && any) {
                ok = wait(o_done[grp], parts);
                ++parts;
            }
            tc_fence_after();
            // ---- the part's rows: the copies' and both groups' outputs, weighed, added through the
            // group's query buffer (its scores are done), 32 dimensions at a time ----
            ml[grp][j] = any ? make_float2(ref, l) : make_float2(-INFINITY, 0.0f);
            if (kv8_rows_any(!ok)) {
                ok = false;
                break;
            }
            const int nl = 256 / span;               // lanes of a row: copies x groups
            float m = -INFINITY, ls = 0.0f;
#pragma unroll 2
            for (int k = 0; k < nl; ++k) m = fmaxf(m, ml[k & 1][(k >> 1) * span + r].x);
            const float at = m == -INFINITY ? 0.0f : m;
#pragma unroll 2
            for (int k = 0; k < nl; ++k) {
                const float2 v = ml[k & 1][(k >> 1) * span + r];
                const float w = kv8_exp2(0.5f * (v.x - at));
                ls = fmaf(v.y * w, w, ls);
            }
            const bool whole = s.t0 == 0 && s.t1 == s.tiles, none = m == -INFINITY && ls == 0.0f;
            const size_t part = (size_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * KR_ROWS;
            float wt = kv8_exp2(0.5f * (ref - at));
            wt = any ? wt * wt : 0.0f;
            if (whole) wt = none ? 0.0f : wt / ls;
            if (grp == 0 && j < span && r < R) {
                if (!whole) part_ml[part + r] = make_float2(m - KR_LEAD, ls);
                else if (a.lse)
                    a.lse[(size_t)(s.row0 + r / G) * a.hq + s.h * G + r % G] = none ? -INFINITY : 0.6931471805599453f * (m - KR_LEAD + log2f(ls));
            }
            // as many dimensions at a time as the rows leave room for: 32 << wl of them
            float4* stage = reinterpret_cast<float4*>(gbase + (seg & 1) * C::QBYTES);
            int wl = 0;
            while ((64 << wl) <= D && (nl * R << (6 + wl)) <= 8192) ++wl;
            const int W = 32 << wl;
            float4* mine = stage + ((j / span * 2 + grp) * R + r) * (W / 4);
#pragma unroll 1
            for (int c = 0; c < D; c += W) {
#pragma unroll 1
                for (int u = 0; u < W; u += 32) {
                    float o[32];
                    kv8_tmem_ld32(to + c + u, o);
                    kv8_tmem_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) asm volatile("" : "+f"(o[e]));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (r < R)
                            mine[u / 4 + (e ^ (r & 7))] = any ? make_float4(o[4 * e] * wt, o[4 * e + 1] * wt, o[4 * e + 2] * wt, o[4 * e + 3] * wt)
                                                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                kv8_rows_any(0);
#pragma unroll 1
                for (int x = threadIdx.x; x < R * (W / 4); x += 256) {
                    const int q = x >> (3 + wl), d = x & (W / 4 - 1), tt = q / G;
                    const float4* from = stage + q * (W / 4) + (d ^ (q & 7));
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
                    for (int k = 0; k < nl; ++k) {
                        const float4 y = from[k * R * (W / 4)];
                        v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
                    }
                    if (whole) {
                        const __nv_bfloat162 y[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
                        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (long long)(s.row0 + tt) * a.o_stride +
                                                  (size_t)(s.h * G + q - tt * G) * D + c + d * 4) = *reinterpret_cast<const uint2*>(y);
                    } else {
                        *reinterpret_cast<float4*>(part_o + (part + q) * D + c + d * 4) = v;
                    }
                }
                if (c + W < D) kv8_rows_any(0);
            }
            // (ml, the buffer: the next group's first are behind a barrier of both groups)
            tc_fence_before();
            if (lane == 0) mbar_arrive(smem_u32(&q_free[seg & 1]));
            ++seg;
        }
        if (!ok) {
            // a bounded wait gave up: the remaining rows of this block become NaN
            abort_flag = 1;
#pragma unroll 1
            do {
                if (threadIdx.x == 0) kv8_note(runs[blockIdx.x], s, begun);
                const size_t part = (size_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * KR_ROWS;
#pragma unroll 1
                for (int q = threadIdx.x; q < s.n * G; q += 256) {
                    const int tt = q / G;
                    if (s.t0 == 0 && s.t1 == s.tiles) {
#pragma unroll 1
                        for (int d = 0; d < D; ++d)
                            static_cast<__nv_bfloat16*>(a.out)[(long long)(s.row0 + tt) * a.o_stride + (size_t)(s.h * G + q - tt * G) * D + d] =
                                __float2bfloat16_rn(__uint_as_float(0x7fc00000u));
                        if (a.lse) a.lse[(size_t)(s.row0 + tt) * a.hq + s.h * G + q - tt * G] = __uint_as_float(0x7fc00000u);
                    } else
                        part_ml[part + q] = make_float2(__uint_as_float(0x7fc00000u), 1.0f);
                }
            } while (walk.next(a, s));
        }
    }
    kv8_finish(after);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && abort_flag) kv8_report(a.err);
    if (warp == 10) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512u) : "memory");
}

template <int D> static cudaError_t rows_launch(const Kv8Attn& a, const Kv8Parts& parts, bool after, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(kv8_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)KrCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    return kv8_launch(kv8_rows_kernel<D>, dim3(KV8_RUNS), KR_THREADS, KrCfg<D>::SMEM, st, a, parts.o, parts.ml, parts.runs, after);
}

cudaError_t kv8_rows_attention(const Kv8Attn& a, int D, const Kv8Parts& parts, bool after, cudaStream_t st) {
    return D == 128 ? rows_launch<128>(a, parts, after, st) : rows_launch<64>(a, parts, after, st);
}

}  // namespace sv
