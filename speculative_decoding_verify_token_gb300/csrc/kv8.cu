// The page plan and the quantising append of the 8-bit paged KV cache.
//
// Plan: block tables, slot maps and row positions of a batch from its lengths, on the
// device, because after a verify pass only the device knows how many drafts were accepted.
//
// Append: per page, head and side the scale is 2^e with the smallest e >= -64 such that the
// largest value is at most 448 * 2^e, over the tokens kept in the page and the new ones.  A
// power of two loses nothing against the exact quotient, since e4m3 is a floating format
// and a scale only moves its range, and it makes re-scaling exact: when new tokens move a
// page's scale, the kept codes only change their exponent (bits are lost only where a code
// falls into the subnormal range).  The scale is a function of the page's tokens alone, so a
// page that held rejected drafts gets back the scale it would have had without them, but not the
// bits of kept codes that fell below the smallest step of a larger draft's scale.
#include <algorithm>

#include <cuda_bf16.h>
#include <cmath>

#include "common.cuh"
#include "host_util.h"
#include "kv8.cuh"

namespace sv {

// ---- plan ---------------------------------------------------------------------------------

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_MAX_B = 8192;
constexpr int PLAN_PER = PLAN_MAX_B / PLAN_THREADS;

struct PlanArgs {
    int B, max_pages, max_rows, free_cap;
    const int *kv_len, *new_len, *held, *free_pages, *n_free;
    int *block_table, *row_start, *kv_out, *held_out;
    long long* slots;
    int *positions, *row_seq, *status;
};

// Inclusive scan over the block of two 64-bit sums per thread.
__device__ __forceinline__ void plan_scan(long long& x, long long& y, long long (&sh)[2][PLAN_THREADS / 32]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(FULL, x, o), b = __shfl_up_sync(FULL, y, o);
        if (lane >= o) { x += a; y += b; }
    }
    __syncthreads();
    if (lane == 31) { sh[0][w] = x; sh[1][w] = y; }
    __syncthreads();
    long long a = 0, b = 0;
    for (int i = 0; i < w; ++i) { a += sh[0][i]; b += sh[1][i]; }
    x += a;
    y += b;
}

// Every block scans all sequences (a few thousand numbers from L2) and then writes its share
// of the tables and rows: one launch, no block waits for another.  Bound by latency up to
// some ten thousand rows, then by the 16 bytes written per row (a call of 32 or of 1,000
// sequences takes 10.5 us, the host's share).
__global__ void __launch_bounds__(PLAN_THREADS) kv8_plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int plan_sh[];
    __shared__ long long sh[2][PLAN_THREADS / 32];
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int failed, used;
    int* s_row = plan_sh;               // [B + 1] first row
    int* s_base = s_row + a.B + 1;      // [B] pages taken by the sequences before
    int* s_held = s_base + a.B;         // [B] pages held before
    int* s_take = s_held + a.B;         // [B] pages taken
    const int per = (a.B + PLAN_THREADS - 1) / PLAN_THREADS;
    const int b0 = threadIdx.x * per;
    const int n_free = min(max(*a.n_free, 0), a.free_cap);
    if (threadIdx.x == 0) failed = used = 0;
    long long need_sum = 0, row_sum = 0;
    int need[PLAN_PER], rows[PLAN_PER], asked[PLAN_PER], held[PLAN_PER], kv[PLAN_PER];
#pragma unroll
    for (int i = 0; i < PLAN_PER; ++i) {
        need[i] = rows[i] = asked[i] = held[i] = kv[i] = 0;
        const int b = b0 + i;
        if (i < per && b < a.B) {
            kv[i] = max(a.kv_len[b], 0);
            asked[i] = max(a.new_len[b], 0);
            held[i] = min(max(a.held[b], 0), a.max_pages);
            const long long want = ((long long)kv[i] + asked[i] + 15) >> 4;
            if (want <= a.max_pages) {
                need[i] = max((int)want - held[i], 0);
                rows[i] = asked[i];
            } else {
                need[i] = -1;           // never granted
            }
            need_sum += max(need[i], 0);
            row_sum += rows[i];
        }
    }
    long long need_end = need_sum, row_end = row_sum;
    plan_scan(need_end, row_end, sh);
    long long np = need_end - need_sum, nr = row_end - row_sum;
    long long got_rows = 0, zero = 0;
#pragma unroll
    for (int i = 0; i < PLAN_PER; ++i) {
        const int b = b0 + i;
        if (i < per && b < a.B) {
            const int nd = max(need[i], 0);
            const bool ok = need[i] >= 0 && (nd == 0 || np + nd <= n_free) && nr + rows[i] <= a.max_rows;
            s_base[b] = (int)min(np, (long long)a.free_cap);
            s_held[b] = held[i];
            s_take[b] = ok ? nd : 0;
            if (!ok && asked[i] > 0) atomicAdd(&failed, 1);
            if (ok && nd > 0) atomicMax(&used, (int)(np + nd));
            np += nd;
            nr += rows[i];
            if (!ok) rows[i] = 0;
            got_rows += rows[i];
        }
    }
    long long got_end = got_rows;
    plan_scan(got_end, zero, sh);
    int first = (int)(got_end - got_rows);
#pragma unroll
    for (int i = 0; i < PLAN_PER; ++i) {
        const int b = b0 + i;
        if (i < per && b < a.B) {
            s_row[b] = first;
            first += rows[i];
            if (b == a.B - 1) s_row[a.B] = first;
            if (blockIdx.x == 0) {
                a.row_start[b] = s_row[b];
                a.kv_out[b] = kv[i] + rows[i];
                a.held_out[b] = held[i] + s_take[b];
                if (b == a.B - 1) a.row_start[a.B] = first;
            }
        }
    }
    __syncthreads();
    const int total = s_row[a.B];
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.status[0] = n_free - used;
        a.status[1] = total;
        a.status[2] = failed;
    }
    // a sequence's new pages: a warp each
    const int lane = threadIdx.x & 31;
    for (int b = blockIdx.x * (PLAN_THREADS / 32) + (threadIdx.x >> 5); b < a.B; b += gridDim.x * (PLAN_THREADS / 32)) {
        const int take = s_take[b], top = n_free - 1 - s_base[b];
        for (int j = lane; j < take; j += 32)
            a.block_table[(size_t)b * a.max_pages + s_held[b] + j] = a.free_pages[top - j];
    }
    // the rows: sequence by bisection, page from the list where it is new
    for (int r = blockIdx.x * PLAN_THREADS + threadIdx.x; r < a.max_rows; r += gridDim.x * PLAN_THREADS) {
        long long slot = -1;
        int pos = 0, b = -1;
        if (r < total) {
            int lo = 0, hi = a.B;       // s_row[lo] <= r < s_row[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_row[mid] <= r) lo = mid; else hi = mid;
            }
            b = lo;
            pos = max(a.kv_len[b], 0) + r - s_row[b];
            const int lp = pos >> 4;
            const int page = lp >= s_held[b] ? a.free_pages[n_free - 1 - s_base[b] - (lp - s_held[b])]
                                             : a.block_table[(size_t)b * a.max_pages + lp];
            if (page >= 0) slot = (long long)page * KV8_PAGE + (pos & 15);
        }
        a.slots[r] = slot;
        a.positions[r] = pos;
        a.row_seq[r] = b;
    }
}

// ---- append -------------------------------------------------------------------------------

// Four consecutive elements as loaded, and as floats.
template <typename T> struct Four;
template <> struct Four<float> {
    float4 x;
    __device__ __forceinline__ void load(const float* p) { x = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void zero() { x = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w; }
    // largest magnitude's bits so far, on top of m
    __device__ __forceinline__ uint32_t top(uint32_t m) const {
        return max(max(max(m, __float_as_uint(x.x) & 0x7fffffffu), max(__float_as_uint(x.y) & 0x7fffffffu, __float_as_uint(x.z) & 0x7fffffffu)),
                   __float_as_uint(x.w) & 0x7fffffffu);
    }
    static __device__ __forceinline__ float top_value(uint32_t m) { return __uint_as_float(m); }
};
template <> struct Four<__nv_bfloat16> {
    uint2 x;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void zero() { x = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float (&f)[4]) const {
        f[0] = __uint_as_float(x.x << 16); f[1] = __uint_as_float(x.x & 0xffff0000u);
        f[2] = __uint_as_float(x.y << 16); f[3] = __uint_as_float(x.y & 0xffff0000u);
    }
    __device__ __forceinline__ uint32_t top(uint32_t m) const {
        return __vmaxu2(m, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu));
    }
    static __device__ __forceinline__ float top_value(uint32_t m) { return __uint_as_float(max(m & 0xffffu, m >> 16) << 16); }
};

__device__ __forceinline__ bool finite_f(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// A kept code's value: 256 * 2^120, which the largest floats round to, is past FLT_MAX.
__device__ __forceinline__ float kept_value(float code, float scale) {
    const float x = code * scale;
    return fabsf(x) == INFINITY ? copysignf(3.402823466e38f, x) : x;
}

// The exponent of the smallest power of two s >= 2^-64 with amax <= 448 s.
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 126 - 9 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, KV8_MIN_EXP);
}

// The bytes of a little-endian word that lie below index n (all from 4 on, none up to 0).
__device__ __forceinline__ uint32_t kv8_first_bytes(int n) { return n >= 4 ? 0xffffffffu : (n <= 0 ? 0u : (1u << (8 * n)) - 1); }

// 4 x 4 bytes transposed: w[j] byte e = u[e] byte j.
__device__ __forceinline__ void kv8_turn4(const uint32_t (&u)[4], uint32_t (&w)[4]) {
    const uint32_t x = __byte_perm(u[0], u[1], 0x5140), y = __byte_perm(u[2], u[3], 0x5140);
    const uint32_t z = __byte_perm(u[0], u[1], 0x7362), q = __byte_perm(u[2], u[3], 0x7362);
    w[0] = __byte_perm(x, y, 0x5410);
    w[1] = __byte_perm(x, y, 0x7632);
    w[2] = __byte_perm(z, q, 0x5410);
    w[3] = __byte_perm(z, q, 0x7632);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

constexpr int APPEND_THREADS = 128;

// One warp takes one (page with a new token, kv head): it reads the page's kept codes and
// its new rows, finds both scales and writes both blocks whole, with zeros behind the last
// token, so that a page in use never holds what its memory held before.  A lane has 4
// dimensions of 16 (D = 64: of 8) tokens; its values' tokens are then consecutive bytes.
// A token with a NaN or an infinity gets NaN keys and zero values: the rows that see it
// become NaN and no other row does (a probability of zero times a NaN would be NaN).
// Blocks take 16 consecutive rows; the pages' first new rows ("leaders") are the items.
// Bound by the bytes read and written; 8k rows of 8 heads of 128 take 14 us of the kernel and 17 of
// a call (46% of the copy rate), 5 rows 5.5 us, mostly three dependent loads (the row's
// sequence, its page, the kept codes).
template <typename T, int D>
__global__ void __launch_bounds__(APPEND_THREADS, sizeof(T) == 2 ? 4 : 2) kv8_append_kernel(const __grid_constant__ Kv8Append a) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int DL = D / 4;                // lanes of one token
    constexpr int NT = 16 * DL / 32;         // tokens of a lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dim = (lane % DL) * 4, t0 = (lane / DL) * NT;
    // sequence and position of row 16 * blockIdx.x + lane (every warp for itself)
    const int r = blockIdx.x * 16 + lane;
    int seq = -1, pos = -1, first = 0, row0 = 0, len = 0;
    if (a.row_start && a.B < 32) {
        // up to 31 sequences: all starts and lengths in one load each, bisected by shuffles
        const int st = lane <= a.B ? a.row_start[lane] : 0x7fffffff, kv = lane < a.B ? a.kv_len[lane] : 0;
        int lo = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int v = __shfl_sync(FULL, st, lo + o);
            if (v <= r) lo += o;
        }
        row0 = __shfl_sync(FULL, st, lo);
        const int end = __shfl_sync(FULL, st, (lo + 1) & 31);
        len = __shfl_sync(FULL, kv, lo);
        if (lane < 16 && r < a.n_rows && lo < a.B && row0 <= r && r < end) {
            seq = lo;
            first = row0 - end + len;
            pos = first + r - row0;
        }
    } else if (lane < 16 && r < a.n_rows) {
        if (a.row_start) {
            if (r >= a.row_start[0] && r < a.row_start[a.B]) {
                int lo = 0, hi = a.B;
#pragma unroll 1
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (a.row_start[mid] <= r) lo = mid; else hi = mid;
                }
                seq = lo;
                row0 = a.row_start[lo];
                len = a.kv_len[lo];
                first = row0 - a.row_start[lo + 1] + len;
                pos = first + r - row0;
            }
        } else if (r < a.B * a.T) {
            row0 = r / a.T * a.T;
            seq = a.seq_ids ? a.seq_ids[r / a.T] : r / a.T;
            if (seq >= 0 && seq < a.n_tables) {
                len = a.kv_len[seq] + a.kv_add;
                first = len - a.T;
                pos = first + r - row0;
            }
        }
    }
    const bool leader = pos >= 0 && ((pos & 15) == 0 || r == row0) && (pos >> 4) < a.max_pages;
    const unsigned todo = __ballot_sync(FULL, leader);
    const int rank = leader ? __popc(todo & ((1u << lane) - 1)) : -1;
    const int n_items = __popc(todo) * a.hkv;
    constexpr int W = APPEND_THREADS / 32;
    const int step = gridDim.y * W;
#pragma unroll 1
    for (int it = blockIdx.y * W + warp; it < n_items; it += step) {
        const int src = __ffs(__ballot_sync(FULL, rank == it / a.hkv)) - 1, h = it % a.hkv;
        const int pos0 = __shfl_sync(FULL, pos, src), len0 = __shfl_sync(FULL, len, src);
        const int r0 = blockIdx.x * 16 + src;
        const int table = __shfl_sync(FULL, seq, src);
        const int page = a.block_table[(size_t)table * a.max_pages + (pos0 >> 4)];
        const int kept = pos0 & 15;                                   // tokens [0, kept) stay
        const int end = min(len0 - (pos0 & ~15), 16);                 // [kept, end) are new
        // both sides' new elements are asked for at once, beside the page's number and kept as they came (a lane of bf16 holds
        // 64 registers of them, so that 16 warps fit an SM)
        Four<T> kr[NT], vr[NT];
        const bool staged = a.stage_pages > 0;
        const long long ks = staged ? D : a.k_stride, vs = staged ? D : a.v_stride;
        const long long at = staged ? ((long long)table * a.stage_pages + (pos0 >> 4) % a.stage_pages) * a.hkv * 16 * D + (long long)h * 16 * D + dim
                                    : (long long)h * D + dim;
        const long long r_at = staged ? 0 : r0 - kept;                // row of token 0
        const T* kp = static_cast<const T*>(a.k) + at;
        const T* vp = static_cast<const T*>(a.v) + at;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int t = t0 + i, row = r0 + t - kept;
            kr[i].zero();
            vr[i].zero();
            if (t >= kept && t < end && row < a.n_rows) {
                kr[i].load(kp + (r_at + t) * ks);
                vr[i].load(vp + (r_at + t) * vs);
            }
        }
        if (page < 0 || page >= a.num_pages) continue;
        uint8_t* kb = a.pool + ((size_t)page * a.hkv + h) * 2 * (16 * D);
        uint8_t* vb = kb + 16 * D;
        float* sc = a.scales + ((size_t)page * a.hkv + h) * 2;
        // the kept tokens' codes, and the page's old scales
        const float sk = kept > 0 ? sc[0] : 0.0f, sv_ = kept > 0 ? sc[1] : 0.0f;
        uint32_t kw[NT], vw[4][NT / 4];
        uint32_t ck = 0, cv = 0;              // largest kept codes, byte by byte
        if (kept > 0) {
#pragma unroll
            for (int i = 0; i < NT / 4; ++i) {
                const uint32_t m = kv8_first_bytes(kept - t0 - 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    vw[j][i] = *reinterpret_cast<const uint32_t*>(vb + (dim + j) * 16 + t0 + i * 4) & m;
                    cv = __vmaxu4(cv, vw[j][i] & 0x7f7f7f7fu);
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                kw[i] = t0 + i < kept ? *reinterpret_cast<const uint32_t*>(kb + kv8_key_off<D>(t0 + i, dim)) : 0u;
                ck = __vmaxu4(ck, kw[i] & 0x7f7f7f7fu);
            }
        }
        // maxima as bit patterns, which order like the magnitudes
        uint32_t tk = 0, tv = 0;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            tk = kr[i].top(tk);
            tv = vr[i].top(tv);
        }
        ck = max(max(ck & 0xff, ck >> 8 & 0xff), max(ck >> 16 & 0xff, ck >> 24));
        cv = max(max(cv & 0xff, cv >> 8 & 0xff), max(cv >> 16 & 0xff, cv >> 24));
        float dk[4], dv[4];
        kv8_decode4(ck, dk);
        kv8_decode4(cv, dv);
        const float nk = Four<T>::top_value(tk), nv = Four<T>::top_value(tv);
        if (__all_sync(FULL, finite_f(nk) && finite_f(nv) && ck != 127 && cv != 127)) {
            // ---- every number finite: kept codes change only when their scale does ----
            const int ek = scale_exp(warp_max(fmaxf(nk, kept > 0 ? kept_value(dk[0], sk) : 0.0f)));
            const int ev = scale_exp(warp_max(fmaxf(nv, kept > 0 ? kept_value(dv[0], sv_) : 0.0f)));
            const float ik = exp2_int(-ek), iv = exp2_int(-ev);
            const bool move_k = kept > 0 && exp2_int(ek) != sk, move_v = kept > 0 && exp2_int(ev) != sv_;
            __syncwarp();                     // every lane has read the kept codes
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                uint32_t w;
                if (t0 + i >= kept) {
                    float f[4];
                    kr[i].get(f);
                    w = kv8_encode4(f[0] * ik, f[1] * ik, f[2] * ik, f[3] * ik);
                } else if (move_k) {
                    float f[4];
                    kv8_decode4(kw[i], f);
                    w = kv8_encode4(kept_value(f[0], sk) * ik, kept_value(f[1], sk) * ik, kept_value(f[2], sk) * ik, kept_value(f[3], sk) * ik);
                } else {
                    continue;
                }
                *reinterpret_cast<uint32_t*>(kb + kv8_key_off<D>(t0 + i, dim)) = w;
            }
#pragma unroll
            for (int i = 0; i < NT; i += 4) {
                uint32_t u[4], w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f[4];
                    vr[i + e].get(f);
                    u[e] = kv8_encode4(f[0] * iv, f[1] * iv, f[2] * iv, f[3] * iv);
                }
                kv8_turn4(u, w);              // from dimensions to tokens
                if (kept > 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t old = vw[j][i / 4];
                        if (move_v) {
                            float f[4];
                            kv8_decode4(old, f);
                            old = kv8_encode4(kept_value(f[0], sv_) * iv, kept_value(f[1], sv_) * iv, kept_value(f[2], sv_) * iv, kept_value(f[3], sv_) * iv);
                        }
                        const uint32_t m = kv8_first_bytes(kept - t0 - i);
                        w[j] = (old & m) | (w[j] & ~m);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) vw[j][i / 4] = w[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (NT == 16)
                    *reinterpret_cast<uint4*>(vb + (dim + j) * 16 + t0) = make_uint4(vw[j][0], vw[j][1], vw[j][2], vw[j][3]);
                else
                    *reinterpret_cast<uint2*>(vb + (dim + j) * 16 + t0) = make_uint2(vw[j][0], vw[j][1]);
            }
            if (lane == 0) {
                sc[0] = exp2_int(ek);
                sc[1] = exp2_int(ev);
            }
            continue;
        }
        // ---- a NaN or an infinity among them ----
        auto key = [&](int i, float (&f)[4]) {
            if (t0 + i < kept) {
                kv8_decode4(kw[i], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = kept_value(f[j], sk);
            } else {
                kr[i].get(f);
            }
        };
        auto value = [&](int i, float (&f)[4]) {
            if (t0 + i < kept) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float g[4];
                    kv8_decode4(vw[j][i / 4] >> (8 * (i & 3)), g);
                    f[j] = kept_value(g[0], sv_);
                }
            } else {
                vr[i].get(f);
            }
        };
        float mk = 0.0f, mv = 0.0f;
        unsigned bad = 0;                     // tokens with a NaN or infinity
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float f[4], g[4];
            key(i, f);
            value(i, g);
            bool fin = true;
#pragma unroll
            for (int j = 0; j < 4; ++j) fin = fin && finite_f(f[j]) && finite_f(g[j]);
            if (!fin) bad |= 1u << (t0 + i);
        }
        bad = __reduce_or_sync(FULL, bad);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float f[4], g[4];
            key(i, f);
            value(i, g);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (!(bad >> (t0 + i) & 1)) {
                    mk = fmaxf(mk, fabsf(f[j]));
                    mv = fmaxf(mv, fabsf(g[j]));
                }
        }
        const int ek = scale_exp(warp_max(mk)), ev = scale_exp(warp_max(mv));
        const float ik = exp2_int(-ek), iv = exp2_int(-ev);
        __syncwarp();                         // every lane has read the kept codes
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float f[4];
            key(i, f);
            uint32_t w = kv8_encode4(f[0] * ik, f[1] * ik, f[2] * ik, f[3] * ik);
            if (bad >> (t0 + i) & 1) w = 0x7f7f7f7fu;
            *reinterpret_cast<uint32_t*>(kb + kv8_key_off<D>(t0 + i, dim)) = w;
        }
        // four tokens at a time, turned from dimensions to tokens
        uint32_t w[4][NT / 4];
#pragma unroll
        for (int i = 0; i < NT; i += 4) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float f[4];
                value(i + e, f);
                u[e] = bad >> (t0 + i + e) & 1 ? 0u : kv8_encode4(f[0] * iv, f[1] * iv, f[2] * iv, f[3] * iv);
            }
            uint32_t q[4];
            kv8_turn4(u, q);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j][i / 4] = q[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (NT == 16)
                *reinterpret_cast<uint4*>(vb + (dim + j) * 16 + t0) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
            else
                *reinterpret_cast<uint2*>(vb + (dim + j) * 16 + t0) = make_uint2(w[j][0], w[j][1]);
        }
        if (lane == 0) {
            sc[0] = exp2_int(ek);
            sc[1] = exp2_int(ev);
        }
    }
}

template <typename T>
static cudaError_t append_launch(const Kv8Append& a, int D, cudaStream_t st) {
    const int x = (a.n_rows + 15) / 16;
    // up to 16 leaders and hkv heads in a block: spread over more blocks while the rows alone do
    // not fill the GPU's warps (just as many as there are pages takes 8k rows 2 us longer: a block of
    // rows where one sequence ends and the next begins has twice the pages)
    const int y = std::max(1, std::min(4 * a.hkv, (2432 + x - 1) / x));
    return D == 128 ? kv8_launch(kv8_append_kernel<T, 128>, dim3(x, y), APPEND_THREADS, 0, st, a)
                    : kv8_launch(kv8_append_kernel<T, 64>, dim3(x, y), APPEND_THREADS, 0, st, a);
}

cudaError_t kv8_append(const Kv8Append& a, bool f32, int D, cudaStream_t st) {
    return f32 ? append_launch<float>(a, D, st) : append_launch<__nv_bfloat16>(a, D, st);
}

}  // namespace sv

using namespace sv;

static int launch_status(const char* what, cudaError_t e) {
    return e == cudaSuccess ? SPEC_OK : set_error(SPEC_E_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

extern "C" int spec_kv8_plan(int B, int max_pages, int max_rows, int free_capacity, const int32_t* kv_len,
                             const int32_t* new_len, const int32_t* held, const int32_t* free_pages,
                             const int32_t* n_free, int32_t* block_table, int32_t* row_start, int32_t* kv_len_out,
                             int32_t* held_out, int64_t* slots, int32_t* positions, int32_t* row_seq, int32_t* status,
                             void* stream) {
    clear_error();
    if (B < 1 || max_pages < 1 || max_rows < 0 || free_capacity < 0) return set_error(SPEC_E_INVAL, "bad sizes");
    if (B > PLAN_MAX_B) return set_error(SPEC_E_RANGE, "B=%d above %d", B, PLAN_MAX_B);
    if (max_pages > SPEC_KV8_MAX_TOKENS / SPEC_PAGE_TOKENS)
        return set_error(SPEC_E_RANGE, "max_pages=%d above %d", max_pages, SPEC_KV8_MAX_TOKENS / SPEC_PAGE_TOKENS);
    if (!kv_len || !new_len || !held || !n_free || !block_table || !row_start || !kv_len_out || !held_out || !status ||
        (free_capacity > 0 && !free_pages) || (max_rows > 0 && (!slots || !positions || !row_seq)))
        return set_error(SPEC_E_INVAL, "NULL required pointer");
    // blocks read the inputs while others write: nothing may lie over anything else
    const size_t i4 = sizeof(int32_t), nb = B, nr = max_rows;
    const struct { const char* name; const void* p; size_t bytes, align; } arrays[] = {
        {"kv_len", kv_len, i4 * nb, 4}, {"new_len", new_len, i4 * nb, 4}, {"held", held, i4 * nb, 4},
        {"free_pages", free_pages, i4 * free_capacity, 4}, {"n_free", n_free, i4, 4},
        {"block_table", block_table, i4 * nb * max_pages, 4}, {"row_start", row_start, i4 * (nb + 1), 4},
        {"kv_len_out", kv_len_out, i4 * nb, 4}, {"held_out", held_out, i4 * nb, 4}, {"slots", slots, 8 * nr, 8},
        {"positions", positions, i4 * nr, 4}, {"row_seq", row_seq, i4 * nr, 4}, {"status", status, i4 * 3, 4}};
    constexpr int N_IN = 5, N = sizeof(arrays) / sizeof(arrays[0]);
    for (int i = 0; i < N; ++i) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(arrays[i].p);
        if (p % arrays[i].align) return set_error(SPEC_E_INVAL, "%s is not aligned to its type", arrays[i].name);
        for (int j = 0; i >= N_IN && j < i; ++j) {
            const uintptr_t q = reinterpret_cast<uintptr_t>(arrays[j].p);
            if (arrays[i].bytes && arrays[j].bytes && p < q + arrays[j].bytes && q < p + arrays[i].bytes)
                return set_error(SPEC_E_INVAL, "%s: %s and %s", j < N_IN ? "an output is one of the inputs" : "two outputs are the same array",
                                 arrays[i].name, arrays[j].name);
        }
    }
    PlanArgs a{B, max_pages, max_rows, free_capacity, kv_len, new_len, held, free_pages, n_free, block_table, row_start,
               kv_len_out, held_out, reinterpret_cast<long long*>(slots), positions, row_seq, status};
    const int blocks = std::max(1, std::min((max_rows + PLAN_THREADS - 1) / PLAN_THREADS, 152));
    const size_t smem = sizeof(int) * (4 * (size_t)B + 1);
    if (B > 2048) {                     // (from 32 KB on: the 48 KB that need no opting in hold the static arrays too)
        const cudaError_t e = cudaFuncSetAttribute(kv8_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)(sizeof(int) * (4 * PLAN_MAX_B + 1)));
        if (e != cudaSuccess) return set_error(SPEC_E_CUDA, "plan attributes: %s", cudaGetErrorString(e));
    }
    return launch_status("spec_kv8_plan", kv8_launch(kv8_plan_kernel, dim3(blocks), PLAN_THREADS, smem, static_cast<cudaStream_t>(stream), a));
}

int sv::kv8_cache_checks(int num_pages, int n_kv_heads, int head_dim, int B, int max_pages, int n_rows,
                         const int32_t* block_table, const void* pool, const void* scales) {
    if (num_pages < 1 || n_kv_heads < 1 || B < 1 || max_pages < 1 || n_rows < 0) return set_error(SPEC_E_INVAL, "bad sizes");
    if (head_dim != 64 && head_dim != 128) return set_error(SPEC_E_INVAL, "head_dim=%d is not 64 or 128", head_dim);
    if (max_pages > SPEC_KV8_MAX_TOKENS / SPEC_PAGE_TOKENS || n_kv_heads > 1024 || n_rows > (1 << 24))
        return set_error(SPEC_E_RANGE, "max_pages=%d, n_kv_heads=%d or n_rows=%d too large", max_pages, n_kv_heads, n_rows);
    if (!block_table || !pool || !scales) return set_error(SPEC_E_INVAL, "NULL required pointer");
    if ((reinterpret_cast<uintptr_t>(pool) & 15) || (reinterpret_cast<uintptr_t>(scales) & 7))
        return set_error(SPEC_E_INVAL, "pool must be 16-byte and scales 8-byte aligned");
    if (reinterpret_cast<uintptr_t>(block_table) & 3) return set_error(SPEC_E_INVAL, "block_table is not aligned");
    return SPEC_OK;
}

extern "C" int spec_kv8_append(int num_pages, int n_kv_heads, int head_dim, int B, int max_pages, int n_rows, uint8_t* pool,
                               float* scales, const int32_t* block_table, const int32_t* row_start,
                               const int32_t* kv_len, const void* k, const void* v, int dtype, int64_t k_stride,
                               int64_t v_stride, void* stream) {
    clear_error();
    const int rc = kv8_cache_checks(num_pages, n_kv_heads, head_dim, B, max_pages, n_rows, block_table, pool, scales);
    if (rc != SPEC_OK) return rc;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return set_error(SPEC_E_INVAL, "dtype=%d", dtype);
    if (!row_start || !kv_len || (n_rows > 0 && (!k || !v))) return set_error(SPEC_E_INVAL, "NULL required pointer");
    const int al = dtype == SPEC_F32 ? 16 : 8;
    if ((reinterpret_cast<uintptr_t>(k) % al) || (reinterpret_cast<uintptr_t>(v) % al) || (n_rows > 1 && (k_stride % 4 || v_stride % 4)))
        return set_error(SPEC_E_INVAL, "k and v must be aligned to 4 elements, and so must their row strides");
    if ((reinterpret_cast<uintptr_t>(row_start) | reinterpret_cast<uintptr_t>(kv_len)) & 3)
        return set_error(SPEC_E_INVAL, "row_start and kv_len must be 4-byte aligned");
    if (n_rows == 0) return SPEC_OK;
    Kv8Append a{pool, scales, block_table, num_pages, n_kv_heads, max_pages, B, B, n_rows, nullptr, row_start, 0,
                 kv_len, 0, k, v, k_stride, v_stride, 0};
    return launch_status("spec_kv8_append", kv8_append(a, dtype == SPEC_F32, head_dim, static_cast<cudaStream_t>(stream)));
}
