// The work lists of the 8-bit cache's attention kernels.
//
// The key tiles of all groups (query rows of one sequence and kv head that share a pass over the
// keys) form one list, cut into equal runs, one per block: ragged batches balance by
// themselves, and no host bound on the lengths is needed.  A run's first and last group may
// be shared with its neighbours; those parts leave (max, sum, output) partials behind.  The list
// counts in units of time, some for each tile and, in front of its tiles, some for what the group's
// queries and output cost, so that no run is the last because it has many short groups or
// more rows: with tiles alone 48 ragged decodes took 102 us in the run with 14 groups and 69
// in those with two.
//
// Two lists: sequences of up to 128 rows per kv head (rows = new tokens x G query heads) have
// one group per kv head ("rows"); longer ones are cut into blocks of 2 x floor(128 / G) tokens
// ("blocks"), whose tiles end at the block's last token.
#pragma once

#include "common.cuh"
#include "kv8.cuh"

namespace sv {

constexpr int KV8_RUNS = 152;           // runs, one per SM of a GB300
constexpr int KV8_TILE = 128;           // keys of a tile
constexpr int KR_ROWS = 128;            // most rows of a group of the rows list
constexpr int KB_ROWS = 256;            // most rows of a group of the blocks list
constexpr int KB_EXTRA = 6;             // units of a group of the blocks list besides its tiles

// ---- the rows list ----

// Tiles of sequence b per kv head.
__device__ __forceinline__ int kr_tiles(const Kv8Attn& a, int b, int& slot, int& row0, int& n, int& len) {
    kv8_sequence(a, b, slot, row0, n, len);
    return n > 0 && (long long)n * (a.hq / a.hkv) <= KR_ROWS ? (len + KV8_TILE - 1) / KV8_TILE : 0;
}

// Units (of some 0.2 us) of a tile and of the rest of a group of R rows, mostly the wait for its queries.  Batches of
// 32 sequences to 16k, D = 128: a tile takes 0.84, 0.98 and 1.4 us, the rest of a group 4.4, 6.2 and 8.1 to 9.3;
// 48 sequences to 8k, D = 64: 0.7, 0.96 and 1.2, and 2.7 to 3.2.  The extras are those whose runs end closest to
// each other (32 verify passes: 152 us with 12, 22 and 26 for both, 143 with these; 48 decodes 80 and 73).
__device__ __forceinline__ int kr_weight(int R) { return R <= 32 ? 4 : (R <= 64 ? 5 : 6); }
template <int D> __device__ __forceinline__ int kr_extra(int R) {
    return D == 64 ? (R <= 32 ? 18 : (R <= 64 ? 26 : 32)) : (R <= 32 ? 24 : (R <= 64 ? 36 : 46));
}

// Units of a kv head of n > 0 tokens, and the first tile of a run that begins at unit u of it.
template <int D> __device__ __forceinline__ int kr_group(const Kv8Attn& a, int n, int tiles) {
    const int R = n * (a.hq / a.hkv);
    return tiles * kr_weight(R) + kr_extra<D>(R);
}
template <int D> __device__ __forceinline__ int kr_tile_of(const Kv8Attn& a, int n, int u) {
    const int R = n * (a.hq / a.hkv), w = kr_weight(R);
    return max(u - kr_extra<D>(R) + w - 1, 0) / w;
}

// Units of all kv heads of sequence b.
template <int D> __device__ __forceinline__ long long kr_units(const Kv8Attn& a, int b) {
    int slot, row0, n, len;
    const int tiles = kr_tiles(a, b, slot, row0, n, len);
    return tiles ? (long long)kr_group<D>(a, n, tiles) * a.hkv : 0;
}

// ---- the blocks list ----

__device__ __forceinline__ int kb_half(const Kv8Attn& a) { return 128 / (a.hq / a.hkv); }    // tokens of 128 rows

// Keys that block rb of a sequence sees, its last token's.
__device__ __forceinline__ int kb_keys(int n, int len, int tb, int rb) {
    return max(0, (int)min((long long)len, (long long)len - n + (long long)tb * (rb + 1)));
}

// Sum of floor((a i + b) / 128) for i < n (a, b >= 0), by the Euclidean recursion on (a, 128): the steps
// are those of the floor sum in public algorithm libraries (the AtCoder Library, CC0).
// n a + b stays below 2^32: a call has at most 2^24 rows, so n a does by 2^24 tokens.
__device__ __forceinline__ long long kv8_floor_sum(uint32_t n, uint32_t a, uint32_t b) {
    uint32_t m = KV8_TILE;
    unsigned long long sum = 0;
#pragma unroll 1
    while (n > 0) {
        if (a >= m) { sum += (unsigned long long)n * (n - 1) / 2 * (a / m); a %= m; }
        if (b >= m) { sum += (unsigned long long)n * (b / m); b %= m; }
        const uint32_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return (long long)sum;
}

// Units of the first k blocks of a sequence of nb blocks.
__device__ __forceinline__ long long kb_prefix(int n, int len, int tb, int nb, int k) {
    long long sum = (long long)k * KB_EXTRA;
    if (k == nb) { sum += (len + KV8_TILE - 1) / KV8_TILE; --k; }
    // block r - 1 (r = 1 .. k) sees len - n + tb r keys, none while that is negative; whole
    // tiles of the keys before the first block (up to 2^27) are taken out of the sum
    const int c = len - n;
    const int r0 = c >= 0 ? 1 : max(1, (-c) / tb);
    if (k >= r0) {
        int first = c + tb * r0, cnt = k - r0 + 1;
        if (first < 0) { first += tb; --cnt; }
        sum += (long long)cnt * (first / KV8_TILE) + kv8_floor_sum(cnt, tb, first % KV8_TILE + KV8_TILE - 1);
    }
    return sum;
}

__device__ __forceinline__ int kb_blocks(const Kv8Attn& a, int n) {
    if (n <= 0 || (long long)n * (a.hq / a.hkv) <= KR_ROWS) return 0;
    const int tb = 2 * kb_half(a);
    return (n + tb - 1) / tb;
}

// Units of all kv heads of sequence b.
__device__ __forceinline__ long long kb_units(const Kv8Attn& a, int b) {
    int slot, row0, n, len;
    kv8_sequence(a, b, slot, row0, n, len);
    const int nb = kb_blocks(a, n);
    return nb > 0 && len > 0 ? kb_prefix(n, len, 2 * kb_half(a), nb, nb) * a.hkv : 0;
}

// ---- both ----

// First unit of run c: equal runs, the first ones a unit longer when `total` is no multiple of
// their number (with fewer units the last are empty).
__device__ __forceinline__ long long kv8_run_begin(long long total, int c) {
    const long long q = (long long)((unsigned long long)total / KV8_RUNS);
    return q * c + min((long long)c, total - q * KV8_RUNS);
}

// All threads of a block (whole warps): the list's length, and the sequence that holds index at(length) of it
// with that sequence's first index (b = a.B when there is none).  count(b) = its units over
// all kv heads; sh: 36 long longs.
template <typename N, typename F>
__device__ __forceinline__ long long kv8_find(int B, long long* sh, N count, F at, int& b_out, long long& base_out) {
    const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nw = (T + 31) >> 5;
    if (B <= 32) {
        // every warp for itself: one round of loads, no barrier (3,700 clocks less of a short call)
        const long long mine = lane < B ? count(lane) : 0;
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL, x, o);
            if (lane >= o) x += y;
        }
        const long long total = __shfl_sync(FULL, x, 31);
        const unsigned past = __ballot_sync(FULL, at(total) < x);
        b_out = past ? __ffs(past) - 1 : B;
        base_out = __shfl_sync(FULL, x - mine, past ? __ffs(past) - 1 : 0);
        return total;
    }
    const int per = (B + T - 1) / T, b0 = tid * per, b1 = min(B, b0 + per);
    long long mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += count(b);
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh[w] = x;
    if (tid == 0) { sh[32] = B; sh[33] = 0; }
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll 1
    for (int i = 0; i < nw; ++i) {
        if (i == w) before = total;
        total += sh[i];
    }
    const long long target = at(total), lo = before + x - mine;
    if (target >= lo && target < lo + mine) {
        long long base = lo;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const long long c = count(b);
            if (target < base + c) { sh[32] = b; sh[33] = base; break; }
            base += c;
        }
    }
    __syncthreads();
    b_out = (int)sh[32];
    base_out = sh[33];
    return total;
}

// Tiles [t0, t1) of a group's `tiles`.
struct Kv8Seg {
    int b, h, rb, t0, t1, tiles, slot, row0, n, len;
};

// What a run leaves for the join of the groups that it shares with others: its first part's place in
// its group, and, when its last part opens a group that others go on with, that group.
constexpr int KV8_NONE = 0, KV8_NEW = 1, KV8_MIDDLE = 2, KV8_END = 3;    // no part; a group's first, an inner, its last part
struct __align__(16) Kv8Run {
    int first, open, row0, n, h, rb, pad[2];
};
// The workspace of a list: per run two parts' outputs and (maximum, sum) pairs, and its note.
struct Kv8Parts {
    float* o;
    float2* ml;
    Kv8Run* runs;
};
__device__ __forceinline__ void kv8_note(Kv8Run& r, const Kv8Seg& s, bool& begun) {
    if (!begun) r.first = s.t0 == 0 ? KV8_NEW : (s.t1 == s.tiles ? KV8_END : KV8_MIDDLE);
    begun = true;
    if (s.t0 == 0 && s.t1 < s.tiles) {
        r.open = 1;
        r.row0 = s.row0; r.n = s.n; r.h = s.h; r.rb = s.rb;
    }
}

// Walks the run [pos, end) of the rows list; b holds pos, its first unit is index base.
template <int D> struct KrWalk {
    long long left;                 // units of the run still to come
    long long at;                   // offset in sequence b's units (of all kv heads)
    int b, tiles, slot, row0, n, len;
    __device__ __forceinline__ void start(const Kv8Attn& a, long long pos, long long end, int b_, long long base) {
        left = end - pos; at = pos - base; b = b_;
        if (left > 0) tiles = kr_tiles(a, b, slot, row0, n, len);
    }
    __device__ __forceinline__ bool next(const Kv8Attn& a, Kv8Seg& s) {
#pragma unroll 1
        while (left > 0) {
#pragma unroll 1
            while (tiles == 0 || at >= (long long)kr_group<D>(a, n, tiles) * a.hkv) {
                at = 0;
                if (++b >= a.B) return false;
                tiles = kr_tiles(a, b, slot, row0, n, len);
            }
            const int units = kr_group<D>(a, n, tiles), h = (int)(at / units), u0 = (int)(at - (long long)h * units);
            const int u1 = left < units - u0 ? u0 + (int)left : units;
            at += u1 - u0;
            left -= u1 - u0;
            s.b = b; s.rb = 0; s.tiles = tiles; s.slot = slot; s.row0 = row0; s.n = n; s.len = len;
            s.h = h;
            s.t0 = kr_tile_of<D>(a, n, u0);
            s.t1 = kr_tile_of<D>(a, n, u1);
            if (s.t1 > s.t0) return true;
        }
        return false;
    }
};

// The blocks list's group at offset `at` of sequence b's units: kv head, block, offset in it.
// Called by whole warps, which try 32 candidates at a time.
__device__ __forceinline__ void kb_locate(const Kv8Attn& a, int n, int len, long long at, int& h, int& rb, int& t) {
    const int tb = 2 * kb_half(a), nb = kb_blocks(a, n), lane = threadIdx.x & 31;
    const long long per = kb_prefix(n, len, tb, nb, nb);
    h = (int)(at / per);
    at -= h * per;
    int lo = 0, hi = nb;                // prefix(lo) <= at < prefix(hi)
    long long before = 0;               // prefix(lo)
#pragma unroll 1
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, mid = lo + lane * step;
        const long long p = mid < hi ? kb_prefix(n, len, tb, nb, mid) : at + 1;
        const int k = 31 - __clz(__ballot_sync(FULL, p <= at));
        before = __shfl_sync(FULL, p, k);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    rb = lo;
    t = (int)(at - before);
}

struct KbWalk {
    long long left;
    int b, h, rb, t, nb, slot, row0, n, len;
    __device__ __forceinline__ void start(const Kv8Attn& a, long long pos, long long end, int b_, long long base) {
        left = end - pos; b = b_;
        if (left > 0) {
            kv8_sequence(a, b, slot, row0, n, len);
            nb = kb_blocks(a, n);
            kb_locate(a, n, len, pos - base, h, rb, t);
        }
    }
    __device__ __forceinline__ bool next(const Kv8Attn& a, Kv8Seg& s) {
#pragma unroll 1
        while (left > 0) {
            if (rb >= nb) {
                rb = 0;
                if (++h >= a.hkv || nb == 0) {
                    h = 0;
                    do {
                        if (++b >= a.B) return false;
                        kv8_sequence(a, b, slot, row0, n, len);
                        nb = len > 0 ? kb_blocks(a, n) : 0;
                    } while (nb == 0);
                }
            }
            const int tiles = (kb_keys(n, len, 2 * kb_half(a), rb) + KV8_TILE - 1) / KV8_TILE, units = tiles + KB_EXTRA, u0 = t;
            const int u1 = left < units - u0 ? u0 + (int)left : units;
            left -= u1 - u0;
            t = u1;
            s.b = b; s.h = h; s.rb = rb; s.tiles = tiles; s.slot = slot; s.row0 = row0; s.n = n; s.len = len;
            s.t0 = max(u0 - KB_EXTRA, 0);
            s.t1 = u1 - KB_EXTRA;
            if (u1 == units) {
                t = 0;
                ++rb;
            }
            if (s.t1 > s.t0) return true;
        }
        return false;
    }
};

}  // namespace sv
