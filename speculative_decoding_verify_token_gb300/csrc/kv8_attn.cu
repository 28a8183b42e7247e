// Causal attention over the 8-bit paged KV cache: the call, and the join of the groups that
// several runs of the work lists share.
#include <cuda_bf16.h>
#include <cmath>
#include <cstdlib>

#include "kv8_mma.cuh"

namespace sv {

// Block (c, y, list) joins the group that run c of the list (0: rows, 1: blocks) opened and did not
// finish, if there is one; the blocks of y take every ny-th row.  Partials are added in
// the order of the runs.  What to join the runs themselves left behind (with every block searching the
// list for its group, ragged prompts took 77 us instead of 60, and small calls 20.5 instead of 18.4).
constexpr int JOIN_THREADS = 512, JOIN_Y = 4, JOIN_Y_PROMPTS = 8;

template <int D>
__global__ void __launch_bounds__(JOIN_THREADS, 2)
kv8_join_kernel(const __grid_constant__ Kv8Attn a, const __grid_constant__ Kv8Parts rows, const __grid_constant__ Kv8Parts blks) {
    const bool blocks = blockIdx.z == 1;
    const int ny = blocks ? gridDim.y : JOIN_Y;
    if ((int)blockIdx.y >= ny) return;
    const int PR = blocks ? KB_ROWS : KR_ROWS, G = a.hq / a.hkv, half = kb_half(a), lane = threadIdx.x & 31;
    const float* part_o = blocks ? blks.o : rows.o;
    const float2* part_ml = blocks ? blks.ml : rows.ml;
    const Kv8Run* runs = blocks ? blks.runs : rows.runs;
    const int c = blockIdx.x;
    pdl_wait();
    // few loads one after the other: the run's note beside those of the next 32, then maxima and sums
    // beside the first outputs
    const Kv8Run note = runs[c];
    const int next = c + 1 + lane < KV8_RUNS ? runs[c + 1 + lane].first : KV8_NONE;
    if (!note.open) return;
    const int row0 = note.row0, n = note.n, h = note.h, rb = note.rb;
    // the run with the group's last part
    int last = c + 1;
    unsigned ends = __ballot_sync(FULL, next == KV8_END);
#pragma unroll 1
    while (!ends && (last += 32) < KV8_RUNS)
        ends = __ballot_sync(FULL, last + lane < KV8_RUNS && runs[last + lane].first == KV8_END);
    if (!ends) return;
    last += __ffs(ends) - 1;
    const int first_flags = __shfl_up_sync(FULL, next, 1);
    // a warp takes a row: lane k the maxima and sums of the k-th run (of up to 32 at a time), then
    // its share of the dimensions over all of them
    constexpr int V = D / 32;
#pragma unroll 1
    for (int j = blockIdx.y + ny * (threadIdx.x >> 5); j < (blocks ? KB_ROWS : n * G); j += ny * (JOIN_THREADS / 32)) {
        int tok, hh;
        if (blocks) {
            const int jj = j & 127;
            tok = (2 * rb + (j >> 7)) * half + jj / G;
            hh = h * G + jj % G;
            if (jj >= half * G || tok >= n) continue;
        } else {
            tok = j / G;
            hh = h * G + j - tok * G;
        }
        auto slot_of = [&](int r) { return (size_t)(2 * r + (r == c ? 1 : 0)) * PR + j; };
        float m = -INFINITY, l = 0.0f, o[V] = {};
        bool bad = false;
#pragma unroll 1
        for (int r0 = c; r0 <= last; r0 += 32) {
            const int r = r0 + lane, k1 = min(32, last - r0 + 1);
            const bool mine = r <= last && (r == c || (r0 == c ? first_flags : runs[r].first) != KV8_NONE);
            const unsigned have = __ballot_sync(FULL, mine);
            const float2 ml = mine ? part_ml[slot_of(r)] : make_float2(-INFINITY, 0.0f);
            auto output = [&](int k, float (&y)[V]) {          // the k-th run's, zeros where it has none
                const float* x = part_o + slot_of(r0 + k) * D + lane * V;
                if (k < k1 && (have >> k & 1)) {
                    if constexpr (V == 4) {
                        const float4 z = *reinterpret_cast<const float4*>(x);
                        y[0] = z.x; y[1] = z.y; y[2] = z.z; y[3] = z.w;
                    } else {
                        const float2 z = *reinterpret_cast<const float2*>(x);
                        y[0] = z.x; y[1] = z.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] = 0.0f;
                }
            };
            float y[2][V];
#pragma unroll
            for (int k = 0; k < 2; ++k) output(k, y[k]);
            bad |= __any_sync(FULL, ml.x != ml.x) != 0;
            float top = fmaxf(m, ml.x);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, x));
            // in two halves: see the kernels
            const float ref = top == -INFINITY ? 0.0f : top, oh = kv8_exp2(0.5f * (m - ref)), wh = kv8_exp2(0.5f * (ml.x - ref));
            m = top;
            const float w = wh * wh;
            l = l * oh * oh + (lane < k1 ? ml.y * wh * wh : 0.0f);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] *= oh * oh;
#pragma unroll 1
            for (int k0 = 0; k0 < k1; k0 += 2) {
                float z[2][V];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int e = 0; e < V; ++e) z[k][e] = y[k][e];
                    if (k0 + 2 < k1) output(k0 + 2 + k, y[k]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float wk = __shfl_sync(FULL, w, k0 + k);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] = fmaf(z[k][e], wk, o[e]);
                }
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(FULL, l, x);
        const bool none = m == -INFINITY && l == 0.0f && !bad;
        const float il = bad ? __uint_as_float(0x7fc00000u) : (none ? 0.0f : 1.0f / l);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (long long)(row0 + tok) * a.o_stride + (size_t)hh * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 2)
            *reinterpret_cast<__nv_bfloat162*>(out + e) = __floats2bfloat162_rn(o[e] * il, o[e + 1] * il);
        if (a.lse && lane == 0)
            a.lse[(size_t)(row0 + tok) * a.hq + hh] = none ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
    }
}

constexpr size_t part_rows(int rows) { return (size_t)2 * KV8_RUNS * rows; }

// Whether a batch of n_rows can hold a sequence of the blocks list.
static bool may_have_blocks(int n_rows, int G) { return (long long)n_rows * G > KR_ROWS; }

// The workspace of one list: outputs, (maximum, sum) pairs, notes of the runs.
static size_t parts_bytes(int rows, int D) {
    return part_rows(rows) * (sizeof(float) * D + sizeof(float2)) + KV8_RUNS * sizeof(Kv8Run);
}
static Kv8Parts parts_at(void* ws, int rows, int D) {
    Kv8Parts p;
    p.o = static_cast<float*>(ws);
    p.ml = reinterpret_cast<float2*>(p.o + part_rows(rows) * D);
    p.runs = reinterpret_cast<Kv8Run*>(p.ml + part_rows(rows));
    return p;
}

static size_t workspace_bytes_of(int n_rows, int G, int D) {
    return parts_bytes(KR_ROWS, D) + (may_have_blocks(n_rows, G) ? parts_bytes(KB_ROWS, D) : 0);
}

template <int D>
static cudaError_t attention_launch(const Kv8Attn& a, void* ws, cudaStream_t st) {
    const bool blocks = may_have_blocks(a.n_rows, a.hq / a.hkv);
    const Kv8Parts rows = parts_at(ws, KR_ROWS, D), blks = parts_at(static_cast<uint8_t*>(ws) + parts_bytes(KR_ROWS, D), KB_ROWS, D);
    cudaError_t e;
    // the list that has little or nothing last, where it fits beside the end of the other: long
    // prompts by the average (32 verify passes with the blocks kernel first: 1 us more)
    const bool blocks_first = blocks && (long long)a.n_rows * (a.hq / a.hkv) > (long long)KR_ROWS * a.B;
    if (blocks_first && (e = kv8_blocks_attention(a, D, blks, false, st)) != cudaSuccess) return e;
    if ((e = kv8_rows_attention(a, D, rows, blocks_first, st)) != cudaSuccess) return e;
    if (blocks && !blocks_first && (e = kv8_blocks_attention(a, D, blks, true, st)) != cudaSuccess) return e;
    return kv8_launch(kv8_join_kernel<D>, dim3(KV8_RUNS, blocks_first ? JOIN_Y_PROMPTS : JOIN_Y, blocks ? 2 : 1), JOIN_THREADS, 0, st, a, rows,
                      blks);
}

cudaError_t kv8_attention(const Kv8Attn& a, int D, void* workspace, cudaStream_t st) {
    return D == 128 ? attention_launch<128>(a, workspace, st) : attention_launch<64>(a, workspace, st);
}

int kv8_attention_kernels(int n_rows, int G) { return may_have_blocks(n_rows, G) ? 3 : 2; }

// (no copy in flight, no tensor memory held)
__global__ void kv8_wait_probe_kernel(int* err, long long cycles) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x != 0) return;
    mbar_init(smem_u32(&bar), 1);
    fence_barrier_init();
    if (!kv8_wait(bar, 0, cycles)) kv8_report(err);
}

cudaError_t kv8_wait_probe(int* err, int budget_ms, cudaStream_t st) {
    kv8_wait_probe_kernel<<<1, 32, 0, st>>>(err, WAIT_CYCLES / 2000 * budget_ms);
    return cudaGetLastError();
}

}  // namespace sv

using namespace sv;

extern "C" size_t spec_kv8_attention_workspace_bytes(int n_rows, int n_q_heads, int n_kv_heads, int head_dim) {
    if (n_rows < 0 || n_kv_heads < 1 || n_q_heads < n_kv_heads || n_q_heads % n_kv_heads ||
        n_q_heads / n_kv_heads > 64 || (head_dim != 64 && head_dim != 128))
        return 0;
    return workspace_bytes_of(n_rows, n_q_heads / n_kv_heads, head_dim);
}

extern "C" int spec_kv8_attention(int num_pages, int n_kv_heads, int head_dim, int B, int max_pages, int n_rows, int n_q_heads,
                                  const uint8_t* pool, const float* scales, const int32_t* block_table,
                                  const int32_t* row_start, const int32_t* kv_len, const void* q, int64_t q_stride,
                                  float scale, void* out, int64_t o_stride, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    clear_error();
    const int rc = kv8_cache_checks(num_pages, n_kv_heads, head_dim, B, max_pages, n_rows, block_table, pool, scales);
    if (rc != SPEC_OK) return rc;
    if (n_q_heads < n_kv_heads || n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 64)
        return set_error(SPEC_E_INVAL, "n_q_heads=%d: a multiple of n_kv_heads=%d, at most 64 of them, is needed",
                         n_q_heads, n_kv_heads);
    if (!row_start || !kv_len || (n_rows > 0 && (!q || !out)) || !workspace)
        return set_error(SPEC_E_INVAL, "NULL required pointer");
    if ((reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(out) & 15) || (n_rows > 1 && (q_stride % 8 || o_stride % 8)))
        return set_error(SPEC_E_INVAL, "q and out must be 16-byte aligned and their strides multiples of 8");
    if ((reinterpret_cast<uintptr_t>(row_start) | reinterpret_cast<uintptr_t>(kv_len) | reinterpret_cast<uintptr_t>(lse)) & 3)
        return set_error(SPEC_E_INVAL, "row_start, kv_len and lse must be 4-byte aligned");
    if (n_rows > 1 && std::llabs(o_stride) < (long long)n_q_heads * head_dim)
        return set_error(SPEC_E_INVAL, "rows of out overlap: o_stride=%lld", (long long)o_stride);
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return set_error(SPEC_E_INVAL, "workspace not 256-byte aligned");
    if (workspace_bytes < workspace_bytes_of(n_rows, n_q_heads / n_kv_heads, head_dim))
        return set_error(SPEC_E_NOMEM, "workspace of %zu bytes is too small", workspace_bytes);
    if (!(scale > -INFINITY && scale < INFINITY)) return set_error(SPEC_E_INVAL, "scale is not finite");
    if (n_rows == 0) return SPEC_OK;
    const Kv8Attn a{pool, scales, block_table, num_pages, n_kv_heads, n_q_heads, max_pages, B, B, n_rows, nullptr, row_start,
                    0, kv_len, 0, q, q_stride, scale, out, o_stride, lse, nullptr};
    const cudaError_t e = kv8_attention(a, head_dim, workspace, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : set_error(SPEC_E_CUDA, "spec_kv8_attention: %s", cudaGetErrorString(e));
}
