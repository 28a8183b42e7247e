// The 8-bit paged KV cache of one layer, shared by its operators (kv8.cu, kv8_attn.cu).
//
// pool [pages][kv heads][2][16 * D] holds e4m3 codes, scales [pages][kv heads][2] what a
// code is multiplied by: one scale per 16-token page, head and side (keys, values).  Both
// blocks are laid out as operands of the tensor cores, so that attention moves them from
// memory to the matrix unit without touching them:
//  * keys: token-major rows of D bytes, in the swizzle of a K-major operand whose rows are
//    D bytes (128-byte swizzle for D = 128, 64-byte for D = 64);
//  * values: dimension-major, the 16 tokens of a dimension in 16 consecutive bytes: eight
//    dimensions are one 128-byte core matrix of an unswizzled K-major operand (K = keys).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace sv {

constexpr int KV8_PAGE = 16;
constexpr int KV8_MIN_EXP = -64;      // smallest exponent of a scale written by the append

// Byte of dimension d of token r in a page's key block.
template <int D> __host__ __device__ __forceinline__ int kv8_key_off(int r, int d) {
    const int x = D == 128 ? (r & 7) : ((r >> 1) & 3);
    return r * D + ((((d >> 4) ^ x) << 4) | (d & 15));
}

// Four e4m3 codes of a word as floats.
__device__ __forceinline__ void kv8_decode4(uint32_t w, float (&f)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[0]), "=f"(f[1]) : "r"(lo));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[2]), "=f"(f[3]) : "r"(hi));
}

// Four floats as e4m3 codes (round to nearest even, saturating; NaN -> 0x7f).
__device__ __forceinline__ uint32_t kv8_encode4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
        "mov.b32 %0, {x, y};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// What the attention kernels read.  Sequence b has rows [row_start[b], row_start[b + 1]) of
// q, or the T rows from b * T on when row_start is nullptr; its keys are the first
// kv_len[slot] + kv_add positions of block table row slot = seq_ids ? seq_ids[b] : b.
struct Kv8Attn {
    const uint8_t* pool;
    const float* scales;
    const int* block_table;
    int num_pages, hkv, hq, max_pages, n_tables, B, n_rows;
    const int* seq_ids;
    const int* row_start;
    int T;
    const int* kv_len;
    int kv_add;
    const void* q;          // bf16, row stride q_stride elements, heads D apart
    long long q_stride;
    float scale;
    void* out;              // bf16, row stride o_stride
    long long o_stride;
    float* lse;             // [n_rows][hq] or nullptr
    int* err;               // status word for a wait that gave up, or nullptr
};

__device__ __forceinline__ int kv8_row_begin(const Kv8Attn& a, int b) { return a.row_start ? a.row_start[b] : b * a.T; }

// Rows and keys of sequence b, held within the buffers whatever the device arrays say.
__device__ __forceinline__ void kv8_sequence(const Kv8Attn& a, int b, int& slot, int& row0, int& n, int& len) {
    row0 = kv8_row_begin(a, b);
    const int end = kv8_row_begin(a, b + 1);
    slot = a.seq_ids ? a.seq_ids[b] : b;
    n = row0 < 0 || end > a.n_rows ? 0 : end - row0;
    if (n < 0) n = 0;
    len = 0;
    if (slot >= 0 && slot < a.n_tables) {
        const long long l = (long long)a.kv_len[slot] + a.kv_add;
        len = (int)(l < 0 ? 0 : (l > (long long)a.max_pages * KV8_PAGE ? (long long)a.max_pages * KV8_PAGE : l));
    }
}

// What the append reads and writes; rows and lengths as above, but with row_start the sequences are the
// rows of the block table (seq_ids and kv_add are for batches of T rows each).
struct Kv8Append {
    uint8_t* pool;
    float* scales;
    const int* block_table;
    int num_pages, hkv, max_pages, n_tables, B, n_rows;
    const int* seq_ids;
    const int* row_start;
    int T;
    const int* kv_len;
    int kv_add;
    const void *k, *v;      // fp32 or bf16, row strides in elements
    long long k_stride, v_stride;
    // > 0: k and v are pages [n_tables * stage_pages][hkv][16][D] instead, the tokens of page p of a
    // slot at their places in page slot * stage_pages + p % stage_pages
    int stage_pages;
};

// The calls without their checks, as the model context makes them.
cudaError_t kv8_append(const Kv8Append& a, bool f32, int D, cudaStream_t st);
cudaError_t kv8_attention(const Kv8Attn& a, int D, void* workspace, cudaStream_t st);
int kv8_attention_kernels(int n_rows, int G);       // kernels that an attention of n_rows rows launches
// One wait of the attention's on a barrier that nothing completes, reported as one of its own.
cudaError_t kv8_wait_probe(int* err, int budget_ms, cudaStream_t st);

// Every kernel of the cache is launched so that it may be set up while the one before it in the
// stream still runs, and waits for that one (griddepcontrol.wait) before it reads or writes anything.
template <typename K, typename... A>
static cudaError_t kv8_launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The refusals that the append and the attention share (SPEC_OK or an error, recorded).
int kv8_cache_checks(int num_pages, int n_kv_heads, int head_dim, int B, int max_pages, int n_rows, const int* block_table,
                     const void* pool, const void* scales);

}  // namespace sv
