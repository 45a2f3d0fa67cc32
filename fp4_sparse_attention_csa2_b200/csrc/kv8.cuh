// The 8-bit key / value cache (csa2_kv8_cache): device view, formats and the
// launch interface between the C ABI (kv8_api.cu) and its kernels.
//
// Codes are E4M3, with one power-of-two scale per (block of tokens, head) for
// keys and one for values.  A power of two loses nothing against amax / 448
// (E4M3 keeps three mantissa bits at any scale) and makes every use of a scale
// exact: dequantisation, the rescaling of held codes when a block's scale
// grows (except where a code becomes subnormal), and the block scores.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

struct CUtensorMap_st;

namespace csa2 {

// A by-value copy of csa2_kv8_cache.
struct DevKv8 {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    uint8_t* k_bounds;
    const int32_t* table;
    const int32_t* seq_lens;
    int32_t batch, max_blocks, bs_log2, heads, dim;
    int64_t n_blocks;
    __host__ __device__ int bs() const { return 1 << bs_log2; }
};

// Query rows of a call: element (b, j, h, d) at q + b * stride_b + j * stride_t
// + h * dim + d (elements); n_q nullable (all T rows of every sequence).
struct Kv8Query {
    const void* q;
    int32_t is_bf16;
    int64_t stride_b, stride_t;
    const int32_t* n_q;
    int32_t T, H;
};

__device__ __forceinline__ int kv8_len(const DevKv8& c, int b, uint32_t* status) {
    const int64_t cap = (int64_t)c.max_blocks << c.bs_log2;
    int L = __ldg(c.seq_lens + b);
    if (L < 0 || L > cap) {
        flag(status, kStatusBounds);
        L = L < 0 ? 0 : (int)cap;
    }
    return L;
}

// Rows of sequence b that a call covers: n[b] clamped to [0, T] (flagged), or T.
__device__ __forceinline__ int kv8_rows(const int32_t* n, int b, int T, uint32_t* status) {
    if (!n) return T;
    int r = __ldg(n + b);
    if (r < 0 || r > T) {
        flag(status, kStatusBounds);
        r = r < 0 ? 0 : T;
    }
    return r;
}

// Physical block of block lb of sequence b, or -1 when the table points
// outside the cache.  The caller guarantees 0 <= lb < max_blocks (checked in
// the debug build).
__device__ __forceinline__ int kv8_block(const DevKv8& c, int b, int lb) {
    if (kDebugBounds && (lb < 0 || lb >= c.max_blocks || b < 0 || b >= c.batch)) return -1;
    const int64_t i = (int64_t)b * c.max_blocks + lb;
    if (!c.table) return (int)i;  // contiguous: the host checked batch * max_blocks <= n_blocks
    const int32_t p = __ldg(c.table + i);
    return (p < 0 || p >= c.n_blocks) ? -1 : p;
}

// A value scale is used by its exponent alone; one that is no power of two (0 is
// that of a block nobody wrote) is flagged in the debug build, like a bad index.
__device__ __forceinline__ void kv8_check_scale(float s, uint32_t* status) {
    if (kDebugBounds && (__float_as_uint(s) & 0x807FFFFFu)) flag(status, kStatusBounds);
}

// The scale of a block whose greatest finite magnitude is amax: the least 2^e,
// -120 <= e <= 120, with amax <= 448 * 2^e (448 = 1.75 * 2^8), from amax's own
// exponent and mantissa.  The limits keep 2^e and 2^-e normal numbers in fp32,
// and the least code times 2^e, 2^-129, a subnormal one; at the top code 256 times
// 2^120 is infinity (rows within 3 % of fp32's greatest number).
__device__ __forceinline__ int kv8_scale_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int x = (int)(u >> 23) - 127;  // subnormal amax: x = -127, clamped below
    const int e = x - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < -120 ? -120 : (e > 120 ? 120 : e);
}

__device__ __forceinline__ float exp2_int(int e) {  // -126 <= e <= 127
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two E4M3 codes in the low (high) half of w -> half2; exact.
__device__ __forceinline__ uint32_t half2_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t half2_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---------------------------------------------------------------- launches
cudaError_t launch_kv8_append(const DevKv8& c, const void* k_new, const void* v_new, int dtype, int64_t stride_b,
                              int64_t stride_t, const int32_t* start, const int32_t* n_new, int T, uint32_t* status,
                              cudaStream_t st);
cudaError_t launch_kv8_read(const DevKv8& c, const int32_t* start, const int32_t* n_rows, int T, void* k_out,
                            void* v_out, int dtype, uint32_t* status, cudaStream_t st);

// Attention over the cache (block_idx == nullptr: every visible position of
// the window; else the listed blocks).  part: the partials of cut items, so
// many floats as the kernel's *_part_floats says.
struct Kv8Attn {
    Kv8Query q;
    const int32_t* block_idx;
    int32_t n_sel, window;
    float sm_scale;
    void* out;
    float* lse;
    float* part;
    uint32_t* status;
};
// The codes as a 2-D byte tensor [blocks * heads * block_size][dim] for TMA
// boxes of box_rows rows; `swizzled`: rows swizzled by their own length (128 or
// 64 B) in shared memory, else dense.
bool kv8_row_map(CUtensorMap_st* map, const DevKv8& c, void* codes, int box_rows, bool swizzled);

// The dense attention runs as the streaming kernel (kv8_attn.cu) for up to 16
// query rows of a key head (tokens x query heads), and for more while its cost is
// small: steps of 16 rows by 128 positions as far as the cache reaches (the lengths
// are on the device), and two an item for its queries and outputs.  Beyond that
// the tensor-core kernel (kv8_prefill.cu) runs, which takes 256 rows a step but
// 10 us more to start.  Measured, streaming against tensor cores: cost 1,536 (64
// rows, 8 sequences of 512) 22.0 and 34.4 us, 2,160 (160 rows, 9 of 82) 24.7 and
// 25.9, 4,536 (328 rows of the same) 42.3 and 28.5; of 24 rows 2,304 (8 sequences of
// 2,048) 29.6 and 41.9, 5,120 (32 of 1,024) 49.0 and 64.0, 16,384 about equal.
constexpr int64_t kKv8StreamRows = 16;
inline bool kv8_streams(const DevKv8& c, const Kv8Attn& a) {
    const int64_t rows = (int64_t)a.q.T * (a.q.H / c.heads);
    if (a.block_idx || rows <= kKv8StreamRows) return true;
    int64_t span = (int64_t)c.max_blocks << c.bs_log2;
    if (a.window && (int64_t)a.window + a.q.T < span) span = (int64_t)a.window + a.q.T;
    return (rows + 15) / 16 * c.batch * c.heads * ((span + 127) / 128 + 2) <= (rows <= 32 ? 5120 : 2560);
}
size_t kv8_attn_part_floats(int dim);
size_t kv8_prefill_part_floats(int dim);
cudaError_t launch_kv8_attn(const DevKv8& c, const Kv8Attn& a, cudaStream_t st);
cudaError_t launch_kv8_prefill(const DevKv8& c, const Kv8Attn& a, cudaStream_t st);

cudaError_t launch_kv8_select(const DevKv8& c, const Kv8Query& q, int n_sel, int n_first, int n_recent,
                              int32_t* block_idx, float* scores, uint32_t* status, cudaStream_t st);

}  // namespace csa2
