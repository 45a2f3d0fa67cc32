// The 8-bit cache written and read: quantise-on-append per block of tokens and
// head, and rows back as values.
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv8.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;

// Eight consecutive channels of a row as they come, kW words: what the
// quantiser needs of them is done on the packed words where it can be.
template <typename T>
struct Raw;

template <>
struct Raw<float> {
    static constexpr int kW = 8;
    static constexpr uint32_t kInf = 0x7F800000u;
    // the greatest magnitude so far, as an integer: finite < infinite < NaN
    static __device__ __forceinline__ uint32_t top(uint32_t m, uint32_t w) { return max(m, w & 0x7FFFFFFFu); }
    static __device__ __forceinline__ uint32_t top(uint32_t m) { return m; }
    static __device__ __forceinline__ float value(uint32_t top) { return __uint_as_float(top); }
    static __device__ __forceinline__ uint32_t lower(uint32_t a, uint32_t b) {
        return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static constexpr uint32_t kHighest = 0x7F800000u, kLowest = 0xFF800000u;
    static __device__ __forceinline__ uint32_t no_nan(uint32_t w) { return (w & 0x7FFFFFFFu) > kInf ? 0u : w; }
    static __device__ __forceinline__ uint32_t finite(uint32_t w) { return (w & 0x7FFFFFFFu) >= kInf ? 0u : w; }
    static __device__ __forceinline__ void floats(const uint32_t* w, float* x) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ float channel(const uint32_t* words, int d) { return __uint_as_float(words[d]); }
};

// Two 16-bit floats a word.
template <uint32_t INF>
struct Raw16 {
    static constexpr int kW = 4;
    static constexpr uint32_t kInf = INF;
    static constexpr uint32_t kHighest = INF * 0x10001u, kLowest = kHighest | 0x80008000u;
    static __device__ __forceinline__ uint32_t top(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
    static __device__ __forceinline__ uint32_t top(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
    static __device__ __forceinline__ uint32_t no_nan(uint32_t w) {
        if ((w & 0x7FFFu) > INF) w &= 0xFFFF0000u;
        if ((w >> 16 & 0x7FFFu) > INF) w &= 0xFFFFu;
        return w;
    }
    static __device__ __forceinline__ uint32_t finite(uint32_t w) {
        if ((w & 0x7FFFu) >= INF) w &= 0xFFFF0000u;
        if ((w >> 16 & 0x7FFFu) >= INF) w &= 0xFFFFu;
        return w;
    }
};

template <>
struct Raw<__nv_bfloat16> : Raw16<0x7F80u> {
    static __device__ __forceinline__ float value(uint32_t top) { return __uint_as_float(top << 16); }
    static __device__ __forceinline__ uint32_t lower(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void floats(const uint32_t* w, float* x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ float channel(const uint32_t* words, int d) {
        return __uint_as_float(d & 1 ? words[d >> 1] & 0xFFFF0000u : words[d >> 1] << 16);
    }
};

template <>
struct Raw<__half> : Raw16<0x7C00u> {
    static __device__ __forceinline__ __half2 half2_of(uint32_t w) {
        __half2 h;
        memcpy(&h, &w, 4);
        return h;
    }
    static __device__ __forceinline__ float value(uint32_t top) { return __low2float(half2_of(top)); }
    static __device__ __forceinline__ uint32_t lower(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void floats(const uint32_t* w, float* x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(half2_of(w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float channel(const uint32_t* words, int d) {
        const float2 f = __half22float2(half2_of(words[d >> 1]));
        return d & 1 ? f.y : f.x;
    }
};

__device__ __forceinline__ void decode8(uint2 codes, float* x) {
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = __half22float2(e4m3x2_to_half2((uint16_t)w[i]));
        const float2 b = __half22float2(e4m3x2_to_half2((uint16_t)(w[i] >> 16)));
        x[4 * i] = a.x;
        x[4 * i + 1] = a.y;
        x[4 * i + 2] = b.x;
        x[4 * i + 3] = b.y;
    }
}

__device__ __forceinline__ uint2 encode8(const float* x) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)cvt_e4m3x2(x[4 * i + 1], x[4 * i]) | ((uint32_t)cvt_e4m3x2(x[4 * i + 3], x[4 * i + 2]) << 16);
    return make_uint2(w[0], w[1]);
}

// One CTA quantises the new rows of one (block, head) of the keys or the
// values: the greatest finite magnitude of those rows gives the scale; a block
// that already holds rows keeps the larger of its own and the new scale, and
// when it grows the held codes are rescaled (value * s_old / s_new, exact
// before its one rounding).  The rows are read once and stay in registers, as
// they came, between the two uses; the store is one byte a channel.  Each
// thread holds eight channels of RPT rows (D / 8 threads a row).  The kernel
// waits for HBM, so the page table is looked up beside the rows and little is
// done per element: the greatest magnitude and the least and greatest value of
// a channel on packed words (the encoder is monotone, so a channel's least
// code is the code of its least value).
template <typename T, int D, int RPT>
__global__ void __launch_bounds__(kThreads) k_kv8_append(DevKv8 c, const T* k_new, const T* v_new, int64_t stride_b,
                                                         int64_t stride_t, const int32_t* start_pos,
                                                         const int32_t* n_new, int n_max, uint32_t* status) {
    using R = Raw<T>;
    constexpr int kVec = D / 8, kLanes = kThreads / kVec, kWarps = kThreads / 32, kW = R::kW, kRow = D * kW / 8;
    __shared__ uint32_t s_top[kWarps];
    __shared__ uint32_t s_lo[kWarps][kRow], s_hi[kWarps][kRow];
    pdl_begin();
    const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y >> 1;
    const bool keys = (blockIdx.y & 1) == 0;
    const int bs = c.bs();
    const int64_t cap = (int64_t)c.max_blocks << c.bs_log2;
    const int n = kv8_rows(n_new, b, n_max, status);
    const int64_t start = __ldg(start_pos + b);
    if (n == 0) return;
    if (start < 0 || start + n > cap) flag(status, kStatusBounds);
    if (start < 0) return;   // none of the rows: where such a call's rows belong is not to be guessed
    const int64_t end = start + n < cap ? start + n : cap;
    const int64_t lb = (start >> c.bs_log2) + blockIdx.x, pos0 = lb << c.bs_log2;
    if (pos0 >= end) return;
    const int r0 = start > pos0 ? (int)(start - pos0) : 0;                   // rows already held
    const int r1 = end - pos0 < bs ? (int)(end - pos0) : bs;                 // rows held after the call

    const int vec = tid % kVec, lane = tid / kVec;
    const T* src = (keys ? k_new : v_new) + (int64_t)b * stride_b + (int64_t)h * D + vec * 8 + (pos0 - start) * stride_t;
    uint32_t x[RPT][kW];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = lane + i * kLanes;
#pragma unroll
        for (int q = 0; q < kW; q += 4) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (r >= r0 && r < r1) u = __ldg(reinterpret_cast<const uint4*>(src + r * stride_t) + q / 4);
            x[i][q] = u.x, x[i][q + 1] = u.y, x[i][q + 2] = u.z, x[i][q + 3] = u.w;
        }
    }
    const int phys = kv8_block(c, b, (int)lb);
    if (phys < 0) {
        flag(status, kStatusBounds);
        return;
    }
    const int64_t unit = (int64_t)phys * c.heads + h;
    uint8_t* codes = (keys ? c.k : c.v) + unit * bs * D;
    float* scale = (keys ? c.k_scale : c.v_scale) + unit;
    const float s_old = r0 ? *scale : 0.0f;

    // the greatest magnitude of the CTA, as an integer
    auto greatest = [&]() {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int q = 0; q < kW; ++q) m = R::top(m, x[i][q]);
        m = __reduce_max_sync(0xFFFFFFFFu, R::top(m));
        __syncthreads();
        if ((tid & 31) == 0) s_top[tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = max(m, s_top[w]);
        return m;
    };
    uint32_t top = greatest();
    uint32_t held[RPT][kW];          // (the rows again, where some are not finite: what the scale does not count)
    if (top >= R::kInf) {            // infinite: saturates below; NaN: stored as 0; neither counts for the scale
        if (tid == 0) flag(status, kStatusNonFinite);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int q = 0; q < kW; ++q) {
                held[i][q] = R::no_nan(x[i][q]);
                x[i][q] = R::finite(x[i][q]);
            }
        top = greatest();
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int q = 0; q < kW; ++q) x[i][q] = held[i][q];
    }
    const float s = fmaxf(exp2_int(kv8_scale_exp(R::value(top))), s_old);
    const float inv = 1.0f / s;                    // exact: a power of two
    if (r0 && s > s_old) {
        const float shrink = s_old * inv;
        for (int r = lane; r < r0; r += kLanes) {
            uint2* p = reinterpret_cast<uint2*>(codes + (int64_t)r * D + vec * 8);
            float y[8];
            decode8(*p, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= shrink;
            *p = encode8(y);
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = lane + i * kLanes;
        if (r >= r0 && r < r1) {
            float y[8];
            R::floats(x[i], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= inv;
            *reinterpret_cast<uint2*>(codes + (int64_t)r * D + vec * 8) = encode8(y);
        }
    }
    if (tid == 0) *scale = s;
    if (!keys || !c.k_bounds) return;

    // the block's bounds in whole units of s: least code rounded down, greatest
    // rounded up, joined with what the held rows had (rescaled outward)
    uint32_t lo[kW], hi[kW];
#pragma unroll
    for (int q = 0; q < kW; ++q) lo[q] = R::kHighest, hi[q] = R::kLowest;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = lane + i * kLanes;
        if (r >= r0 && r < r1) {
#pragma unroll
            for (int q = 0; q < kW; ++q) {
                lo[q] = R::lower(lo[q], x[i][q]);
                hi[q] = R::upper(hi[q], x[i][q]);
            }
        }
    }
#pragma unroll
    for (int o = kVec; o < 32; o <<= 1)
#pragma unroll
        for (int q = 0; q < kW; ++q) {
            lo[q] = R::lower(lo[q], __shfl_xor_sync(0xFFFFFFFFu, lo[q], o));
            hi[q] = R::upper(hi[q], __shfl_xor_sync(0xFFFFFFFFu, hi[q], o));
        }
    if ((tid & 31) < kVec) {
#pragma unroll
        for (int q = 0; q < kW; ++q) {
            s_lo[tid >> 5][vec * kW + q] = lo[q];
            s_hi[tid >> 5][vec * kW + q] = hi[q];
        }
    }
    __syncthreads();
    if (tid < 2 * D) {
        const int d = tid % D;
        const bool upper = tid >= D;
        float v = upper ? R::channel(s_hi[0], d) : R::channel(s_lo[0], d);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = upper ? fmaxf(v, R::channel(s_hi[w], d)) : fminf(v, R::channel(s_lo[w], d));
        v = e4m3_to_float((uint8_t)cvt_e4m3x2(0.0f, v * inv));
        v = upper ? ceilf(v) : floorf(v);
        uint8_t* p = c.k_bounds + unit * 2 * D + tid;
        if (r0) {
            const float o = e4m3_to_float(*p) * (s_old * inv);
            v = upper ? fmaxf(v, ceilf(o)) : fminf(v, floorf(o));
        }
        *p = (uint8_t)cvt_e4m3x2(0.0f, v);
    }
}

// Cached rows as values: 16 channels (16 code bytes) a thread at a time, the
// scale applied in fp32 (exact) and rounded once to the output type.  It
// streams; kUnits independent loads a thread keep HBM busy (8 sequences of 8,192
// tokens: one 73.6 us, two 63.5 = 6.3 TB/s, eight 64.2), and a 16-bit output
// leaves in one 32-byte store, so that no sector is written in halves.
constexpr int kUnits = 2;

__device__ __forceinline__ void store8w(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float* x);

template <>
__device__ __forceinline__ void store16<float>(float* p, const float* x) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[i]);
    store8w(p, w);
    store8w(p + 8, w + 8);
}

template <>
__device__ __forceinline__ void store16<__half>(__half* p, const float* x) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        memcpy(&w[i], &h, 4);
    }
    store8w(p, w);
}

template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        memcpy(&w[i], &h, 4);
    }
    store8w(p, w);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_kv8_read(DevKv8 c, const int32_t* start_pos, const int32_t* n_rows,
                                                       int n_max, T* k_out, T* v_out, uint32_t* status) {
    pdl_begin();
    const int b = blockIdx.z;
    const int kvec = c.dim / 16, per_row = c.heads * kvec;
    const int n = kv8_rows(n_rows, b, n_max, status);
    const int64_t cap = (int64_t)c.max_blocks << c.bs_log2, start = __ldg(start_pos + b);
    const uint8_t* codes = blockIdx.y ? c.v : c.k;
    const float* scales = blockIdx.y ? c.v_scale : c.k_scale;
    T* out = (blockIdx.y ? v_out : k_out) + (int64_t)b * n_max * per_row * 16;
    const int64_t units = (int64_t)n * per_row;
    const int step_i = kThreads / per_row, step_r = kThreads - step_i * per_row;
    for (int64_t u0 = (int64_t)blockIdx.x * kThreads * kUnits + threadIdx.x; u0 < units;
         u0 += (int64_t)gridDim.x * kThreads * kUnits) {
        int64_t i = (u0 | per_row) >> 32 ? u0 / per_row : (uint32_t)u0 / (uint32_t)per_row;
        int r = (int)(u0 - i * per_row);
        uint4 w[kUnits];
        float s[kUnits];
#pragma unroll
        for (int x = 0; x < kUnits; ++x) {
            w[x] = make_uint4(0, 0, 0, 0);        // outside the cache: zeros
            s[x] = 0.0f;
            if (u0 + x * kThreads < units) {
                const int64_t pos = start + i;
                const int h = r / kvec, v = r - h * kvec;
                const int phys = pos >= 0 && pos < cap ? kv8_block(c, b, (int)(pos >> c.bs_log2)) : -1;
                if (phys < 0) {
                    flag(status, kStatusBounds);
                } else {
                    const int64_t unit = (int64_t)phys * c.heads + h;
                    w[x] = __ldg(reinterpret_cast<const uint4*>(
                        codes + ((unit << c.bs_log2) + (pos & (c.bs() - 1))) * c.dim + v * 16));
                    s[x] = __ldg(scales + unit);
                }
            }
            r += step_r;
            i += step_i;
            if (r >= per_row) r -= per_row, ++i;
        }
#pragma unroll
        for (int x = 0; x < kUnits; ++x) {
            if (u0 + x * kThreads >= units) break;
            float y[16];
            decode8(make_uint2(w[x].x, w[x].y), y);
            decode8(make_uint2(w[x].z, w[x].w), y + 8);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] *= s[x];
            store16<T>(out + (u0 + x * kThreads) * 16, y);
        }
    }
}

template <typename T, int D>
cudaError_t append_d(const DevKv8& c, const void* k, const void* v, int64_t sb, int64_t st, const int32_t* start,
                     const int32_t* n_new, int n_max, uint32_t* status, cudaStream_t stream) {
    const int bs = c.bs();
    const int nb = (int)(((int64_t)n_max + bs - 2) / bs + 1);
    const dim3 grid(nb < c.max_blocks ? nb : c.max_blocks, 2 * c.heads, c.batch);
    const T* kn = static_cast<const T*>(k);
    const T* vn = static_cast<const T*>(v);
    constexpr int kLanes = kThreads / (D / 8);
    const int rpt = (bs + kLanes - 1) / kLanes;
#define CSA2_KV8_APPEND(R) \
    return launch_pdl(k_kv8_append<T, D, R>, grid, kThreads, 0, stream, c, kn, vn, sb, st, start, n_new, n_max, status)
    if (rpt <= 1) CSA2_KV8_APPEND(1);
    if (rpt <= 2) CSA2_KV8_APPEND(2);
    if (rpt <= 4) CSA2_KV8_APPEND(4);
    CSA2_KV8_APPEND(8);
#undef CSA2_KV8_APPEND
}

}  // namespace

cudaError_t launch_kv8_append(const DevKv8& c, const void* k, const void* v, int dtype, int64_t sb, int64_t st,
                              const int32_t* start, const int32_t* n_new, int T, uint32_t* status,
                              cudaStream_t stream) {
    switch (dtype) {
        case 0:
            return c.dim == 64 ? append_d<float, 64>(c, k, v, sb, st, start, n_new, T, status, stream)
                               : append_d<float, 128>(c, k, v, sb, st, start, n_new, T, status, stream);
        case 1:
            return c.dim == 64 ? append_d<__nv_bfloat16, 64>(c, k, v, sb, st, start, n_new, T, status, stream)
                               : append_d<__nv_bfloat16, 128>(c, k, v, sb, st, start, n_new, T, status, stream);
        default:
            return c.dim == 64 ? append_d<__half, 64>(c, k, v, sb, st, start, n_new, T, status, stream)
                               : append_d<__half, 128>(c, k, v, sb, st, start, n_new, T, status, stream);
    }
}

cudaError_t launch_kv8_read(const DevKv8& c, const int32_t* start, const int32_t* n_rows, int T, void* k_out,
                            void* v_out, int dtype, uint32_t* status, cudaStream_t st) {
    const int64_t vecs = (int64_t)T * c.heads * (c.dim / 16);
    int64_t gx = (vecs + kThreads * kUnits - 1) / (kThreads * kUnits);
    if (gx > 65536) gx = 65536;
    const dim3 grid((unsigned)gx, 2, c.batch);
    switch (dtype) {
        case 0:
            return launch_pdl(k_kv8_read<float>, grid, kThreads, 0, st, c, start, n_rows, T, (float*)k_out,
                              (float*)v_out, status);
        case 1:
            return launch_pdl(k_kv8_read<__nv_bfloat16>, grid, kThreads, 0, st, c, start, n_rows, T,
                              (__nv_bfloat16*)k_out, (__nv_bfloat16*)v_out, status);
        default:
            return launch_pdl(k_kv8_read<__half>, grid, kThreads, 0, st, c, start, n_rows, T, (__half*)k_out,
                              (__half*)v_out, status);
    }
}

}  // namespace csa2
