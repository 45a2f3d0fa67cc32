// The 8-bit cache written and read: quantise-on-append per block of tokens and
// head, and rows back as values.
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv8.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;

// Eight consecutive channels of a row at the caller's type, as floats.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x);

template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float* x) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h;
        memcpy(&h, &w[i], 4);
        const float2 f = __half22float2(h);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <>
__device__ __forceinline__ void load8<float>(const float* p, float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
        x[4 * i] = f.x;
        x[4 * i + 1] = f.y;
        x[4 * i + 2] = f.z;
        x[4 * i + 3] = f.w;
    }
}

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
// before its one rounding).  The rows are read once and stay in registers
// between the two uses; the store is one byte a channel.  Each thread holds
// eight channels of RPT rows (D / 8 threads a row).
template <typename T, int D, int RPT>
__global__ void __launch_bounds__(kThreads) k_kv8_append(DevKv8 c, const T* k_new, const T* v_new, int64_t stride_b,
                                                         int64_t stride_t, const int32_t* start_pos,
                                                         const int32_t* n_new, int n_max, uint32_t* status) {
    constexpr int kVec = D / 8, kLanes = kThreads / kVec, kWarps = kThreads / 32;
    __shared__ float s_amax[kWarps];
    __shared__ float s_lo[kWarps][D], s_hi[kWarps][D];
    pdl_begin();
    const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y >> 1;
    const bool keys = (blockIdx.y & 1) == 0;
    const int bs = c.bs();
    const int64_t cap = (int64_t)c.max_blocks << c.bs_log2;
    const int n = kv8_rows(n_new, b, n_max, status);
    const int64_t start = __ldg(start_pos + b);
    if (n == 0) return;
    if (start < 0 || start + n > cap) flag(status, kStatusBounds);
    if (start < 0) return;
    const int64_t end = start + n < cap ? start + n : cap;
    const int64_t lb = (start >> c.bs_log2) + blockIdx.x, pos0 = lb << c.bs_log2;
    if (pos0 >= end) return;
    const int phys = kv8_block(c, b, (int)lb);
    if (phys < 0) {
        flag(status, kStatusBounds);
        return;
    }
    const int r0 = start > pos0 ? (int)(start - pos0) : 0;                   // rows already held
    const int r1 = end - pos0 < bs ? (int)(end - pos0) : bs;                 // rows held after the call
    const int64_t unit = (int64_t)phys * c.heads + h;
    uint8_t* codes = (keys ? c.k : c.v) + unit * bs * D;
    float* scale = (keys ? c.k_scale : c.v_scale) + unit;
    const float s_old = r0 ? *scale : 0.0f;

    const int vec = tid % kVec, lane = tid / kVec;
    const T* src = (keys ? k_new : v_new) + (int64_t)b * stride_b + (int64_t)h * D + vec * 8;
    float x[RPT][8];
    float amax = 0.0f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = lane + i * kLanes;
        if (r >= r0 && r < r1) load8<T>(src + (pos0 + r - start) * stride_t, x[i]);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = lane + i * kLanes;
        if (r >= r0 && r < r1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = fabsf(x[i][j]);
                if (a <= 3.4028235e38f) amax = fmaxf(amax, a);
                else {
                    bad = true;                    // infinite: saturates below; NaN: stored as 0
                    if (isnan(a)) x[i][j] = 0.0f;
                }
            }
        }
    }
    if (bad) flag(status, kStatusNonFinite);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if ((tid & 31) == 0) s_amax[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, s_amax[w]);
    const int e_new = kv8_scale_exp(amax);
    const float s = fmaxf(exp2_int(e_new), s_old);
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
    float lo[8], hi[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) lo[j] = 448.0f, hi[j] = -448.0f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = lane + i * kLanes;
        if (r >= r0 && r < r1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= inv;
            const uint2 w = encode8(x[i]);
            *reinterpret_cast<uint2*>(codes + (int64_t)r * D + vec * 8) = w;
            if (keys) {
                decode8(w, x[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    lo[j] = fminf(lo[j], x[i][j]);
                    hi[j] = fmaxf(hi[j], x[i][j]);
                }
            }
        }
    }
    if (tid == 0) *scale = s;
    if (!keys || !c.k_bounds) return;

    // the block's bounds in whole units of s: least code rounded down, greatest
    // rounded up, joined with what the held rows had (rescaled outward)
#pragma unroll
    for (int o = kVec; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lo[j] = fminf(lo[j], __shfl_xor_sync(0xFFFFFFFFu, lo[j], o));
            hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xFFFFFFFFu, hi[j], o));
        }
    if ((tid & 31) < kVec) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s_lo[tid >> 5][vec * 8 + j] = lo[j];
            s_hi[tid >> 5][vec * 8 + j] = hi[j];
        }
    }
    __syncthreads();
    if (tid < 2 * D) {
        const int d = tid % D;
        const bool upper = tid >= D;
        float v = upper ? s_hi[0][d] : s_lo[0][d];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = upper ? fmaxf(v, s_hi[w][d]) : fminf(v, s_lo[w][d]);
        v = upper ? ceilf(v) : floorf(v);
        uint8_t* p = c.k_bounds + unit * 2 * D + tid;
        if (r0) {
            const float o = e4m3_to_float(*p) * (s_old * inv);
            v = upper ? fmaxf(v, ceilf(o)) : fminf(v, floorf(o));
        }
        *p = (uint8_t)cvt_e4m3x2(0.0f, v);
    }
}

// Cached rows as values: 16 channels (16 code bytes) a thread, the scale
// applied in fp32 (exact) and rounded once to the output type.
template <typename T>
__device__ __forceinline__ void store16(T* p, const float* x);

template <>
__device__ __forceinline__ void store16<float>(float* p, const float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}

template <>
__device__ __forceinline__ void store16<__half>(__half* p, const float* x) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        memcpy(&w[i], &h, 4);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        memcpy(&w[i], &h, 4);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
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
    T* out = blockIdx.y ? v_out : k_out;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < (int64_t)n * per_row;
         u += (int64_t)gridDim.x * kThreads) {
        const int i = (int)(u / per_row), r = (int)(u - (int64_t)i * per_row), h = r / kvec, v = r - h * kvec;
        const int64_t pos = start + i;
        float x[16];
        const int phys = pos >= 0 && pos < cap ? kv8_block(c, b, (int)(pos >> c.bs_log2)) : -1;
        if (phys < 0) {
            flag(status, kStatusBounds);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = 0.0f;
        } else {
            const int64_t unit = (int64_t)phys * c.heads + h;
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(
                codes + ((unit << c.bs_log2) + (pos & (c.bs() - 1))) * c.dim + v * 16));
            const float s = __ldg(scales + unit);
            decode8(make_uint2(w.x, w.y), x);
            decode8(make_uint2(w.z, w.w), x + 8);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] *= s;
        }
        store16<T>(out + (((int64_t)b * n_max + i) * c.heads + h) * c.dim + v * 16, x);
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
    int64_t gx = (vecs + kThreads - 1) / kThreads;
    if (gx > 4096) gx = 4096;
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
