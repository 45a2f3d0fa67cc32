// Block selection over the 8-bit cache: a cheap score per (query token, key
// head, block) from the block's key bounds, and the best blocks of every row.
//
// The score of a block is the greatest q . k that its bounds allow, over the
// query heads of the key head:
//     max_g 2^e_g s_block sum_d (min(qi_d, 0) lo_d + max(qi_d, 0) hi_d),
// qi = q rounded to whole numbers of at most 127 in units of 2^e_g, lo and hi
// the bounds, whole numbers of at most 448 in units of the key scale.  That is
// one dot product of length 2 D with the bounds as stored.  Every partial sum
// is a whole number below 128 * 127 * 448 < 2^23, so fp32 accumulation on the
// tensor cores is exact in any order and the two powers of two change nothing:
// the selection is reproducible, and equal scores are equal bits.
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv8.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTiles = 4;                          // tiles of 16 blocks a warp scores
constexpr int kCtaBlocks = kWarps * kTiles * 16;

struct Params {
    DevKv8 c;
    Kv8Query q;
    int G, n_sel, n_first, n_recent;
    int32_t* idx;
    float* scores;   // [batch][T][heads][max_blocks]
    uint32_t* status;
};

// Eight query rows in operand layout: whole numbers, the negative part against
// the lower bounds, the positive against the upper.
// b[half of bounds][chunk][k step][register].
template <int D>
struct QueryRows {
    static constexpr int kC = D / 64;
    uint32_t b[2][kC][4][2];
    float unit[2];   // 2^e of rows 2c and 2c + 1

    // Two 16-bit values as floats, what is not finite as 0.
    static __device__ __forceinline__ float2 both(uint32_t w, int is_bf16) {
        float2 f;
        if (is_bf16) {
            f = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        } else {
            __half2 h;
            memcpy(&h, &w, 4);
            f = __half22float2(h);
        }
        if (!(fabsf(f.x) <= 3.4028235e38f)) f.x = 0.0f;
        if (!(fabsf(f.y) <= 3.4028235e38f)) f.y = 0.0f;
        return f;
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        const __half2 h = __floats2half2_rn(x, y);
        uint32_t w;
        memcpy(&w, &h, 4);
        return w;
    }
    // Heads g0 + r of key head h (lane column c holds chunks c, c + 4).
    __device__ __forceinline__ void load(const Params& p, int bq, int j, int h, int g0, int r, int c) {
        const int g = g0 + r;
        const bool ok = g < p.G;
        uint32_t raw[kC][8];
        const uint16_t* src = static_cast<const uint16_t*>(p.q.q) + (int64_t)bq * p.q.stride_b +
                              (int64_t)j * p.q.stride_t + (int64_t)(h * p.G + g) * D;
#pragma unroll
        for (int k = 0; k < kC; ++k) {
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (ok) {
                const uint4* s4 = reinterpret_cast<const uint4*>(src + (c + 4 * k) * 16);
                x = __ldg(s4);
                y = __ldg(s4 + 1);
            }
            raw[k][0] = x.x, raw[k][1] = x.y, raw[k][2] = x.z, raw[k][3] = x.w;
            raw[k][4] = y.x, raw[k][5] = y.y, raw[k][6] = y.z, raw[k][7] = y.w;
        }
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < kC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = both(raw[k][i], p.q.is_bf16);
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        // the least e with amax <= 127 * 2^e (127 = 1.984375 * 2^6)
        const uint32_t u = __float_as_uint(amax);
        int e = (int)(u >> 23) - 127 - 6 + ((u & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
        e = e < -118 ? -118 : e;
        const float mine = ok ? exp2_int(e) : -INFINITY, down = exp2_int(-e);
        unit[0] = __shfl_sync(0xFFFFFFFFu, mine, 2 * c * 4);
        unit[1] = __shfl_sync(0xFFFFFFFFu, mine, (2 * c + 1) * 4);
#pragma unroll
        for (int k = 0; k < kC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {   // word i: channels 2i, 2i + 1 of the chunk, k step i / 2
                const float2 f = both(raw[k][i], p.q.is_bf16);
                const float x = rintf(f.x * down), y = rintf(f.y * down);
                b[0][k][i >> 1][i & 1] = pack(fminf(x, 0.0f), fminf(y, 0.0f));
                b[1][k][i >> 1][i & 1] = pack(fmaxf(x, 0.0f), fmaxf(y, 0.0f));
            }
    }
};

// The row of a CTA: sequence b, token j, key head h; false beyond the call's rows.
__device__ __forceinline__ bool row_of(const Params& p, int row, int& b, int& j, int& h, int& visible, bool report) {
    h = row % p.c.heads;
    const int bj = row / p.c.heads;
    b = bj / p.q.T;
    j = bj - b * p.q.T;
    uint32_t* status = report ? p.status : nullptr;
    const int L = kv8_len(p.c, b, status), n = kv8_rows(p.q.n_q, b, p.q.T, status);
    const int pos = L - n + j;
    visible = pos < 0 ? 0 : (pos >> p.c.bs_log2) + 1;
    return j < n;
}

// Scores of kCtaBlocks blocks of one row: a warp takes four tiles of 16 blocks
// (the rows of the matrix tile; the query heads are its 8 columns), 2 D bytes a
// block straight from global memory into operand registers (four lanes read 64
// adjacent bytes of a block at a time), the next tile's loads in flight while
// one is multiplied.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) k_kv8_score(const __grid_constant__ Params p) {
    constexpr int kC = D / 64;
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
    int b, j, h, visible;
    if (!row_of(p, blockIdx.x, b, j, h, visible, blockIdx.y == 0 && threadIdx.x == 0)) return;
    const int first = (blockIdx.y * kWarps + warp) * kTiles * 16;
    if (first >= visible) return;
    int unit[kTiles][2];   // physical block * heads + head of blocks r and r + 8 of every tile, -1: none
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int lb = first + i * 16 + half * 8 + r;
            unit[i][half] = lb < visible ? kv8_block(p.c, b, lb) : -2;
        }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (unit[i][half] == -1 && c == 0) flag(p.status, kStatusBounds);
            if (unit[i][half] >= 0) unit[i][half] = unit[i][half] * p.c.heads + h;
        }
    auto load = [&](uint4 (&w)[2][2][kC], const int (&u)[2]) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int k = 0; k < kC; ++k) {
                    w[half][m][k] = make_uint4(0, 0, 0, 0);
                    if (u[half] >= 0)
                        w[half][m][k] = __ldg(reinterpret_cast<const uint4*>(p.c.k_bounds + (int64_t)u[half] * 2 * D + m * D) + c + 4 * k);
                }
    };
    float best[kTiles][2];   // blocks r and r + 8 of every tile
#pragma unroll
    for (int i = 0; i < kTiles; ++i) best[i][0] = best[i][1] = -INFINITY;
    for (int g0 = 0; g0 < p.G; g0 += 8) {
        uint4 w[2][2][2][kC];
        load(w[0], unit[0]);
        QueryRows<D> q;
        q.load(p, b, j, h, g0, r, c);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            if (i + 1 < kTiles) load(w[(i + 1) & 1], unit[i + 1]);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int k = 0; k < kC; ++k) {
                    const uint4 &x = w[i & 1][0][m][k], &y = w[i & 1][1][m][k];
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint32_t a[4] = {half2_lo(xs[s]), half2_lo(ys[s]), half2_hi(xs[s]), half2_hi(ys[s])};
                        mma_16816(acc, a, q.b[m][k][s][0], q.b[m][k][s][1]);
                    }
                }
            // rows without a query head hold 0 * -inf: fmaxf drops the NaN
            best[i][0] = fmaxf(best[i][0], fmaxf(acc[0] * q.unit[0], acc[1] * q.unit[1]));
            best[i][1] = fmaxf(best[i][1], fmaxf(acc[2] * q.unit[0], acc[3] * q.unit[1]));
        }
    }
    float* out = p.scores + (int64_t)blockIdx.x * p.c.max_blocks;
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v = best[i][half];
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
            const int lb = first + i * 16 + half * 8 + r;
            if (c == 0 && lb < visible)
                out[lb] = unit[i][half] < 0 ? -INFINITY : v * __ldg(p.c.k_scale + unit[i][half]);
        }
}

// ---------------------------------------------------------------- the best blocks of a row
constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kCand = 2048;      // candidates resolved by rank
constexpr int kMostSel = 2048;

struct SelSmem {
    uint32_t hist[kBins];
    uint32_t cand_key[kCand];
    int cand_idx[kCand];
    int chosen[kMostSel];
    uint32_t red[kSelThreads / 32][2];
    uint32_t cut_key;
    int cut_idx, n_cand, n_chosen, bin, above;
};

__device__ __forceinline__ uint32_t block_sum(uint32_t v, SelSmem& s) {
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[warp][0] = v;
    __syncthreads();
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) t += s.red[w][0];
    return t;
}

// One CTA per row.  The blocks that compete are those between the first and
// the newest ones; `want` of them are taken: linear bins between the least and
// the greatest score find the bin with the cut, whose members are ranked
// exactly by (score, lower index first).  Many equal scores (a bin too full
// to rank) are cut by bisection over the score's bits and then over the index.
// The chosen are put in ascending order by counting.  KPT keys a thread stay in
// registers; KPT == 0: rows of any length, keys kept in the scores' place.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) k_kv8_select(const __grid_constant__ Params p) {
    __shared__ SelSmem s;
    pdl_begin();
    const int tid = threadIdx.x;
    int b, j, h, visible;
    if (!row_of(p, blockIdx.x, b, j, h, visible, false)) return;
    int32_t* out = p.idx + (int64_t)blockIdx.x * p.n_sel;
    const int k = p.n_sel < visible ? p.n_sel : visible;
    if (visible <= p.n_sel) {
        for (int i = tid; i < p.n_sel; i += kSelThreads) out[i] = i < k ? i : -1;
        return;
    }
    const int c0 = p.n_first, c1 = visible - p.n_recent;       // competing blocks [c0, c1); c0 <= c1 as n_sel < visible
    const int want = k - p.n_first - p.n_recent;
    uint32_t* row = reinterpret_cast<uint32_t*>(p.scores + (int64_t)blockIdx.x * p.c.max_blocks);
    uint32_t reg[KPT ? KPT : 1];
    auto key_of = [](uint32_t bits) {
        const float f = __uint_as_float(bits);
        return isnan(f) ? 0u : ordered_key(f);
    };
    // every competing (index, key) of this thread
    auto each = [&](auto&& f) {
        if (KPT) {
#pragma unroll
            for (int i = 0; i < (KPT ? KPT : 1); ++i) {
                const int at = c0 + i * kSelThreads + tid;
                if (at < c1) f(at, reg[i]);
            }
        } else {
#pragma unroll 4
            for (int at = c0 + tid; at < c1; at += kSelThreads) f(at, row[at]);
        }
    };
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    if (KPT) {
#pragma unroll
        for (int i = 0; i < (KPT ? KPT : 1); ++i) {
            const int at = c0 + i * kSelThreads + tid;
            reg[i] = at < c1 ? row[at] : 0u;
        }
#pragma unroll
        for (int i = 0; i < (KPT ? KPT : 1); ++i) reg[i] = key_of(reg[i]);
    } else {
        for (int at = c0 + tid; at < c1; at += kSelThreads) row[at] = key_of(row[at]);
    }
    each([&](int, uint32_t key) {
        lo = min(lo, key);
        hi = max(hi, key);
    });
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if ((tid & 31) == 0) s.red[tid >> 5][0] = lo, s.red[tid >> 5][1] = hi;
    for (int i = tid; i < kBins; i += kSelThreads) s.hist[i] = 0;
    if (tid == 0) s.n_cand = s.n_chosen = 0;
    __syncthreads();
    lo = __reduce_min_sync(0xFFFFFFFFu, s.red[tid & 31][0]);   // 32 warps
    hi = __reduce_max_sync(0xFFFFFFFFu, s.red[tid & 31][1]);
    const float flo = lo ? key_score(lo) : -INFINITY, fhi = hi ? key_score(hi) : -INFINITY;
    const float per = (float)(kBins - 1) / (fhi - flo);
    const bool linear = fhi - flo > 0.0f && fhi - flo < INFINITY && per < INFINITY;
    uint32_t cut_key = 0;      // chosen: key > cut_key, or key == cut_key with index <= cut_idx
    int cut_idx = -1;
    bool ranked = false;
    if (want > 0 && linear) {
        auto bin_of = [&](uint32_t key) {
            const int v = (int)((key_score(key) - flo) * per);
            return v < 0 ? 0 : (v > kBins - 1 ? kBins - 1 : v);
        };
        each([&](int, uint32_t key) { atomicAdd(&s.hist[bin_of(key)], 1u); });
        __syncthreads();
        {   // the bin in which the running count from the top reaches `want`: two bins a thread
            const uint32_t n0 = s.hist[kBins - 1 - 2 * tid], n1 = s.hist[kBins - 2 - 2 * tid], n = n0 + n1;
            uint32_t inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if ((tid & 31) >= o) inc += v;
            }
            if ((tid & 31) == 31) s.red[tid >> 5][0] = inc;
            __syncthreads();
            uint32_t w = s.red[tid & 31][0];
            w = __reduce_add_sync(0xFFFFFFFFu, (tid & 31) < (tid >> 5) ? w : 0u);
            const uint32_t after = w + inc, before = after - n;
            if (before < (uint32_t)want && after >= (uint32_t)want) {
                const bool second = before + n0 < (uint32_t)want;
                s.bin = kBins - 1 - 2 * tid - (second ? 1 : 0);
                s.above = (int)(before + (second ? n0 : 0u));
            }
        }
        __syncthreads();
        const int bin = s.bin, need = want - s.above;
        const int members = (int)s.hist[bin];
        if (members <= kCand) {
            each([&](int at, uint32_t key) {
                if (bin_of(key) == bin) {
                    const int i = atomicAdd(&s.n_cand, 1);
                    s.cand_key[i] = key;
                    s.cand_idx[i] = at;
                }
            });
            __syncthreads();
            // the need-th best member is the cut: keys of higher bins are greater
            for (int i = tid; i < members; i += kSelThreads) {
                const uint32_t key = s.cand_key[i];
                const int at = s.cand_idx[i];
                int rank = 0;
                for (int o = 0; o < members; ++o) {
                    const uint32_t ko = s.cand_key[o];
                    rank += ko > key || (ko == key && s.cand_idx[o] < at);
                }
                if (rank == need - 1) s.cut_key = key, s.cut_idx = at;
            }
            __syncthreads();
            cut_key = s.cut_key;
            cut_idx = s.cut_idx;
            ranked = true;
        }
    }
    if (want > 0 && !ranked) {
        // the greatest key with at least `want` keys >= it, then the index of the last tie taken
        uint32_t a = lo, z = hi;
        while (a < z) {
            const uint32_t mid = a + (z - a) / 2 + 1;
            uint32_t n = 0;
            each([&](int, uint32_t key) { n += key >= mid; });
            if (block_sum(n, s) >= (uint32_t)want) a = mid;
            else z = mid - 1;
        }
        cut_key = a;
        uint32_t n = 0;
        each([&](int, uint32_t key) { n += key > cut_key; });
        const uint32_t need = (uint32_t)want - block_sum(n, s);
        int x = c0, y = c1 - 1;
        while (x < y) {
            const int mid = (x + y) / 2;
            n = 0;
            each([&](int at, uint32_t key) { n += at <= mid && key == cut_key; });
            if (block_sum(n, s) >= need) y = mid;
            else x = mid + 1;
        }
        cut_idx = x;
    }
    // the chosen competitors, then all in ascending order
    if (want > 0)
        each([&](int at, uint32_t key) {
            if (key > cut_key || (key == cut_key && at <= cut_idx)) {
                const int i = atomicAdd(&s.n_chosen, 1);
                if (i < kMostSel) s.chosen[i] = at;
            }
        });
    __syncthreads();
    for (int i = tid; i < p.n_first; i += kSelThreads) out[i] = i;
    for (int i = tid; i < p.n_recent; i += kSelThreads) out[p.n_first + want + i] = c1 + i;
    for (int i = tid; i < want; i += kSelThreads) {
        const int v = s.chosen[i];
        int rank = 0;
        for (int o = 0; o < want; ++o) rank += s.chosen[o] < v;
        out[p.n_first + rank] = v;
    }
}

}  // namespace

cudaError_t launch_kv8_select(const DevKv8& c, const Kv8Query& q, int n_sel, int n_first, int n_recent,
                              int32_t* block_idx, float* scores, uint32_t* status, cudaStream_t st) {
    Params p;
    p.c = c;
    p.q = q;
    p.G = q.H / c.heads;
    p.n_sel = n_sel;
    p.n_first = n_first;
    p.n_recent = n_recent;
    p.idx = block_idx;
    p.scores = scores;
    p.status = status;
    const unsigned rows = (unsigned)((int64_t)c.batch * q.T * c.heads);
    const dim3 grid(rows, (c.max_blocks + kCtaBlocks - 1) / kCtaBlocks);
    cudaError_t e = c.dim == 64 ? launch_pdl(k_kv8_score<64>, grid, kThreads, 0, st, p)
                                : launch_pdl(k_kv8_score<128>, grid, kThreads, 0, st, p);
    if (e != cudaSuccess) return e;
    if (c.max_blocks <= 2 * kSelThreads) return launch_pdl(k_kv8_select<2>, dim3(rows), kSelThreads, 0, st, p);
    if (c.max_blocks <= 8 * kSelThreads) return launch_pdl(k_kv8_select<8>, dim3(rows), kSelThreads, 0, st, p);
    if (c.max_blocks <= 17 * kSelThreads) return launch_pdl(k_kv8_select<17>, dim3(rows), kSelThreads, 0, st, p);
    return launch_pdl(k_kv8_select<0>, dim3(rows), kSelThreads, 0, st, p);
}

}  // namespace csa2
