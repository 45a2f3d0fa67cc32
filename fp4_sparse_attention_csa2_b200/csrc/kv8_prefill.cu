// Attention over the 8-bit cache for many query rows per sequence (prompt
// chunks, wide verification) on the 5th-generation tensor cores.
//
// With the query rows of all tokens and the query heads of a key head as the
// rows of a matrix (256 of them a CTA, two tiles of 128), both products are
// GEMM-shaped and the tensor cores bound the kernel: 4 * 256 * 128 * D flop per
// 128 positions.  One CTA per SM, four warpgroups:
//   - two softmax warpgroups, one per row tile, a thread a row: read S from
//     TMEM, keep the running maximum and sum, write the weights as fp16 over S
//     (the second product takes them from TMEM), and rescale O on the rare step
//     that moves the maximum by more than 2^4;
//   - a converter warpgroup: the codes of the next 128 positions from global
//     memory through registers to fp16 operand tiles (E4M3 values are exact in
//     fp16; 1.5 % of a step's instructions), two stages deep;
//   - one thread that issues every tcgen05.mma.  It alternates the row tiles
//     (O0 += P0 V, S0 = Q0 K, O1 += P1 V, S1 = Q1 K), so one tile's products
//     run while the other's softmax does.
// Key scales multiply S per block; value scales enter the weights' exponent,
// weight = 2^(z + log2(vs) - M), so the fp16 weights stay in range whatever the
// blocks' scales are, and the sum takes them back out per block (exact powers
// of two).
//
// Work split as in kv8_attn.cu: the (row block, head, 128 positions) steps of
// the batch form one line cut into equal pieces, cut items are merged by
// k_kv8_prefill_combine.
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv8.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kRows = 256, kTileRows = 128, kPos = 128;
constexpr int kThreads = 512;
constexpr int kMaxCtas = 148;
constexpr float kNone = -3.0e38f;
constexpr float kHeadroom = 8.0f;   // weights are 2^(z - M + 8): full fp16 precision down to 2^-22
constexpr float kLazy = 4.0f;       // and at most 2^12 before the maximum is moved

struct Params {
    DevKv8 c;
    Kv8Attn a;
    int G, ctas, row_blocks;        // row blocks of a sequence with all T rows
    uint32_t wait_limit;
};

template <int D>
struct Part {   // of a cut item: outputs [256][D], per row (m, l, M), then what the merge needs of the item
    static constexpr int kStats = kRows * D, kDesc = kStats + kRows * 3, kFloats = kDesc + 32;
};

// One step of the line: sequence b, row block rb, head h, positions lo + 128 *
// step ...; rows: row0 .. row0 + rows - 1 of the sequence's (token, group) rows.
struct Cursor {
    int pair, b, rb, h, step, steps;
    int L, n, lo, row0, rows;
};

struct Line {
    const Params& p;
    __device__ explicit Line(const Params& p) : p(p) {}
    __device__ __forceinline__ void load(Cursor& k, int pair, uint32_t* status) const {
        k.pair = pair;
        k.h = k.step = k.steps = k.rows = 0;
        k.b = pair / p.row_blocks;
        k.rb = pair - k.b * p.row_blocks;
        if (k.b >= p.c.batch) return;
        k.L = kv8_len(p.c, k.b, status);
        k.n = kv8_rows(p.a.q.n_q, k.b, p.a.q.T, status);
        k.row0 = k.rb * kRows;
        const int left = k.n * p.G - k.row0;
        if (left <= 0) return;
        k.rows = left < kRows ? left : kRows;
        const int64_t p0 = (int64_t)k.L - k.n + k.row0 / p.G, p1 = (int64_t)k.L - k.n + (k.row0 + k.rows - 1) / p.G;
        const int64_t first = p.a.window ? p0 - p.a.window + 1 : 0;
        k.lo = first > 0 ? (int)first / kPos * kPos : 0;
        const int64_t seen = p1 + 1 - k.lo;
        k.steps = seen > 0 ? (int)((seen + kPos - 1) / kPos) : 1;  // an empty row still has to be written
    }
    __device__ __forceinline__ int64_t total(const Cursor& k) const { return (int64_t)p.c.heads * k.steps; }
    __device__ __forceinline__ void next_item(Cursor& k) const {
        k.step = 0;
        if (++k.h < p.c.heads) return;
        const int pairs = p.c.batch * p.row_blocks;
        int pair = k.pair;
        do load(k, ++pair, nullptr);
        while (pair < pairs && k.steps == 0);
    }
};

// Prefix sums of the line by thread, kThreads + 1 words; the total.
__device__ int64_t line_sums(const Line& w, int64_t* sums, uint32_t* status) {
    const int tid = threadIdx.x, pairs = w.p.c.batch * w.p.row_blocks, per = (pairs + kThreads - 1) / kThreads;
    int64_t s = 0;
    for (int i = 0; i < per; ++i) {
        const int pair = tid * per + i;
        if (pair < pairs) {
            Cursor k;
            w.load(k, pair, status);
            s += w.total(k);
        }
    }
    int64_t inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if ((tid & 31) >= o) inc += v;
    }
    sums[tid + 1] = inc;
    __syncthreads();
    int64_t base = 0;
    for (int i = 0; i < (tid >> 5); ++i) base += sums[(i + 1) * 32];
    __syncthreads();
    sums[tid + 1] = base + inc;
    if (tid == 0) sums[0] = 0;
    __syncthreads();
    return sums[kThreads];
}

__device__ void line_find(const Line& w, const int64_t* sums, int64_t u, Cursor& k) {
    const int pairs = w.p.c.batch * w.p.row_blocks, per = (pairs + kThreads - 1) / kThreads;
    int lo = 0, hi = kThreads;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= u) lo = mid;
        else hi = mid;
    }
    u -= sums[lo];
    for (int pair = lo * per;; ++pair) {
        w.load(k, pair, nullptr);
        const int64_t t = w.total(k);
        if (u < t || pair + 1 >= pairs) break;
        u -= t;
    }
    k.h = k.steps ? (int)(u / k.steps) : 0;
    k.step = k.steps ? (int)(u - (int64_t)k.h * k.steps) : 0;
}

template <int D>
struct Smem {
    static constexpr int kPanels = D / 64;                    // 64 channels (128 bytes of fp16) a panel
    static constexpr int kPanel = kPos * 128;                 // bytes of one panel of 128 rows
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int q = 0;                               // [row tile][panel]
    static constexpr int k = q + 2 * kTile;                   // [stage][panel]
    static constexpr int v = k + 2 * kTile;                   // [stage][panel]
    static constexpr int sc = v + 2 * kTile;                  // [4][8] (key scale, log2 value scale)
    static constexpr int bars = sc + 4 * 8 * 8;
    static constexpr int misc = bars + 16 * 8;                // TMEM base, dead
    static constexpr int sums = misc + 16;
    static constexpr int bytes = sums + (kThreads + 1) * 8 + 1024;
};

enum Bar { kQ = 0, kKFull = 1, kKEmpty = 3, kVFull = 5, kVEmpty = 7, kS = 9, kP = 11, kO = 13, kDrain = 14 };  // pairs by stage or tile; kO one

constexpr uint32_t kColO = 256;      // TMEM columns: S0, S1 (P over them), O0, O1

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_prefill(const __grid_constant__ Params p) {
    using S = Smem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::bars);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + S::misc);
    int64_t* sums = reinterpret_cast<int64_t*>(smem + S::sums);
    float2* sc = reinterpret_cast<float2*>(smem + S::sc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = tid >> 7, wt = tid & 127;
    const int bs = p.c.bs(), G = p.G, T = p.a.q.T, H = p.a.q.H;

    // A bounded wait; once one ran out, every later wait of the CTA gives up too.
    auto wait = [&](int bar, uint32_t parity) {
        for (uint32_t i = 0; i < p.wait_limit; ++i) {
            if (tc::mbar_try_wait(bars + bar, parity)) return true;
            if (misc[1]) return false;
        }
        misc[1] = 1;
        flag(p.a.status, kStatusTimeout);
        return false;
    };

    if (tid == 0) {
        tc::mbar_init(bars + kQ, 256);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bars + kKFull + i, 128);
            tc::mbar_init(bars + kKEmpty + i, 1);
            tc::mbar_init(bars + kVFull + i, 128);
            tc::mbar_init(bars + kVEmpty + i, 1);
            tc::mbar_init(bars + kS + i, 1);
            tc::mbar_init(bars + kP + i, 128);
        }
        tc::mbar_init(bars + kO, 1);
        tc::mbar_init(bars + kDrain, 1);
        tc::fence_mbar_init();
        misc[1] = 0;
    }
    pdl_begin();
    if (warp == 12) tc::tmem_alloc(const_cast<uint32_t*>(misc), 512);
    const Line line(p);
    const int64_t total = line_sums(line, sums, blockIdx.x == 0 ? p.a.status : nullptr);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = misc[0];
    const int64_t share = total < p.ctas ? (total < 1 ? 1 : total) : p.ctas;
    int* desc = reinterpret_cast<int*>(p.a.part + ((int64_t)blockIdx.x * 2 + 1) * Part<D>::kFloats + Part<D>::kDesc);
    if (tid == 0) desc[4] = 0;
    const bool any = blockIdx.x < share && total > 0;
    const int64_t u0 = any ? total * blockIdx.x / share : 0, u1 = any ? total * (blockIdx.x + 1) / share : 0;
    Cursor cur;
    if (any) line_find(line, sums, u0, cur);

    if (wg < 2) {
        // ---------------------------------------------------------------- softmax: row wt of tile wg
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t col_s = lanes + wg * 128, col_o = lanes + kColO + wg * D;
        uint32_t tile = 0, s_phase = 0, o_phase = 0;   // tiles done by the CTA; parities
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok;) {
            const bool from_start = cur.step == 0;
            const int left = cur.steps - cur.step;
            const int todo = u1 - u < left ? (int)(u1 - u) : left;
            const bool to_end = todo == left, used = wg * kTileRows < cur.rows;
            const int row = wg * kTileRows + wt;
            const bool mine = row < cur.rows;
            const int j = (cur.row0 + row) / G, g = cur.row0 + row - j * G;
            const int pos = mine ? cur.L - cur.n + j : -1;
            const int first = p.a.window ? pos - p.a.window + 1 : 0;
            float zs = p.a.sm_scale * 1.4426950408889634f;
            {   // the query row as fp16, K-major; bf16 scaled by the power of two that takes its greatest
                // finite magnitude to [2^14, 2^15)
                const uint16_t* src = static_cast<const uint16_t*>(p.a.q.q) + (int64_t)cur.b * p.a.q.stride_b +
                                      (int64_t)j * p.a.q.stride_t + (int64_t)(cur.h * G + g) * D;
                uint8_t* dst = smem + S::q + wg * S::kTile;
                float up = 1.0f;
                if (p.a.q.is_bf16) {
                    float amax = 0.0f;
                    if (mine) {
#pragma unroll 4
                        for (int i = 0; i < D / 8; ++i) {
                            const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + i);
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float a = fabsf(__uint_as_float(w[q] << 16)), b = fabsf(__uint_as_float(w[q] & 0xFFFF0000u));
                                if (a <= 3.4028235e38f) amax = fmaxf(amax, a);
                                if (b <= 3.4028235e38f) amax = fmaxf(amax, b);
                            }
                        }
                    }
                    int e = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
                    e = e > 126 ? 126 : e;
                    up = exp2_int(e);
                    zs *= exp2_int(-e);
                }
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (mine) x = __ldg(reinterpret_cast<const uint4*>(src) + i);
                    if (p.a.q.is_bf16) {
                        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const __half2 h = __floats2half2_rn(__uint_as_float(w[q] << 16) * up,
                                                                __uint_as_float(w[q] & 0xFFFF0000u) * up);
                            memcpy(&w[q], &h, 4);
                        }
                        x = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    *reinterpret_cast<uint4*>(dst + (i >> 3) * S::kPanel + tc::sw128_offset(wt, i & 7)) = x;
                }
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(bars + kQ);
            }
            float M = kNone, l = 0.0f, e0 = 0.0f;
            for (int i = 0; i < todo; ++i, ++tile) {
                if (!used) continue;
                const int t0 = cur.lo + (cur.step + i) * kPos;
                ok = __all_sync(0xFFFFFFFFu, wait(kS + wg, s_phase));
                if (!ok) break;
                s_phase ^= 1;
                tc::fence_after_sync();
                const float2* f2 = sc + (tile & 3) * 8;
                if (i == 0) {
                    e0 = f2[0].y;
                    e0 = e0 < -100.0f ? -100.0f : (e0 > 100.0f ? 100.0f : e0);
                }
                const bool full = __all_sync(0xFFFFFFFFu, (!mine) || (t0 + kPos - 1 <= pos && t0 >= first));
                // ---- the greatest logit + log2(value scale) of the row
                float top = -INFINITY;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t r[32];
                    tc::tmem_ld32_nowait(col_s + q * 32, r);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        const float2 f = f2[q * 2 + hb];
                        const float ev = f.y == -120.0f ? e0 : f.y;
                        float m = -INFINITY;
                        if (full) {
#pragma unroll
                            for (int x = 0; x < 16; ++x) m = fmaxf(m, __uint_as_float(r[hb * 16 + x]));
                        } else {
#pragma unroll
                            for (int x = 0; x < 16; ++x) {
                                const int t = t0 + q * 32 + hb * 16 + x;
                                if (t <= pos && t >= first) m = fmaxf(m, __uint_as_float(r[hb * 16 + x]));
                            }
                        }
                        top = fmaxf(top, m * (zs * f.x) + ev);
                    }
                }
                if (__any_sync(0xFFFFFFFFu, top > M + kLazy)) {
                    const float M1 = fmaxf(M, top), f = ex2(M - M1);
                    l *= f;
                    M = M1;
                    if (i > 0) {
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t r[32];
                            tc::tmem_ld32_nowait(col_o + q * 32, r);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int x = 0; x < 32; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * f);
                            tc::tmem_st32_nowait(col_o + q * 32, r);
                        }
                    }
                }
                // ---- weights over S, two to a column
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t r[32], w[16];
                    tc::tmem_ld32_nowait(col_s + q * 32, r);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        const float2 f = f2[q * 2 + hb];
                        const float ev = f.y == -120.0f ? e0 : f.y;
                        const float a = zs * f.x, d = ev - M + kHeadroom;
                        float sum = 0.0f;
#pragma unroll
                        for (int x = 0; x < 16; x += 2) {
                            const int t = t0 + q * 32 + hb * 16 + x;
                            float w0 = ex2(__uint_as_float(r[hb * 16 + x]) * a + d);
                            float w1 = ex2(__uint_as_float(r[hb * 16 + x + 1]) * a + d);
                            if (!full) {
                                if (!(t <= pos && t >= first)) w0 = 0.0f;
                                if (!(t + 1 <= pos && t + 1 >= first)) w1 = 0.0f;
                            }
                            sum += w0 + w1;
                            const __half2 h = __floats2half2_rn(w0, w1);
                            memcpy(&w[hb * 8 + x / 2], &h, 4);
                        }
                        // back from 2^(z + log2 vs - M + 8) to 2^(z + e0 - M + 8), exactly
                        const float de = e0 - ev;
                        l += sum * exp2_int(de < -126.0f ? -126 : (de > 126.0f ? 126 : (int)de));
                    }
                    tc::tmem_st16_nowait(col_s + q * 16, w);
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                tc::mbar_arrive(bars + kP + wg);
            }
            if (!ok) break;
            // ---- the outputs
            ok = __all_sync(0xFFFFFFFFu, wait(kO, o_phase));
            if (!ok) break;
            o_phase ^= 1;
            tc::fence_after_sync();
            const bool whole = from_start && to_end;
            float* part = p.a.part + ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * Part<D>::kFloats;
            const int64_t at = ((int64_t)cur.b * T + j) * H + cur.h * G + g;
            const float f = l == 0.0f ? 0.0f : exp2_int((int)e0) / l;
            if (used) {
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t r[32];
                    tc::tmem_ld32_nowait(col_o + q * 32, r);
                    tc::tmem_ld_wait();
                    if (!mine) continue;
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + at * D + q * 32);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t w[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float o0 = __uint_as_float(r[x * 8 + y * 2]) * f, o1 = __uint_as_float(r[x * 8 + y * 2 + 1]) * f;
                                if (p.a.q.is_bf16) {
                                    const __nv_bfloat162 h = __floats2bfloat162_rn(o0, o1);
                                    memcpy(&w[y], &h, 4);
                                } else {
                                    const __half2 h = __floats2half2_rn(o0, o1);
                                    memcpy(&w[y], &h, 4);
                                }
                            }
                            dst[x] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        // by 16-byte columns across the rows, so that a warp's stores are dense
                        float4* dst = reinterpret_cast<float4*>(part) + (int64_t)q * 8 * kRows + row;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            dst[x * kRows] = make_float4(__uint_as_float(r[x * 4]), __uint_as_float(r[x * 4 + 1]),
                                                         __uint_as_float(r[x * 4 + 2]), __uint_as_float(r[x * 4 + 3]));
                    }
                }
                if (mine) {
                    if (whole) {
                        if (p.a.lse)
                            p.a.lse[at] = l == 0.0f ? -INFINITY : (M - e0 - kHeadroom + log2f(l)) * 0.6931471805599453f;
                    } else {
                        float* s3 = part + Part<D>::kStats + row * 3;
                        s3[0] = l == 0.0f ? kNone : M - e0 - kHeadroom;
                        s3[1] = l;
                        s3[2] = M - kHeadroom;
                    }
                }
            }
            if (from_start && !to_end && tid == 0) {
                const int64_t last_u = u + left - 1;
                const int64_t last = ((last_u + 1) * share + total - 1) / total - 1;
                desc[0] = cur.b;
                desc[1] = cur.h;
                desc[2] = cur.row0;
                desc[3] = cur.rows;
                desc[4] = (int)(last - blockIdx.x) + 1;
            }
            tc::fence_before_sync();
            u += todo;
            cur.step += todo - 1;
            if (++cur.step >= cur.steps) line.next_item(cur);
        }
    } else if (wg == 2) {
        // ---------------------------------------------------------------- codes to fp16 operand tiles
        constexpr int kPer = D / 16;             // 16-byte pieces of a row, and of this thread in a tile
        uint32_t tile = 0, k_phase = 0, v_phase = 0;
        uint4 kr[kPer], vr[kPer];
        int phys[kPer];
        float ks = 0.0f, vs = 1.0f;
        int t0 = 0, lim = 0, h = 0, my_phys = -1;
        int64_t ahead_u = u0;
        // the blocks of the tile at `cur`, which moves on
        auto look = [&]() {
            t0 = cur.lo + cur.step * kPos;
            lim = cur.L;
            h = cur.h;
            my_phys = -1;
#pragma unroll
            for (int i = 0; i < kPer; ++i) phys[i] = -1;
            if (ahead_u >= u1) return;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int t = t0 + (i * 128 + wt) / kPer;
                if (t < lim) {
                    phys[i] = kv8_block(p.c, cur.b, t >> p.c.bs_log2);
                    if (phys[i] < 0) flag(p.a.status, kStatusBounds);
                }
            }
            if (wt < 8 && t0 + wt * 16 < lim) my_phys = kv8_block(p.c, cur.b, (t0 + wt * 16) >> p.c.bs_log2);
            ++ahead_u;
            if (++cur.step >= cur.steps) line.next_item(cur);
        };
        auto fetch = [&](uint4 (&r)[kPer], const uint8_t* codes) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int x = i * 128 + wt, t = t0 + x / kPer;
                r[i] = make_uint4(0, 0, 0, 0);      // behind the sequence's end: zeros, whatever the block holds
                if (phys[i] >= 0) {
                    const int64_t row = (((int64_t)phys[i] * p.c.heads + h) << p.c.bs_log2) + (t & (bs - 1));
                    r[i] = __ldg(reinterpret_cast<const uint4*>(codes + row * D) + x % kPer);
                }
            }
        };
        auto store = [&](const uint4 (&r)[kPer], uint8_t* dst) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int x = i * 128 + wt, row = x / kPer, piece = x % kPer;
                const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
                uint4 a, b;
                a.x = half2_lo(w[0]), a.y = half2_hi(w[0]), a.z = half2_lo(w[1]), a.w = half2_hi(w[1]);
                b.x = half2_lo(w[2]), b.y = half2_hi(w[2]), b.z = half2_lo(w[3]), b.w = half2_hi(w[3]);
                uint8_t* panel = dst + (piece >> 2) * S::kPanel;
                const uint32_t c0 = (piece & 3) * 2;
                // the two panels share banks: their pieces go in opposite order
                if (piece & 4) {
                    *reinterpret_cast<uint4*>(panel + tc::sw128_offset(row, c0 + 1)) = b;
                    *reinterpret_cast<uint4*>(panel + tc::sw128_offset(row, c0)) = a;
                } else {
                    *reinterpret_cast<uint4*>(panel + tc::sw128_offset(row, c0)) = a;
                    *reinterpret_cast<uint4*>(panel + tc::sw128_offset(row, c0 + 1)) = b;
                }
            }
        };
        auto scales = [&]() {
            ks = 0.0f;
            vs = 1.0f;
            if (my_phys >= 0) {
                const int64_t unit = (int64_t)my_phys * p.c.heads + h;
                ks = __ldg(p.c.k_scale + unit);
                vs = __ldg(p.c.v_scale + unit);
            }
        };
        bool ok = true;
        if (u0 < u1) {
            look();
            fetch(kr, p.c.k);
            fetch(vr, p.c.v);
            scales();
        }
        for (int64_t u = u0; u < u1; ++u, ++tile) {
            const uint32_t st = tile & 1;
            if (tile >= 2) {
                ok = __all_sync(0xFFFFFFFFu, wait(kKEmpty + st, (k_phase >> st) & 1u));
                if (!ok) break;
                k_phase ^= 1u << st;
            }
            store(kr, smem + S::k + st * S::kTile);
            if (wt < 8) sc[(tile & 3) * 8 + wt] = make_float2(ks, (float)((int)(__float_as_uint(vs) >> 23) - 127));
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(bars + kKFull + st);
            look();
            fetch(kr, p.c.k);
            scales();
            if (tile >= 2) {
                ok = __all_sync(0xFFFFFFFFu, wait(kVEmpty + st, (v_phase >> st) & 1u));
                if (!ok) break;
                v_phase ^= 1u << st;
            }
            store(vr, smem + S::v + st * S::kTile);
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(bars + kVFull + st);
            fetch(vr, p.c.v);
        }
    } else if (warp == 12 && lane == 0) {
        // ---------------------------------------------------------------- every tcgen05.mma of the CTA
        constexpr uint32_t idesc_s = tc::idesc_f16_f32(128, kPos);
        constexpr uint32_t idesc_o = tc::idesc_f16_f32(128, D, false, true);
        const uint64_t dq = tc::desc_sw128(tc::smem_u32(smem + S::q)), dk = tc::desc_sw128(tc::smem_u32(smem + S::k));
        const uint64_t dv = tc::desc_mn_sw128(tc::smem_u32(smem + S::v), S::kPanel, 1024);
        uint32_t tile = 0, q_phase = 0, p_phase = 0;
        bool ok = true;
        auto scores = [&](int t, uint32_t st) {      // S_t = Q_t K^T
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                const uint32_t off = (x >> 2) * S::kPanel + (x & 3) * 32;
                tc::mma_f16(tmem + t * 128, tc::desc_at(dq, t * S::kTile + off), tc::desc_at(dk, st * S::kTile + off), idesc_s, x > 0);
            }
        };
        auto outputs = [&](int t, uint32_t st, bool more) {   // O_t += P_t V
#pragma unroll
            for (int x = 0; x < kPos / 16; ++x)
                tc::mma_f16_ta(tmem + kColO + t * D, tmem + t * 128 + x * 8, tc::desc_at(dv, st * S::kTile + x * 2048), idesc_o,
                               more || x > 0);
        };
        for (int64_t u = u0; u < u1 && ok;) {
            const int left = cur.steps - cur.step;
            const int todo = u1 - u < left ? (int)(u1 - u) : left;
            const int tiles = cur.rows > kTileRows ? 2 : 1;
            ok = wait(kQ, q_phase);
            q_phase ^= 1;
            for (int i = 0; i <= todo && ok; ++i) {
                const uint32_t st = tile & 1, prev = st ^ 1;     // stage of tile i, and of tile i - 1
                if (i < todo) ok = wait(kKFull + st, (tile >> 1) & 1u);
                if (i > 0) ok = ok && wait(kVFull + prev, ((tile - 1) >> 1) & 1u);
                for (int t = 0; t < tiles && ok; ++t) {
                    if (i > 0) {
                        ok = wait(kP + t, (p_phase >> t) & 1u);
                        if (!ok) break;
                        p_phase ^= 1u << t;
                        tc::fence_after_sync();
                        outputs(t, prev, i > 1);
                        if (t == tiles - 1) tc::mma_commit(bars + kVEmpty + prev);
                    } else {
                        tc::fence_after_sync();
                    }
                    if (i < todo) {
                        scores(t, st);
                        tc::mma_commit(bars + kS + t);
                        if (t == tiles - 1) tc::mma_commit(bars + kKEmpty + st);
                    }
                }
                if (i < todo) ++tile;
            }
            if (ok) tc::mma_commit(bars + kO);
            u += todo;
            cur.step += todo - 1;
            if (++cur.step >= cur.steps) line.next_item(cur);
        }
        if (!ok) {
            // the products already issued still write: a last commit, waited for with the full limit
            tc::mma_commit(bars + kDrain);
            tc::mbar_wait(bars + kDrain, 0);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 12) tc::tmem_dealloc(tmem, 512);
}

// The items that the line's cuts went through: CTA x merges the item that
// starts in piece x, 16 bytes of a row a thread, the parts in order.
template <int D>
__global__ void __launch_bounds__(256) k_kv8_prefill_combine(const __grid_constant__ Params p) {
    pdl_begin();
    const int x = blockIdx.x;
    const float* first = p.a.part + ((int64_t)x * 2 + 1) * Part<D>::kFloats;
    const int* desc = reinterpret_cast<const int*>(first + Part<D>::kDesc);
    const int parts = desc[4], rows = desc[3], row = threadIdx.x, q4 = blockIdx.y;
    if (parts < 2 || row >= rows) return;
    auto part = [&](int i) { return i == 0 ? first : p.a.part + (int64_t)(x + i) * 2 * Part<D>::kFloats; };
    float m = kNone, M = kNone, l = 0.0f;
    for (int i = 0; i < parts; ++i) {
        const float* s3 = part(i) + Part<D>::kStats + row * 3;
        m = fmaxf(m, s3[0]);
        M = fmaxf(M, s3[2]);
    }
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < parts; ++i) {
        const float* b = part(i);
        const float* s3 = b + Part<D>::kStats + row * 3;
        const float4 v = reinterpret_cast<const float4*>(b)[(int64_t)q4 * kRows + row];
        l += s3[1] * ex2(s3[0] - m);
        const float f = ex2(s3[2] - M);
        s.x += v.x * f;
        s.y += v.y * f;
        s.z += v.z * f;
        s.w += v.w * f;
    }
    const int j = (desc[2] + row) / p.G, g = desc[2] + row - j * p.G;
    const int64_t at = ((int64_t)desc[0] * p.a.q.T + j) * p.a.q.H + desc[1] * p.G + g;
    const float f = l == 0.0f ? 0.0f : ex2(M - m) / l;
    uint32_t w[2];
    if (p.a.q.is_bf16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(s.x * f, s.y * f), b = __floats2bfloat162_rn(s.z * f, s.w * f);
        memcpy(&w[0], &a, 4);
        memcpy(&w[1], &b, 4);
    } else {
        const __half2 a = __floats2half2_rn(s.x * f, s.y * f), b = __floats2half2_rn(s.z * f, s.w * f);
        memcpy(&w[0], &a, 4);
        memcpy(&w[1], &b, 4);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.a.out) + at * D + q4 * 4) = make_uint2(w[0], w[1]);
    if (p.a.lse && q4 == 0) p.a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch(const Params& p, cudaStream_t st) {
    using S = Smem<D>;
    static_assert(S::bytes <= 227 * 1024, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(k_kv8_prefill<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_kv8_prefill<D>, p.ctas, kThreads, S::bytes, st, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_kv8_prefill_combine<D>, dim3(p.ctas, D / 4), kRows, 0, st, p);
}

}  // namespace

size_t kv8_prefill_part_floats(int dim) { return (size_t)2 * kMaxCtas * (dim == 64 ? Part<64>::kFloats : Part<128>::kFloats); }

cudaError_t launch_kv8_prefill(const DevKv8& c, const Kv8Attn& a, cudaStream_t st) {
    Params p;
    p.c = c;
    p.a = a;
    p.G = a.q.H / c.heads;
    p.row_blocks = (int)(((int64_t)a.q.T * p.G + kRows - 1) / kRows);
    p.wait_limit = wait_limit();
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    p.ctas = sms < kMaxCtas ? sms : kMaxCtas;
    return c.dim == 64 ? launch<64>(p, st) : launch<128>(p, st);
}

}  // namespace csa2
