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
constexpr int kSlots = 5, kRowBytes = 16 * 128, kSlot = kRowBytes + 128;   // a warp's ring: lines of 16 blocks, their scales and pages
// CTAs an SM.  5 with four slots: 20.2 against 19.7 us (16,384 blocks of one sequence), 20.1
// against 18.7 us (32 sequences); 3, or 80 registers a thread, cost 3 us.
constexpr int kPerSm = 4;

struct Params {
    DevKv8 c;
    Kv8Query q;
    int G, n_sel, n_first, n_recent;
    int32_t* idx;
    float* scores;   // [batch][T][heads][max_blocks]
    uint32_t* status;
};

// Two 16-bit values as floats.
__device__ __forceinline__ float2 both(uint32_t w, int is_bf16) {
    if (is_bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}

// Eight query heads in operand layout: whole numbers of at most 127 in units of
// 2^e.  The 2 D bytes of a block's bounds are one k axis, of which lane column
// c holds bytes 128 x + 32 c .. + 31: for D = 128 the same 32 channels' lower
// (x = 0) and upper (x = 1) bounds, for D = 64 lower (c < 2) or upper ones.
template <int D>
struct QueryRows {
    uint32_t b[16];                      // two channels a word
    float unit[2];                       // 2^e of rows 2c and 2c + 1

    // Heads g0 + r of key head h.
    __device__ __forceinline__ void load(const Params& p, int bq, int j, int h, int g0, int r, int c) {
        const int g = g0 + r;
        const uint16_t* src = static_cast<const uint16_t*>(p.q.q) + (int64_t)bq * p.q.stride_b +
                              (int64_t)j * p.q.stride_t + (int64_t)(h * p.G + g) * D + (D == 128 ? c : c & 1) * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (g < p.G) x = __ldg(reinterpret_cast<const uint4*>(src) + i);
            b[4 * i] = x.x, b[4 * i + 1] = x.y, b[4 * i + 2] = x.z, b[4 * i + 3] = x.w;
        }
    }
    __device__ __forceinline__ void round(const Params& p, int g0, int r, int c) {
        const uint32_t inf = p.q.is_bf16 ? 0x7F80u : 0x7C00u;
        uint32_t odd = 0;                // what is not finite counts as 0: rare, out of the way
#pragma unroll
        for (int i = 0; i < 16; ++i) odd |= (uint32_t)((b[i] & inf) == inf) | (uint32_t)((b[i] >> 16 & inf) == inf);
        if (__any_sync(0xFFFFFFFFu, odd)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if ((b[i] & inf) == inf) b[i] &= 0xFFFF0000u;
                if ((b[i] >> 16 & inf) == inf) b[i] &= 0xFFFFu;
            }
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f = both(b[i], p.q.is_bf16);
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        // the least e with amax <= 127 * 2^e (127 = 1.984375 * 2^6)
        const uint32_t u = __float_as_uint(amax);
        int e = (int)(u >> 23) - 127 - 6 + ((u & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
        e = e < -118 ? -118 : e;
        const float mine = g0 + r < p.G ? exp2_int(e) : -INFINITY, down = exp2_int(-e);
        unit[0] = __shfl_sync(0xFFFFFFFFu, mine, 2 * c * 4);
        unit[1] = __shfl_sync(0xFFFFFFFFu, mine, (2 * c + 1) * 4);
        constexpr float kWhole = 12582912.0f;   // 1.5 * 2^23: adding it rounds to whole numbers, ties to even
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f = both(b[i], p.q.is_bf16);
            __half2 h = __floats2half2_rn(__fmaf_rn(f.x, down, kWhole) - kWhole, __fmaf_rn(f.y, down, kWhole) - kWhole);
            if (D == 64) {   // this lane's half of the k axis is all lower or all upper bounds
                const __half2 z = __floats2half2_rn(0.0f, 0.0f);
                h = c < 2 ? __hmin2(h, z) : __hmax2(h, z);
            }
            memcpy(&b[i], &h, 4);
        }
    }
    // Word w as it meets the lower (x = 0) or upper bounds.
    __device__ __forceinline__ uint32_t part(int x, int w) const {
        if (D == 64) return b[w];
        uint32_t lo, hi;
        asm("min.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(b[w]), "r"(0u));
        asm("max.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b[w]), "r"(0u));
        return x ? hi : lo;
    }
};

// Asynchronous copies of 16 (4) bytes; zeros where `there` is false.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Blocks that query row (b, j) sees; false beyond the call's rows.
__device__ __forceinline__ bool row_of(const Params& p, int b, int j, int& visible, bool report) {
    uint32_t* status = report ? p.status : nullptr;
    const int L = kv8_len(p.c, b, status), n = kv8_rows(p.q.n_q, b, p.q.T, status);
    const int pos = L - n + j;
    visible = pos < 0 ? 0 : (pos >> p.c.bs_log2) + 1;
    return j < n;
}

// Scores of all rows.  The tiles of 16 blocks of every row (token, key head) of
// every sequence form one line that the grid's warps cut into equal runs (the
// lengths are on the device: every warp sums them itself), since rows of one
// batch differ in length and a warp has only a few tiles.  A tile's blocks are the
// rows of the matrix tile, eight query heads its columns; the 2 D bytes a block
// go by asynchronous copies into a ring of the warp's own, four lines ahead,
// whole lines at a time: an SM asks for about 340 lines a microsecond, whatever
// part of a line it asks for.  (Loads to registers, one line ahead: 20.9 against
// 19.7 us, 22.3 against 18.7 us.)  With the bounds in L2 it takes as long: what
// bounds it is the instructions of a line, and those before the first, which
// have to be fetched; hence the short loops.
template <int D>
__global__ void __launch_bounds__(kThreads, kPerSm) k_kv8_score(const __grid_constant__ Params p) {
    constexpr int kLines = D / 64;
    extern __shared__ __align__(16) uint8_t rings[];
    pdl_begin();
    uint8_t* ring = rings + (threadIdx.x >> 5) * kSlots * kSlot;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int nb = p.c.batch, per = (nb + 31) >> 5, heads = p.c.heads;
    struct Seq {
        int L, n, tiles;      // positions, query rows, tiles that its last row sees
    };
    auto sequence = [&](int b, uint32_t* status) {
        Seq q = {0, 0, 0};
        if (b < nb) {
            q.L = kv8_len(p.c, b, status);
            q.n = kv8_rows(p.q.n_q, b, p.q.T, status);
            if (q.L > 0) q.tiles = ((q.L - 1) >> (p.c.bs_log2 + 4)) + 1;
        }
        return q;
    };
    uint32_t* report = blockIdx.x == 0 && threadIdx.x < 32 ? p.status : nullptr;
    Seq mine = {0, 0, 0};
    int64_t sum = 0;
    for (int i = 0; i < per; ++i) {
        mine = sequence(lane * per + i, report);
        sum += (int64_t)mine.n * heads * mine.tiles;
    }
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    const int64_t before = upto - sum, total = __shfl_sync(0xFFFFFFFFu, upto, 31);
    const int warps = gridDim.x * kWarps, id = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int share = total < warps ? (int)total : warps;
    if (id >= share) return;
    const int64_t size = total / share, more = total - size * share;
    int64_t u = size * id + (id < more ? id : more);
    const int64_t u1 = u + size + (id < more ? 1 : 0);
    // the sequence, row and tile of step u
    const int at = 31 - __clz(__ballot_sync(0xFFFFFFFFu, before <= u));
    int64_t off = u - __shfl_sync(0xFFFFFFFFu, before, at);
    int b = at * per;
    Seq seq;
    if (per == 1) {
        seq.L = __shfl_sync(0xFFFFFFFFu, mine.L, at);
        seq.n = __shfl_sync(0xFFFFFFFFu, mine.n, at);
        seq.tiles = __shfl_sync(0xFFFFFFFFu, mine.tiles, at);
    } else {
        for (;; ++b) {
            seq = sequence(b, nullptr);
            const int64_t t = (int64_t)seq.n * heads * seq.tiles;
            if (off < t) break;
            off -= t;
        }
    }
    int row = (int)(off / seq.tiles), t0 = (int)(off - (int64_t)row * seq.tiles);

    while (u < u1) {
        const int j = row / heads, h = row - j * heads;
        const int nt = seq.tiles - t0 < u1 - u ? seq.tiles - t0 : (int)(u1 - u), first = t0 * 16;
        const int pos = seq.L - seq.n + j, visible = pos < 0 ? 0 : (pos >> p.c.bs_log2) + 1;
        // pages of tiles t and t + 1: lanes 0 .. 15 and 16 .. 31
        auto pages = [&](int t) {
            const int lb = first + t * 16 + lane;
            return t + (lane >> 4) < nt && lb < visible ? kv8_block(p.c, b, lb) : -1;
        };
        const uint8_t* base = p.c.k_bounds + h * 2 * D + (lane & 7) * 16;
        float* out = p.scores + ((int64_t)(b * p.q.T + j) * heads + h) * p.c.max_blocks;
        for (int g0 = 0; g0 < p.G && first < visible; g0 += 8) {
            int now = pages(0), next = pages(2), sent = 0, to = 0;   // line `sent` goes to slot `to` next
            auto send = [&] {
                const int t = sent / kLines, x = sent - t * kLines;
                uint8_t* slot = ring + to * kSlot;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = i * 4 + (lane >> 3), phys = __shfl_sync(0xFFFFFFFFu, now, (t & 1) * 16 + row);
                    copy16(slot + row * 128 + (((lane & 7) ^ (row & 7)) << 4),
                           base + (int64_t)(phys < 0 ? 0 : phys) * heads * 2 * D + x * 128, phys >= 0);
                }
                if (x == kLines - 1) {       // the tile's pages and key scales, with its last line
                    const int phys = __shfl_sync(0xFFFFFFFFu, now, (t & 1) * 16 + (lane & 15));
                    if (lane < 16) {
                        copy4(slot + kRowBytes + lane * 4, p.c.k_scale + (int64_t)(phys < 0 ? 0 : phys) * heads + h, phys >= 0);
                        reinterpret_cast<int*>(slot + kRowBytes + 64)[lane] = phys;
                    }
                    if (t & 1) {
                        now = next;
                        next = pages(t + 3);
                    }
                }
                ++sent;
                if (++to == kSlots) to = 0;
            };
            QueryRows<D> q;
            q.load(p, b, j, h, g0, r, c);
            const int lines = nt * kLines;
#pragma unroll 1
            for (int s = 0; s < kSlots - 1; ++s) {
                if (s < lines) send();
                copies_commit();
            }
            q.round(p, g0, r, c);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            int t = 0, x = 0, at = 0;
#pragma unroll 1
            for (int s = 0; s < lines; ++s) {
                copies_wait<kSlots - 2>();
                __syncwarp();                       // everyone's copies are there, and the slot before has been read
                if (sent < lines) send();
                copies_commit();
                const uint8_t* slot = ring + at * kSlot;
                uint4 w[2][2];
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        w[half][i] = *reinterpret_cast<const uint4*>(slot + (half * 8 + r) * 128 + (((2 * c + i) ^ r) << 4));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t u0 = word(w[0][i >> 2], i & 3), u1 = word(w[1][i >> 2], i & 3);
                    const uint32_t a[4] = {half2_lo(u0), half2_lo(u1), half2_hi(u0), half2_hi(u1)};
                    mma_16816(acc, a, q.part(x, 2 * i), q.part(x, 2 * i + 1));
                }
                if (++at == kSlots) at = 0;
                if (++x < kLines) continue;
                x = 0;
                // rows without a query head hold 0 * -inf: fmaxf drops the NaN
                float best[2] = {fmaxf(acc[0] * q.unit[0], acc[1] * q.unit[1]), fmaxf(acc[2] * q.unit[0], acc[3] * q.unit[1])};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    best[half] = fmaxf(best[half], __shfl_xor_sync(0xFFFFFFFFu, best[half], 1));
                    best[half] = fmaxf(best[half], __shfl_xor_sync(0xFFFFFFFFu, best[half], 2));
                    const int lb = first + t * 16 + half * 8 + r;
                    if (c == 0 && lb < visible) {
                        const bool here = reinterpret_cast<const int*>(slot + kRowBytes + 64)[half * 8 + r] >= 0;
                        if (!here) flag(p.status, kStatusBounds);
                        const float score = here ? best[half] * reinterpret_cast<const float*>(slot + kRowBytes)[half * 8 + r] : -INFINITY;
                        out[lb] = g0 ? fmaxf(score, out[lb]) : score;
                    }
                }
                acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
                ++t;
            }
            copies_wait<0>();
            __syncwarp();                           // the ring is free
        }
        u += nt;
        t0 = 0;
        if (++row >= seq.n * heads) {
            row = 0;
            do seq = sequence(++b, nullptr);
            while (b < nb && (seq.n == 0 || seq.tiles == 0));
        }
    }
}

// ---------------------------------------------------------------- the best blocks of a row
constexpr int kCand = 2048;      // candidates resolved by rank

template <int THREADS>
struct SelSmem {
    static constexpr int kBins = 2 * THREADS, kWarps = THREADS / 32;
    uint32_t hist[kBins];
    uint32_t cand_key[kCand];
    int cand_idx[kCand];
    uint32_t red[kWarps][2];
    int n_cand, bin, above;
};

template <int THREADS>
__device__ __forceinline__ uint32_t block_sum(uint32_t v, SelSmem<THREADS>& s) {
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5][0] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(0xFFFFFFFFu, lane < THREADS / 32 ? s.red[lane][0] : 0u);
}

// One CTA per row.  The blocks that compete are those between the first and
// the newest ones; `want` of them are taken: linear bins between the least and
// the greatest score find the bin with the cut, whose members are ranked
// exactly by (score, lower index first).  Many equal scores (a bin too full
// to rank) are cut by bisection over the score's bits and then over the index.
// The chosen are bits of a map over the row's blocks, read out in order.  KPT
// keys a thread stay in registers, fetched before the row's length is known;
// KPT == 0: rows of any length, keys kept in the scores' place.
template <int KPT, int THREADS>
__global__ void __launch_bounds__(THREADS) k_kv8_select(const __grid_constant__ Params p) {
    constexpr int kBins = SelSmem<THREADS>::kBins, kSelWarps = THREADS / 32;
    __shared__ SelSmem<THREADS> s;
    extern __shared__ uint32_t map[];                          // a bit a block
    pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t* row = reinterpret_cast<uint32_t*>(p.scores + (int64_t)blockIdx.x * p.c.max_blocks);
    constexpr int kKeys = KPT ? KPT : 1;
    uint32_t reg[kKeys];
    if (KPT) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int at = i * THREADS + tid;
            reg[i] = at < p.c.max_blocks ? row[at] : 0u;
        }
    }
    const int bj = blockIdx.x / p.c.heads, b = bj / p.q.T;
    int visible;
    if (!row_of(p, b, bj - b * p.q.T, visible, false)) return;
    int32_t* out = p.idx + (int64_t)blockIdx.x * p.n_sel;
    if (visible <= p.n_sel) {
        for (int i = tid; i < p.n_sel; i += THREADS) out[i] = i < visible ? i : -1;
        return;
    }
    const int c0 = p.n_first, c1 = visible - p.n_recent;       // competing blocks [c0, c1); c0 <= c1 as n_sel < visible
    const int want = p.n_sel - p.n_first - p.n_recent, words = (visible + 31) >> 5;
    auto key_of = [](uint32_t bits) {
        const float f = __uint_as_float(bits);
        return isnan(f) ? 0u : ordered_key(f);
    };
    // every competing (index, key) of this thread
    auto each = [&](auto&& f) {
        if (KPT) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                const int at = i * THREADS + tid;
                if (at >= c0 && at < c1) f(at, reg[i]);
            }
        } else {
#pragma unroll 4
            for (int at = c0 + tid; at < c1; at += THREADS) f(at, row[at]);
        }
    };
    auto choose = [&](int at) { atomicOr(map + (at >> 5), 1u << (at & 31)); };
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    if (KPT) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) reg[i] = key_of(reg[i]);
    } else {
        for (int at = c0 + tid; at < c1; at += THREADS) row[at] = key_of(row[at]);
    }
    each([&](int, uint32_t key) {
        lo = min(lo, key);
        hi = max(hi, key);
    });
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if (lane == 0) s.red[warp][0] = lo, s.red[warp][1] = hi;
    for (int i = tid; i < kBins; i += THREADS) s.hist[i] = 0;
    for (int i = tid; i < words; i += THREADS) {           // the first and the newest are chosen
        uint32_t m = 0;
        for (int x = i * 32; x < i * 32 + 32; ++x)
            if (x < c0 || (x >= c1 && x < visible)) m |= 1u << (x & 31);
        map[i] = m;
    }
    if (tid == 0) s.n_cand = 0;
    __syncthreads();
    lo = __reduce_min_sync(0xFFFFFFFFu, lane < kSelWarps ? s.red[lane][0] : 0xFFFFFFFFu);
    hi = __reduce_max_sync(0xFFFFFFFFu, lane < kSelWarps ? s.red[lane][1] : 0u);
    const float flo = lo ? key_score(lo) : -INFINITY, fhi = hi ? key_score(hi) : -INFINITY;
    const float per = (float)(kBins - 1) / (fhi - flo);
    const bool linear = fhi - flo > 0.0f && fhi - flo < INFINITY && per < INFINITY;
    bool done = want == 0;
    if (!done && linear) {
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
                if (lane >= o) inc += v;
            }
            if (lane == 31) s.red[warp][0] = inc;
            __syncthreads();
            const uint32_t w = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s.red[lane][0] : 0u);
            const uint32_t after = w + inc, before = after - n;
            if (before < (uint32_t)want && after >= (uint32_t)want) {
                const bool second = before + n0 < (uint32_t)want;
                s.bin = kBins - 1 - 2 * tid - (second ? 1 : 0);
                s.above = (int)(before + (second ? n0 : 0u));
            }
        }
        __syncthreads();
        const int bin = s.bin, need = want - s.above, members = (int)s.hist[bin];
        if (members <= kCand) {
            each([&](int at, uint32_t key) {     // higher bins are chosen, members of this one ranked
                const int v = bin_of(key);
                if (v > bin) choose(at);
                if (v == bin) {
                    const int i = atomicAdd(&s.n_cand, 1);
                    s.cand_key[i] = key;
                    s.cand_idx[i] = at;
                }
            });
            __syncthreads();
            for (int i = warp; i < members; i += kSelWarps) {          // a warp a member
                const uint32_t key = s.cand_key[i];
                const int at = s.cand_idx[i];
                int rank = 0;
                for (int o = lane; o < members; o += 32) {
                    const uint32_t ko = s.cand_key[o];
                    rank += ko > key || (ko == key && s.cand_idx[o] < at);
                }
                rank = __reduce_add_sync(0xFFFFFFFFu, rank);
                if (lane == 0 && rank < need) choose(at);
            }
            done = true;
        }
    }
    if (!done) {
        // the greatest key with at least `want` keys >= it, then the index of the last tie taken
        uint32_t a = lo, z = hi;
        while (a < z) {
            const uint32_t mid = a + (z - a) / 2 + 1;
            uint32_t n = 0;
            each([&](int, uint32_t key) { n += key >= mid; });
            if (block_sum(n, s) >= (uint32_t)want) a = mid;
            else z = mid - 1;
        }
        uint32_t n = 0;
        each([&](int, uint32_t key) { n += key > a; });
        const uint32_t need = (uint32_t)want - block_sum(n, s);
        int x = c0, y = c1 - 1;
        while (x < y) {
            const int mid = (x + y) / 2;
            n = 0;
            each([&](int at, uint32_t key) { n += at <= mid && key == a; });
            if (block_sum(n, s) >= need) y = mid;
            else x = mid + 1;
        }
        each([&](int at, uint32_t key) {
            if (key > a || (key == a && at <= x)) choose(at);
        });
    }
    __syncthreads();
    // ---- the map in order: THREADS words at a time
    int base = 0;
    for (int i0 = 0; i0 < words; i0 += THREADS) {
        uint32_t m = i0 + tid < words ? map[i0 + tid] : 0u;
        const uint32_t n = __popc(m);
        uint32_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s.red[warp][1] = inc;
        __syncthreads();
        const uint32_t w = lane < kSelWarps ? s.red[lane][1] : 0u;
        int at = base + (int)(__reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0u) + inc - n);
        base += (int)__reduce_add_sync(0xFFFFFFFFu, w);
        for (; m; m &= m - 1) {
            if (at < p.n_sel) out[at] = (i0 + tid) * 32 + __ffs(m) - 1;
            ++at;
        }
        if (i0 + THREADS < words) __syncthreads();
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
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t most = ((int64_t)rows * ((c.max_blocks + 15) / 16) + kWarps - 1) / kWarps;   // CTAs with a tile a warp
    const unsigned ctas = (unsigned)(most < sms * kPerSm ? most : sms * kPerSm);
    const int ring = kWarps * kSlots * kSlot;
    e = c.dim == 64 ? launch_pdl(k_kv8_score<64>, ctas, kThreads, ring, st, p)
                    : launch_pdl(k_kv8_score<128>, ctas, kThreads, ring, st, p);
    if (e != cudaSuccess) return e;
    // rows of up to 512 blocks by 256 threads each, so that more of them run at once: 4,096 rows
    // of 256 blocks, with the scores, 104 us with 1,024 threads and 59 with 256, one row of 8 heads
    // over 512 blocks 8.0 and 7.2 (512 rows of 768 blocks 36.4 and 37.7)
    // A thread's keys stay in registers, as few as the row's blocks need, since every one of them is
    // looked at whether it is there or not; keys kept in the scores' place have no limit but are read
    // again.  Scores and selection for 8 rows, us, by keys a thread (0: in place): 2,048 blocks 2: 7.9,
    // 8: 9.2, 17: 11.3, 0: 9.2; 4,096 blocks 8: 10.5, 17: 12.8, 0: 10.9; 8,192 blocks 8: 11.6, 17: 13.7,
    // 0: 13.0; 12,000 blocks 17: 14.6, 24: 16.5, 0: 15.1; 17,408 blocks 17: 16.9, 24: 18.4, 0: 19.7; of 128
    // rows, 17,408 blocks 17: 78.6, 24: 82.4, 0: 96.8.  24,000 blocks 24: 20.5, 0: 24.0.
    const bool small = c.max_blocks <= 512;
    const auto select = small                       ? k_kv8_select<2, 256>
                        : c.max_blocks <= 2 * 1024  ? k_kv8_select<2, 1024>
                        : c.max_blocks <= 8 * 1024  ? k_kv8_select<8, 1024>
                        : c.max_blocks <= 17 * 1024 ? k_kv8_select<17, 1024>
                                                    : k_kv8_select<0, 1024>;
    const int map_bytes = (c.max_blocks + 31) / 32 * 4;
    if (map_bytes > 16 * 1024) e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, map_bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(select, dim3(rows), small ? 256 : 1024, map_bytes, st, p);
}

}  // namespace csa2
