// Attention over the 8-bit cache for few query rows per sequence (decode and
// short verification), dense or over listed blocks.
//
// One query row needs two products with every cached row, so up to the 32
// rows a pass holds the kernel is bound by the codes' bytes (2 * D a position
// and head) and its work is moving them: the codes go by TMA into a ring of
// each warp's own (no synchronisation between warps while they stream; the
// rows swizzled, so that the loads below are free of bank conflicts), from
// there as 16-byte loads straight into the operand layout of mma.m16n8k16,
// converted to fp16 by bit placement (exact).  The layouts need no
// transposition: a product's k order may be permuted as long as both operands
// agree, so a lane's 16 bytes of a key row are four k steps, and the
// probabilities leave the first product in the layout the second one reads.
// tcgen05 would take the codes as they are (kind::f8f6f4) but wants the
// probabilities as E4M3 terms and 128 rows a tile; with at most 32 rows it
// has nothing to win over a kernel that already waits for HBM.
//
// Work split: a step is 64 positions of one (sequence, head, row tile); the
// steps of the whole batch form one line, which the CTAs cut into equal
// pieces (the lengths are on the device, so every CTA sums them itself).  A
// CTA finishes what lies inside its piece; an item that is cut leaves
// partials (output, running maxima and sum), merged by k_kv8_combine in a
// fixed order, so results do not vary from run to run.
#include <cuda.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv8.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 16;                 // positions a warp takes at a time
constexpr int kStep = kWarps * kTile;     // positions a CTA takes at a time
constexpr float kNone = -3.0e38f;         // running maximum before any position
// Weights are 2^(z - M + 8) in fp16: the greatest is a power of two (exact, so
// that a row with one dominant position rounds only once), and weights down to
// 2^-22 of it keep fp16's full precision.  The 2^8 cancels the 2^-8 of the
// value codes' bit placement.
constexpr float kHeadroom = 8.0f;
constexpr int kMaxCtas = 3 * 148;

struct Params {
    DevKv8 c;
    Kv8Attn a;
    int G, gt, ctas;   // query heads of a key head; row tiles of a token (listed blocks)
    uint32_t wait_limit;
};

// Where a step lies: sequence b, head h, row tile rt (of the sequence's rows
// (token, query head of h); of one token's rows when blocks are listed), step `step` of `steps`.  L, n: the sequence's positions
// and query rows; lo: its first position, on a tile boundary.
struct Cursor {
    int b, h, rt, step;
    int steps, tiles, L, n, lo;
};

template <int MT, bool LIST>
struct Work {
    const Params& p;
    __device__ explicit Work(const Params& p) : p(p) {}

    // Rows of item k, and the (token, head of the group) of its row i.
    __device__ __forceinline__ int rows(const Cursor& k) const {
        const int left = LIST ? p.G - k.rt % p.gt * 16 * MT : k.n * p.G - k.rt * 16 * MT;
        return left < 16 * MT ? left : 16 * MT;
    }
    __device__ __forceinline__ int2 token(const Cursor& k, int i) const {
        if (LIST) {
            const int j = k.rt / p.gt;
            return make_int2(j, (k.rt - j * p.gt) * 16 * MT + i);
        }
        const int j = (k.rt * 16 * MT + i) / p.G;
        return make_int2(j, k.rt * 16 * MT + i - j * p.G);
    }
    // The shape of sequence b's items.
    __device__ __forceinline__ void load(Cursor& k, int b, uint32_t* status) const {
        k.b = b;
        k.h = k.rt = k.step = 0;
        k.steps = k.tiles = k.L = k.n = k.lo = 0;
        if (b >= p.c.batch) return;
        k.L = kv8_len(p.c, b, status);
        k.n = kv8_rows(p.a.q.n_q, b, p.a.q.T, status);
        if (k.n == 0) return;
        if (LIST) {
            const int vis = k.L > 0 ? ((k.L - 1) >> p.c.bs_log2) + 1 : 0;
            const int e = vis < p.a.n_sel ? vis : p.a.n_sel;
            k.steps = ((e << p.c.bs_log2) + kStep - 1) / kStep;
            k.tiles = k.n * p.gt;
        } else {
            if (p.a.window) {
                const int64_t first = (int64_t)k.L - k.n - p.a.window + 1;
                k.lo = first > 0 ? (int)first / kTile * kTile : 0;
            }
            k.steps = (k.L - k.lo + kStep - 1) / kStep;
            k.tiles = (k.n * p.G + 16 * MT - 1) / (16 * MT);
        }
        if (k.steps < 1) k.steps = 1;  // an empty row still has to be written
    }
    __device__ __forceinline__ int64_t total(const Cursor& k) const {
        return (int64_t)p.c.heads * k.tiles * k.steps;
    }
    __device__ __forceinline__ void seek(Cursor& k, int64_t u) const {  // step u of the sequence
        const int64_t item = u / k.steps;
        k.step = (int)(u - item * k.steps);
        k.h = (int)(item / k.tiles);
        k.rt = (int)(item - (int64_t)k.h * k.tiles);
    }
    __device__ __forceinline__ void next_item(Cursor& k) const {
        k.step = 0;
        if (++k.rt < k.tiles) return;
        k.rt = 0;
        if (++k.h < p.c.heads) return;
        int b = k.b;
        do load(k, ++b, nullptr);
        while (b < p.c.batch && k.tiles == 0);
    }
};

// The line of all steps: its length, and the sequence that holds step u with
// the steps before it.  Every thread of the CTA calls it; `sums` is kThreads + 1
// words of shared memory.
template <int MT, bool LIST>
__device__ int64_t line_sums(const Work<MT, LIST>& w, int64_t* sums, uint32_t* status) {
    const int tid = threadIdx.x, nb = w.p.c.batch, per = (nb + kThreads - 1) / kThreads;
    int64_t s = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < nb) {
            Cursor k;
            w.load(k, b, status);
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

// The step u (0 <= u < total) as a cursor.
template <int MT, bool LIST>
__device__ void line_find(const Work<MT, LIST>& w, const int64_t* sums, int64_t u, Cursor& k) {
    const int nb = w.p.c.batch, per = (nb + kThreads - 1) / kThreads;
    int lo = 0, hi = kThreads;  // sums[lo] <= u < sums[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= u) lo = mid;
        else hi = mid;
    }
    u -= sums[lo];
    int b = lo * per;
    for (;; ++b) {
        w.load(k, b, nullptr);
        const int64_t t = w.total(k);
        if (u < t || b + 1 >= nb) break;
        u -= t;
    }
    w.seek(k, u);
}

// How many CTAs share `total` steps: all, but no fewer than two steps each.
__device__ __forceinline__ int64_t sharing(int64_t total, int ctas) {
    const int64_t most = (total + 1) / 2;
    return most < ctas ? (most < 1 ? 1 : most) : ctas;
}

template <int D, int MT>
struct Smem {
    static constexpr int kRows = kTile * D;          // bytes of one tile's keys (or values)
    // three CTAs an SM with one row tile, two with two: 2 or more tiles in flight a warp
    static constexpr int kStages = (MT == 1 ? 3 : 5) * (128 / D);
    static constexpr int kNt = D / 8;
    static constexpr int ring = 0;                                            // [warp][stage][K, V]
    static constexpr int merge = ring + kWarps * kStages * 2 * kRows;         // [warp][2][kNt][32] floats
    static constexpr int stats = merge + kWarps * 2 * kNt * 32 * 4;           // [warp][16 * MT][3] floats
    static constexpr int slots = stats + kWarps * 16 * MT * 3 * 4;            // [warp][stage] int2
    static constexpr int bars = slots + kWarps * kStages * 8;                 // [warp][stage]
    static constexpr int sums = bars + kWarps * kStages * 8;                  // kThreads + 1
    static constexpr int bytes = sums + (kThreads + 1) * 8 + 1024;            // base aligned to 1024
};

// Partial of a cut item: [32 rows][D] outputs, per row (m, l, M), then what
// k_kv8_combine needs of the item: b, h, rt, rows, and how many pieces it has.
template <int D>
struct Part {
    static constexpr int kStats = 32 * D, kDesc = kStats + 32 * 3, kFloats = kDesc + 32;
};

// N adjacent outputs x * f, rounded once to the query's type.
template <int N>
__device__ __forceinline__ void store_out(void* out, int is_bf16, int64_t at, const float* x, float f) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        if (is_bf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i] * f, x[2 * i + 1] * f);
            memcpy(&w[i], &h, 4);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i] * f, x[2 * i + 1] * f);
            memcpy(&w[i], &h, 4);
        }
    }
    uint16_t* dst = static_cast<uint16_t*>(out) + at;
    if (N == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[N / 2 - 2], w[N / 2 - 1]);
    else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

template <int D, int MT, bool LIST>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 3 : 2) k_kv8_attn(const __grid_constant__ Params p,
                                                                         const __grid_constant__ CUtensorMap kmap,
                                                                         const __grid_constant__ CUtensorMap vmap) {
    using S = Smem<D, MT>;
    constexpr int kChunks = D / 64;   // 16-byte chunks of a key row per lane
    constexpr int kNt = D / 8;        // n tiles of the second product; a lane's bytes of a value row
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + S::ring + warp * kStages * 2 * S::kRows;
    int2* slots = reinterpret_cast<int2*>(smem + S::slots) + warp * kStages;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::bars) + warp * kStages;
    int64_t* sums = reinterpret_cast<int64_t*>(smem + S::sums);
    const int bs = p.c.bs(), G = p.G, T = p.a.q.T, H = p.a.q.H;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) tc::mbar_init(bars + i, 1);
        tc::fence_mbar_init();
    }
    pdl_begin();
    const Work<MT, LIST> work(p);
    const int64_t total = line_sums(work, sums, blockIdx.x == 0 ? p.a.status : nullptr);
    const int64_t share = sharing(total, p.ctas);
    int* desc = reinterpret_cast<int*>(p.a.part + ((int64_t)blockIdx.x * 2 + 1) * Part<D>::kFloats + Part<D>::kDesc);
    if (tid == 0) desc[4] = 0;
    if (blockIdx.x >= share) return;
    const int64_t u0 = total * blockIdx.x / share, u1 = total * (blockIdx.x + 1) / share;
    if (u0 >= u1) return;

    Cursor cur, ahead;
    line_find(work, sums, u0, cur);
    ahead = cur;

    // ---- the copies: the ring runs ahead of the tiles by kStages - 1.  A
    // tile's block is looked up two tiles before its copy is issued (the list
    // entry) and one tile before (the page table), so neither load is waited for.
    int64_t ahead_u = u0;
    int look_b, look_h, look_t0, look_lb;
    auto peek = [&]() {      // describe the tile at `ahead`, start its list load, move on
        look_lb = -1;
        look_b = ahead.b;
        look_h = ahead.h;
        if (ahead_u >= u1) return;
        const int off = ahead.step * kStep + warp * kTile;
        if (LIST) {
            const int e = off >> p.c.bs_log2;
            look_t0 = off & (bs - 1);
            if (e < p.a.n_sel) {
                const int32_t* l = p.a.block_idx +
                                   (((int64_t)ahead.b * T + ahead.rt / p.gt) * p.c.heads + ahead.h) * p.a.n_sel + e;
                const int v = __ldg(l), prev = e ? __ldg(l - 1) : -1;
                const int pos = ahead.L - ahead.n + ahead.rt / p.gt;
                if (v >= 0) {
                    // strictly ascending, visible, nothing behind padding: anything else is skipped and flagged
                    if (pos < 0 || v > (pos >> p.c.bs_log2) || (e && v <= prev) || (e && prev < 0)) {
                        if (lane == 0) flag(p.a.status, kStatusBounds);
                    } else {
                        look_lb = v;
                    }
                } else if (v < -1 && lane == 0) {
                    flag(p.a.status, kStatusBounds);
                }
            }
        } else {
            const int t = ahead.lo + off;
            if (t < ahead.L) {
                look_lb = t >> p.c.bs_log2;
                look_t0 = t & (bs - 1);
            }
        }
        ++ahead_u;
        if (++ahead.step >= ahead.steps) work.next_item(ahead);
    };
    int hand_phys = -1, hand_h = 0, hand_t0 = 0, hand_lb = 0;
    auto lookup = [&]() {    // the page of the tile peeked at
        hand_phys = -1;
        hand_h = look_h;
        hand_lb = look_lb;
        hand_t0 = look_t0;
        if (look_lb >= 0) {
            hand_phys = kv8_block(p.c, look_b, look_lb);
            if (hand_phys < 0 && lane == 0) flag(p.a.status, kStatusBounds);
        }
    };
    bool alive = true;       // false once a wait ran out: no further copies, no further results
    uint32_t issued = 0;     // copies by slot still to be waited for (bit mask)
    auto issue = [&](int slot) {
        if (lane == 0) {
            int2 d = make_int2(-1, 0);
            if (hand_phys >= 0 && alive) {
                const int64_t unit = (int64_t)hand_phys * p.c.heads + hand_h;
                const int row = (int)((unit << p.c.bs_log2) + hand_t0);
                tc::mbar_arrive_expect_tx(bars + slot, 2 * S::kRows);
                tc::tma_load_2d(ring + slot * 2 * S::kRows, &kmap, 0, row, bars + slot);
                tc::tma_load_2d(ring + slot * 2 * S::kRows + S::kRows, &vmap, 0, row, bars + slot);
                d = make_int2((int)unit, (hand_lb << p.c.bs_log2) + hand_t0);
            }
            slots[slot] = d;
        }
    };

    peek();
    lookup();
    peek();
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
        issue(i);
        lookup();
        peek();
    }
    __syncwarp();
    int slot = 0;
    uint32_t phase = 0;      // parity of each slot's barrier (bit mask)
    int2 here = slots[0];
    float ks = here.x >= 0 ? __ldg(p.c.k_scale + here.x) : 0.0f;
    float vs = here.x >= 0 ? __ldg(p.c.v_scale + here.x) : 0.0f;

    int64_t u = u0;
    while (u < u1) {
        const bool from_start = cur.step == 0;
        const int item_left = cur.steps - cur.step;
        const int todo = u1 - u < item_left ? (int)(u1 - u) : item_left;
        const bool to_end = todo == item_left;
        const int rows = work.rows(cur);

        // ---- the query rows of this lane (r and r + 8 of every row tile) in operand layout
        uint32_t qa[MT][kChunks * 4][4];
        float zs[MT][2];     // factor from the product to a base-2 logit, without the key scale
        int pos[MT][2];      // position of the row's token (-1: no row)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = mt * 16 + half * 8 + r;
                const bool ok = row < rows;
                const int2 jg = work.token(cur, row);
                pos[mt][half] = ok ? cur.L - cur.n + jg.x : -1;
                uint32_t raw[kChunks][8];
                const uint16_t* src = static_cast<const uint16_t*>(p.a.q.q) + (int64_t)cur.b * p.a.q.stride_b +
                                      (int64_t)jg.x * p.a.q.stride_t + (int64_t)(cur.h * G + jg.y) * D;
#pragma unroll
                for (int k = 0; k < kChunks; ++k) {
                    uint4 x = make_uint4(0, 0, 0, 0), y = x;
                    if (ok) {
                        const uint4* s4 = reinterpret_cast<const uint4*>(src + (c * kChunks + k) * 16);
                        x = __ldg(s4);
                        y = __ldg(s4 + 1);
                    }
                    raw[k][0] = x.x, raw[k][1] = x.y, raw[k][2] = x.z, raw[k][3] = x.w;
                    raw[k][4] = y.x, raw[k][5] = y.y, raw[k][6] = y.z, raw[k][7] = y.w;
                }
                float back = 1.0f;
                if (p.a.q.is_bf16) {
                    // bf16 -> fp16: the row scaled by the power of two that takes its greatest finite
                    // magnitude to [2^14, 2^15), so that its eight bits survive down to 2^-28 of it
                    float amax = 0.0f;
#pragma unroll
                    for (int k = 0; k < kChunks; ++k)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float a = fabsf(__uint_as_float(raw[k][i] << 16));
                            const float b = fabsf(__uint_as_float(raw[k][i] & 0xFFFF0000u));
                            if (a <= 3.4028235e38f) amax = fmaxf(amax, a);
                            if (b <= 3.4028235e38f) amax = fmaxf(amax, b);
                        }
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
                    int e = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
                    e = e > 126 ? 126 : e;
                    const float up = exp2_int(e);
                    back = exp2_int(-e);
#pragma unroll
                    for (int k = 0; k < kChunks; ++k)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const __half2 h = __floats2half2_rn(__uint_as_float(raw[k][i] << 16) * up,
                                                                __uint_as_float(raw[k][i] & 0xFFFF0000u) * up);
                            memcpy(&raw[k][i], &h, 4);
                        }
                }
                // 2^8: what the codes' bit placement leaves out
                zs[mt][half] = back * 256.0f * p.a.sm_scale * 1.4426950408889634f;
#pragma unroll
                for (int k = 0; k < kChunks; ++k)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {  // k step s: channels 4s, 4s+2 | 4s+1, 4s+3 of the chunk
                        const uint32_t w0 = raw[k][2 * s], w1 = raw[k][2 * s + 1];
                        qa[mt][k * 4 + s][half] = __byte_perm(w0, w1, 0x5410);
                        qa[mt][k * 4 + s][2 + half] = __byte_perm(w0, w1, 0x7632);
                    }
            }

        float o[MT][kNt][4];
        float m[MT][2], l[MT][2], M[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int i = 0; i < kNt; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.0f;
#pragma unroll
            for (int half = 0; half < 2; ++half) m[mt][half] = M[mt][half] = kNone, l[mt][half] = 0.0f;
        }

#pragma unroll 1
        for (int i = 0; i < todo; ++i) {
            // refill the slot that was read last, then look at the next tile's scales
            {
                const int fill = slot == 0 ? kStages - 1 : slot - 1;
                issue(fill);
                lookup();
                peek();
            }
            const int unit = here.x, t0 = here.y;
            const float ks_now = ks, vs_now = vs;
            const int now = slot;
            slot = slot + 1 == kStages ? 0 : slot + 1;
            __syncwarp();
            here = slots[slot];
            if (here.x >= 0) {
                ks = __ldg(p.c.k_scale + here.x);
                vs = __ldg(p.c.v_scale + here.x);
            }
            if (unit < 0) continue;
            if (alive) {
                alive = tc::mbar_wait(bars + now, (phase >> now) & 1u, p.wait_limit);
                if (!alive && lane == 0) flag(p.a.status, kStatusTimeout);
            }
            alive = __all_sync(0xFFFFFFFFu, alive);
            if (!alive) {
                issued |= 1u << now;
                continue;
            }
            phase ^= 1u << now;
            const uint8_t* kt = ring + now * 2 * S::kRows;
            const uint8_t* vt = kt + S::kRows;

            // ---- S = Q K^T, two n tiles of eight positions
            float s[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.0f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int k = 0; k < kChunks; ++k) {
                    const uint32_t row = nt * 8 + r, chunk = c * kChunks + k;
                    const uint4 w = *reinterpret_cast<const uint4*>(
                        kt + (D == 128 ? tc::sw128_offset(row, chunk) : tc::sw64_offset(row, chunk)));
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint32_t even, odd;
                        e4m3x4_to_half(ww[q4], even, odd);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) mma_16816(s[mt][nt], qa[mt][k * 4 + q4], even, odd);
                    }
                }

            // ---- base-2 logits, masked; a vote tells whether a running maximum moves at all.  m: maximum of the logits (for l), M: of logit + log2(value scale) (for the output)
            const float ev = (float)((int)(__float_as_uint(vs_now) >> 23) - 127);
            bool over = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float f = zs[mt][half] * ks_now;
                    const int pr = pos[mt][half];
                    const int first = !LIST && p.a.window ? pr - p.a.window + 1 : 0;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int t = t0 + nt * 8 + 2 * c + e;
                            float z = s[mt][nt][half * 2 + e] * f;
                            z = t <= pr && t >= first ? z : -INFINITY;
                            s[mt][nt][half * 2 + e] = z;
                            over |= z > m[mt][half] || z + ev > M[mt][half];
                        }
                }
            if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float z = fmaxf(fmaxf(s[mt][0][half * 2], s[mt][0][half * 2 + 1]),
                                        fmaxf(s[mt][1][half * 2], s[mt][1][half * 2 + 1]));
                        z = fmaxf(z, __shfl_xor_sync(0xFFFFFFFFu, z, 1));
                        z = fmaxf(z, __shfl_xor_sync(0xFFFFFFFFu, z, 2));
                        const float m1 = fmaxf(m[mt][half], z), M1 = fmaxf(M[mt][half], z + ev);
                        l[mt][half] *= ex2(m[mt][half] - m1);
                        const float fo = ex2(M[mt][half] - M1);
                        m[mt][half] = m1;
                        M[mt][half] = M1;
#pragma unroll
                        for (int i2 = 0; i2 < kNt; ++i2) {
                            o[mt][i2][half * 2] *= fo;
                            o[mt][i2][half * 2 + 1] *= fo;
                        }
                    }
            }
            uint32_t pa[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const float z0 = s[mt][nt][half * 2], z1 = s[mt][nt][half * 2 + 1];
                        l[mt][half] += ex2(z0 - m[mt][half]) + ex2(z1 - m[mt][half]);
                        // fp16 keeps 11 bits of a weight: no fewer than the output's type keeps
                        const float d = ev - M[mt][half] + kHeadroom;
                        const __half2 h = __floats2half2_rn(ex2(z0 + d), ex2(z1 + d));
                        memcpy(&pa[mt][nt * 2 + half], &h, 4);
                    }

            // ---- O += P V: value rows 2c, 2c+1, 8+2c, 9+2c, this lane's D / 8 channels
            uint32_t vw[4][kNt / 4];
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) {
                const uint32_t row = 2 * c + (i2 & 1) + (i2 >> 1) * 8;
                if (D == 128) {
                    const uint4 w = *reinterpret_cast<const uint4*>(vt + tc::sw128_offset(row, r));
                    vw[i2][0] = w.x, vw[i2][1] = w.y, vw[i2][kNt / 4 - 2] = w.z, vw[i2][kNt / 4 - 1] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(vt + tc::sw64_offset(row, r >> 1) + (r & 1) * 8);
                    vw[i2][0] = w.x, vw[i2][1] = w.y;
                }
            }
#pragma unroll
            for (int i2 = 0; i2 < kNt / 4; ++i2) {
                const uint32_t a0 = vw[0][i2], a1 = vw[1][i2], b0 = vw[2][i2], b1 = vw[3][i2];
                const uint32_t f0 = e4m3_pair<0>(a0, a1), g0 = e4m3_pair<0>(b0, b1);
                const uint32_t f1 = e4m3_pair<1>(a0, a1), g1 = e4m3_pair<1>(b0, b1);
                const uint32_t f2 = e4m3_pair<2>(a0, a1), g2 = e4m3_pair<2>(b0, b1);
                const uint32_t f3 = e4m3_pair<3>(a0, a1), g3 = e4m3_pair<3>(b0, b1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma_16816(o[mt][i2 * 4 + 0], pa[mt], f0, g0);
                    mma_16816(o[mt][i2 * 4 + 1], pa[mt], f1, g1);
                    mma_16816(o[mt][i2 * 4 + 2], pa[mt], f2, g2);
                    mma_16816(o[mt][i2 * 4 + 3], pa[mt], f3, g3);
                }
            }
            __syncwarp();
        }

        // ---- the four warps' parts of this item become one
        float* stats = reinterpret_cast<float*>(smem + S::stats);
        float* buf = reinterpret_cast<float*>(smem + S::merge);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                l[mt][half] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][half], 1);
                l[mt][half] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][half], 2);
                if (c == 0) {
                    float* s3 = stats + (warp * 16 * MT + mt * 16 + half * 8 + r) * 3;
                    s3[0] = m[mt][half];
                    s3[1] = l[mt][half];
                    s3[2] = M[mt][half];
                }
            }
        __syncthreads();
        float mx[MT][2], lx[MT][2], Mx[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float* s3 = stats + (mt * 16 + half * 8 + r) * 3;
                float a = kNone, B = kNone, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    a = fmaxf(a, s3[w * 48 * MT]);
                    B = fmaxf(B, s3[w * 48 * MT + 2]);
                }
#pragma unroll
                for (int w = 0; w < kWarps; ++w) sum += s3[w * 48 * MT + 1] * ex2(s3[w * 48 * MT] - a);
                mx[mt][half] = a;
                lx[mt][half] = sum;
                Mx[mt][half] = B;
                const float f = ex2(M[mt][half] - B);
#pragma unroll
                for (int i2 = 0; i2 < kNt; ++i2) {
                    o[mt][i2][half * 2] *= f;
                    o[mt][i2][half * 2 + 1] *= f;
                }
            }
        // eight rows (r, half `half` of a row tile) a pass: warp w sums register e = w & 1 of half the n
        // tiles, that is kNt / 2 adjacent channels of lane column 2c + e
        const bool whole = from_start && to_end;
        float* part = p.a.part + ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * Part<D>::kFloats;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (mt * 16 + half * 8 >= rows) continue;
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i2 = 0; i2 < kNt; ++i2)
                        buf[((warp * 2 + e) * kNt + i2) * 32 + lane] = o[mt][i2][half * 2 + e];
                __syncthreads();
                const int row = mt * 16 + half * 8 + r, e = warp & 1, n0 = (warp >> 1) * (kNt / 2);
                const int ch = (2 * c + e) * kNt + n0;
                if (row >= rows || !alive) continue;
                float x[kNt / 2];
#pragma unroll
                for (int i2 = 0; i2 < kNt / 2; ++i2) {
                    x[i2] = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) x[i2] += buf[((w * 2 + e) * kNt + n0 + i2) * 32 + lane];
                }
                const float lr = lx[mt][half], mr = mx[mt][half], Mr = Mx[mt][half];
                if (whole) {
                    const int2 jg = work.token(cur, row);
                    const int64_t at = ((int64_t)cur.b * T + jg.x) * H + cur.h * G + jg.y;
                    const float f = lr == 0.0f ? 0.0f : ex2(Mr - mr) / lr;
                    store_out<kNt / 2>(p.a.out, p.a.q.is_bf16, at * D + ch, x, f);
                    if (p.a.lse && c == 0 && warp == 0)
                        p.a.lse[at] = lr == 0.0f ? -INFINITY : (mr + log2f(lr)) * 0.6931471805599453f;
                } else {
                    float4* dst = reinterpret_cast<float4*>(part + row * D + ch);
#pragma unroll
                    for (int i2 = 0; i2 < kNt / 2; i2 += 4)
                        dst[i2 / 4] = make_float4(x[i2], x[i2 + 1], x[i2 + 2], x[i2 + 3]);
                    if (c == 0 && warp == 0) {
                        float* s3 = part + Part<D>::kStats + row * 3;
                        s3[0] = mr;
                        s3[1] = lr;
                        s3[2] = Mr;
                    }
                }
            }
        if (from_start && !to_end && tid == 0) {  // the pieces up to the one with the item's last step
            const int64_t last_u = u + item_left - 1;
            const int64_t last = ((last_u + 1) * share + total - 1) / total - 1;
            desc[0] = cur.b;
            desc[1] = cur.h;
            desc[2] = cur.rt;
            desc[3] = rows;
            desc[4] = (int)(last - blockIdx.x) + 1;
        }
        u += todo;
        cur.step += todo - 1;
        if (++cur.step >= cur.steps) work.next_item(cur);
        __syncthreads();
    }
    // copies that were given up on still land in this CTA's memory
    if (!alive) {
        for (int i = 0; i < kStages; ++i)
            if ((issued >> i) & 1u) tc::mbar_wait(bars + i, (phase >> i) & 1u);
    }
}

// The items that the line's cuts went through: CTA x merges the item that
// starts in piece x and goes on behind it, four rows per blockIdx.y, the parts
// of a row in four shares, each in the order of the pieces.
template <int D, int MT, bool LIST>
__global__ void __launch_bounds__(4 * D) k_kv8_combine(const __grid_constant__ Params p) {
    constexpr int kLanes = D / 4, kShares = 4, kRows = 4;
    __shared__ float4 acc[kRows][kShares][kLanes];
    __shared__ float stat[kRows][kShares][3];
    pdl_begin();
    const int x = blockIdx.x, tid = threadIdx.x;
    const float* first = p.a.part + ((int64_t)x * 2 + 1) * Part<D>::kFloats;
    const int* desc = reinterpret_cast<const int*>(first + Part<D>::kDesc);
    const int parts = desc[4], rows = desc[3];
    if (parts < 2 || (int)blockIdx.y * kRows >= rows) return;
    const int ri = tid / (kShares * kLanes), sh = tid / kLanes % kShares, q4 = tid % kLanes;
    const int row = blockIdx.y * kRows + ri;
    auto part = [&](int i) { return i == 0 ? first : p.a.part + (int64_t)(x + i) * 2 * Part<D>::kFloats; };
    float m = kNone, M = kNone, l = 0.0f;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row < rows) {
        // every share finds the row's maxima over all parts itself: three words a part, from L2
        for (int i = q4; i < parts; i += kLanes) {
            const float* s3 = part(i) + Part<D>::kStats + row * 3;
            m = fmaxf(m, s3[0]);
            M = fmaxf(M, s3[2]);
        }
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    }
    if (row < rows) {
#pragma unroll 8
        for (int i = sh; i < parts; i += kShares) {
            const float* b = part(i);
            const float* s3 = b + Part<D>::kStats + row * 3;
            const float4 v = *reinterpret_cast<const float4*>(b + row * D + q4 * 4);
            l += s3[1] * ex2(s3[0] - m);
            const float f = ex2(s3[2] - M);
            s.x += v.x * f;
            s.y += v.y * f;
            s.z += v.z * f;
            s.w += v.w * f;
        }
    }
    acc[ri][sh][q4] = s;
    if (q4 == 0) stat[ri][sh][0] = l;
    __syncthreads();
    if (sh || row >= rows) return;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < kShares; ++i) {
        const float4 v = acc[ri][i][q4];
        l += stat[ri][i][0];
        y[0] += v.x;
        y[1] += v.y;
        y[2] += v.z;
        y[3] += v.w;
    }
    const Work<MT, LIST> work(p);
    Cursor k;
    k.rt = desc[2];
    const int2 jg = work.token(k, row);
    const int64_t at = ((int64_t)desc[0] * p.a.q.T + jg.x) * p.a.q.H + desc[1] * p.G + jg.y;
    store_out<4>(p.a.out, p.a.q.is_bf16, at * D + q4 * 4, y, l == 0.0f ? 0.0f : ex2(M - m) / l);
    if (p.a.lse && q4 == 0) p.a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, int MT, bool LIST>
cudaError_t launch(Params& p, cudaStream_t st) {
    using S = Smem<D, MT>;
    static_assert(S::bytes * (MT == 1 ? 3 : 2) <= 227 * 1024, "CTAs per SM");
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    p.ctas = sms * (MT == 1 ? 3 : 2);
    if (p.ctas > kMaxCtas) p.ctas = kMaxCtas;
    p.gt = (p.G + 16 * MT - 1) / (16 * MT);
    CUtensorMap kmap, vmap;
    if (!kv8_row_map(&kmap, p.c, p.c.k, kTile) || !kv8_row_map(&vmap, p.c, p.c.v, kTile)) return cudaErrorNotSupported;
    e = cudaFuncSetAttribute(k_kv8_attn<D, MT, LIST>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_kv8_attn<D, MT, LIST>, p.ctas, kThreads, S::bytes, st, p, kmap, vmap);
    if (e != cudaSuccess) return e;
    const int most = LIST ? (p.G < 16 * MT ? p.G : 16 * MT) : ((int64_t)p.a.q.T * p.G < 16 * MT ? p.a.q.T * p.G : 16 * MT);
    return launch_pdl(k_kv8_combine<D, MT, LIST>, dim3(p.ctas, (most + 3) / 4), 4 * D, 0, st, p);
}

}  // namespace

namespace {
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (EncodeTiled) nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}
}  // namespace

bool kv8_row_map(CUtensorMap_st* map, const DevKv8& c, void* codes, int box_rows) {
    EncodeTiled enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t gdim[2] = {(cuuint64_t)c.dim, ((cuuint64_t)c.n_blocks * c.heads) << c.bs_log2};
    const cuuint64_t gstride[1] = {(cuuint64_t)c.dim};
    const cuuint32_t box[2] = {(cuuint32_t)c.dim, (cuuint32_t)box_rows}, estride[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, gdim, gstride, box, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE, c.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int kv8_attn_parts() { return 2 * kMaxCtas; }
size_t kv8_part_floats(int dim) { return dim == 64 ? Part<64>::kFloats : Part<128>::kFloats; }

cudaError_t launch_kv8_attn(const DevKv8& c, const Kv8Attn& a, cudaStream_t st) {
    Params p;
    p.c = c;
    p.a = a;
    p.G = a.q.H / c.heads;
    p.wait_limit = wait_limit();
    if (a.block_idx) return c.dim == 64 ? launch<64, 1, true>(p, st) : launch<128, 1, true>(p, st);
    if ((int64_t)a.q.T * p.G <= 16) return c.dim == 64 ? launch<64, 1, false>(p, st) : launch<128, 1, false>(p, st);
    return c.dim == 64 ? launch<64, 2, false>(p, st) : launch<128, 2, false>(p, st);
}

}  // namespace csa2
