// Attention over the 8-bit cache for few query rows per sequence (decode and
// short verification), dense or over listed blocks.
//
// One query row needs two products with every cached row, so up to the 16
// rows a pass holds the kernel is bound by the codes' bytes (2 * D a position
// and head) and its work is moving them: the codes go by TMA into a ring of
// each warp's own (no synchronisation between warps while they stream; the
// rows swizzled, so that the loads below are free of bank conflicts), from
// there as 16-byte loads into the operand layout of mma.m16n8k16, converted to
// fp16 two at a time (exact).
//
// Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T: positions
// and channels fill the 16 rows of a tile and the query rows its 8 columns, so
// that the usual group of up to 8 query heads wastes nothing.  No operand is
// transposed in memory: the order of a product's k index may be permuted as
// long as both operands agree, so a lane's 16 bytes of a key row are four k
// steps, and of a value row the same channel of two positions is one byte
// permutation; the weights turn around in registers (movmatrix).
// tcgen05 would take the codes as they are (kind::f8f6f4) but wants the
// weights as E4M3 terms and 128 rows a tile; with at most 16 rows it has
// nothing to win over a kernel that already waits for HBM.
//
// Work split: a step is 128 positions of one (sequence, head, row tile); the
// steps of the whole batch form one line, which the CTAs cut into equal
// pieces (the lengths are on the device, so every warp sums them itself).  A
// CTA finishes what lies inside its piece; an item that is cut leaves
// partials (output, running maxima and sum), merged by k_kv8_combine in a
// fixed order, so results do not vary from run to run.  (Merges by the CTA
// that comes last, in the same launch, groups of eight pieces and then the
// groups, were slower: 17.0 against 12.4 us for 64 blocks of one sequence, 183
// against 175 us for a million positions; one CTA reads the parts where the
// second launch reads them with many.)
//
// A CTA is four computing warps and one that looks ahead: it walks the line,
// looks up list entries, pages and scales, and issues the copies into the four
// warps' rings (a lane a warp).  With that in the computing warps themselves the
// registers it needs made 16 query rows spill (281 against 158 us for 32
// sequences of up to 16,384 positions) and its instructions were a third of a tile's.
#include <cuda.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv8.cuh"
#include "kv8_tc.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 4, kThreads = (kWarps + 1) * 32;   // computing warps, and the one that looks ahead
constexpr int kGroup = 16;                // positions of one matrix tile
constexpr int kTile = 2 * kGroup;         // positions a warp takes at a time
constexpr int kStep = kWarps * kTile;     // positions a CTA takes at a time
constexpr float kNone = -3.0e38f;         // running maximum before any position
// Weights are 2^(z - M + 8) in fp16: the greatest is a power of two (exact, so
// that a row with one dominant position rounds only once), and weights down to
// 2^-22 of it keep fp16's full precision.  The 2^8 cancels the 2^-8 of the
// value codes' bit placement.
constexpr float kHeadroom = 8.0f;
// Two CTAs an SM with three stages a warp (192 KB in flight or in use): three CTAs
// with two stages take 117 against 112 us for 32 sequences of up to 16,384 tokens.
constexpr int kPerSm = 2;
constexpr int kMaxCtas = kPerSm * 148;
constexpr int kMergeWarps = 16;           // of a CTA of k_kv8_combine_few
constexpr int kFewItems = 16, kFewSteps = 16;   // it merges where an item can have as many pieces, and as many steps

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

// a / b for a >= 0, b > 0: in 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

template <int NT, bool LIST>
struct Work {
    const Params& p;
    __device__ explicit Work(const Params& p) : p(p) {}

    // Rows of item k, and the (token, head of the group) of its row i.
    __device__ __forceinline__ int rows(const Cursor& k) const {
        const int left = LIST ? p.G - k.rt % p.gt * 8 * NT : k.n * p.G - k.rt * 8 * NT;
        return left < 8 * NT ? left : 8 * NT;
    }
    __device__ __forceinline__ int2 token(const Cursor& k, int i) const {
        if (LIST) {
            const int j = k.rt / p.gt;
            return make_int2(j, (k.rt - j * p.gt) * 8 * NT + i);
        }
        const int j = (k.rt * 8 * NT + i) / p.G;
        return make_int2(j, k.rt * 8 * NT + i - j * p.G);
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
            k.tiles = (k.n * p.G + 8 * NT - 1) / (8 * NT);
        }
        if (k.steps < 1) k.steps = 1;  // an empty row still has to be written
    }
    __device__ __forceinline__ int64_t total(const Cursor& k) const {
        return (int64_t)p.c.heads * k.tiles * k.steps;
    }
    __device__ __forceinline__ void seek(Cursor& k, int64_t u) const {  // step u of the sequence
        const int64_t item = quotient(u, k.steps);
        k.step = (int)(u - item * k.steps);
        k.h = (int)quotient(item, k.tiles);
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

// The line of all steps, by one warp (every warp on its own, no barrier): lane
// x holds `per` sequences from x * per on, and the steps before them.
template <int NT, bool LIST>
struct LineOf {
    int64_t before, total;
    int per;
    Cursor mine;    // of this lane's sequence when per == 1

    __device__ __forceinline__ LineOf(const Work<NT, LIST>& w, uint32_t* status) {
        const int lane = threadIdx.x & 31, nb = w.p.c.batch;
        per = (nb + 31) >> 5;
        int64_t s = 0;
        for (int i = 0; i < per; ++i) {
            w.load(mine, lane * per + i, status);
            s += w.total(mine);
        }
        int64_t inc = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        before = inc - s;
        total = __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    // The step u (0 <= u < total) as a cursor.
    __device__ __forceinline__ void find(const Work<NT, LIST>& w, int64_t u, Cursor& k) const {
        const int at = 31 - __clz(__ballot_sync(0xFFFFFFFFu, before <= u));
        u -= __shfl_sync(0xFFFFFFFFu, before, at);
        if (per == 1) {
            k.b = at;
            k.steps = __shfl_sync(0xFFFFFFFFu, mine.steps, at);
            k.tiles = __shfl_sync(0xFFFFFFFFu, mine.tiles, at);
            k.L = __shfl_sync(0xFFFFFFFFu, mine.L, at);
            k.n = __shfl_sync(0xFFFFFFFFu, mine.n, at);
            k.lo = __shfl_sync(0xFFFFFFFFu, mine.lo, at);
        } else {
            for (int b = at * per;; ++b) {
                w.load(k, b, nullptr);
                const int64_t t = w.total(k);
                if (u < t || b + 1 >= w.p.c.batch) break;
                u -= t;
            }
        }
        w.seek(k, u);
    }
};

// The line in `share` pieces: the first `more` of them one step longer than `size`.
struct Pieces {
    int64_t size, more;
    int share;
    __device__ __forceinline__ Pieces(int64_t total, int ctas) {
        share = total < ctas ? (total < 1 ? 1 : (int)total) : ctas;
        size = quotient(total, share);
        more = total - size * share;
    }
    __device__ __forceinline__ int64_t start(int x) const { return size * x + (x < more ? x : more); }
    __device__ __forceinline__ int holding(int64_t u) const {   // the piece with step u
        const int64_t longer = more * (size + 1);
        return (int)(u < longer ? quotient(u, size + 1) : more + quotient(u - longer, size));
    }
};

// What a computing warp is told of a tile: the first position of both groups of
// 16 (-1: nothing there) and their scales; and of an item.
struct Tile {
    int t0, t1;
    float ks0, ks1, vs0, vs1;
};
struct Item {
    Cursor k;
    int todo, flags;        // steps of the piece; 1: from the item's first step, 2: to its last
    int parts;              // pieces the item lies in, from this one on
};

template <int D, int NT>
struct Smem {
    static constexpr int kRows = kTile * D;          // bytes of one tile's keys (or values)
    static constexpr int kStages = 3 * (128 / D);
    static constexpr int kItems = 4;                 // items looked ahead
    static constexpr int ring = 0;                                            // [warp][stage][K, V]
    static constexpr int merge = ring + kWarps * kStages * 2 * kRows;         // [warp][16][32] floats
    static constexpr int stats = merge + kWarps * 16 * 32 * 4;                // [warp][8 * NT][3] floats
    static constexpr int tiles = stats + kWarps * 8 * NT * 3 * 4;             // [warp][stage]
    static constexpr int items = tiles + kWarps * kStages * 32;               // [kItems]
    static constexpr int bars = items + kItems * 64;                          // full, empty [warp][stage]; items full, empty
    static constexpr int bytes = bars + (2 * kWarps * kStages + 2 * kItems) * 8 + 1024;   // base aligned to 1024
};

// Partial of a cut item: [16 rows][D] outputs, per row (m, l, M), then what
// k_kv8_combine needs of the item: b, h, rt, rows, and how many pieces it has.
template <int D>
struct Part {
    static constexpr int kStats = 16 * D, kDesc = kStats + 16 * 3, kFloats = kDesc + 16;
};

// Four adjacent outputs x * 2^(M - m - 8) / l, rounded once to the query's type.
// M - m is as low as the least value scale, -120, and 2^-128 / l nothing in fp32:
// there the power of two goes in two parts.
__device__ __forceinline__ void store_out(void* out, int is_bf16, int64_t at, float* x, float m, float l, float M) {
    constexpr float kLow = -100.0f;
    const float e = M - m - kHeadroom, f = l == 0.0f ? 0.0f : ex2(fmaxf(e, kLow)) / l;
    if (e < kLow) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= ex2(e - kLow);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (is_bf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i] * f, x[2 * i + 1] * f);
            memcpy(&w[i], &h, 4);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i] * f, x[2 * i + 1] * f);
            memcpy(&w[i], &h, 4);
        }
    }
    uint16_t* dst = static_cast<uint16_t*>(out) + at;
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// NT: tiles of eight query rows.
template <int D, int NT, bool LIST>
__global__ void __launch_bounds__(kThreads, kPerSm) k_kv8_attn(const __grid_constant__ Params p,
                                                               const __grid_constant__ CUtensorMap kmap,
                                                               const __grid_constant__ CUtensorMap vmap) {
    using S = Smem<D, NT>;
    constexpr int kChunks = D / 64;   // 16-byte chunks of a key row per lane
    constexpr int kCh = D / 8;        // channels of a value row per lane
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::bars);          // full [warp][stage]
    uint64_t* empty = bars + kWarps * kStages;                             // [warp][stage]
    uint64_t* item_full = empty + kWarps * kStages;                        // [kItems]
    uint64_t* item_empty = item_full + S::kItems;
    Item* items = reinterpret_cast<Item*>(smem + S::items);
    const int bs = p.c.bs(), G = p.G, T = p.a.q.T, H = p.a.q.H;
    if (tid == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) {
            tc::mbar_init(bars + i, 1);
            tc::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < S::kItems; ++i) {
            tc::mbar_init(item_full + i, 1);
            tc::mbar_init(item_empty + i, kWarps);
        }
        tc::fence_mbar_init();
    }
    pdl_begin();
    __syncthreads();
    const Work<NT, LIST> work(p);
    int* desc = reinterpret_cast<int*>(p.a.part + ((int64_t)blockIdx.x * 2 + 1) * Part<D>::kFloats + Part<D>::kDesc);

    if (warp == kWarps) {
        // ------------------------------------------------------------ the warp that looks ahead
        if (lane == 0) desc[4] = 0;
        const LineOf<NT, LIST> line(work, blockIdx.x == 0 ? p.a.status : nullptr);
        const Pieces pieces(line.total, p.ctas);
        const bool any = line.total > 0 && blockIdx.x < pieces.share;
        const int64_t u0 = any ? pieces.start(blockIdx.x) : 0, u1 = any ? pieces.start(blockIdx.x + 1) : 0;
        int steps = (int)(u1 - u0);
        Cursor cur;
        if (any) line.find(work, u0, cur);
        const bool pairs = bs == kGroup;      // a tile is two blocks
        const int w = lane & (kWarps - 1);    // this lane's warp (lanes 0 .. 3 act)
        bool alive = true;
        uint32_t copies = 0;                  // slots with a copy in flight that nobody waits for (bit mask)

        // A step goes through four stages, each a load that the next one needs: list entries, pages,
        // scales, and the copy; the steps behind it are one stage further back.
        struct Look {
            int b, h, row, lb[2], phys[2];
            float ks[2], vs[2];
        };
        int64_t ahead_u = u0;
        int item_no = 0;
        Cursor at = cur;
        int todo_left = steps, in_item = 0;   // steps of the piece not yet looked at; of the item at `at`
        auto entries = [&](Look& k) {         // stage 1, and the items as they come up
            k.lb[0] = k.lb[1] = -1;
            k.b = at.b;
            k.h = at.h;
            k.row = 0;
            if (todo_left == 0) return;
            if (in_item == 0) {
                const int left = at.steps - at.step, todo = todo_left < left ? todo_left : left, i = item_no % S::kItems;
                if (item_no >= S::kItems && alive) {
                    alive = tc::mbar_wait(item_empty + i, ((item_no / S::kItems) - 1) & 1, p.wait_limit);
                    if (!alive && lane == 0) flag(p.a.status, kStatusTimeout);
                    alive = __all_sync(0xFFFFFFFFu, alive);
                }
                if (lane == 0) {
                    items[i].k = at;
                    items[i].todo = todo;
                    items[i].flags = (at.step == 0 ? 1 : 0) | (todo == left ? 2 : 0);
                    items[i].parts = pieces.holding(ahead_u + left - 1) - (int)blockIdx.x + 1;
                    tc::mbar_arrive(item_full + i);
                }
                __syncwarp();
                ++item_no;
                in_item = todo;
            }
            const int off = at.step * kStep + w * kTile;
            if (LIST) {
                const int j = at.rt / p.gt, pos = at.L - at.n + j;
                const int32_t* l = p.a.block_idx + (((int64_t)at.b * T + j) * p.c.heads + at.h) * p.a.n_sel;
                k.row = off & (bs - 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int e = (off >> p.c.bs_log2) + i;
                    if ((i && !pairs) || e >= p.a.n_sel) break;
                    const int v = __ldg(l + e), prev = e ? __ldg(l + e - 1) : -1;
                    if (v >= 0) {
                        // strictly ascending, visible, nothing behind padding: anything else is skipped and flagged
                        if (pos < 0 || v > (pos >> p.c.bs_log2) || (e && v <= prev) || (e && prev < 0)) {
                            if (lane < kWarps) flag(p.a.status, kStatusBounds);
                        } else {
                            k.lb[i] = v;
                        }
                    } else if (v < -1 && lane < kWarps) {
                        flag(p.a.status, kStatusBounds);
                    }
                }
            } else {
                const int t = at.lo + off;
                k.row = t & (bs - 1);
                const int lb = t >> p.c.bs_log2;
                // a block of 16 before every row's window is not looked up: its page may be gone
                if (t < at.L && !(pairs && p.a.window && t + kGroup <= at.L - at.n - p.a.window + 1)) k.lb[0] = lb;
                if (pairs && t + kGroup < at.L) k.lb[1] = lb + 1;
            }
            ++ahead_u;
            --todo_left;
            --in_item;
            if (++at.step >= at.steps) work.next_item(at);
        };
        auto pages = [&](Look& k) {           // stage 2
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                k.phys[i] = k.lb[i] >= 0 ? kv8_block(p.c, k.b, k.lb[i]) : -1;
                if (k.lb[i] >= 0 && k.phys[i] < 0 && lane < kWarps) flag(p.a.status, kStatusBounds);
            }
        };
        auto scales = [&](Look& k) {          // stage 3
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                k.ks[i] = k.vs[i] = 1.0f;
                if (k.phys[i] >= 0) {
                    const int64_t unit = (int64_t)k.phys[i] * p.c.heads + k.h;
                    k.ks[i] = __ldg(p.c.k_scale + unit);
                    k.vs[i] = __ldg(p.c.v_scale + unit);
                    kv8_check_scale(k.ks[i], p.a.status);
                    kv8_check_scale(k.vs[i], p.a.status);
                }
            }
        };
        Look k1, k2, k3;
        entries(k1);
        k2 = k1;
        pages(k2);
        entries(k1);
        k3 = k2;
        scales(k3);
        k2 = k1;
        pages(k2);
        entries(k1);
        int slot = 0, round = 0;
#pragma unroll 1
        for (int s = 0; s < steps; ++s) {
            if (round > 0 && alive && lane < kWarps) {   // the warp has read the slot's last tile
                alive = tc::mbar_wait(empty + w * kStages + slot, (round - 1) & 1, p.wait_limit);
                if (!alive) flag(p.a.status, kStatusTimeout);
            }
            alive = __all_sync(0xFFFFFFFFu, alive);
            if (!alive) break;
            if (lane < kWarps) {
                uint8_t* kd = smem + S::ring + (w * kStages + slot) * 2 * S::kRows;
                uint64_t* bar = bars + w * kStages + slot;
                const int n = pairs ? (k3.phys[0] >= 0) + (k3.phys[1] >= 0) : k3.phys[0] >= 0 ? 2 : 0;   // groups that arrive
                tc::mbar_expect_tx(bar, n * S::kRows);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (k3.phys[i] < 0) continue;
                    const int row = ((k3.phys[i] * p.c.heads + k3.h) << p.c.bs_log2) + k3.row;
                    tc::tma_load_2d(kd + i * kGroup * D, &kmap, 0, row, bar);
                    tc::tma_load_2d(kd + S::kRows + i * kGroup * D, &vmap, 0, row, bar);
                }
                Tile d = {-1, -1, k3.ks[0], k3.ks[1], k3.vs[0], k3.vs[1]};
                if (k3.phys[0] >= 0) d.t0 = (k3.lb[0] << p.c.bs_log2) + k3.row;
                if (pairs) {
                    if (k3.phys[1] >= 0) d.t1 = k3.lb[1] << p.c.bs_log2;
                } else {
                    if (n) d.t1 = d.t0 + kGroup;
                    d.ks1 = d.ks0;
                    d.vs1 = d.vs0;
                }
                reinterpret_cast<Tile*>(smem + S::tiles + (w * kStages + slot) * 32)[0] = d;
                tc::mbar_arrive(bar);
                copies |= 1u << slot;
            }
            if (++slot == kStages) slot = 0, ++round;
            k3 = k2;
            scales(k3);
            k2 = k1;
            pages(k2);
            entries(k1);
        }
        // the end of the line: an item without steps
        if (alive) {
            const int i = item_no % S::kItems;
            if (item_no >= S::kItems) alive = __all_sync(0xFFFFFFFFu, tc::mbar_wait(item_empty + i, ((item_no / S::kItems) - 1) & 1, p.wait_limit));
            if (lane == 0 && alive) {
                items[i].todo = 0;
                tc::mbar_arrive(item_full + i);
            }
        }
        // what was copied last still lands in this CTA's memory
        if (lane < kWarps) {
            for (int i = 0; i < kStages; ++i) {
                const int last_round = i < slot ? round : round - 1;   // of the slot's last copy
                if ((copies >> i) & 1u) tc::mbar_wait(bars + w * kStages + i, last_round & 1);
            }
        }
        return;
    }

    // ---------------------------------------------------------------- a computing warp
    const int r = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + S::ring + warp * kStages * 2 * S::kRows;
    bars += warp * kStages;
    empty += warp * kStages;
    // The computing warps meet; they all leave together once a wait of one of them ran out.
    auto meet = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    bool alive = true;       // false once a wait ran out: no further results
    int slot = 0;
    uint32_t phase = 0;      // parity of each slot's barrier (bit mask)
    for (int item_no = 0;; ++item_no) {
        Item* item = items + item_no % S::kItems;
        {
            bool ok = tc::mbar_wait(item_full + item_no % S::kItems, (item_no / S::kItems) & 1, p.wait_limit) && alive;
            if (!ok) flag(p.a.status, kStatusTimeout);
            int go;
            asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %1, 0;\n\t"
                         "barrier.cta.red.and.pred b, 1, 128, a;\n\tselp.b32 %0, 1, 0, b;\n\t}"
                         : "=r"(go) : "r"((int)ok) : "memory");
            if (!go) return;
        }
        const Cursor cur = item->k;
        const int todo = item->todo;
        if (todo == 0) return;
        const int rows = work.rows(cur);

        // ---- query row r of every tile of eight, in operand layout
        uint32_t qb[NT][kChunks * 4][2];
        float zs[NT][2];     // rows 2c, 2c + 1: factor from the product to a base-2 logit, without the key scale
        int pos[NT][2];      // and the position of their token (-1: no row)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = nt * 8 + r;
            const bool ok = row < rows;
            const int2 jg = work.token(cur, row);
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
            const float z = back * p.a.sm_scale * 1.4426950408889634f;
            const int pr = ok ? cur.L - cur.n + jg.x : -1;
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // row 2c + e is held by the lanes with r = 2c + e
                zs[nt][e] = __shfl_sync(0xFFFFFFFFu, z, (2 * c + e) * 4);
                pos[nt][e] = __shfl_sync(0xFFFFFFFFu, pr, (2 * c + e) * 4);
            }
#pragma unroll
            for (int k = 0; k < kChunks; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    qb[nt][k * 4 + s][0] = raw[k][2 * s];
                    qb[nt][k * 4 + s][1] = raw[k][2 * s + 1];
                }
        }
        // a tile inside [see0, see1] is visible to every row of the item
        const int see1 = cur.L - cur.n + work.token(cur, 0).x;
        const int see0 = !LIST && p.a.window ? cur.L - cur.n + work.token(cur, rows - 1).x - p.a.window + 1 : 0;

        float o[NT][kCh / 2][4];
        float m[NT][2], l[NT][2], M[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < kCh / 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) m[nt][e] = M[nt][e] = kNone, l[nt][e] = 0.0f;
        }

#pragma unroll 1
        for (int i = 0; i < todo; ++i) {
            if (alive) {
                alive = tc::mbar_wait(bars + slot, (phase >> slot) & 1u, p.wait_limit);
                if (!alive && lane == 0) flag(p.a.status, kStatusTimeout);
            }
            alive = __all_sync(0xFFFFFFFFu, alive);
            if (!alive) break;
            phase ^= 1u << slot;
            const Tile tile = *reinterpret_cast<const Tile*>(smem + S::tiles + (warp * kStages + slot) * 32);
            uint8_t* kt = ring + slot * 2 * S::kRows;
            uint8_t* vt = kt + S::kRows;
            uint64_t* done = empty + slot;
            slot = slot + 1 == kStages ? 0 : slot + 1;
            if (tile.t0 < 0 && tile.t1 < 0) {
                if (lane == 0) tc::mbar_arrive(done);
                continue;
            }
            const float ks_now[2] = {tile.ks0, tile.ks1}, vs_now[2] = {tile.vs0, tile.vs1};
            const bool inside = tile.t0 >= 0 && tile.t1 >= 0 && tile.t0 >= see0 && tile.t1 + kGroup - 1 <= see1;
            if (!inside) {
                // what lies behind the sequence's end, or was not copied, may be any code: NaN times a
                // weight of 0 is NaN, so those value rows are cleared
                bool cleared = false;
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    for (int x = lane; x < kGroup * (D / 16); x += 32) {
                        const int row = x / (D / 16);
                        if ((g ? tile.t1 : tile.t0) < 0 || (g ? tile.t1 : tile.t0) + row >= cur.L) {
                            *reinterpret_cast<uint4*>(vt + g * kGroup * D + x * 16) = make_uint4(0, 0, 0, 0);
                            cleared = true;
                        }
                    }
                if (cleared) tc::fence_proxy_async_smem();   // before a later copy into this slot
                __syncwarp();
            }

            // ---- S^T = K Q^T: group g, positions r and r + 8 of it, query rows 2c and 2c + 1 of every tile
            float s[2][NT][4];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[g][nt][e] = 0.0f;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                uint32_t w[2][2][4];
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t row = g * kGroup + half * 8 + r, chunk = c * kChunks + k;
                        const uint4 x = *reinterpret_cast<const uint4*>(
                            kt + (D == 128 ? tc::sw128_offset(row, chunk) : tc::sw64_offset(row, chunk)));
                        w[g][half][0] = x.x, w[g][half][1] = x.y, w[g][half][2] = x.z, w[g][half][3] = x.w;
                    }
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint32_t a[4] = {half2_lo(w[g][0][q4]), half2_lo(w[g][1][q4]), half2_hi(w[g][0][q4]),
                                               half2_hi(w[g][1][q4])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816(s[g][nt], a, qb[nt][k * 4 + q4][0], qb[nt][k * 4 + q4][1]);
                    }
            }

            // ---- base-2 logits; a vote tells whether a running maximum moves at all.  m: maximum of the
            // logits (for l), M: of logit + log2(value scale) (for the output)
            float ev[2];
            bool over = false;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                ev[g] = (float)((int)(__float_as_uint(vs_now[g]) >> 23) - 127);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = zs[nt][e] * ks_now[g];
                        s[g][nt][e] *= f;
                        s[g][nt][2 + e] *= f;
                    }
            }
            if (!inside) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const bool there = (g ? tile.t1 : tile.t0) >= 0;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = (g ? tile.t1 : tile.t0) + r + (e >> 1) * 8, pr = pos[nt][e & 1];
                            const bool in = there && t <= pr && (LIST || !p.a.window || t > pr - p.a.window);
                            s[g][nt][e] = in ? s[g][nt][e] : -INFINITY;
                        }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float z0 = fmaxf(s[0][nt][e], s[0][nt][2 + e]), z1 = fmaxf(s[1][nt][e], s[1][nt][2 + e]);
                    over |= fmaxf(z0, z1) > m[nt][e] || fmaxf(z0 + ev[0], z1 + ev[1]) > M[nt][e];
                }
            if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float z0 = fmaxf(s[0][nt][e], s[0][nt][2 + e]), z1 = fmaxf(s[1][nt][e], s[1][nt][2 + e]);
                        float z = fmaxf(z0, z1), Z = fmaxf(z0 + ev[0], z1 + ev[1]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) {
                            z = fmaxf(z, __shfl_xor_sync(0xFFFFFFFFu, z, x));
                            Z = fmaxf(Z, __shfl_xor_sync(0xFFFFFFFFu, Z, x));
                        }
                        z = fmaxf(m[nt][e], z);
                        Z = fmaxf(M[nt][e], Z);
                        l[nt][e] *= ex2(m[nt][e] - z);
                        const float f = ex2(M[nt][e] - Z);
                        m[nt][e] = z;
                        M[nt][e] = Z;
#pragma unroll
                        for (int i2 = 0; i2 < kCh / 2; ++i2) {
                            o[nt][i2][e] *= f;
                            o[nt][i2][2 + e] *= f;
                        }
                    }
            }
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float d0 = ev[g] - M[nt][0] + kHeadroom, d1 = ev[g] - M[nt][1] + kHeadroom;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float z0 = s[g][nt][half * 2], z1 = s[g][nt][half * 2 + 1];
                        l[nt][0] += ex2(z0 - m[nt][0]);
                        l[nt][1] += ex2(z1 - m[nt][1]);
                        // fp16 keeps 11 bits of a weight: no fewer than the output's type keeps
                        const __half2 h = __floats2half2_rn(ex2(z0 + d0), ex2(z1 + d1));
                        uint32_t x;
                        memcpy(&x, &h, 4);
                        pb[g][nt][half] = transpose8x8(x);
                    }
                }

            // ---- O^T += V^T P^T: positions 2c, 2c+1, 8+2c, 9+2c of a group, this lane's D / 8 channels
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t w[4][kCh / 4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t row = g * kGroup + 2 * c + (x & 1) + (x >> 1) * 8;
                    if (D == 128) {
                        const uint4 y = *reinterpret_cast<const uint4*>(vt + tc::sw128_offset(row, r));
                        w[x][0] = y.x, w[x][1] = y.y, w[x][kCh / 4 - 2] = y.z, w[x][kCh / 4 - 1] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2*>(vt + tc::sw64_offset(row, r >> 1) + (r & 1) * 8);
                        w[x][0] = y.x, w[x][1] = y.y;
                    }
                }
#pragma unroll
                for (int i2 = 0; i2 < kCh / 4; ++i2) {
                    // one channel of two positions side by side
                    const uint32_t x01 = __byte_perm(w[0][i2], w[1][i2], 0x5140), x23 = __byte_perm(w[0][i2], w[1][i2], 0x7362);
                    const uint32_t y01 = __byte_perm(w[2][i2], w[3][i2], 0x5140), y23 = __byte_perm(w[2][i2], w[3][i2], 0x7362);
                    const uint32_t a01[4] = {half2_lo(x01), half2_hi(x01), half2_lo(y01), half2_hi(y01)};
                    const uint32_t a23[4] = {half2_lo(x23), half2_hi(x23), half2_lo(y23), half2_hi(y23)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_16816(o[nt][i2 * 2], a01, pb[g][nt][0], pb[g][nt][1]);
                        mma_16816(o[nt][i2 * 2 + 1], a23, pb[g][nt][0], pb[g][nt][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(done);
        }

        // ---- the four warps' parts of this item become one
        float* stats = reinterpret_cast<float*>(smem + S::stats);
        float* buf = reinterpret_cast<float*>(smem + S::merge);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], x);
                if (r == 0) {
                    float* s3 = stats + (warp * 8 * NT + nt * 8 + 2 * c + e) * 3;
                    s3[0] = m[nt][e];
                    s3[1] = l[nt][e];
                    s3[2] = M[nt][e];
                }
            }
        meet();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float* s3 = stats + (nt * 8 + 2 * c + e) * 3;
                float a = kNone, B = kNone, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    a = fmaxf(a, s3[w * 24 * NT]);
                    B = fmaxf(B, s3[w * 24 * NT + 2]);
                }
#pragma unroll
                for (int w = 0; w < kWarps; ++w) sum += s3[w * 24 * NT + 1] * ex2(s3[w * 24 * NT] - a);
                const float f = ex2(M[nt][e] - B);
                m[nt][e] = a;
                l[nt][e] = sum;
                M[nt][e] = B;
#pragma unroll
                for (int i2 = 0; i2 < kCh / 2; ++i2) {
                    o[nt][i2][e] *= f;
                    o[nt][i2][2 + e] *= f;
                }
            }
        // a pass: eight rows, eight of each lane's channels; warp w sums four of them for row 2c + (w & 1)
        const bool from_start = (item->flags & 1) != 0, to_end = (item->flags & 2) != 0, whole = from_start && to_end;
        float* part = p.a.part + ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * Part<D>::kFloats;
        const int e = warp & 1, hh = warp >> 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt * 8 >= rows) continue;
#pragma unroll
            for (int ps = 0; ps < kCh / 8; ++ps) {
#pragma unroll
                for (int x = 0; x < 16; ++x) buf[(warp * 16 + x) * 32 + lane] = o[nt][ps * 4 + x / 4][x & 3];
                meet();
                const int row = nt * 8 + 2 * c + e;
                if (row < rows && alive) {
                    float y[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int reg = (hh * 2 + x / 2) * 4 + (x & 1) * 2 + e;
                        y[x] = 0.0f;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) y[x] += buf[(w * 16 + reg) * 32 + lane];
                    }
                    const int ch = r * kCh + ps * 8 + hh * 4;
                    const float lr = e ? l[nt][1] : l[nt][0], mr = e ? m[nt][1] : m[nt][0],
                                Mr = e ? M[nt][1] : M[nt][0];
                    const bool first = ps == 0 && r == 0 && hh == 0;
                    if (whole) {
                        const int2 jg = work.token(cur, row);
                        const int64_t at = ((int64_t)cur.b * T + jg.x) * H + cur.h * G + jg.y;
                        store_out(p.a.out, p.a.q.is_bf16, at * D + ch, y, mr, lr, Mr);
                        if (p.a.lse && first) p.a.lse[at] = lr == 0.0f ? -INFINITY : (mr + log2f(lr)) * 0.6931471805599453f;
                    } else {
                        *reinterpret_cast<float4*>(part + row * D + ch) = make_float4(y[0], y[1], y[2], y[3]);
                        if (first) {
                            float* s3 = part + Part<D>::kStats + row * 3;
                            s3[0] = mr;
                            s3[1] = lr;
                            s3[2] = Mr;
                        }
                    }
                }
                meet();
            }
        }
        if (from_start && !to_end && tid == 0) {  // the pieces up to the one with the item's last step
            desc[0] = cur.b;
            desc[1] = cur.h;
            desc[2] = cur.rt;
            desc[3] = rows;
            desc[4] = item->parts;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(item_empty + item_no % S::kItems);
    }
}

// The items that the line's cuts went through: CTA x merges the item that
// starts in piece x and goes on behind it, four rows per blockIdx.y, the parts
// of a row in four shares, each in the order of the pieces.
template <int D, int NT, bool LIST>
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
    const Work<NT, LIST> work(p);
    Cursor k;
    k.rt = desc[2];
    const int2 jg = work.token(k, row);
    const int64_t at = ((int64_t)desc[0] * p.a.q.T + jg.x) * p.a.q.H + desc[1] * p.G + jg.y;
    store_out(p.a.out, p.a.q.is_bf16, at * D + q4 * 4, y, m, l, M);
    if (p.a.lse && q4 == 0) p.a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// The same for few items, each in many pieces: blockIdx.x counts the items that
// were cut, a CTA merges one row, warp w the parts w, w + 16, .. in this order, the
// first warp the sixteen.  With k_kv8_combine two heads of 24,415 positions, 148
// parts each, take 27.7 us, with this 14.5; 8 heads of a million positions 173.1
// and 168.9; two heads of 64 blocks (32 parts) 11.3 and 9.9; but four heads of
// 1,000 positions (8 parts) 8.4 and 9.1.
template <int D, int NT, bool LIST>
__global__ void __launch_bounds__(kMergeWarps * 32) k_kv8_combine_few(const __grid_constant__ Params p) {
    constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;     // lanes of a part's row, parts a warp reads at once
    static_assert(kMaxCtas <= kMergeWarps * 32, "a thread a piece, a lane a part");
    __shared__ float4 acc[kMergeWarps][kLanes];
    __shared__ float stat[kMergeWarps][3];
    __shared__ int starts[kMergeWarps], found[6];
    pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int parts = 0;                                           // a thread a piece
    int4 item = make_int4(0, 0, 0, 0);                       // b, h, rt, rows
    if (tid < p.ctas) {
        const float* d = p.a.part + ((int64_t)tid * 2 + 1) * Part<D>::kFloats + Part<D>::kDesc;
        item = *reinterpret_cast<const int4*>(d);
        parts = reinterpret_cast<const int*>(d)[4];
    }
    const uint32_t cut = __ballot_sync(0xFFFFFFFFu, parts >= 2);
    if (lane == 0) starts[warp] = __popc(cut);
    if (tid == 0) found[0] = -1;
    __syncthreads();
    const int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? starts[lane] : 0) + __popc(cut & ((1u << lane) - 1));
    if (parts >= 2 && before == (int)blockIdx.x) {
        found[0] = tid, found[1] = parts;
        found[2] = item.x, found[3] = item.y, found[4] = item.z, found[5] = item.w;
    }
    __syncthreads();
    const int x = found[0], row = blockIdx.y;
    if (x < 0 || row >= found[5]) return;
    parts = found[1];
    const int q4 = lane % kLanes;
    auto part = [&](int i) { return p.a.part + ((int64_t)(x + i) * 2 + (i == 0 ? 1 : 0)) * Part<D>::kFloats; };
    const int n = warp < parts ? (parts - warp - 1) / kMergeWarps + 1 : 0;    // this warp's, a lane each
    float pl = 0.0f, pm = kNone, pM = kNone;
    if (lane < n) {
        const float* s3 = part(warp + lane * kMergeWarps) + Part<D>::kStats + row * 3;
        pm = s3[0], pl = s3[1], pM = s3[2];
    }
    float m = pm, M = pM;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    }
    float l = pl * ex2(pm - m);
    const float f = ex2(pM - M);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int k = 0; k < n; k += kAtOnce) {
        const int at = k + lane / kLanes;
        const float w = __shfl_sync(0xFFFFFFFFu, f, at & 31);
        if (at < n) {
            const float4 v = *reinterpret_cast<const float4*>(part(warp + at * kMergeWarps) + row * D + q4 * 4);
            s.x += v.x * w;
            s.y += v.y * w;
            s.z += v.z * w;
            s.w += v.w * w;
        }
    }
    if (kAtOnce == 2) {
        s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, 16);
        s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, 16);
        s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, 16);
        s.w += __shfl_xor_sync(0xFFFFFFFFu, s.w, 16);
    }
    if (lane < kLanes) acc[warp][q4] = s;
    if (lane == 0) stat[warp][0] = m, stat[warp][1] = l, stat[warp][2] = M;
    __syncthreads();
    if (warp || lane >= kLanes) return;
    for (int i = 1; i < kMergeWarps; ++i) {
        m = fmaxf(m, stat[i][0]);
        M = fmaxf(M, stat[i][2]);
    }
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    l = 0.0f;
    for (int i = 0; i < kMergeWarps; ++i) {
        const float4 v = acc[i][q4];
        const float f = ex2(stat[i][2] - M);
        l += stat[i][1] * ex2(stat[i][0] - m);
        y[0] += v.x * f;
        y[1] += v.y * f;
        y[2] += v.z * f;
        y[3] += v.w * f;
    }
    const Work<NT, LIST> work(p);
    Cursor k;
    k.rt = found[4];
    const int2 jg = work.token(k, row);
    const int64_t at = ((int64_t)found[2] * p.a.q.T + jg.x) * p.a.q.H + found[3] * p.G + jg.y;
    store_out(p.a.out, p.a.q.is_bf16, at * D + q4 * 4, y, m, l, M);
    if (p.a.lse && q4 == 0) p.a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, int NT, bool LIST>
cudaError_t launch(Params& p, cudaStream_t st) {
    using S = Smem<D, NT>;
    static_assert(S::bytes * kPerSm + kPerSm * 1024 <= 228 * 1024, "CTAs per SM");
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    p.ctas = sms * kPerSm < kMaxCtas ? sms * kPerSm : kMaxCtas;
    p.gt = (p.G + 8 * NT - 1) / (8 * NT);
    CUtensorMap kmap, vmap;
    const int box = p.c.bs() < kTile ? p.c.bs() : kTile;
    if (!kv8_row_map(&kmap, p.c, p.c.k, box, true) || !kv8_row_map(&vmap, p.c, p.c.v, box, true)) return cudaErrorNotSupported;
    e = cudaFuncSetAttribute(k_kv8_attn<D, NT, LIST>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_kv8_attn<D, NT, LIST>, p.ctas, kThreads, S::bytes, st, p, kmap, vmap);
    if (e != cudaSuccess) return e;
    const int64_t rows = LIST ? p.G : (int64_t)p.a.q.T * p.G;
    const int most = rows < 8 * NT ? (int)rows : 8 * NT;
    // items that can be cut: no more than there are, and than there are pieces
    const int64_t tiles = LIST ? (int64_t)p.a.q.T * p.gt : (rows + 8 * NT - 1) / (8 * NT);
    const int64_t items = (int64_t)p.c.batch * p.c.heads * tiles;
    // pieces an item can be in: no more than its steps
    const int64_t span = LIST ? (int64_t)p.a.n_sel << p.c.bs_log2 : (int64_t)p.c.max_blocks << p.c.bs_log2;
    const int64_t seen = !LIST && p.a.window && (int64_t)p.a.window + p.a.q.T < span ? (int64_t)p.a.window + p.a.q.T : span;
    if (items * kFewItems <= p.ctas && seen >= kFewSteps * kStep)
        return launch_pdl(k_kv8_combine_few<D, NT, LIST>, dim3((unsigned)items, most), kMergeWarps * 32, 0, st, p);
    return launch_pdl(k_kv8_combine<D, NT, LIST>, dim3(p.ctas, (most + 3) / 4), 4 * D, 0, st, p);
}

template <int D>
cudaError_t launch_d(Params& p, cudaStream_t st) {
    if (p.a.block_idx) return p.G <= 8 ? launch<D, 1, true>(p, st) : launch<D, 2, true>(p, st);
    const int64_t rows = (int64_t)p.a.q.T * p.G;
    if (rows <= 8) return launch<D, 1, false>(p, st);
    return launch<D, 2, false>(p, st);
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

bool kv8_row_map(CUtensorMap_st* map, const DevKv8& c, void* codes, int box_rows, bool swizzled) {
    EncodeTiled enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t gdim[2] = {(cuuint64_t)c.dim, ((cuuint64_t)c.n_blocks * c.heads) << c.bs_log2};
    const cuuint64_t gstride[1] = {(cuuint64_t)c.dim};
    const cuuint32_t box[2] = {(cuuint32_t)c.dim, (cuuint32_t)box_rows}, estride[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, gdim, gstride, box, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : c.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t kv8_attn_part_floats(int dim) {
    return (size_t)2 * kMaxCtas * (dim == 64 ? Part<64>::kFloats : Part<128>::kFloats);
}

cudaError_t launch_kv8_attn(const DevKv8& c, const Kv8Attn& a, cudaStream_t st) {
    Params p;
    p.c = c;
    p.a = a;
    p.G = a.q.H / c.heads;
    p.wait_limit = wait_limit();
    return c.dim == 64 ? launch_d<64>(p, st) : launch_d<128>(p, st);
}

}  // namespace csa2
