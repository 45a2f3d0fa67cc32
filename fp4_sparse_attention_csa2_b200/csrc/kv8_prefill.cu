// Attention over the 8-bit cache for many query rows per sequence (prompt
// chunks, wide verification) on the 5th-generation tensor cores.
//
// With the query rows of all tokens and the query heads of a key head as the
// rows of a matrix (256 of them a CTA, two tiles of 128), both products are
// GEMM-shaped and the tensor cores bound the kernel: 4 * 256 * 128 * D flop per
// 128 positions.  One CTA per SM, six warpgroups:
//   - four softmax warpgroups, two per row tile, a thread half a row (two
//     halves a row keep a thread's 64 values in registers and halve the time
//     from S to the weights, which is what the products wait for): read S from
//     TMEM, work out the weights with the maximum so far, and write them as
//     fp16 over S (the second product takes them from TMEM) unless a weight
//     came out above 2^7 of the maximum: then, rarely but for an item's first
//     step, the halves agree on the new maximum, O is rescaled and the weights
//     are worked out again;
//   - a converter warpgroup: the codes of the next 128 positions from where TMA
//     put them to fp16 operand tiles (E4M3 values are exact in fp16), two
//     stages deep;
//   - one warp that issues every tcgen05.mma.  It alternates the row tiles
//     (O0 += P0 V, S0 = Q0 K, O1 += P1 V, S1 = Q1 K), so one tile's products
//     run while the other's softmax does.  An item of at most 128 rows has one
//     row tile: its even and odd steps then take the two places, each with a
//     maximum, sum and output of its own, added up at the end;
//   - one warp that looks up pages and issues the TMA loads.
// Key scales multiply S per block; value scales enter the weights' exponent,
// weight = 2^(z + log2(vs) - M), so the fp16 weights stay in range whatever the
// blocks' scales are.  The sum of 2^z does not depend on them, and takes them
// back out per block (exact powers of two) where they lie within 2^kSpread of
// the item's first block's: a weight that fp32 cannot hold is then nothing to
// the sum either.  A tile with another scale (a block of zeros has the least,
// 2^-120, but so have values of 1e-35), and every tile behind one with a far
// greater scale, has its sum worked out from S for itself, without the value
// scales (2,048 tokens over 8,192 positions with zeros for every other block's
// values: 401 us, without 260).
//
// Work split as in kv8_attn.cu: the (row block, head, 128 positions) steps of
// the batch, and kItem units an item, form one line cut into equal pieces; cut
// items are merged by k_kv8_prefill_combine.  2,048 tokens over 8,192 positions
// (32 / 8 heads of 128): 268 to 282 us on different boards, 285 called from Python
// = 0.84 PFLOP/s, half the measured bf16 rate.  A
// step of a row tile is a chain of about 4,100 cycles (S to registers 250, weights
// 1,500, the halves' agreement and the store 500, both products 1,100, looks at
// barriers the rest), of which the other tile's covers a half.
#include <cuda.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv8.cuh"
#include "kv8_tc.cuh"

namespace csa2 {
namespace {

constexpr int kRows = 256, kTileRows = 128, kPos = 128;
constexpr int kThreads = 768, kConv = 128, kSoftmax = 512;   // all, converter's, softmax's
constexpr int kMaxCtas = 148;
constexpr int kMmaWarp = 20, kLoadWarp = 21;
constexpr int kMergeWarps = 16, kFewItems = 16;   // of a CTA of k_kv8_prefill_combine_few; pieces an item from which it merges
constexpr float kNone = -3.0e38f;
constexpr float kHeadroom = 8.0f;   // weights are 2^(z - M + 8): full fp16 precision down to 2^-22
constexpr float kLazy = 7.0f;       // and at most 2^15 (fp16: 65504) before the maximum is moved
// log2 of how far a block's value scale may be from the sums' unit 2^e0 for the
// weights to carry the sum.  With scales within 2^48 of each other a weight that
// underflows, 2^-126, is below 2^-86 of the greatest term of the sum.
constexpr int kSpread = 24;
constexpr float kApart = 64.0f;     // log2 of how far a sum's unit may be from another for it to be kept in that

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

// Units of the line that an item costs besides its steps: queries, the first
// products and the outputs, with nothing else under way.  Without them the piece
// with the most short items was the last by far: a prompt of 2,000 tokens, 32 / 8
// heads, took 279 us, with 3 units 115, with 6 or 10 95 (8 and rows by whole lines:
// 92); 2,048 tokens over 8,192 positions 278, 277, 275 and 272.
constexpr int kItem = 8;

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
    __device__ __forceinline__ int64_t total(const Cursor& k) const { return (int64_t)p.c.heads * (k.steps ? k.steps + kItem : 0); }
    // Whether position t's block is to be looked up: it holds positions, and not only
    // such as lie before every row's window (their page may be gone).
    __device__ __forceinline__ bool seen(const Cursor& k, int t) const {
        const int64_t first = p.a.window ? (int64_t)k.L - k.n + k.row0 / p.G - p.a.window + 1 : 0;
        return t < k.L && ((((int64_t)t >> p.c.bs_log2) + 1) << p.c.bs_log2) > first;
    }
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

// The item and step of unit u, and the units before its first step that are left.
__device__ int line_find(const Line& w, const int64_t* sums, int64_t u, Cursor& k) {
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
    if (k.steps == 0) return 0;
    k.h = (int)(u / (k.steps + kItem));
    const int at = (int)(u - (int64_t)k.h * (k.steps + kItem));
    k.step = at > kItem ? at - kItem : 0;
    return at < kItem ? kItem - at : 0;
}

// Steps among `units` units from cursor k on, `ahead` of them before its first step.
__device__ int line_steps(const Line& w, Cursor k, int64_t units, int ahead) {
    const int pairs = w.p.c.batch * w.p.row_blocks;
    int64_t n = 0;
    while (units > ahead) {
        units -= ahead;
        const int64_t here = units < k.steps - k.step ? units : k.steps - k.step;
        n += here;
        units -= here;
        if (units == 0) break;
        // the other heads have the same steps
        const int64_t each = k.steps + kItem, rest = w.p.c.heads - 1 - k.h, whole = units / each < rest ? units / each : rest;
        n += whole * k.steps;
        units -= whole * each;
        if (whole < rest) {
            if (units > kItem) n += units - kItem;
            break;
        }
        int pair = k.pair;
        do w.load(k, ++pair, nullptr);
        while (pair < pairs && k.steps == 0);
        if (pair >= pairs) break;
        ahead = kItem;
    }
    return (int)n;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// log2 of the value scale that an item's sums are kept in: its first block's.
// The least scale is mostly that of a block of zeros and says nothing of the
// others: 1 then, which is as right as any and nearer to most.
__device__ __forceinline__ int sum_scale(float vs) {
    const int e = (int)(__float_as_uint(vs) >> 23) - 127;
    return e <= -120 ? 0 : (e > 120 ? 120 : e);
}

// A sum l of 2^z in units of 2^(M - 8 - e0 - x), x a whole number and mostly 0.
struct Sum {
    float l, x;
    // l to [1, 2), where it is a number that has an exponent.
    __device__ __forceinline__ void normalise() {
        const int u = __float_as_int(l), e = u >> 23;
        if (e > 0 && e < 255) {
            l = __int_as_float((u & 0x7FFFFF) | 0x3F800000);
            x -= (float)(e - 127);
        }
    }
    // The maximum M rises by d.
    __device__ __forceinline__ void rise(float d) {
        if (l < 0x1p-40f) normalise();
        if (d <= kApart || l == 0.0f) {
            l *= ex2(-d);
        } else {
            const float k = rintf(d);
            l *= ex2(k - d);
            x += k;
        }
    }
    // A sum with the same M.
    __device__ __forceinline__ void add(Sum o) {
        if (x == 0.0f && o.x == 0.0f) {
            l += o.l;
            return;
        }
        normalise();
        o.normalise();
        const float to = l == 0.0f ? o.x : o.l == 0.0f ? x : fminf(x, o.x);
        l = l * ex2(fminf(to - x, 0.0f)) + o.l * ex2(fminf(to - o.x, 0.0f));
        x = to;
        if (fabsf(x) <= kApart) {
            l *= ex2(-x);
            x = 0.0f;
        }
    }
};

template <int D>
struct Smem {
    static constexpr int kPanels = D / 64;                    // 64 channels (128 bytes of fp16) a panel
    static constexpr int kPanel = kPos * 128;                 // bytes of one panel of 128 rows
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int q = 0;                               // [row tile][panel]
    static constexpr int k = q + 2 * kTile;                   // [stage][panel]
    static constexpr int v = k + 2 * kTile;                   // [stage][panel]
    static constexpr int codes = v + 2 * kTile;               // K, V as stored
    static constexpr int sums = codes;                        // kThreads + 1 words, before the first load
    static constexpr int sc = codes + 2 * kPos * D;           // [8][8] key scale, log2 of the value scale
    static constexpr int sg = sc + 8 * 8 * 8;                 // [8][8] 2^(e0 - that); 0: the weights do not carry the sum
    static constexpr int lims = sg + 8 * 8 * 4;               // [8] positions of a tile that are values
    static constexpr int xch = lims + 8 * 4;                  // [tile][half][128] floats: halves of a row agree
    static constexpr int bars = xch + 4 * 128 * 4;
    static constexpr int misc = bars + 20 * 8;                // TMEM base, dead
    static constexpr int bytes = misc + 16;
};

// Barriers, in pairs by stage or row tile (kLFull, kLEmpty: K, V).
enum Bar { kQ = 0, kKFull = 1, kKEmpty = 3, kVFull = 5, kVEmpty = 7, kS = 9, kP = 11, kLFull = 13, kLEmpty = 15, kO = 17, kDrain = 18 };

constexpr uint32_t kColO = 256;      // TMEM columns: S0, S1 (P over them), O0, O1

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_prefill(const __grid_constant__ Params p,
                                                             const __grid_constant__ CUtensorMap kmap,
                                                             const __grid_constant__ CUtensorMap vmap) {
    using S = Smem<D>;
    extern __shared__ __align__(1024) uint8_t smem[];   // no static shared memory: it starts on such a boundary
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::bars);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + S::misc);
    int64_t* sums = reinterpret_cast<int64_t*>(smem + S::sums);
    float2* sc = reinterpret_cast<float2*>(smem + S::sc);
    float* sg = reinterpret_cast<float*>(smem + S::sg);
    volatile int* lims = reinterpret_cast<volatile int*>(smem + S::lims);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // A bounded wait of a warp for up to three barriers (< 0: none); once one ran out, every later wait
    // of the CTA gives up too.  A look at a barrier takes some 400 cycles here even when its phase is
    // over, so looks at several go out together and without a time limit of their own (292 -> 278 us
    // for 2,048 tokens over 8,192 positions).
    auto wait_all = [&](int bar0, uint32_t parity0, int bar1, uint32_t parity1, int bar2, uint32_t parity2) {
        uint32_t n = 0;
        bool ok;
        do {
            const bool a = bar0 < 0 || tc::mbar_try_wait_brief(bars + bar0, parity0);
            const bool b = bar1 < 0 || tc::mbar_try_wait_brief(bars + bar1, parity1);
            const bool c = bar2 < 0 || tc::mbar_try_wait_brief(bars + bar2, parity2);
            ok = p.wait_limit && __all_sync(0xFFFFFFFFu, a && b && c);
        } while (!ok && ++n < p.wait_limit && !misc[1]);
        if (!ok) {
            if (!misc[1]) flag(p.a.status, kStatusTimeout);
            misc[1] = 1;
        }
        return ok;
    };
    auto wait_warp = [&](int bar, uint32_t parity) { return wait_all(bar, parity, -1, 0, -1, 0); };

    if (tid == 0) {
        tc::mbar_init(bars + kQ, kSoftmax);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bars + kKFull + i, kConv);
            tc::mbar_init(bars + kKEmpty + i, 1);
            tc::mbar_init(bars + kVFull + i, kConv);
            tc::mbar_init(bars + kVEmpty + i, 1);
            tc::mbar_init(bars + kS + i, 1);
            tc::mbar_init(bars + kP + i, kSoftmax / 2);
            tc::mbar_init(bars + kLFull + i, 1);
            tc::mbar_init(bars + kLEmpty + i, kConv);
        }
        tc::mbar_init(bars + kO, 1);
        tc::mbar_init(bars + kDrain, 1);
        tc::fence_mbar_init();
        misc[1] = 0;
    }
    pdl_begin();
    if (warp == kMmaWarp) tc::tmem_alloc(const_cast<uint32_t*>(misc), 512);
    const Line line(p);
    const int64_t total = line_sums(line, sums, blockIdx.x == 0 ? p.a.status : nullptr);
    const int64_t share = total < p.ctas ? (total < 1 ? 1 : total) : p.ctas;
    int* desc = reinterpret_cast<int*>(p.a.part + ((int64_t)blockIdx.x * 2 + 1) * Part<D>::kFloats + Part<D>::kDesc);
    if (tid == 0) desc[4] = 0;
    const bool any = blockIdx.x < share && total > 0;
    const int64_t u0 = any ? total * blockIdx.x / share : 0, u1 = any ? total * (blockIdx.x + 1) / share : 0;
    Cursor cur;
    int piece_steps = 0;
    if (any) {
        const int ahead = line_find(line, sums, u0, cur);
        piece_steps = line_steps(line, cur, u1 - u0, ahead);
    }
    tc::fence_before_sync();
    __syncthreads();   // TMEM is there, the barriers are, and `sums` becomes the codes' place
    tc::fence_after_sync();
    const uint32_t tmem = misc[0];

    // registers by role: 4 * 96 + 56 + 40 = 6 * 80, what the CTA is launched with
    if (warp < 16) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
        // ---------------------------------------------------------------- softmax: half `half` of a row of tile `t`
        const int G = p.G, T = p.a.q.T, H = p.a.q.H;
        const int t = warp >> 3, half = (warp >> 2) & 1, rt = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t col_s = lanes + t * 128, col_o = lanes + kColO + t * D + half * (D / 2);
        volatile float* xch = reinterpret_cast<volatile float*>(smem + S::xch) + t * 256;
        // Meetings of the threads of a tile (both halves of its rows) and of both tiles.  Whether all are
        // well is part of the barrier itself, so that everyone goes the same way.  (A barrier for each two
        // warps that share 32 rows, 64 threads, was slower, 343 against 314 us for 2,048 tokens over 8,192
        // positions: warps of a tile that drift apart delay the tile's products.)
        auto meet = [](int id, int threads, bool v) {
            int r;
            asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %1, 0;\n\t"
                         "barrier.cta.red.and.pred b, %2, %3, a;\n\tselp.b32 %0, 1, 0, b;\n\t}"
                         : "=r"(r) : "r"((int)v), "r"(id), "r"(threads) : "memory");
            return r != 0;
        };
        auto agree = [&](bool v) { return meet(1 + t, 256, v); };
        auto both_tiles = [&](bool v) { return meet(3, 512, v); };
        uint32_t tile = 0, s_phase = 0, o_phase = 0;   // tiles done by the CTA; parities
        bool ok = true;
        // Between items only this much of the cursor is kept (registers): the rest is worked out again.
        int pair = cur.pair, head = cur.h, step = cur.step, todo_all = piece_steps;
        auto item = [&]() {
            asm volatile("" : "+r"(pair));   // not to be kept from the time before
            Cursor k;
            line.load(k, pair, nullptr);
            k.h = head;
            k.step = step;
            return k;
        };
        while (todo_all > 0) {
            int todo, pos, first;
            bool dual;      // one row tile, even and odd steps apart
            float e0;       // log2 of the value scale that sums are kept in
            float zs = p.a.sm_scale * 1.4426950408889634f;
            {   // half a query row as fp16, K-major; bf16 scaled by the power of two that takes the row's
                // greatest finite magnitude to [2^14, 2^15)
                constexpr int kVec = D / 16;
                const Cursor cur = item();
                todo = todo_all < cur.steps - cur.step ? todo_all : cur.steps - cur.step;
                dual = cur.rows <= kTileRows;
                const int row = dual ? rt : t * kTileRows + rt;
                const bool mine = row < cur.rows;
                const int at0 = cur.lo + cur.step * kPos;
                const int block0 = line.seen(cur, at0) ? kv8_block(p.c, cur.b, at0 >> p.c.bs_log2) : -1;
                const float vs0 = block0 >= 0 ? __ldg(p.c.v_scale + (int64_t)block0 * p.c.heads + cur.h) : 1.0f;
                e0 = (float)sum_scale(vs0);
                const int j = (cur.row0 + row) / G, g = cur.row0 + row - j * G;
                pos = mine ? cur.L - cur.n + j : -1;
                pos = pos < -1 ? -1 : pos;     // before the sequence: nothing is seen either way
                first = p.a.window ? pos - p.a.window + 1 : 0;
                // as seen from this half's first column of the item's first step
                pos -= cur.lo + cur.step * kPos + half * 64;
                first -= cur.lo + cur.step * kPos + half * 64;
                if (!mine) pos = 0x7FFFFFFF, first = -0x7FFFFFFF;   // rows without a token: anything, without the mask
                // a warp's 32 half rows by whole lines: kVec lanes a row, 32 / kVec rows at a time
                const int64_t from = (int64_t)cur.b * p.a.q.stride_b + (int64_t)j * p.a.q.stride_t + (int64_t)(cur.h * G + g) * D;
                const uint32_t live = __ballot_sync(0xFFFFFFFFu, mine);
                const int piece = lane % kVec;
                uint4 x[kVec];
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const int at = i * (32 / kVec) + lane / kVec;
                    const int64_t src = __shfl_sync(0xFFFFFFFFu, from, at);
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (live >> at & 1)
                        x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.a.q.q) + src + half * (D / 2)) + piece);
                }
                if (p.a.q.is_bf16) {
                    float amax[kVec];
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
                        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                        amax[i] = 0.0f;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float a = fabsf(__uint_as_float(w[q] << 16)), b = fabsf(__uint_as_float(w[q] & 0xFFFF0000u));
                            if (a <= 3.4028235e38f) amax[i] = fmaxf(amax[i], a);
                            if (b <= 3.4028235e38f) amax[i] = fmaxf(amax[i], b);
                        }
#pragma unroll
                        for (int o = 1; o < kVec; o <<= 1) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xFFFFFFFFu, amax[i], o));
                    }
                    ok = agree(ok);              // the sums of the item before have been read
                    const int r0 = (warp & 3) * 32;
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        if (piece == 0) xch[half * 128 + r0 + i * (32 / kVec) + lane / kVec] = amax[i];
                    ok = agree(ok);
                    auto up_of = [&](float m) {
                        const int e = 14 - ((int)(__float_as_uint(m) >> 23) - 127);
                        return e > 126 ? 126 : e;
                    };
                    zs *= exp2_int(-up_of(fmaxf(xch[rt], xch[128 + rt])));
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
                        const float up = exp2_int(up_of(fmaxf(amax[i], xch[(half ^ 1) * 128 + r0 + i * (32 / kVec) + lane / kVec])));
                        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const __half2 h = __floats2half2_rn(__uint_as_float(w[q] << 16) * up,
                                                                __uint_as_float(w[q] & 0xFFFF0000u) * up);
                            memcpy(&w[q], &h, 4);
                        }
                        x[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                uint8_t* dst = smem + S::q + t * S::kTile;
                const int c = half * kVec + piece;
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    *reinterpret_cast<uint4*>(dst + (c >> 3) * S::kPanel +
                                              tc::sw128_offset((warp & 3) * 32 + i * (32 / kVec) + lane / kVec, c & 7)) = x[i];
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(bars + kQ);
            }
            float M = kNone;
            Sum sum = {0.0f, 0.0f};
            bool started = false;      // O holds something
            bool wide = false;         // the sum is in a unit of its own
            int i = 0;
            while (i < todo) {
                for (; !wide && i < todo; ++i, ++tile) {
                    if (dual && (i & 1) != t) continue;
                    const int t0 = i * kPos;
                    ok = wait_warp(kS + t, s_phase) && ok;
                    s_phase ^= 1;
                    tc::fence_after_sync();
                    const float2* f2 = sc + (tile & 7) * 8 + half * 4;
                    const float* g1 = sg + (tile & 7) * 8 + half * 4;
                    const bool edge = !__all_sync(0xFFFFFFFFu, t0 + 63 <= pos && t0 >= first);
                    if (ok && g1[0] == 0.0f) break;        // goes on below (everyone where a wait ran out goes the same way)
                    uint32_t w[32];        // weights, two a word
                    float l1;
#pragma unroll 1
                    for (;;) {
                        uint32_t r[64];
                        tc::tmem_ld32_nowait(col_s + half * 64, r);
                        tc::tmem_ld32_nowait(col_s + half * 64 + 32, r + 32);
                        tc::tmem_ld_wait();
                        if (edge) {
#pragma unroll
                            for (int x = 0; x < 64; ++x)
                                if (t0 + x > pos || t0 + x < first) r[x] = 0xFF800000u;
                        }
                        float top = -INFINITY;     // the greatest logit + log2(value scale) of the half row
                        l1 = 0.0f;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t* v = r + q * 16;
                            const float2 f = f2[q];
                            // at least the least normal number: 0 times a masked -inf would be NaN, and what is
                            // added to a logit, |S| < 2^31, is below 2^-95
                            const float a = fmaxf(zs * f.x, 1.17549435e-38f), d = f.y - M + kHeadroom;
                            const uint64_t ff = pack2(a, a), dd = pack2(d, d);
                            uint64_t acc = 0;
                            float m = __uint_as_float(v[0]);
#pragma unroll
                            for (int x = 0; x < 16; x += 2) {
                                m = x ? max3(m, __uint_as_float(v[x]), __uint_as_float(v[x + 1])) : fmaxf(m, __uint_as_float(v[1]));
                                const float2 z = unpack2(fma2(pack2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), ff, dd));
                                const float2 e = make_float2(ex2(z.x), ex2(z.y));
                                acc = add2(acc, pack2(e.x, e.y));
                                const __half2 h = __floats2half2_rn(e.x, e.y);
                                memcpy(&w[q * 8 + x / 2], &h, 4);
                            }
                            top = fmaxf(top, m * a + f.y);
                            // back from 2^(z + log2 vs - M + 8) to 2^(z + e0 - M + 8), exactly
                            const float2 s2 = unpack2(acc);
                            l1 += (s2.x + s2.y) * g1[q];
                        }
                        // all of S is in registers from here: the weights may go over it
                        if (agree(ok && !(top > M + kLazy))) break;
                        xch[half * 128 + rt] = top;
                        ok = agree(ok);
                        if (!ok) break;
                        const float M1 = fmaxf(M, fmaxf(top, xch[(half ^ 1) * 128 + rt])), f = ex2(M - M1);
                        sum.l *= f;
                        M = M1;
                        if (started) {
#pragma unroll 1
                            for (int q = 0; q < D / 2; q += 16) {
                                uint32_t o[16];
                                tc::tmem_ld16_nowait(col_o + q, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                                tc::tmem_st16_nowait(col_o + q, o);
                            }
                        }
                        ok = agree(ok);            // the other half has read this one's maximum
                        if (!ok) break;
                    }
                    if (!ok) break;
                    sum.l += l1;
                    started = true;
                    tc::tmem_st16_nowait(col_s + half * 32, w);
                    tc::tmem_st16_nowait(col_s + half * 32 + 16, w + 16);
                    tc::tmem_st_wait();
                    tc::fence_before_sync();
                    tc::mbar_arrive(bars + kP + t);
                }
                if (!ok || i >= todo) break;
                // A step whose weights do not carry the sum, or the sum is in another unit: S is read for both maxima
                // first, then for the weights and the sum's terms, whose greatest is near 1.
                if (!(dual && (i & 1) != t)) {
                    const int t0 = i * kPos;
                    if (wide) {
                        ok = wait_warp(kS + t, s_phase);
                        s_phase ^= 1;
                        tc::fence_after_sync();
                    }
                    const float2* f2 = sc + (tile & 7) * 8 + half * 4;
                    const bool edge = !__all_sync(0xFFFFFFFFu, t0 + 63 <= pos && t0 >= first);
                    auto logits = [&](int q, uint32_t* v) {        // 16 columns of S, and the factor to a logit
                        tc::tmem_ld16_nowait(col_s + half * 64 + q * 16, v);
                        tc::tmem_ld_wait();
                        if (edge) {
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                if (t0 + q * 16 + x > pos || t0 + q * 16 + x < first) v[x] = 0xFF800000u;
                        }
                        return fmaxf(zs * f2[q].x, 1.17549435e-38f);
                    };
                    float top = -INFINITY, most = -INFINITY;       // of logit + log2(value scale), and of the logits
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t v[16];
                        const float a = logits(q, v);
                        float m = __uint_as_float(v[0]);
#pragma unroll
                        for (int x = 1; x < 15; x += 2) m = max3(m, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
                        m = fmaxf(m, __uint_as_float(v[15]));
                        top = fmaxf(top, m * a + f2[q].y);
                        most = fmaxf(most, m * a);
                    }
                    if (!agree(ok && !(top > M + kLazy))) {
                        xch[half * 128 + rt] = top;
                        ok = agree(ok);
                        if (!ok) break;
                        const float M1 = fmaxf(M, fmaxf(top, xch[(half ^ 1) * 128 + rt])), f = ex2(M - M1);
                        sum.rise(M1 - M);
                        M = M1;
                        if (started) {
#pragma unroll 1
                            for (int q = 0; q < D / 2; q += 16) {
                                uint32_t o[16];
                                tc::tmem_ld16_nowait(col_o + q, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                                tc::tmem_st16_nowait(col_o + q, o);
                            }
                        }
                    }
                    Sum own = {0.0f, 0.0f};
                    const float off = most == -INFINITY ? 0.0f : M - kHeadroom - e0 - most;
                    if (!(fabsf(off) <= kApart)) own.x = rintf(off);
                    const float d = kHeadroom - M + e0 + own.x;
                    uint32_t w[32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t v[16];
                        const float a = logits(q, v), dw = f2[q].y - M + kHeadroom;
                        const uint64_t ff = pack2(a, a), dd = pack2(d, d), ww = pack2(dw, dw);
                        uint64_t acc = 0;
#pragma unroll
                        for (int x = 0; x < 16; x += 2) {
                            const float2 z = unpack2(fma2(pack2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), ff, dd));
                            acc = add2(acc, pack2(ex2(z.x), ex2(z.y)));
                        }
                        const float2 s2 = unpack2(acc);
                        own.l += s2.x + s2.y;
                        if (__all_sync(0xFFFFFFFFu, most + dw < -25.5f)) {    // zeros in fp16: no need to work them out
#pragma unroll
                            for (int x = 0; x < 8; ++x) w[q * 8 + x] = 0;
                            continue;
                        }
#pragma unroll
                        for (int x = 0; x < 16; x += 2) {
                            const float2 z = unpack2(fma2(pack2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), ff, ww));
                            const __half2 h = __floats2half2_rn(ex2(z.x), ex2(z.y));
                            memcpy(&w[q * 8 + x / 2], &h, 4);
                        }
                    }
                    ok = agree(ok);                // S has been read, and the other half's maximum
                    if (!ok) break;
                    started = true;
                    tc::tmem_st16_nowait(col_s + half * 32, w);
                    tc::tmem_st16_nowait(col_s + half * 32 + 16, w + 16);
                    tc::tmem_st_wait();
                    tc::fence_before_sync();
                    tc::mbar_arrive(bars + kP + t);
                    sum.add(own);
                    wide = !agree(ok && sum.x == 0.0f);
                }
                ++i, ++tile;
            }
            // ---- the outputs, half the channels
            ok = ok && wait_warp(kO, o_phase);
            o_phase ^= 1;
            tc::fence_after_sync();
            {   // the row's other half's sum; and its unit, where there are any but 2^e0
                xch[half * 128 + rt] = sum.l;
                const bool plain = agree(ok && sum.x == 0.0f);
                Sum other = {xch[(half ^ 1) * 128 + rt], 0.0f};
                if (!plain) {
                    ok = agree(ok);
                    xch[half * 128 + rt] = sum.x;
                    ok = agree(ok);
                    other.x = xch[(half ^ 1) * 128 + rt];
                }
                sum.add(other);
            }
            Cursor cur = item();
            const int row = dual ? rt : t * kTileRows + rt;
            const bool mine = row < cur.rows;
            const int j = (cur.row0 + row) / G, g = cur.row0 + row - j * G, left = cur.steps - cur.step;
            const bool from_start = cur.step == 0, to_end = todo == left;
            const bool whole = from_start && to_end;
            float* part = p.a.part + ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * Part<D>::kFloats;
            const int64_t at = ((int64_t)cur.b * T + j) * H + cur.h * G + g;
            float f0 = 1.0f, f1 = 0.0f;            // factors of this tile's output and, dual, of the odd steps'
            if (dual) {
                float* odd = reinterpret_cast<float*>(smem + S::q);     // the odd steps' output [D][128], over the queries
                volatile float* stats = reinterpret_cast<volatile float*>(smem + S::xch) + 256;   // their M and l
                ok = agree(ok);
                if (t == 1) {
#pragma unroll 1
                    for (int q = 0; q < D / 2; q += 16) {
                        uint32_t o[16];
                        tc::tmem_ld16_nowait(col_o + q, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            odd[(half * (D / 2) + q + x) * 128 + rt] = started ? __uint_as_float(o[x]) : 0.0f;
                    }
                    if (half == 0) stats[rt] = M, stats[128 + rt] = sum.l;
                }
                const bool plain = both_tiles(ok && (t == 0 || sum.x == 0.0f));
                const float M1 = stats[rt];
                Sum other = {stats[128 + rt], 0.0f};
                if (!plain) {
                    ok = both_tiles(ok);
                    if (t == 1 && half == 0) stats[rt] = sum.x;
                    ok = both_tiles(ok);
                    other.x = stats[rt];
                }
                if (t == 0) {
                    const float top = fmaxf(M, M1);
                    f0 = ex2(M - top);
                    f1 = ex2(M1 - top);
                    sum.rise(top - M);
                    other.rise(top - M1);
                    sum.add(other);
                    M = top;
                }
            }
            // parts to be merged, whose units differ, by their own magnitude
            if (!whole || !(fabsf(e0 + sum.x) <= 100.0f)) sum.normalise();
            // outputs: O 2^e / l, -136 < e <= 120, in two factors, of which the first stays a normal number
            const float l = sum.l, e = e0 + sum.x, scale = ex2(fminf(e + 100.0f, 0.0f));
            const float f = l == 0.0f ? 0.0f : ex2(fmaxf(e, -100.0f)) / l;
            if (ok && (!dual || t == 0)) {
                const float* odd = reinterpret_cast<const float*>(smem + S::q);
                const uint32_t live = __ballot_sync(0xFFFFFFFFu, mine);
#pragma unroll 1
                for (int q = 0; q < D / 2; q += 32) {
                    uint32_t r[32];
                    tc::tmem_ld32_nowait(col_o + q, r);
                    tc::tmem_ld_wait();
                    const int ch = half * (D / 2) + q;
                    if (dual) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            r[x] = __float_as_uint(__uint_as_float(r[x]) * f0 + odd[(ch + x) * 128 + rt] * f1);
                    }
                    if (__any_sync(0xFFFFFFFFu, scale != 1.0f)) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * (whole ? scale : 1.0f));
                    }
                    if (whole) {
                        // through shared memory, two rows of 64 bytes in 128, so that they leave by lines: over the
                        // queries, or over what this warp alone has read of the odd steps' output
                        __syncwarp();
                        auto stage = [&](int row, int chunk) {
                            const int pair = row >> 1;
                            uint8_t* at = dual ? smem + S::q + ((ch + pair) * 128 + (warp & 3) * 32) * 4
                                               : smem + S::q + t * S::kTile + (warp & 7) * 2048 + pair * 128;
                            return reinterpret_cast<uint4*>(at + (row & 1) * 64 + ((chunk ^ (pair & 3)) << 4));
                        };
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
                            *stage(lane, x) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int from = x * 8 + (lane >> 2);
                            const int64_t to = __shfl_sync(0xFFFFFFFFu, at, from);
                            if (live >> from & 1)
                                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + to * D + ch + (lane & 3) * 8) =
                                    *stage(from, lane & 3);
                        }
                    } else if (mine) {
                        // by 16-byte columns across the rows, so that a warp's stores are dense
                        float4* dst = reinterpret_cast<float4*>(part) + (int64_t)(ch / 4) * kRows + row;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            dst[x * kRows] = make_float4(__uint_as_float(r[x * 4]), __uint_as_float(r[x * 4 + 1]),
                                                         __uint_as_float(r[x * 4 + 2]), __uint_as_float(r[x * 4 + 3]));
                    }
                }
                if (mine && half == 0) {
                    if (whole) {
                        if (p.a.lse)
                            p.a.lse[at] = l == 0.0f ? -INFINITY : (M - e - kHeadroom + log2f(l)) * 0.6931471805599453f;
                    } else {
                        float* s3 = part + Part<D>::kStats + row * 3;
                        s3[0] = l == 0.0f ? kNone : M - e - kHeadroom;
                        s3[1] = l;
                        s3[2] = M - kHeadroom;
                    }
                }
            }
            if (ok && from_start && !to_end && tid == 0) {
                const int64_t last_u = u1 - todo_all + left - 1;
                const int64_t last = ((last_u + 1) * share + total - 1) / total - 1;
                desc[0] = cur.b;
                desc[1] = cur.h;
                desc[2] = cur.row0;
                desc[3] = cur.rows;
                desc[4] = (int)(last - blockIdx.x) + 1;
            }
            tc::fence_before_sync();
            ok = both_tiles(ok);       // (and the odd steps' outputs have been read: queries may go over them)
            if (!ok) break;
            todo_all -= todo;
            if (todo_all > 0) {      // an item that goes on behind this piece is the last of it
                line.next_item(cur);
                pair = cur.pair;
                head = cur.h;
                step = 0;
            }
        }
    } else if (warp < kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // ---------------------------------------------------------------- codes to fp16 operand tiles
        const int ct = tid - kSoftmax, l8 = ct & 7;
        // Piece (16 codes, two 16-byte chunks of fp16) `x` of this thread: eight lanes load 128 dense bytes'
        // worth of distinct banks and store to eight distinct ones.
        auto convert = [&](const uint8_t* src, uint8_t* dst, bool clear, int lead, int lim) {
#pragma unroll 4
            for (int x = 0; x < D / 16; ++x) {
                const int row = D == 128 ? 2 * ((ct >> 3) + 16 * (x >> 1)) + ((l8 >> 2) ^ (x & 1)) : (ct >> 2) + 32 * x;
                const int piece = D == 128 ? l8 : ct & 3;
                uint4 w = *reinterpret_cast<const uint4*>(src + row * D + piece * 16);
                if (clear && (row < lead || row >= lim)) w = make_uint4(0, 0, 0, 0);
                uint8_t* panel = dst + (piece >> 2) * S::kPanel;
                const uint32_t c = (piece & 3) * 2;
                *reinterpret_cast<uint4*>(panel + tc::sw128_offset(row, c)) =
                    make_uint4(half2_lo(w.x), half2_hi(w.x), half2_lo(w.y), half2_hi(w.y));
                *reinterpret_cast<uint4*>(panel + tc::sw128_offset(row, c + 1)) =
                    make_uint4(half2_lo(w.z), half2_hi(w.z), half2_lo(w.w), half2_hi(w.w));
            }
        };
        const int steps = piece_steps;
        for (int tile = 0; tile < steps; ++tile) {
            const uint32_t st = tile & 1;
            bool ok = wait_warp(kLFull, st);
            if (tile >= 2) ok = ok && wait_warp(kKEmpty + st, ((tile >> 1) - 1) & 1);
            if (!ok) break;
            const int lim = lims[tile & 7] & 255, lead = lims[tile & 7] >> 8;
            convert(smem + S::codes, smem + S::k + st * S::kTile, false, 0, 0);
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(bars + kLEmpty);
            tc::mbar_arrive(bars + kKFull + st);
            ok = wait_warp(kLFull + 1, st);
            if (tile >= 2) ok = ok && wait_warp(kVEmpty + st, ((tile >> 1) - 1) & 1);
            if (!ok) break;
            // values behind the sequence's end, and where nothing was copied, are zeros: a weight of 0 times NaN is NaN
            if (lim < kPos || lead) convert(smem + S::codes + kPos * D, smem + S::v + st * S::kTile, true, lead, lim);
            else convert(smem + S::codes + kPos * D, smem + S::v + st * S::kTile, false, 0, 0);
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(bars + kLEmpty + 1);
            tc::mbar_arrive(bars + kVFull + st);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------ pages, scales and the codes' loads
            const int box = p.c.bs() < kPos ? p.c.bs() : kPos, boxes = kPos / box;
            uint32_t issued = 0, steps = (uint32_t)piece_steps;
            int phys = -1, lim = 0, h = 0, e0 = 0;  // lim: positions before the sequence's end, and (<< 8) how many are not looked up
            bool fresh = true, item_ends = true;    // the tile is the first of its item in this piece
            bool high = false;                      // a tile of the item had a value scale far above the sums' unit
            auto look = [&](bool there) {    // lane x < 8: the block of positions 16 x .. of the tile at `cur`
                phys = -1;
                fresh = item_ends;
                if (!there) return;
                const int t0 = cur.lo + cur.step * kPos;
                lim = cur.L - t0 < kPos ? (cur.L > t0 ? cur.L - t0 : 0) : kPos;
                h = cur.h;
                const bool there_too = lane < 8 && line.seen(cur, t0 + lane * 16);
                if (there_too) {
                    phys = kv8_block(p.c, cur.b, (t0 + lane * 16) >> p.c.bs_log2);
                    if (phys < 0) flag(p.a.status, kStatusBounds);
                }
                const uint32_t some = __ballot_sync(0xFFFFFFFFu, there_too);
                lim |= (some ? __ffs(some) - 1 : 0) << 12;      // 16 of them a block
                item_ends = ++cur.step >= cur.steps;
                if (item_ends) line.next_item(cur);
            };
            bool ok = true;
            if (steps) look(true);
            for (uint32_t tile = 0; tile < steps; ++tile) {
                const int now = phys, now_h = h, now_lim = lim;
                const bool first = fresh;
                look(tile + 1 < steps);
                float ks = 1.0f, vs = 1.0f;
                if (now >= 0) {
                    const int64_t unit = (int64_t)now * p.c.heads + now_h;
                    ks = __ldg(p.c.k_scale + unit);
                    vs = __ldg(p.c.v_scale + unit);
                    kv8_check_scale(ks, p.a.status);
                    kv8_check_scale(vs, p.a.status);
                }
                if (first) e0 = sum_scale(__shfl_sync(0xFFFFFFFFu, vs, 0));
                // lane x < boxes copies box x: the block of its first 16 positions
                const int mine = __shfl_sync(0xFFFFFFFFu, now, (lane * (box / 16)) & 7);
                const bool copy = lane < boxes && mine >= 0;
                const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, copy));
                const int row = copy ? (mine * p.c.heads + now_h) << p.c.bs_log2 : 0;
#pragma unroll
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    if (tile >= 1) ok = wait_warp(kLEmpty + kv, (tile - 1) & 1);
                    if (!ok) break;
                    if (lane == 0) tc::mbar_expect_tx(bars + kLFull + kv, n * box * D);
                    __syncwarp();
                    if (copy)
                        tc::tma_load_2d(smem + S::codes + kv * kPos * D + lane * box * D, kv ? &vmap : &kmap, 0, row, bars + kLFull + kv);
                    if (kv == 0) {     // the scales, while the codes are under way
                        const int ev = now >= 0 ? (int)(__float_as_uint(vs) >> 23) - 127 : e0;
                        high = (high && !first) || __any_sync(0xFFFFFFFFu, ev - e0 > kSpread);
                        const bool apart = high || __any_sync(0xFFFFFFFFu, e0 - ev > kSpread);
                        if (lane < 8) {
                            sc[(tile & 7) * 8 + lane] = make_float2(ks, (float)ev);
                            sg[(tile & 7) * 8 + lane] = apart ? 0.0f : exp2_int(e0 - ev);
                        }
                        if (lane == 0) lims[tile & 7] = now_lim;
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bars + kLFull + kv);
                    __syncwarp();
                    ++issued;
                }
                if (!ok) break;
            }
            // loads that nobody waits for any more still land in this CTA's memory
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t done = (issued + 1 - kv) / 2;
                if (done) tc::mbar_wait(bars + kLFull + kv, (done - 1) & 1);
            }
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------------------ every tcgen05.mma of the CTA
            constexpr uint32_t idesc_s = tc::idesc_f16_f32(128, kPos);
            constexpr uint32_t idesc_o = tc::idesc_f16_f32(128, D, false, true);
            const uint64_t dq = tc::desc_sw128(tc::smem_u32(smem + S::q)), dk = tc::desc_sw128(tc::smem_u32(smem + S::k));
            const uint64_t dv = tc::desc_mn_sw128(tc::smem_u32(smem + S::v), S::kPanel, 1024);
            const uint32_t tmem0 = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            uint32_t tile = 0, q_phase = 0, p_phase = 0;
            bool ok = true;
            auto scores = [&](int t, int q, uint32_t st) {      // S_t = Q_q K^T
                const uint64_t a = tc::desc_at(dq, q * S::kTile), b = tc::desc_at(dk, st * S::kTile);
#pragma unroll 1
                for (int x = 0; x < S::kPanels; ++x) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t off = x * S::kPanel + y * 32;
                        tc::mma_f16(tmem0 + t * 128, tc::desc_at(a, off), tc::desc_at(b, off), idesc_s, x + y > 0);
                    }
                }
            };
            auto outputs = [&](int t, uint32_t st, bool more) {   // O_t += P_t V
                const uint64_t b = tc::desc_at(dv, st * S::kTile);
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        tc::mma_f16_ta(tmem0 + kColO + t * D, tmem0 + t * 128 + x * 32 + y * 8, tc::desc_at(b, (x * 4 + y) * 2048),
                                       idesc_o, more || x + y > 0);
                }
            };
            int pair = cur.pair, head = cur.h, step = cur.step, todo_all = piece_steps;
            while (todo_all > 0 && ok) {
                int todo, tiles;
                {
                    line.load(cur, pair, nullptr);
                    todo = cur.steps - step < todo_all ? cur.steps - step : todo_all;
                    tiles = cur.rows > kTileRows ? 2 : 1;
                    todo_all -= todo;
                    cur.h = head;
                    line.next_item(cur);
                    pair = cur.pair;
                    head = cur.h;
                    step = 0;
                }
                todo = __shfl_sync(0xFFFFFFFFu, todo, 0);
                tiles = __shfl_sync(0xFFFFFFFFu, tiles, 0);
                ok = wait_warp(kQ, q_phase);
                q_phase ^= 1;
                if (tiles == 1) {
                    // steps alternate between the two places; a step's outputs come two steps later
                    for (int i = 0; i < todo + 2 && ok; ++i, ++tile) {
                        const int t = i & 1;
                        const uint32_t st = tile & 1;            // stage of step i, and of step i - 2
                        const bool out = i >= 2, in = i < todo;
                        if (!out && !in) continue;
                        ok = wait_all(in ? kKFull + (int)st : -1, (tile >> 1) & 1u, out ? kVFull + (int)st : -1, ((tile - 2) >> 1) & 1u,
                                      out ? kP + t : -1, (p_phase >> t) & 1u);
                        if (!ok) break;
                        if (out) p_phase ^= 1u << t;
                        tc::fence_after_sync();
                        if (tc::elect_one()) {
                            if (out) {
                                outputs(t, st, i >= 4);
                                tc::mma_commit(bars + kVEmpty + st);
                            }
                            if (in) {
                                scores(t, 0, st);
                                tc::mma_commit(bars + kS + t);
                                tc::mma_commit(bars + kKEmpty + st);
                            }
                        }
                        __syncwarp();
                    }
                    tile -= 2;                                   // there is nothing behind the last step
                } else
                for (int i = 0; i <= todo && ok; ++i) {
                    const uint32_t st = tile & 1, prev = st ^ 1;     // stage of tile i, and of tile i - 1
                    const bool out = i > 0, in = i < todo;
                    for (int t = 0; t < 2 && ok; ++t) {
                        if (t == 0)
                            ok = wait_all(in ? kKFull + (int)st : -1, (tile >> 1) & 1u, out ? kVFull + (int)prev : -1, ((tile - 1) >> 1) & 1u,
                                          out ? kP : -1, p_phase & 1u);
                        else if (out) ok = wait_warp(kP + 1, p_phase >> 1);
                        if (!ok) break;
                        if (out) p_phase ^= 1u << t;
                        tc::fence_after_sync();
                        if (tc::elect_one()) {
                            if (out) {
                                outputs(t, prev, i > 1);
                                if (t == 1) tc::mma_commit(bars + kVEmpty + prev);
                            }
                            if (in) {
                                scores(t, t, st);
                                tc::mma_commit(bars + kS + t);
                                if (t == 1) tc::mma_commit(bars + kKEmpty + st);
                            }
                        }
                        __syncwarp();
                    }
                    if (in) ++tile;
                }
                if (ok && tc::elect_one()) tc::mma_commit(bars + kO);
                __syncwarp();
            }
            if (!ok) {
                // the products already issued still write: a last commit, waited for with the full limit
                if (tc::elect_one()) tc::mma_commit(bars + kDrain);
                __syncwarp();
                tc::mbar_wait(bars + kDrain, 0);
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// Four channels of a merged row, and its logarithm of the sum.
template <int D>
__device__ __forceinline__ void store_row(const Params& p, int b, int h, int row, int q4, const float4& s, float m, float M, float l) {
    const int j = row / p.G, g = row - j * p.G;
    const int64_t at = ((int64_t)b * p.a.q.T + j) * p.a.q.H + h * p.G + g;
    // 2^(M - m) / l in two factors: the first stays a normal number
    const float f = l == 0.0f ? 0.0f : ex2(fmaxf(M - m, -100.0f)) / l, f2 = ex2(fminf(M - m + 100.0f, 0.0f));
    const float x = s.x * f2 * f, y = s.y * f2 * f, z = s.z * f2 * f, u = s.w * f2 * f;
    uint32_t w[2];
    if (p.a.q.is_bf16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x, y), b2 = __floats2bfloat162_rn(z, u);
        memcpy(&w[0], &a, 4);
        memcpy(&w[1], &b2, 4);
    } else {
        const __half2 a = __floats2half2_rn(x, y), b2 = __floats2half2_rn(z, u);
        memcpy(&w[0], &a, 4);
        memcpy(&w[1], &b2, 4);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.a.out) + at * D + q4 * 4) = make_uint2(w[0], w[1]);
    if (p.a.lse && q4 == 0) p.a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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
    store_row<D>(p, desc[0], desc[1], desc[2] + row, q4, s, m, M, l);
}

// The same for few items, each in many pieces: blockIdx.x counts the items that
// were cut; a lane is a row, warp w takes the parts w, w + 16, .. in this order
// and the first warp adds the sixteen up.  One head with 32 rows over 24,415
// positions, 148 parts: 67.2 us with the kernel above, 23.0 with this; with 256
// rows over 131,072 positions 93.7 and 44.5.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) k_kv8_prefill_combine_few(const __grid_constant__ Params p) {
    static_assert(kMaxCtas <= kMergeWarps * 32, "a thread a piece");
    __shared__ float4 acc[kMergeWarps][32];
    __shared__ float stat[kMergeWarps][3][32];
    __shared__ int starts[kMergeWarps], found[2];
    pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = blockIdx.y;
    auto desc = [&](int x) {
        return reinterpret_cast<const int*>(p.a.part + ((int64_t)x * 2 + 1) * Part<D>::kFloats + Part<D>::kDesc);
    };
    const int own = tid < p.ctas ? desc(tid)[4] : 0;
    const uint32_t cut = __ballot_sync(0xFFFFFFFFu, own >= 2);
    if (lane == 0) starts[warp] = __popc(cut);
    if (tid == 0) found[0] = -1;
    __syncthreads();
    const int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? starts[lane] : 0) + __popc(cut & ((1u << lane) - 1));
    if (own >= 2 && before == (int)blockIdx.x) found[0] = tid, found[1] = own;
    __syncthreads();
    const int x = found[0], parts = found[1];
    if (x < 0) return;
    const int* item = desc(x);
    const int rows = item[3], row = blockIdx.z * 32 + lane;
    if ((int)blockIdx.z * 32 >= rows) return;
    auto part = [&](int i) { return p.a.part + ((int64_t)(x + i) * 2 + (i == 0 ? 1 : 0)) * Part<D>::kFloats; };
    float m = kNone, M = kNone, l = 0.0f;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row < rows) {
#pragma unroll 8
        for (int i = warp; i < parts; i += kMergeWarps) {
            const float* s3 = part(i) + Part<D>::kStats + row * 3;
            m = fmaxf(m, s3[0]);
            M = fmaxf(M, s3[2]);
        }
#pragma unroll 4
        for (int i = warp; i < parts; i += kMergeWarps) {
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
    }
    acc[warp][lane] = s;
    stat[warp][0][lane] = m, stat[warp][1][lane] = l, stat[warp][2][lane] = M;
    __syncthreads();
    if (warp || row >= rows) return;
    for (int i = 1; i < kMergeWarps; ++i) {
        m = fmaxf(m, stat[i][0][lane]);
        M = fmaxf(M, stat[i][2][lane]);
    }
    l = 0.0f;
    s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < kMergeWarps; ++i) {
        const float4 v = acc[i][lane];
        l += stat[i][1][lane] * ex2(stat[i][0][lane] - m);
        const float f = ex2(stat[i][2][lane] - M);
        s.x += v.x * f;
        s.y += v.y * f;
        s.z += v.z * f;
        s.w += v.w * f;
    }
    store_row<D>(p, item[0], item[1], item[2] + row, q4, s, m, M, l);
}

template <int D>
cudaError_t launch(const Params& p, cudaStream_t st) {
    using S = Smem<D>;
    static_assert(S::bytes <= 227 * 1024, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(k_kv8_prefill<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
    if (e != cudaSuccess) return e;
    CUtensorMap kmap, vmap;
    const int box = p.c.bs() < kPos ? p.c.bs() : kPos;
    if (!kv8_row_map(&kmap, p.c, p.c.k, box, false) || !kv8_row_map(&vmap, p.c, p.c.v, box, false)) return cudaErrorNotSupported;
    e = launch_pdl(k_kv8_prefill<D>, p.ctas, kThreads, S::bytes, st, p, kmap, vmap);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)p.c.batch * p.c.heads * p.row_blocks;
    if (items * kFewItems <= p.ctas) {
        const int64_t rows = (int64_t)p.a.q.T * p.G;
        return launch_pdl(k_kv8_prefill_combine_few<D>, dim3((unsigned)items, D / 4, (unsigned)((rows < kRows ? rows : kRows) + 31) / 32),
                          kMergeWarps * 32, 0, st, p);
    }
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
    const uint32_t tries = wait_limit();
    p.wait_limit = tries < 1u << 28 ? tries * 16 : 0xFFFFFFFFu;   // looks of 4 us, not 65
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    p.ctas = sms < kMaxCtas ? sms : kMaxCtas;
    return c.dim == 64 ? launch<64>(p, st) : launch<128>(p, st);
}

}  // namespace csa2
