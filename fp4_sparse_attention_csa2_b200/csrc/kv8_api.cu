// Host side of the csa2_kv8_* calls: argument checks, workspace layout and
// dispatch.  Every call validates on the host, then only enqueues work.
#include <cmath>

#include "abi_checks.h"
#include "kernels.h"
#include "kv8.cuh"

using namespace csa2;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int kMostSel = 2048;
constexpr int kMostScoreBlocks = 1 << 20;  // the selection's map of chosen blocks in shared memory

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

csa2_status check_cache(const csa2_kv8_cache* c) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !c->seq_lens) return CSA2_ERR_INVALID_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_bounds, 16)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(c->block_table, 4) || !aligned(c->seq_lens, 4))
        return CSA2_ERR_INVALID_ARG;
    if (c->batch < 1 || c->batch > 65535 || c->max_blocks < 1 || c->n_blocks < 1) return CSA2_ERR_INVALID_ARG;
    if (c->n_kv_heads < 1 || c->n_kv_heads > 32767 || c->head_dim < 1) return CSA2_ERR_INVALID_ARG;
    if (c->block_size != 16 && c->block_size != 32 && c->block_size != 64 && c->block_size != 128)
        return CSA2_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return CSA2_ERR_UNSUPPORTED;
    if (!c->block_table && (int64_t)c->batch * c->max_blocks > c->n_blocks) return CSA2_ERR_INVALID_ARG;
    if (c->n_blocks >= kMaxRows || c->n_blocks * c->n_kv_heads >= kMaxRows ||
        c->n_blocks * c->n_kv_heads * c->block_size >= kMaxRows)
        return CSA2_ERR_UNSUPPORTED;
    if ((int64_t)c->max_blocks * c->block_size > (int64_t)1 << 30) return CSA2_ERR_UNSUPPORTED;
    return CSA2_OK;
}

DevKv8 dev_kv8(const csa2_kv8_cache* c) {
    DevKv8 d;
    d.k = c->k_codes;
    d.v = c->v_codes;
    d.k_scale = c->k_scale;
    d.v_scale = c->v_scale;
    d.k_bounds = c->k_bounds;
    d.table = c->block_table;
    d.seq_lens = c->seq_lens;
    d.batch = c->batch;
    d.max_blocks = c->max_blocks;
    d.bs_log2 = c->block_size == 16 ? 4 : c->block_size == 32 ? 5 : c->block_size == 64 ? 6 : 7;
    d.heads = c->n_kv_heads;
    d.dim = c->head_dim;
    d.n_blocks = c->n_blocks;
    return d;
}

// Workspace: status word (256 B) | attention partials | block scores.
struct Layout {
    size_t part, scores, total;
};

bool make_layout(const csa2_kv8_cache* c, int T, int H, int n_sel, Layout* L) {
    if (check_cache(c) != CSA2_OK || T < 1 || H < 1 || H % c->n_kv_heads || n_sel < 0) return false;
    if ((int64_t)T * H >= kMaxRows || (int64_t)c->batch * T * H >= kMaxRows) return false;
    size_t off = 256;
    L->part = off;
    const bool wide = (int64_t)T * (H / c->n_kv_heads) > kKv8StreamRows;
    const size_t stream = kv8_attn_part_floats(c->head_dim), prefill = kv8_prefill_part_floats(c->head_dim);
    off += (wide && prefill > stream ? prefill : stream) * sizeof(float);
    off = (off + 255) / 256 * 256;
    L->scores = off;
    if (n_sel) off += (size_t)c->batch * T * c->n_kv_heads * c->max_blocks * sizeof(float);
    L->total = (off + 255) / 256 * 256;
    return true;
}

template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

csa2_status cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

// The arguments every query call shares; fills q and the workspace layout.
csa2_status check_query(const csa2_kv8_cache* c, const void* q, csa2_dtype q_dtype, int64_t stride_b,
                        int64_t stride_t, int T, int H, const int32_t* n_q, int n_sel, void* ws, size_t ws_bytes,
                        Kv8Query* out, Layout* L) {
    const csa2_status s = check_cache(c);
    if (s != CSA2_OK) return s;
    if (!q || !aligned(q, 16) || !aligned(n_q, 4) || stride_b % 8 || stride_t % 8) return CSA2_ERR_INVALID_ARG;
    if (q_dtype != CSA2_BF16 && q_dtype != CSA2_F16) return CSA2_ERR_INVALID_ARG;
    if (!make_layout(c, T, H, n_sel, L)) return CSA2_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 16) || ws_bytes < L->total) return CSA2_ERR_INVALID_ARG;
    out->q = q;
    out->is_bf16 = q_dtype == CSA2_BF16;
    out->stride_b = stride_b;
    out->stride_t = stride_t;
    out->n_q = n_q;
    out->T = T;
    out->H = H;
    return CSA2_OK;
}

csa2_status attention(const csa2_kv8_cache* c, const Kv8Query& q, const int32_t* block_idx, int n_sel, int window,
                      float sm_scale, void* out, float* lse, void* ws, const Layout& L, void* stream) {
    Kv8Attn a;
    a.q = q;
    a.block_idx = block_idx;
    a.n_sel = n_sel;
    a.window = window;
    a.sm_scale = sm_scale > 0.0f ? sm_scale : 1.0f / std::sqrt((float)c->head_dim);
    a.out = out;
    a.lse = lse;
    a.part = at<float>(ws, L.part);
    a.status = at<uint32_t>(ws, 0);
    const DevKv8 d = dev_kv8(c);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(kv8_streams(d, a) ? launch_kv8_attn(d, a, st) : launch_kv8_prefill(d, a, st));
}

}  // namespace

extern "C" {

size_t csa2_kv8_workspace_bytes(const csa2_kv8_cache* cache, int T, int H, int n_sel) {
    CSA2_RANGE("csa2_kv8_workspace_bytes");
    Layout L;
    return make_layout(cache, T, H, n_sel, &L) ? L.total : 0;
}

csa2_status csa2_kv8_append(const csa2_kv8_cache* cache, const void* k_new, const void* v_new, csa2_dtype dtype,
                            int64_t stride_b, int64_t stride_t, int T, const int32_t* start_pos,
                            const int32_t* n_new, void* ws, void* stream) {
    CSA2_RANGE("csa2_kv8_append");
    const csa2_status s = check_cache(cache);
    if (s != CSA2_OK) return s;
    if (T == 0) return CSA2_OK;   // nothing to append, and tensors without rows have no address
    if (!k_new || !v_new || !start_pos || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(start_pos, 4) ||
        !aligned(n_new, 4) || !aligned(ws, 16))
        return CSA2_ERR_INVALID_ARG;
    if (dtype != CSA2_BF16 && dtype != CSA2_F16 && dtype != CSA2_F32) return CSA2_ERR_INVALID_ARG;
    if (stride_b % 8 || stride_t % 8 || T < 0 || T > 1 << 30) return CSA2_ERR_INVALID_ARG;
    return cuda_status(launch_kv8_append(dev_kv8(cache), k_new, v_new, dtype, stride_b, stride_t, start_pos, n_new, T,
                                         static_cast<uint32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

csa2_status csa2_kv8_read(const csa2_kv8_cache* cache, const int32_t* start_pos, const int32_t* n_rows, int T,
                          void* k_out, void* v_out, csa2_dtype dtype, void* ws, void* stream) {
    CSA2_RANGE("csa2_kv8_read");
    const csa2_status s = check_cache(cache);
    if (s != CSA2_OK) return s;
    if (T == 0) return CSA2_OK;
    if (!k_out || !v_out || !start_pos || !aligned(k_out, 32) || !aligned(v_out, 32) || !aligned(start_pos, 4) ||
        !aligned(n_rows, 4) || !aligned(ws, 16))
        return CSA2_ERR_INVALID_ARG;
    if (dtype != CSA2_BF16 && dtype != CSA2_F16 && dtype != CSA2_F32) return CSA2_ERR_INVALID_ARG;
    if (T < 0 || T > 1 << 30) return CSA2_ERR_INVALID_ARG;
    return cuda_status(launch_kv8_read(dev_kv8(cache), start_pos, n_rows, T, k_out, v_out, dtype,
                                       static_cast<uint32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

csa2_status csa2_kv8_attn(const csa2_kv8_cache* cache, const void* q, csa2_dtype q_dtype, int64_t stride_b,
                          int64_t stride_t, int T, int H, const int32_t* n_q, int window, float sm_scale, void* out,
                          float* lse, void* ws, size_t ws_bytes, void* stream) {
    CSA2_RANGE("csa2_kv8_attn");
    Kv8Query k;
    Layout L;
    const csa2_status s = check_query(cache, q, q_dtype, stride_b, stride_t, T, H, n_q, 0, ws, ws_bytes, &k, &L);
    if (s != CSA2_OK) return s;
    if (!out || !aligned(out, 16) || !aligned(lse, 4) || window < 0) return CSA2_ERR_INVALID_ARG;
    if (window >= (int64_t)cache->max_blocks * cache->block_size) window = 0;   // no position is outside it
    return attention(cache, k, nullptr, 0, window, sm_scale, out, lse, ws, L, stream);
}

csa2_status csa2_kv8_select_blocks(const csa2_kv8_cache* cache, const void* q, csa2_dtype q_dtype, int64_t stride_b,
                                   int64_t stride_t, int T, int H, const int32_t* n_q, int n_sel, int n_first,
                                   int n_recent, int32_t* block_idx, void* ws, size_t ws_bytes, void* stream) {
    CSA2_RANGE("csa2_kv8_select_blocks");
    if (n_sel < 1 || n_sel > kMostSel || n_first < 0 || n_recent < 0 || n_first > n_sel || n_recent > n_sel - n_first)
        return CSA2_ERR_INVALID_ARG;
    Kv8Query k;
    Layout L;
    const csa2_status s = check_query(cache, q, q_dtype, stride_b, stride_t, T, H, n_q, n_sel, ws, ws_bytes, &k, &L);
    if (s != CSA2_OK) return s;
    if (!cache->k_bounds || !block_idx || !aligned(block_idx, 4)) return CSA2_ERR_INVALID_ARG;
    if (cache->max_blocks > kMostScoreBlocks) return CSA2_ERR_UNSUPPORTED;
    return cuda_status(launch_kv8_select(dev_kv8(cache), k, n_sel, n_first, n_recent, block_idx,
                                         at<float>(ws, L.scores), at<uint32_t>(ws, 0),
                                         static_cast<cudaStream_t>(stream)));
}

csa2_status csa2_kv8_block_attn(const csa2_kv8_cache* cache, const void* q, csa2_dtype q_dtype, int64_t stride_b,
                                int64_t stride_t, int T, int H, const int32_t* n_q, const int32_t* block_idx,
                                int n_sel, float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                                void* stream) {
    CSA2_RANGE("csa2_kv8_block_attn");
    Kv8Query k;
    Layout L;
    const csa2_status s = check_query(cache, q, q_dtype, stride_b, stride_t, T, H, n_q, 0, ws, ws_bytes, &k, &L);
    if (s != CSA2_OK) return s;
    if (!block_idx || !aligned(block_idx, 4) || n_sel < 1) return CSA2_ERR_INVALID_ARG;
    if (!out || !aligned(out, 16) || !aligned(lse, 4)) return CSA2_ERR_INVALID_ARG;
    return attention(cache, k, block_idx, n_sel, 0, sm_scale, out, lse, ws, L, stream);
}

}  // extern "C"
