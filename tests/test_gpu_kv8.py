"""The 8-bit key / value cache on the GPU against the 64-bit reference of
kv8_ref.py: codes, scales, bounds and chosen blocks bit-exact, attention within
the bounds derived there."""
import math

import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa2_b200 as csa2
import kv8_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def both_caches(B, heads, D, bs, max_blocks, seed=0, paged=True, spare=3):
    """A device cache and its reference with the same (scattered) block table,
    every byte of the codes 0x7F / 0xFF first: what nobody wrote must not enter."""
    rng = np.random.default_rng(seed)
    n_blocks = B * max_blocks + (spare if paged else 0)
    table = rng.permutation(n_blocks)[:B * max_blocks].reshape(B, max_blocks).astype(np.int32) if paged else None
    dev = csa2.KV8Cache(B, heads, D, max_blocks, [0] * B, block_size=bs, n_blocks=n_blocks, block_table=table)
    r = ref.Cache(B, heads, D, max_blocks, bs, n_blocks, table)
    for t in (dev.k, dev.v):
        t.fill_(0x7F)
        t[::2] = 0xFF
    dev.k_scale.fill_(float("nan"))
    dev.v_scale.fill_(float("nan"))
    r.k[:], r.v[:] = dev.k.cpu().numpy(), dev.v.cpu().numpy()
    return dev, r


def fill(dev, r, lens, seed=1, dtype=torch.bfloat16, spread=1.0):
    """Rows of every sequence through one append; per-block magnitudes vary by 2^spread."""
    g = torch.Generator().manual_seed(seed)
    B, T = dev.batch, max(max(lens), 1)
    x = [torch.randn(B, T, dev.n_kv_heads, dev.head_dim, generator=g) for _ in range(2)]
    for a in x:
        nb = (T + dev.block_size - 1) // dev.block_size
        e = torch.round(torch.randn(B, nb, dev.n_kv_heads, 1, generator=g) * spread)
        a *= torch.exp2(e).repeat_interleave(dev.block_size, 1)[:, :T]
    x = [a.to(dtype) for a in x]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    csa2.kv8_append(dev, x[0].cuda(), x[1].cuda(), i32([0] * B), n_new=i32(lens), ws=ws)
    assert csa2.read_device_status(ws) == csa2.OK
    for b in range(B):
        if lens[b]:
            r.append(b, 0, x[0][b, :lens[b]].double().numpy(), x[1][b, :lens[b]].double().numpy())
    dev.seq_lens.copy_(i32(lens))


def same_cache(dev, r):
    for name in ("k", "v"):
        assert np.array_equal(getattr(dev, name).cpu().numpy(), getattr(r, name)), name
    for name, want in (("k_scale", r.ks), ("v_scale", r.vs)):
        got = getattr(dev, name).cpu().numpy()
        assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(got)]), name
        assert np.all(want[np.isnan(got)] == 0), name
    assert np.array_equal(dev.k_bounds.cpu().numpy(), r.kb)


def workspace(dev, T, H, n_sel=0):
    ws = torch.empty(csa2.kv8_workspace_bytes(dev, T, H, n_sel), dtype=torch.uint8, device="cuda")
    csa2.workspace_init(ws)
    return ws


# ---------------------------------------------------------------- append and read
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,bs", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128)])
def test_append_in_pieces(dtype, D, bs):
    B, heads, mb = 3, 2, 6 if bs < 128 else 3
    dev, r = both_caches(B, heads, D, bs, mb, seed=D + bs)
    g = torch.Generator().manual_seed(bs)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    at = [0, 5, bs - 1]
    for b in (1, 2):   # sequences that begin inside a block still own the rows before it
        x = torch.randn(2, 1, at[b], heads, D, generator=g).to(DT[dtype])
        rows = [torch.zeros(B, at[b], heads, D, dtype=DT[dtype]) for _ in range(2)]
        rows[0][b], rows[1][b] = x[0, 0], x[1, 0]
        n = [0] * B
        n[b] = at[b]
        csa2.kv8_append(dev, rows[0].cuda(), rows[1].cuda(), i32([0] * B), n_new=i32(n), ws=ws)
        r.append(b, 0, x[0, 0].double().numpy(), x[1, 0].double().numpy())
    for step, T in enumerate((1, 1, 3, bs, 1, 2 * bs + 1, 7)):
        # magnitudes that grow, shrink and jump, so that held blocks are rescaled by several powers of two
        k, v = (torch.randn(B, T, heads, D, generator=g) * 4.0 ** ((step * 5) % 7 - 3) for _ in range(2))
        k, v = k.to(DT[dtype]), v.to(DT[dtype])
        n = [T, max(0, T - step), T]
        n = [min(n[b], mb * bs - at[b]) for b in range(B)]
        csa2.kv8_append(dev, k.cuda(), v.cuda(), i32(at), n_new=i32(n), ws=ws)
        for b in range(B):
            if n[b]:
                r.append(b, at[b], k[b, :n[b]].double().numpy(), v[b, :n[b]].double().numpy())
            at[b] += n[b]
    assert csa2.read_device_status(ws) == csa2.OK
    same_cache(dev, r)


@pytest.mark.parametrize("paged", [True, False])
def test_append_from_a_fused_projection(paged):
    B, T, H, heads, D = 2, 9, 4, 2, 64
    dev, r = both_caches(B, heads, D, 16, 4, paged=paged)
    qkv = torch.randn(B, T, H + 2 * heads, D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    k, v = qkv[:, :, H:H + heads], qkv[:, :, H + heads:]
    csa2.kv8_append(dev, k, v, i32([0, 30]))
    # sequence 1 starts inside a block that nobody filled: only sequence 0 has a defined scale
    r.append(0, 0, k[0].cpu().double().numpy(), v[0].cpu().double().numpy())
    blk = r.table[0, 0]
    assert np.array_equal(dev.k[blk].cpu().numpy(), r.k[blk])
    assert np.array_equal(dev.v[blk].cpu().numpy(), r.v[blk])
    assert np.array_equal(dev.k_bounds[blk].cpu().numpy(), r.kb[blk])


def test_append_extremes_and_nonfinite():
    dev, r = both_caches(1, 1, 64, 16, 8)
    x = torch.zeros(1, 128, 1, 64)
    x[0, 0:16] = 1e-40                      # below the least scale's grid: zeros
    x[0, 16:32] = 3.3e38
    x[0, 32:48, 0, ::2] = 448.0 * 2.0 ** -120
    x[0, 48:64] = torch.linspace(-448, 448, 64)
    x[0, 64:80] = 448.0000305               # just above: the next power of two
    x[0, 80:96] = torch.tensor([-0.0, 0.0]).repeat(32)
    x[0, 96:112] = torch.randn(16, 1, 64) * 1e-3
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    csa2.kv8_append(dev, x.cuda(), -x.cuda(), i32([0]), ws=ws)
    assert csa2.read_device_status(ws) == csa2.OK
    r.append(0, 0, x[0].double().numpy(), -x[0].double().numpy())
    same_cache(dev, r)
    y = torch.randn(1, 4, 1, 64, generator=torch.Generator().manual_seed(5))
    y[0, 1, 0, 3], y[0, 2, 0, 7], y[0, 3, 0, 9] = math.inf, -math.inf, math.nan
    csa2.kv8_append(dev, y.cuda(), y.cuda(), i32([100]), ws=ws)
    assert csa2.read_device_status(ws) == csa2.ERR_NONFINITE
    assert csa2.read_device_status(ws) == csa2.OK       # sticky until read
    r.append(0, 100, y[0].double().numpy(), y[0].double().numpy())
    same_cache(dev, r)


def test_append_outside_the_cache_is_skipped_and_flagged():
    dev, r = both_caches(2, 1, 64, 16, 2)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x = torch.randn(2, 8, 1, 64, generator=torch.Generator().manual_seed(6))
    csa2.kv8_append(dev, x.cuda(), x.cuda(), i32([-1, 27]), ws=ws)   # before the start; five rows fit
    assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS
    assert np.array_equal(dev.k[r.table[0]].cpu().numpy(), r.k[r.table[0]])
    blk = r.table[1, 1]                                              # a scale nobody set: NaN counts as none
    got = ref.e4m3_value(dev.k[blk, 0, 11:].cpu().numpy()) * float(dev.k_scale[blk, 0])
    s = ref.scale_of(x[1, :5].double().numpy())
    assert np.array_equal(got, ref.e4m3_value(ref.e4m3_encode(x[1, :5, 0].double().numpy() / s)) * s)
    for bad in ([0, 9], [0, -1]):
        csa2.kv8_append(dev, x.cuda(), x.cuda(), i32([0, 0]), n_new=i32(bad), ws=ws)
        assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS
    dev.block_table.fill_(1 << 20)
    before = dev.k.clone()
    csa2.kv8_append(dev, x.cuda(), x.cuda(), i32([0, 0]), ws=ws)
    assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS
    assert torch.equal(before, dev.k)
    csa2.kv8_append(dev, x.cuda(), x.cuda(), i32([0, 0]))            # without a workspace: silently


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 64)])
def test_read(dtype, D, bs):
    B, heads = 3, 3
    dev, r = both_caches(B, heads, D, bs, 4)
    lens = [3 * bs + 5, 1, 2 * bs]
    fill(dev, r, lens)
    T = 2 * bs + 3
    start, n = [bs + 2, 0, 0], [2 * bs + 3, 1, 2 * bs]
    k, v = (torch.full((B, T, heads, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    csa2.kv8_read(dev, i32(start), k, v, n_rows=i32(n), ws=ws)
    assert csa2.read_device_status(ws) == csa2.OK
    for b in range(B):
        for h in range(heads):
            want = r.rows(b, h, np.arange(start[b], start[b] + n[b]))
            for got, w in zip((k, v), want):
                assert torch.equal(got[b, :n[b], h].cpu(), torch.from_numpy(w).to(DT[dtype]))
        assert bool((k[b, n[b]:] == 7).all()) and bool((v[b, n[b]:] == 7).all())
    csa2.kv8_read(dev, i32([4 * bs - 1, -2, 0]), k, v, ws=ws)        # outside: zeros, flagged
    assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS
    assert bool((k[0, 1:] == 0).all()) and bool((v[1, :2] == 0).all())


# ---------------------------------------------------------------- attention
def check_attn(dev, r, q, out, lse, n, sm, visible, lens):
    """Every live row against the reference; `visible(b, j, h, p)`: the positions row (b, j) sees."""
    eps = torch.finfo(q.dtype).eps
    B, T, H, D = q.shape
    G = H // r.heads
    qd = q.double().cpu().numpy()
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        for j in range(n[b]):
            p = lens[b] - n[b] + j
            for h in range(H):
                t = visible(b, j, h // G, p)
                wo, wl, wv, zmax, vmax = r.attend(b, h // G, qd[b, j, h], t, sm)
                bo, bl = ref.bounds(wo, wl, wv, zmax, vmax, len(t), eps)
                if len(t) == 0:
                    assert l[b, j, h] == -math.inf and not o[b, j, h].any()
                    continue
                assert abs(l[b, j, h] - wl) <= bl, (b, j, h, l[b, j, h], wl, bl)
                worst = np.max(np.abs(o[b, j, h] - wo) - bo)
                assert worst <= 0, (b, j, h, worst, np.max(np.abs(o[b, j, h] - wo)))


def attend(dev, r, lens, T, H, n=None, window=0, sm=None, dtype=torch.bfloat16, seed=9, q_scale=1.0):
    D = r.D
    q = (torch.randn(dev.batch, T, H, D, generator=torch.Generator().manual_seed(seed)) * q_scale).to(dtype).cuda()
    out = torch.full_like(q, 5.0)
    lse = torch.full((dev.batch, T, H), 5.0, device="cuda")
    ws = workspace(dev, T, H)
    csa2.kv8_attn(dev, q, out, ws, lse=lse, window=window, n_q=None if n is None else i32(n), sm_scale=sm or 0.0)
    assert csa2.read_device_status(ws) == csa2.OK
    n = [T] * dev.batch if n is None else n
    check_attn(dev, r, q, out, lse, n, sm or 1 / math.sqrt(D),
               lambda b, j, h, p: np.arange(max(0, p - window + 1) if window else 0, p + 1), lens)
    for b in range(dev.batch):
        assert bool((out[b, n[b]:] == 5).all()) and bool((lse[b, n[b]:] == 5).all())
    return q, out, lse


# heads, group, D, block, lengths, T
SHAPES = [
    (2, 1, 64, 16, [1, 17, 40], 1), (1, 8, 128, 64, [1000], 1), (4, 5, 128, 32, [63, 64, 65], 1),
    (3, 16, 64, 128, [300, 129], 1), (1, 20, 128, 64, [200, 33], 1), (2, 4, 128, 64, [70, 500], 4),
    (2, 8, 128, 16, [90, 200], 3), (1, 3, 64, 64, [700, 91], 37), (2, 16, 128, 128, [260], 5), (1, 64, 128, 64, [150], 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,G,D,bs,lens,T", SHAPES)
def test_attn(heads, G, D, bs, lens, T, dtype):
    T = min(T, min(lens))
    mb = (max(lens) + bs - 1) // bs + 1
    dev, r = both_caches(len(lens), heads, D, bs, mb)
    fill(dev, r, lens)
    attend(dev, r, lens, T, heads * G, dtype=DT[dtype])


@pytest.mark.parametrize("window", [1, 15, 16, 100, 1000])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_attn_window(window, T):
    lens = [40, 257, 513]
    dev, r = both_caches(3, 2, 128, 64, 9)
    fill(dev, r, lens)
    attend(dev, r, lens, T, 8, window=window)


def test_attn_padded_batch_and_rows_that_see_nothing():
    # lengths 0 and 1; a padded batch; more query rows than positions (the first see nothing)
    lens, n = [0, 1, 3, 200, 90], [0, 1, 5, 7, 3]
    dev, r = both_caches(5, 2, 128, 32, 8)
    fill(dev, r, lens)
    attend(dev, r, lens, 7, 8, n=n)
    attend(dev, r, lens, 7, 8, n=n, window=2)
    attend(dev, r, lens, 7, 8, n=[0] * 5)


@pytest.mark.parametrize("q_scale,spread", [(2.0 ** -60, 1.0), (2.0 ** 20, 0.0), (1.0, 12.0), (6.0, 3.0)])
def test_attn_magnitudes(q_scale, spread):
    # tiny and large queries, value scales that differ by many powers of two between blocks
    lens = [777]
    dev, r = both_caches(1, 2, 128, 64, 13)
    fill(dev, r, lens, spread=spread)
    if spread > 4:   # keys of one size, values of many: the keys' own scales aside
        k = dev.k_scale.clone()
        dev.k_scale.copy_(torch.where(torch.isnan(k), k, torch.full_like(k, 2.0 ** -6)))
        r.ks[:] = 2.0 ** -6
    attend(dev, r, lens, 1, 16, q_scale=q_scale, sm=2.0 ** -20 if q_scale > 8 else None)


def test_attn_contiguous_cache_without_bounds_and_a_window_beyond_it():
    lens, D = [200, 77], 128
    dev = csa2.KV8Cache(2, 2, D, 5, [0, 0], block_size=64, bounds=False)
    r = ref.Cache(2, 2, D, 5, 64, 10, None)
    x = [torch.randn(2, 200, 2, D, generator=torch.Generator().manual_seed(i)).bfloat16() for i in range(2)]
    csa2.kv8_append(dev, x[0].cuda(), x[1].cuda(), i32([0, 0]), n_new=i32(lens))
    for b in range(2):
        r.append(b, 0, x[0][b, :lens[b]].double().numpy(), x[1][b, :lens[b]].double().numpy())
    dev.seq_lens.copy_(i32(lens))
    for T in (1, 20):
        for window in (0, 320, 2 ** 31 - 1):
            attend(dev, r, lens, T, 8, window=window)
    idx = torch.zeros(2, 1, 2, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(csa2.CSA2Error):
        csa2.kv8_select_blocks(dev, x[0][:, :1].repeat(1, 1, 4, 1).cuda(), idx, workspace(dev, 1, 8, 4))


@pytest.mark.parametrize("T", [1, 12])
def test_many_sequences(T):
    # more sequences than a warp has lanes, some of them empty: every call's split of the batch
    rng = np.random.default_rng(T)
    lens = [int(x) for x in rng.integers(T, 90, 75)]
    for b in (0, 31, 32, 74):
        lens[b] = T
    dev, r = both_caches(75, 2, 64, 16, 7)
    fill(dev, r, lens)
    n = [int(x) for x in rng.integers(0, T + 1, 75)]
    n[1], n[2] = T, 0
    attend(dev, r, lens, T, 8, n=n)
    q = torch.randn(75, T, 8, 64, generator=torch.Generator().manual_seed(8)).half().cuda()
    idx = torch.full((75, T, 2, 3), -7, dtype=torch.int32, device="cuda")
    ws = workspace(dev, T, 8, 3)
    out, lse = torch.zeros_like(q), torch.zeros(75, T, 8, device="cuda")
    csa2.kv8_select_blocks(dev, q, idx, ws, n_first=1, n_q=i32(n))
    check_select(r, q, idx, lens, n, 1, 1)
    csa2.kv8_block_attn(dev, q, idx, out, ws, lse=lse, n_q=i32(n))
    assert csa2.read_device_status(ws) == csa2.OK
    chosen = idx.cpu().numpy()

    def visible(b, j, h, p):
        c = chosen[b, j, h]
        t = (c[c >= 0][:, None] * 16 + np.arange(16)).reshape(-1)
        return t[t <= p]
    check_attn(dev, r, q, out, lse, n, 1 / 8, visible, lens)


def test_attn_strided_query_and_no_lse():
    lens, H, heads, D = [100, 60], 4, 2, 64
    dev, r = both_caches(2, heads, D, 16, 8)
    fill(dev, r, lens)
    fused = torch.randn(2, 3, H + 2 * heads, D, generator=torch.Generator().manual_seed(4)).half().cuda()
    q = fused[:, :, :H]
    out, out2 = torch.zeros(2, 3, H, D, dtype=torch.float16, device="cuda"), torch.zeros(2, 3, H, D, dtype=torch.float16, device="cuda")
    ws = workspace(dev, 3, H)
    csa2.kv8_attn(dev, q, out, ws)
    csa2.kv8_attn(dev, q.contiguous(), out2, ws)
    assert torch.equal(out, out2)


def test_attn_nonfinite_query_stays_in_its_row():
    lens = [500]
    dev, r = both_caches(1, 1, 128, 64, 8)
    fill(dev, r, lens)
    q, out, lse = attend(dev, r, lens, 1, 8)
    q2 = q.clone()
    q2[0, 0, 3, 5], q2[0, 0, 6, 1] = math.nan, math.inf
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    csa2.kv8_attn(dev, q2, out2, workspace(dev, 1, 8), lse=lse2)
    keep = [0, 1, 2, 4, 5, 7]
    assert torch.equal(out[:, :, keep], out2[:, :, keep]) and torch.equal(lse[:, :, keep], lse2[:, :, keep])
    assert bool(out2[0, 0, 3].isnan().all()) and not bool(out2[0, 0, 6].isfinite().all())


def test_attn_same_every_time_and_on_two_streams():
    lens = [3000, 17, 900]
    dev, r = both_caches(3, 2, 128, 64, 47)
    fill(dev, r, lens)
    q = torch.randn(3, 1, 16, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    ws = [workspace(dev, 1, 16) for _ in range(2)]
    want, got = torch.zeros_like(q), [torch.zeros_like(q) for _ in range(2)]
    csa2.kv8_attn(dev, q, want, ws[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            csa2.kv8_attn(dev, q, got[i], ws[i], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)


def test_attn_bad_pages_and_lengths_are_flagged():
    lens = [200]
    dev, r = both_caches(1, 1, 64, 16, 14)
    fill(dev, r, lens)
    q = torch.randn(1, 1, 4, 64).half().cuda()
    out, ws = torch.zeros_like(q), workspace(dev, 1, 4)
    table = dev.block_table.clone()
    for bad in (-1, 1 << 20):
        dev.block_table[0, 3] = bad
        csa2.kv8_attn(dev, q, out, ws)
        assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS
    dev.block_table.copy_(table)
    for bad in (-1, 14 * 16 + 1):
        dev.seq_lens.fill_(bad)
        csa2.kv8_attn(dev, q, out, ws)
        assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS
    dev.seq_lens.fill_(200)
    csa2.kv8_attn(dev, q, out, ws, n_q=i32([2]))
    assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS


def test_attn_wait_that_runs_out():
    lens = [5000]
    dev, r = both_caches(1, 2, 128, 64, 80)
    fill(dev, r, lens)
    q = torch.randn(1, 1, 16, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want, out, ws = torch.zeros_like(q), torch.zeros_like(q), workspace(dev, 1, 16)
    csa2.kv8_attn(dev, q, want, ws)
    csa2.debug_set_wait_limit(0)
    try:
        csa2.kv8_attn(dev, q, out, ws)
    finally:
        csa2.debug_set_wait_limit()
    assert csa2.read_device_status(ws) == csa2.ERR_TIMEOUT
    csa2.kv8_attn(dev, q, out, ws)
    assert csa2.read_device_status(ws) == csa2.OK and torch.equal(out, want)


# ---------------------------------------------------------------- many query rows (the tensor-core kernel)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,G,D,bs,lens,T,window", [
    (1, 8, 128, 64, [400], 100, 0),          # several row blocks, the last not full
    (2, 4, 64, 16, [130, 257, 90], 70, 0),   # ragged, head_dim 64, blocks of 16
    (3, 5, 128, 128, [300, 220], 60, 0),     # groups that do not divide a row block
    (1, 33, 128, 32, [64, 40], 8, 0),
    (2, 8, 128, 64, [1500], 40, 200), (1, 4, 64, 32, [700, 300], 130, 129), (2, 2, 128, 16, [515], 515, 0),
    (1, 1, 128, 64, [33, 2000], 33, 0),
])
def test_attn_many_rows(heads, G, D, bs, lens, T, window, dtype):
    T = min(T, min(lens))
    dev, r = both_caches(len(lens), heads, D, bs, (max(lens) + bs - 1) // bs + 1)
    fill(dev, r, lens)
    attend(dev, r, lens, T, heads * G, window=window, dtype=DT[dtype])


def test_attn_many_rows_padded_and_empty():
    # padded batch; a sequence without rows, one shorter than its rows (the first rows see nothing), length 0
    lens, n = [300, 500, 20, 0, 129], [60, 0, 50, 64, 1]
    dev, r = both_caches(5, 2, 128, 64, 9)
    fill(dev, r, lens)
    for window in (0, 3):
        attend(dev, r, lens, 64, 8, n=n, window=window)
    attend(dev, r, lens, 64, 8, n=[0] * 5)


@pytest.mark.parametrize("q_scale,spread", [(2.0 ** -60, 1.0), (1.0, 7.0), (6.0, 3.0)])
def test_attn_many_rows_magnitudes(q_scale, spread):
    lens = [777]
    dev, r = both_caches(1, 2, 128, 64, 13)
    fill(dev, r, lens, spread=spread)
    k = dev.k_scale.clone()
    dev.k_scale.copy_(torch.where(torch.isnan(k), k, torch.full_like(k, 2.0 ** -6)))
    r.ks[:] = 2.0 ** -6
    attend(dev, r, lens, 24, 8, q_scale=q_scale)


def test_attn_many_rows_zero_values():
    # a block of zero values has the least scale there is and still counts in the sum
    lens, D = [256], 128
    dev, r = both_caches(1, 1, D, 64, 5)
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn(1, 256, 1, D, generator=g), torch.randn(1, 256, 1, D, generator=g)
    v[:, :64] = 0
    v[:, 128:192] = 0
    csa2.kv8_append(dev, k.cuda(), v.cuda(), i32([0]))
    r.append(0, 0, k[0].double().numpy(), v[0].double().numpy())
    dev.seq_lens.fill_(256)
    attend(dev, r, lens, 64, 4)
    attend(dev, r, lens, 1, 4)


def test_attn_many_rows_wait_that_runs_out():
    lens = [900]
    dev, r = both_caches(1, 2, 128, 64, 16)
    fill(dev, r, lens)
    q = torch.randn(1, 100, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want, out, ws = torch.zeros_like(q), torch.zeros_like(q), workspace(dev, 100, 8)
    csa2.kv8_attn(dev, q, want, ws)
    csa2.debug_set_wait_limit(0)
    try:
        csa2.kv8_attn(dev, q, out, ws)
    finally:
        csa2.debug_set_wait_limit()
    assert csa2.read_device_status(ws) == csa2.ERR_TIMEOUT
    csa2.kv8_attn(dev, q, out, ws)
    assert csa2.read_device_status(ws) == csa2.OK and torch.equal(out, want)


# ---------------------------------------------------------------- the same rows of a cache with room for far more
# positions (the kernel for many rows is chosen by how far the cache reaches, not by the lengths), every table entry
# behind the sequences outside the cache
@pytest.fixture
def with_room(monkeypatch):
    near = both_caches

    def far(B, heads, D, bs, max_blocks, *args, **kw):
        dev, r = near(B, heads, D, bs, max_blocks, *args, **kw)
        table = torch.full((B, (1 << 20) // bs), -1, dtype=torch.int32, device="cuda")
        table[:, :max_blocks] = dev.block_table
        return csa2.KV8Cache.wrap(dev.k, dev.v, dev.k_scale, dev.v_scale, dev.seq_lens, dev.k_bounds, table), r
    monkeypatch.setitem(globals(), "both_caches", far)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,G,D,bs,lens,T", [
    (1, 8, 128, 64, [400], 100), (2, 4, 64, 16, [130, 257, 90], 70), (3, 5, 128, 128, [300, 220], 60),
    (1, 33, 128, 32, [64, 40], 8), (2, 2, 128, 16, [515], 515), (1, 1, 128, 64, [33, 2000], 33),
    (1, 4, 64, 32, [5000], 9), (1, 16, 128, 64, [6000], 3), (2, 8, 128, 128, [2600], 33),
])
def test_attn_many_rows_with_room(with_room, heads, G, D, bs, lens, T, dtype):
    test_attn_many_rows(heads, G, D, bs, lens, T, 0, dtype)


@pytest.mark.parametrize("heads,G,D,bs,lens,T,window", [
    (2, 8, 128, 64, [400, 257, 350], 256, 129), (2, 16, 64, 32, [300, 280], 255, 33), (1, 16, 128, 16, [900], 500, 200)])
def test_attn_many_rows_window(with_room, heads, G, D, bs, lens, T, window):
    test_attn_many_rows(heads, G, D, bs, lens, T, window, "bf16")


def test_attn_many_rows_with_room_padded_and_empty(with_room):
    test_attn_many_rows_padded_and_empty()


@pytest.mark.parametrize("q_scale,spread", [(2.0 ** -60, 1.0), (1.0, 7.0), (6.0, 3.0)])
def test_attn_many_rows_with_room_magnitudes(with_room, q_scale, spread):
    test_attn_many_rows_magnitudes(q_scale, spread)


def test_attn_many_rows_with_room_zero_values(with_room):
    test_attn_many_rows_zero_values()


def test_attn_many_rows_with_room_wait_that_runs_out(with_room):
    test_attn_many_rows_wait_that_runs_out()


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("bs,lens,T,G,window", [
    (16, [500, 90], 1, 4, 20), (16, [500, 333], 3, 4, 77), (64, [700], 2, 8, 65), (16, [900, 613], 60, 8, 70),
    (32, [900, 400, 385], 130, 16, 129), (64, [1000, 700], 200, 8, 300), (128, [1000, 999], 260, 8, 200)])
def test_attn_window_with_the_pages_before_it_gone(request, bs, lens, T, G, window, room):
    if room:
        request.getfixturevalue("with_room")
    dev, r = both_caches(len(lens), 2, 128, bs, (max(lens) + bs - 1) // bs)
    fill(dev, r, lens)
    q, out, lse = attend(dev, r, lens, T, 2 * G, window=window)
    for b, L in enumerate(lens):
        gone = max(0, L - T - window + 1) // bs          # blocks that no row sees
        dev.block_table[b, :gone] = -1
        assert gone
    out2, lse2, ws = torch.zeros_like(out), torch.zeros_like(lse), workspace(dev, T, 2 * G)
    csa2.kv8_attn(dev, q, out2, ws, lse=lse2, window=window)
    assert csa2.read_device_status(ws) == csa2.OK
    assert torch.allclose(out2.float(), out.float(), atol=2.0 ** -7, rtol=2.0 ** -7)
    assert torch.allclose(lse2, lse, atol=2.0 ** -12, rtol=2.0 ** -12)


def test_attn_many_rows_nonfinite_bad_pages_and_lengths(with_room):
    lens, T = [500], 40
    dev, r = both_caches(1, 2, 128, 64, 8)
    fill(dev, r, lens)
    q, out, lse = attend(dev, r, lens, T, 16)
    again, ws = torch.zeros_like(out), workspace(dev, T, 16)
    for _ in range(10):
        csa2.kv8_attn(dev, q, again, ws)
        assert torch.equal(again, out)
    q2 = q.clone()
    q2[0, 7, 3, 5], q2[0, 30, 6, 1] = math.nan, math.inf
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    csa2.kv8_attn(dev, q2, out2, ws, lse=lse2)
    assert csa2.read_device_status(ws) == csa2.OK
    keep = torch.ones(1, T, 16, dtype=torch.bool, device="cuda")
    keep[0, 7, 3] = keep[0, 30, 6] = False
    assert bool(out2[~keep].isnan().any(-1).all())
    assert bool(out2[keep].isfinite().all())
    assert torch.allclose(out2[keep].float(), out[keep].float(), atol=2.0 ** -7, rtol=2.0 ** -7)
    table = dev.block_table.clone()
    for bad in (-1, 1 << 20):
        dev.block_table[0, 3] = bad
        csa2.kv8_attn(dev, q, out2, ws)
        assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS
    dev.block_table.copy_(table)
    for n_q, L in (([T + 1], 500), ([-1], 500), (None, -1), (None, (1 << 20) + 1)):
        dev.seq_lens.fill_(L)
        csa2.kv8_attn(dev, q, out2, ws, n_q=None if n_q is None else i32(n_q))
        assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("T", [1, 16, 24])
@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -40, 2.0 ** -15])
def test_attn_zero_keys_and_small_queries(with_room, T, q_scale):
    # the product of the query's and a zero block's scale is below what fp32 holds
    lens, D = [200, 64], 64
    dev, r = both_caches(2, 2, D, 64, 5)
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn(2, 200, 2, D, generator=g), torch.randn(2, 200, 2, D, generator=g)
    k[:, :64] = 0
    k[:, 128:192] = 0
    csa2.kv8_append(dev, k.cuda(), v.cuda(), i32([0, 0]), n_new=i32(lens))
    for b in range(2):
        r.append(b, 0, k[b, :lens[b]].double().numpy(), v[b, :lens[b]].double().numpy())
    dev.seq_lens.copy_(i32(lens))
    for dtype in (torch.bfloat16, torch.float16):
        attend(dev, r, lens, T, 4, q_scale=q_scale, dtype=dtype)


@pytest.mark.parametrize("heads,G,D,bs,lens,T,window", [
    (1, 8, 128, 64, [5000], 1, 0), (2, 3, 64, 16, [4100, 2500], 1, 0), (1, 16, 64, 128, [9000], 2, 0),
    (3, 5, 128, 32, [2100], 3, 0), (1, 1, 128, 64, [30000, 1], 1, 0), (2, 8, 128, 64, [8000], 1, 3000)])
def test_attn_few_items_in_many_pieces(heads, G, D, bs, lens, T, window):
    dev, r = both_caches(len(lens), heads, D, bs, (max(lens) + bs - 1) // bs + 1)
    fill(dev, r, lens)
    attend(dev, r, lens, T, heads * G, window=window)


def test_offsets_beyond_32_bits():
    # codes of more than 4 GiB a side: the sequence's blocks lie at the far end
    heads, D, bs, mb = 8, 128, 64, 5
    n_blocks = (1 << 32) // (heads * D * bs) + 64
    table = np.arange(n_blocks - mb, n_blocks, dtype=np.int32)[::-1].reshape(1, mb).copy()
    z = torch.empty(n_blocks, heads, bs, D, dtype=torch.uint8, device="cuda")
    dev = csa2.KV8Cache.wrap(z, torch.empty_like(z), torch.zeros(n_blocks, heads, device="cuda"),
                             torch.zeros(n_blocks, heads, device="cuda"), i32([0]),
                             k_bounds=torch.zeros(n_blocks, heads, 2, D, dtype=torch.uint8, device="cuda"),
                             block_table=i32(table))
    r = ref.Cache(1, heads, D, mb, bs, mb, np.arange(mb)[None])
    lens = [260]
    fill(dev, r, lens)
    attend(dev, r, lens, 1, 16)
    k, v = (torch.zeros(1, 260, heads, D, dtype=torch.float32, device="cuda") for _ in range(2))
    csa2.kv8_read(dev, i32([0]), k, v)
    for h in range(heads):
        want = r.rows(0, h, np.arange(260))
        assert np.array_equal(k[0, :, h].cpu().numpy(), want[0]) and np.array_equal(v[0, :, h].cpu().numpy(), want[1])
    idx = torch.empty(1, 1, heads, 3, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 16, D, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    csa2.kv8_select_blocks(dev, q, idx, workspace(dev, 1, 16, 3))
    check_select(r, q, idx, lens, [1], 0, 1)


# ---------------------------------------------------------------- selection and the attention over it
def check_select(r, q, idx, lens, n, first, recent):
    qd, got = q.double().cpu().numpy(), idx.cpu().numpy()
    G = q.shape[2] // r.heads
    for b in range(q.shape[0]):
        for j in range(n[b]):
            for h in range(r.heads):
                want = r.select(b, h, qd[b, j, h * G:(h + 1) * G], lens[b] - n[b] + j, idx.shape[-1], first, recent)
                assert np.array_equal(got[b, j, h], want), (b, j, h, got[b, j, h], want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,G,D,bs,lens,T,n_sel,first,recent", [
    (2, 4, 128, 16, [900, 500], 1, 8, 1, 2), (1, 16, 64, 64, [2000], 2, 5, 0, 1), (3, 5, 64, 32, [600, 1, 33], 3, 4, 2, 2),
    (2, 20, 128, 16, [700], 1, 16, 0, 0), (1, 1, 128, 128, [128 * 30], 1, 1, 0, 0), (1, 2, 128, 16, [640], 1, 64, 1, 1),
])
def test_select(heads, G, D, bs, lens, T, n_sel, first, recent, dtype):
    T = min(T, min(lens))
    dev, r = both_caches(len(lens), heads, D, bs, (max(lens) + bs - 1) // bs + 1)
    fill(dev, r, lens)
    q = torch.randn(len(lens), T, heads * G, D, generator=torch.Generator().manual_seed(8)).to(DT[dtype]).cuda()
    idx = torch.full((len(lens), T, heads, n_sel), -7, dtype=torch.int32, device="cuda")
    ws = workspace(dev, T, heads * G, n_sel)
    csa2.kv8_select_blocks(dev, q, idx, ws, n_first=first, n_recent=recent)
    assert csa2.read_device_status(ws) == csa2.OK
    check_select(r, q, idx, lens, [T] * len(lens), first, recent)


@pytest.mark.parametrize("bs,L", [(16, 70000), (64, 200000), (16, 650000)])
@pytest.mark.parametrize("ties", [0, 1, 2])
def test_select_among_many_blocks_and_equal_scores(bs, L, ties):
    # bounds written directly: random (0), all blocks equal (1), two values with the cut inside a tie (2);
    # 650,000 positions make 40,625 blocks, more than the row's keys in shared memory
    mb = (L + bs - 1) // bs
    D, heads, n_sel = 64, 1, 100
    rng = np.random.default_rng(bs + ties)
    z = torch.zeros(mb, heads, bs, D, dtype=torch.uint8, device="cuda")
    lo = rng.integers(-200, 0, (mb, heads, D)).astype(float)
    hi = lo + rng.integers(0, 200, (mb, heads, D))
    if ties == 1:
        lo[:], hi[:] = lo[:1], hi[:1]
    if ties == 2:
        pick = rng.random(mb) < 0.4
        lo[pick], hi[pick] = lo[0], hi[0]
        lo[~pick], hi[~pick] = lo[0] - 1, hi[0] - 1
    kb = np.stack([ref.e4m3_encode(np.floor(lo)), ref.e4m3_encode(np.ceil(hi))], 2)
    ks = np.ones((mb, heads)) if ties else np.exp2(rng.integers(-3, 2, (mb, heads)))
    dev = csa2.KV8Cache.wrap(z, z, torch.from_numpy(ks).float().cuda(), torch.ones(mb, heads, device="cuda"), i32([L]),
                             k_bounds=torch.from_numpy(kb).cuda())
    r = ref.Cache(1, heads, D, mb, bs, 1, np.arange(mb)[None])
    r.kb, r.ks = kb, ks
    q = torch.randn(1, 1, 2, D, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    idx = torch.empty(1, 1, heads, n_sel, dtype=torch.int32, device="cuda")
    csa2.kv8_select_blocks(dev, q, idx, workspace(dev, 1, 2, n_sel), n_first=2, n_recent=3)
    check_select(r, q, idx, [L], [1], 2, 3)


@pytest.mark.parametrize("bs,L", [(64, 30000), (16, 20000), (16, 200000)])
@pytest.mark.parametrize("ties", [0, 1, 2])
def test_select_among_fewer_blocks(bs, L, ties):
    # rows of every width that the selection has a form for
    test_select_among_many_blocks_and_equal_scores(bs, L, ties)


def test_select_nonfinite_query_and_padding():
    lens, n = [300, 400], [2, 0]
    dev, r = both_caches(2, 1, 64, 16, 26)
    fill(dev, r, lens)
    q = torch.randn(2, 3, 2, 64, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    q[0, 0, 0, 3], q[0, 1, 1, 4], q[0, 1] = math.nan, math.inf, q[0, 1] * 1e30
    idx = torch.full((2, 3, 1, 6), -7, dtype=torch.int32, device="cuda")
    csa2.kv8_select_blocks(dev, q, idx, workspace(dev, 3, 2, 6), n_q=i32(n))
    check_select(r, q, idx, lens, n, 0, 1)
    assert bool((idx[0, 2:] == -7).all()) and bool((idx[1] == -7).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,G,D,bs,lens,T,n_sel", [
    (2, 4, 128, 16, [900, 500], 1, 8), (1, 16, 64, 64, [2000], 2, 5), (3, 5, 64, 32, [600, 1, 33], 3, 4),
    (2, 20, 128, 16, [700], 1, 16), (1, 8, 128, 128, [128 * 20], 2, 3), (2, 4, 128, 64, [64 * 40], 1, 64)])
def test_selected_attention(heads, G, D, bs, lens, T, n_sel, dtype):
    T = min(T, min(lens))
    B, H = len(lens), heads * G
    dev, r = both_caches(B, heads, D, bs, (max(lens) + bs - 1) // bs + 1)
    fill(dev, r, lens)
    q = torch.randn(B, T, H, D, generator=torch.Generator().manual_seed(8)).to(DT[dtype]).cuda()
    idx = torch.empty(B, T, heads, n_sel, dtype=torch.int32, device="cuda")
    ws = workspace(dev, T, H, n_sel)
    out, lse = torch.zeros_like(q), torch.zeros(B, T, H, device="cuda")
    csa2.kv8_select_blocks(dev, q, idx, ws, n_recent=1)
    csa2.kv8_block_attn(dev, q, idx, out, ws, lse=lse)
    assert csa2.read_device_status(ws) == csa2.OK
    chosen = idx.cpu().numpy()

    def visible(b, j, h, p):
        i = chosen[b, j, h]
        t = (i[i >= 0][:, None] * bs + np.arange(bs)).reshape(-1)
        return t[t <= p]
    check_attn(dev, r, q, out, lse, [T] * B, 1 / math.sqrt(D), visible, lens)


def test_listed_blocks_that_break_the_rules_are_flagged():
    lens = [200]
    dev, r = both_caches(1, 1, 64, 16, 14)
    fill(dev, r, lens)
    q = torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(8)).half().cuda()
    out, lse, ws = torch.zeros_like(q), torch.zeros(1, 1, 4, device="cuda"), workspace(dev, 1, 4)
    for bad in ([3, 3, 5], [5, 3, 7], [0, 13, -1], [0, -1, 4], [-2, 1, 2], [1, 2, 1 << 30]):
        csa2.kv8_block_attn(dev, q, i32(bad).view(1, 1, 1, -1), out, ws, lse=lse)
        assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS, bad
    # nothing listed: an empty row; a list longer than the sequence has blocks: padding
    csa2.kv8_block_attn(dev, q, i32([-1, -1]).view(1, 1, 1, -1), out, ws, lse=lse)
    assert csa2.read_device_status(ws) == csa2.OK
    assert not bool(out.any()) and bool((lse == -math.inf).all())
    full, short = torch.zeros_like(q), torch.zeros_like(q)
    csa2.kv8_block_attn(dev, q, i32(list(range(13)) + [-1] * 50).view(1, 1, 1, -1), full, ws)
    csa2.kv8_attn(dev, q, short, ws)
    assert csa2.read_device_status(ws) == csa2.OK
    assert torch.allclose(full.float(), short.float(), atol=2e-3)


def test_decode_loop_as_a_graph():
    """Tokens joining a cache, selecting and attending, as a serving loop runs
    them: captured once, replayed per token, against the reference per token."""
    B, heads, G, D, bs, steps, n_sel = 2, 2, 4, 64, 16, 20, 4
    H = heads * G
    dev, r = both_caches(B, heads, D, bs, 12)
    lens = [101, 60]
    fill(dev, r, lens)
    g = torch.Generator().manual_seed(11)
    k, v = (torch.randn(steps, B, 1, heads, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(steps, B, 1, H, D, generator=g).bfloat16()
    kb, vb, qb = k[0].cuda(), v[0].cuda(), q[0].cuda()
    idx = torch.empty(B, 1, heads, n_sel, dtype=torch.int32, device="cuda")
    ws = workspace(dev, 1, H, n_sel)
    dense, sparse = torch.zeros_like(qb), torch.zeros_like(qb)
    dl, sl = (torch.zeros(B, 1, H, device="cuda") for _ in range(2))
    start = i32(lens)

    def step():
        csa2.kv8_append(dev, kb, vb, start, ws=ws)
        dev.seq_lens.add_(1)
        csa2.kv8_select_blocks(dev, qb, idx, ws, n_first=1, n_recent=1)
        csa2.kv8_block_attn(dev, qb, idx, sparse, ws, lse=sl)
        csa2.kv8_attn(dev, qb, dense, ws, lse=dl)
        start.add_(1)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for i in range(steps):
        kb.copy_(k[i]), vb.copy_(v[i]), qb.copy_(q[i])
        graph.replay()
        for b in range(B):
            r.append(b, lens[b], k[i, b].double().numpy(), v[i, b].double().numpy())
            lens[b] += 1
        check_select(r, qb, idx, lens, [1] * B, 1, 1)
        check_attn(dev, r, qb, dense, dl, [1] * B, 1 / math.sqrt(D), lambda b, j, h, p: np.arange(p + 1), lens)
        chosen = idx.cpu().numpy()

        def visible(b, j, h, p):
            c = chosen[b, j, h]
            t = (c[c >= 0][:, None] * bs + np.arange(bs)).reshape(-1)
            return t[t <= p]
        check_attn(dev, r, qb, sparse, sl, [1] * B, 1 / math.sqrt(D), visible, lens)
    same_cache(dev, r)
    assert csa2.read_device_status(ws) == csa2.OK
