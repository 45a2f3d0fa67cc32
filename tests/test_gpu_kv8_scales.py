"""Attention over blocks whose value scales are the least there is, or lie far
apart, on both kernels of csa2_kv8_attn: the scale says nothing of whether a
block's codes are zero, and the softmax sum does not depend on it."""
import math

import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa2_b200 as csa2
import kv8_ref as ref
from test_gpu_kv8 import both_caches, i32, workspace

pytestmark = pytest.mark.gpu


def with_values(heads, D, bs, lens, mags, room, seed=3):
    """A cache of rows in fp32: keys of one size, block i's values of about mags[i % len(mags)]."""
    B, mb = len(lens), (max(lens) + bs - 1) // bs + 1
    dev, r = both_caches(B, heads, D, bs, mb)
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B, max(lens), heads, D, generator=g) for _ in range(2))
    for i in range(mb):
        v[:, i * bs:(i + 1) * bs] *= mags[i % len(mags)]
    csa2.kv8_append(dev, k.cuda(), v.cuda(), i32([0] * B), n_new=i32(lens))
    for b, n in enumerate(lens):
        r.append(b, 0, k[b, :n].double().numpy(), v[b, :n].double().numpy())
    dev.seq_lens.copy_(i32(lens))
    if room:       # a table that reaches far: the kernel for many rows is chosen by that
        table = torch.full((B, (1 << 20) // bs), -1, dtype=torch.int32, device="cuda")
        table[:, :mb] = dev.block_table
        dev = csa2.KV8Cache.wrap(dev.k, dev.v, dev.k_scale, dev.v_scale, dev.seq_lens, dev.k_bounds, table)
    return dev, r


def kernels(call):
    """Names of this library's kernels that a call launches."""
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return " ".join(e.name for e in p.events() if "csa2" in e.name)


def check(dev, r, lens, T, H, seed=9, q_scale=1.0):
    """Every row against the definition in 64 bits.

    Bounds as kv8_ref.bounds derives them, with two differences.  The weights'
    fp16 rounding below the normal range, 2^-33 of the greatest, is of the greatest
    weight times value scale, since that is what is rounded: a channel has at most
    448 of it from each position.  The last term is half bf16's own least step,
    2^-134, not fp16's.
    """
    B, D, heads, sm = dev.batch, r.D, r.heads, 1 / math.sqrt(r.D)
    G = H // heads
    q = (torch.randn(B, T, H, D, generator=torch.Generator().manual_seed(seed)) * q_scale).bfloat16().cuda()
    out, lse = torch.full_like(q, 5.0), torch.full((B, T, H), 5.0, device="cuda")
    ws = workspace(dev, T, H)
    names = kernels(lambda: csa2.kv8_attn(dev, q, out, ws, lse=lse))
    assert csa2.read_device_status(ws) == csa2.OK
    assert ("k_kv8_prefill" in names) == (T * G > 16), names
    eps = torch.finfo(torch.bfloat16).eps
    for b in range(B):
        L, t = lens[b], np.arange(lens[b])
        seen = torch.from_numpy(t[None] <= L - T + np.arange(T)[:, None]).cuda()[None, :]       # [1, T, L]
        for h in range(heads):
            k, v = (torch.from_numpy(x).cuda() for x in r.rows(b, h, t))
            vs = torch.from_numpy(r.vs[r.table[b, t // r.bs], h]).cuda()
            x = q[b, :, h * G:(h + 1) * G].double().transpose(0, 1)                              # [G, T, D]
            z = torch.where(seen, x @ k.T * sm, -math.inf)
            zmax = torch.where(seen, x.abs() @ k.abs().T * sm, 0).amax(-1)
            wl, w = torch.logsumexp(z, -1), torch.softmax(z, -1)
            n = seen.sum(-1).expand(G, T)
            dz = 2.0 ** -18 * zmax + 2.0 ** -20
            want = w @ v
            o = (2.0 ** -11 + 2 * dz + 2.0 ** -17)[..., None] * (w @ v.abs())
            o = o + (n * 2.0 ** -33 * 448 * (w * vs).amax(-1))[..., None]
            o = o + eps / 2 * (want.abs() + o) + 2.0 ** -134
            got = out[b, :, h * G:(h + 1) * G].double().transpose(0, 1)
            assert bool(((got - want).abs() <= o).all()), (b, h, float(((got - want).abs() / o).max()))
            off = (lse[b, :, h * G:(h + 1) * G].double().T - wl).abs()
            assert bool((off <= dz + 2.0 ** -18 + 2.0 ** -22 * wl.abs()).all()), (b, h, float(off.max()))


TINY = [[1e-35], [1e-35, 1.0], [1.0, 1e-35], [1.0, 1.0, 0.0, 1e-35], [0.0, 1e-35], [0.0, 0.0, 1.0], [3e-34, 4e-34]]
APART = [[2.0 ** 60, 2.0 ** -80], [2.0 ** -80, 2.0 ** 60], [2.0 ** 100, 1.0, 2.0 ** -100], [1.0, 2.0 ** 40, 2.0 ** -40],
         [1.0] * 9 + [2.0 ** 110], [2.0 ** 20, 1.0, 2.0 ** -20], [2.0 ** 110, 2.0 ** -105, 0.0]]


@pytest.mark.parametrize("mags", TINY)
@pytest.mark.parametrize("heads,G,D,bs,T", [(1, 4, 128, 64, 1), (2, 8, 64, 16, 2), (1, 4, 128, 64, 64),
                                            (2, 4, 64, 16, 20), (1, 8, 128, 128, 40)])
def test_least_value_scale(mags, heads, G, D, bs, T):
    lens = [300, 257]
    dev, r = with_values(heads, D, bs, lens, mags, room=T * G > 16)
    check(dev, r, lens, T, heads * G)


@pytest.mark.parametrize("mags", APART)
@pytest.mark.parametrize("heads,G,D,bs,T", [(1, 4, 128, 64, 1), (2, 8, 64, 16, 2), (1, 4, 128, 32, 64),
                                            (2, 4, 64, 16, 20), (1, 8, 128, 128, 40)])
def test_value_scales_far_apart(mags, heads, G, D, bs, T):
    lens = [700, 513]
    dev, r = with_values(heads, D, bs, lens, mags, room=T * G > 16)
    check(dev, r, lens, T, heads * G)


@pytest.mark.parametrize("mags", [[1e-35, 1.0, 0.0], [0.0, 0.0, 0.0, 1e-35], [1.0, 2.0 ** 90, 2.0 ** -90],
                                  [2.0 ** -90] * 12 + [1.0]])
@pytest.mark.parametrize("D,T,G", [(128, 300, 4), (64, 30, 4)])
def test_scales_in_items_of_many_steps(mags, D, T, G):
    # enough items that a piece of the line holds several, and whole ones: two row tiles (300 tokens) or one
    lens = [900, 700, 450, 333] * (1 if T == 300 else 4)
    dev, r = with_values(8, D, 32, lens, mags, room=True)
    check(dev, r, lens, T, 8 * G)


@pytest.mark.parametrize("T,G,room", [(1, 8, False), (60, 4, True)])
def test_least_scale_over_many_pieces(T, G, room):
    # one item cut into pieces that a second launch merges
    for mags in ([1e-35], [1e-35, 2.0 ** -7, 0.0], [2.0 ** 70, 2.0 ** -70]):
        dev, r = with_values(1, 128, 64, [9000], mags, room=room)
        check(dev, r, [9000], T, G)


@pytest.mark.parametrize("q_scale", [1.0, 16.0])
@pytest.mark.parametrize("mags", [[1.0, 2.0 ** 72, 2.0 ** 56, 1.0, 2.0 ** -60, 2.0 ** 10],
                                  [2.0 ** 64, 2.0 ** 64, 1.0, 1.0, 1.0, 2.0 ** -64, 2.0 ** 30],
                                  [1.0, 1.0, 1.0, 1.0, 2.0 ** -100, 2.0 ** -36, 2.0 ** 28, 2.0 ** 92]])
@pytest.mark.parametrize("L,T,G,heads", [(9000, 60, 4, 1), (2300, 70, 8, 4), (2300, 20, 4, 8),
                                         (9000, 1, 8, 1), (2300, 4, 4, 4)])
def test_parts_and_halves_with_units_of_their_own(L, T, G, heads, mags, q_scale):
    # the parts of a row, its halves and its even and odd steps are added up whatever units their sums are in;
    # logits of up to some hundred make one of them count for nothing here and there
    dev, r = with_values(heads, 128, 64, [L], mags, room=T * G > 16)
    check(dev, r, [L], T, heads * G, q_scale=q_scale)
