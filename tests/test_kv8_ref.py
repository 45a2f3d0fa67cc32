"""Pins of the 8-bit cache's reference (tests/kv8_ref.py), on the CPU."""
import math

import numpy as np
import torch

from kv8_ref import Cache, e4m3_encode, e4m3_value, scale_of


def test_e4m3_values_and_encoder_agree_with_torch():
    codes = np.arange(256, dtype=np.uint8)
    ok = (codes & 0x7F) != 0x7F
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3_value(codes)[ok], want[ok])
    x = torch.randn(200000, generator=torch.Generator().manual_seed(1)) * 100
    mids = torch.from_numpy((e4m3_value(np.arange(0x7E)) + e4m3_value(np.arange(1, 0x7F))) / 2).float()
    x = torch.cat([x, mids, -mids, torch.tensor([0.0, -0.0, 448.0, 463.9, 1e9, -1e9])]).clamp(-448, 448)
    assert np.array_equal(e4m3_encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scale_is_the_least_power_of_two():
    for a in (448.0, 448.0000001, 1.0, 1e-3, 3e38, 1e-37, 0.0):
        s = scale_of(np.array([a, -a / 2]))
        e = math.log2(s)
        assert e == int(e) and -120 <= e <= 120
        assert a <= 448 * s or e == 120
        assert e == -120 or a > 448 * s / 2
    assert scale_of(np.array([np.inf, 3.0, np.nan])) == scale_of(np.array([3.0]))


def test_token_by_token_equals_one_call_in_scales_and_covers_in_bounds():
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(2, 70, 2, 64)) * np.exp2(np.arange(70) / 20)[:, None, None]
    one, many = (Cache(1, 2, 64, 5, 16, 5, None) for _ in range(2))
    one.append(0, 0, k, v)
    for i in range(70):
        many.append(0, i, k[i:i + 1], v[i:i + 1])
    assert np.array_equal(one.ks, many.ks) and np.array_equal(one.vs, many.vs)
    t = np.arange(70)
    for h in range(2):
        a, b = one.rows(0, h, t)[0], many.rows(0, h, t)[0]
        assert np.all(np.abs(a - k[:, h]) <= np.maximum(np.abs(k[:, h]) * 2.0 ** -4, one.ks[t // 16, h][:, None] * 2.0 ** -10))
        # a rescaled code is rounded twice
        assert np.all(np.abs(b - k[:, h]) <= np.maximum(np.abs(k[:, h]) * 2.0 ** -3, many.ks[t // 16, h][:, None] * 2.0 ** -9))
        for c, x in ((one, a), (many, b)):
            lo, hi = (e4m3_value(c.kb[t // 16, h, i]) * c.ks[t // 16, h][:, None] for i in range(2))
            assert np.all(lo <= x) and np.all(x <= hi)


def test_block_score_bounds_every_product():
    rng = np.random.default_rng(3)
    c = Cache(1, 1, 64, 8, 16, 8, None)
    c.append(0, 0, rng.normal(size=(128, 1, 64)), rng.normal(size=(128, 1, 64)))
    q = np.rint(rng.normal(size=(1, 64)) * 40)          # whole numbers: no rounding of q
    keys = c.rows(0, 0, np.arange(128))[0]
    best = (keys @ q[0]).reshape(8, 16).max(1)
    blk = c.table[0]
    up = (e4m3_value(c.kb[blk, 0, 0]) @ np.minimum(q[0], 0) + e4m3_value(c.kb[blk, 0, 1]) @ np.maximum(q[0], 0)) * c.ks[blk, 0]
    assert np.all(up >= best)
    got = c.select(0, 0, q, 127, 3, 0, 1)
    assert list(got) == sorted(set(got)) and got[-1] == 7
    assert set(got[:2]) == set(np.argsort(-up[:7], kind="stable")[:2])
