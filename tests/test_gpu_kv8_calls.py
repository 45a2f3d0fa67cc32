"""Calls of the 8-bit cache at the edges of what its documentation allows."""
import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa2_b200 as csa2
from test_gpu_kv8 import attend, both_caches, check_attn, fill, i32, same_cache, workspace

pytestmark = pytest.mark.gpu


def test_a_new_tensor_of_lengths_or_blocks_is_used():
    lens = [100, 37]
    dev, r = both_caches(2, 2, 64, 16, 8)
    fill(dev, r, lens)
    attend(dev, r, lens, 1, 8)
    fewer = [60, 37]
    dev.seq_lens = dev.seq_lens - i32([40, 0])
    attend(dev, r, fewer, 1, 8)
    wide = torch.full((2, 12), -1, dtype=torch.int32, device="cuda")
    wide[:, :8] = dev.block_table
    dev.block_table = wide                                        # the old table is freed
    other = torch.full((2, 8), 1 << 20, dtype=torch.int32, device="cuda")
    attend(dev, r, fewer, 1, 8)
    attend(dev, r, fewer, 24, 8)
    assert int(other[0, 0]) == 1 << 20


def test_many_rows_captured_once_and_replayed_as_lengths_change():
    B, T, H = 3, 40, 8
    dev, r = both_caches(B, 2, 64, 16, 512)
    full = [700, 300, 90]
    fill(dev, r, full)
    q = torch.randn(B, T, H, 64, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    out, lse, n = torch.zeros_like(q), torch.zeros(B, T, H, device="cuda"), i32([T] * B)
    ws, side = workspace(dev, T, H), torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            csa2.kv8_attn(dev, q, out, ws, lse=lse, n_q=n)
    for lens, rows in ((full, [40, 40, 40]), ([513, 1, 64], [7, 1, 40]), ([0, 300, 17], [0, 33, 0]), (full, [1, 0, 40])):
        dev.seq_lens.copy_(i32(lens))
        n.copy_(i32(rows))
        out.fill_(5.0), lse.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert csa2.read_device_status(ws) == csa2.OK
        check_attn(dev, r, q, out, lse, rows, 1 / 8, lambda b, j, h, p: np.arange(p + 1), lens)
        for b in range(B):
            assert bool((out[b, rows[b]:] == 5).all()) and bool((lse[b, rows[b]:] == 5).all())


def test_append_at_a_negative_start_drops_that_sequences_rows_alone():
    # rows 3 .. 9 of sequence 0 would lie inside the cache
    dev, r = both_caches(2, 1, 64, 16, 2)
    x = torch.randn(2, 10, 1, 64, generator=torch.Generator().manual_seed(6))
    before, ws = dev.k[r.table[0]].clone(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    csa2.kv8_append(dev, x.cuda(), x.cuda(), i32([-3, 0]), ws=ws)
    assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS
    assert torch.equal(dev.k[r.table[0]], before)
    r.append(1, 0, x[1].double().numpy(), x[1].double().numpy())
    same_cache(dev, r)


def test_rows_near_the_ends_of_fp32_read_back():
    # 240 * 2^120 is the greatest that comes back finite; at the other end a code is worth 2^-129 and more
    dev, r = both_caches(1, 1, 64, 16, 3)
    x = torch.zeros(1, 33, 1, 64)
    x[0, 0, 0, :6] = torch.tensor([3.2e38, 3.29e38, 3.2964e38, 3.4e38, -3.4e38, 1.0])
    x[0, 16, 0, :4] = torch.tensor([1e-35, 2.0 ** -129, 2.0 ** -131, -3e-34])
    x[0, 32, 0, :3] = torch.tensor([240.0 * 2.0 ** 120, 247.9 * 2.0 ** 120, 248.0 * 2.0 ** 120])
    csa2.kv8_append(dev, x.cuda(), x.cuda(), i32([0]))
    r.append(0, 0, x[0].double().numpy(), x[0].double().numpy())
    same_cache(dev, r)
    k, v = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    csa2.kv8_read(dev, i32([0]), k, v)
    want = torch.from_numpy(r.rows(0, 0, np.arange(33))[0])[None, :, None].float()      # 256 * 2^120: infinity
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    top = 240.0 * 2.0 ** 120
    assert k[0, 0, 0, :6].tolist()[:2] == [top, top] and bool(k[0, 0, 0, 3:5].isinf().all())
    assert k[0, 32, 0, :3].tolist() == [top, top, float("inf")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_append_and_read_of_no_rows(dtype):
    dev, r = both_caches(2, 2, 64, 16, 3)
    fill(dev, r, [20, 7])
    rows, ws = torch.empty(2, 0, 2, 64, dtype=dtype, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    csa2.kv8_append(dev, rows, rows, i32([20, 7]), ws=ws)
    csa2.kv8_append(dev, rows, rows, i32([20, 7]), n_new=i32([0, 0]))
    csa2.kv8_read(dev, i32([0, 0]), rows, torch.empty_like(rows), ws=ws)
    assert csa2.read_device_status(ws) == csa2.OK
    same_cache(dev, r)
