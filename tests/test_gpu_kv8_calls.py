"""Calls of the 8-bit cache at the edges of what its documentation allows."""
import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa2_b200 as csa2
from test_gpu_kv8 import both_caches, fill, i32, same_cache, workspace

pytestmark = pytest.mark.gpu


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
