"""The tensor-core kernel of csa2_kv8_attn on caches and batches that only it
can get: a contiguous cache, and more (sequence, row block) pairs than a CTA has
threads.  Each test says which kernel it means to run, and checks that it did."""
import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa2_b200 as csa2
from test_gpu_kv8 import attend, both_caches, fill
from test_gpu_kv8_scales import kernels

pytestmark = pytest.mark.gpu


def by_tensor_cores(call):
    names = kernels(call)
    assert "k_kv8_prefill" in names and "k_kv8_attn" not in names, names


@pytest.mark.parametrize("D,bs,T,window", [(128, 64, 130, 0), (64, 16, 97, 0), (128, 128, 300, 500), (128, 32, 40, 0)])
def test_contiguous_cache(D, bs, T, window):
    # one tile or several of query rows, blocks smaller than a step and as large; room for 8,192 positions
    lens = [700, 131]
    dev, r = both_caches(2, 2, D, bs, 8192 // bs, paged=False)
    fill(dev, r, lens)
    assert dev.block_table is None
    by_tensor_cores(lambda: attend(dev, r, lens, T, 8, window=window))


@pytest.mark.parametrize("window", [0, 20])
def test_more_sequences_than_threads(window):
    B, T = 800, 10
    rng = np.random.default_rng(B + window)
    lens, n = rng.integers(0, 90, B), rng.integers(0, T + 1, B)
    lens[:8], n[:8] = [0, 1, 10, 89, 0, 5, 60, 64], [0, 1, 10, 0, 10, 10, 1, 10]
    n[100:180] = 0                       # a run of sequences without rows, and one without positions
    lens[300:350] = 0
    dev, r = both_caches(B, 1, 64, 16, 6)
    lens, n = lens.tolist(), n.tolist()
    fill(dev, r, lens)
    by_tensor_cores(lambda: attend(dev, r, lens, T, 4, n=n, window=window))


def test_more_row_blocks_than_threads():
    # 520 rows of a sequence are three row blocks: 400 sequences have 1,200, most of them empty
    B, T = 400, 130
    rng = np.random.default_rng(B)
    n = rng.integers(0, 4, B)
    n[[0, 17, 18, 255, 256, 398, 399]] = [130, 64, 65, 128, 129, 1, 130]
    lens = n + rng.integers(0, 60, B)
    dev, r = both_caches(B, 1, 128, 32, 7)
    lens, n = lens.tolist(), n.tolist()
    fill(dev, r, lens)
    by_tensor_cores(lambda: attend(dev, r, lens, T, 4, n=n))


def test_the_last_of_many_sequences_alone_has_rows():
    B, T = 1600, 9
    lens, n = [40] * B, [0] * B
    n[-1] = T
    dev, r = both_caches(B, 1, 64, 16, 3)
    fill(dev, r, lens)
    by_tensor_cores(lambda: attend(dev, r, lens, T, 4, n=n))
