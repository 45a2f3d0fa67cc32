"""The 8-bit cache's calls on the debug build (libcsa2_debug.so), whose kernels
also check block indexes and scales: the same results, and bad input flagged in
the status word.  The tests run in a child process that loads it
(CSA2_LIBRARY=debug)."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CASES = ["tests/test_gpu_kv8.py::" + t for t in (
    "test_append_outside_the_cache_is_skipped_and_flagged", "test_read[128-64-bf16]", "test_attn[2-4-128-64-lens5-4-bf16]",
    "test_attn_padded_batch_and_rows_that_see_nothing", "test_attn_many_rows_with_room[2-4-64-16-lens1-70-bf16]",
    "test_attn_bad_pages_and_lengths_are_flagged", "test_attn_many_rows_nonfinite_bad_pages_and_lengths",
    "test_attn_window_with_the_pages_before_it_gone[16-lens1-3-4-77-False]",
    "test_attn_window_with_the_pages_before_it_gone[16-lens3-60-8-70-True]", "test_select[3-5-64-32-lens2-3-4-2-2-bf16]",
    "test_listed_blocks_that_break_the_rules_are_flagged", "test_decode_loop_as_a_graph")] + [
    "tests/test_gpu_kv8_debug_build.py::test_scales_that_are_no_powers_of_two_are_flagged"]


@pytest.mark.parametrize("T,room", [(1, False), (40, True)])
def test_scales_that_are_no_powers_of_two_are_flagged(T, room):
    if os.environ.get("CSA2_LIBRARY") != "debug":
        pytest.skip("runs inside the debug-build child process")
    import fp4_sparse_attention_csa2_b200 as csa2
    from test_gpu_kv8 import workspace
    from test_gpu_kv8_scales import with_values
    dev, r = with_values(2, 64, 16, [200], [1.0], room)
    q = torch.randn(1, T, 8, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out, ws = torch.zeros_like(q), workspace(dev, T, 8)
    csa2.kv8_attn(dev, q, out, ws)
    assert csa2.read_device_status(ws) == csa2.OK
    at = int(r.table[0, 3])
    for scales in (dev.k_scale, dev.v_scale):
        was = scales[at, 1].clone()
        for bad in (0.75, -0.5, float("nan"), 1e-40):
            scales[at, 1] = bad
            csa2.kv8_attn(dev, q, out, ws)
            assert csa2.read_device_status(ws) == csa2.ERR_DEVICE_BOUNDS, bad
        scales[at, 1] = was
    csa2.kv8_attn(dev, q, out, ws)
    assert csa2.read_device_status(ws) == csa2.OK


def test_kv8_under_the_debug_build():
    from fp4_sparse_attention_csa2_b200 import build
    build.build(debug=True)
    env = dict(os.environ, CSA2_LIBRARY="debug")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", *CASES], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout and "skipped" not in r.stdout
