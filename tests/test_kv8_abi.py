"""Refusals of the csa2_kv8_* calls: on the host, before anything is launched
(none of these calls reaches a device)."""
import ctypes

import pytest
import torch

import fp4_sparse_attention_csa2_b200 as csa2
from fp4_sparse_attention_csa2_b200 import build as _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return csa2.lib()


def fake(**kw):
    d = dict(k_codes=0x10000, v_codes=0x20000, k_scale=0x30000, v_scale=0x40000, k_bounds=0x50000, block_table=0x60000,
             seq_lens=0x70000, batch=2, max_blocks=64, block_size=64, n_kv_heads=4, head_dim=128, n_blocks=128)
    d.update(kw)
    return csa2.csa2_kv8_cache(**d)


BAD_CACHES = [
    (dict(k_codes=None), csa2.ERR_INVALID_ARG), (dict(v_codes=0x20008), csa2.ERR_INVALID_ARG),
    (dict(k_scale=None), csa2.ERR_INVALID_ARG), (dict(v_scale=0x40002), csa2.ERR_INVALID_ARG),
    (dict(k_bounds=0x50004), csa2.ERR_INVALID_ARG), (dict(seq_lens=None), csa2.ERR_INVALID_ARG),
    (dict(block_table=0x60001), csa2.ERR_INVALID_ARG), (dict(batch=0), csa2.ERR_INVALID_ARG),
    (dict(batch=65536), csa2.ERR_INVALID_ARG), (dict(max_blocks=0), csa2.ERR_INVALID_ARG),
    (dict(n_kv_heads=0), csa2.ERR_INVALID_ARG), (dict(block_size=48), csa2.ERR_UNSUPPORTED),
    (dict(block_size=256), csa2.ERR_UNSUPPORTED), (dict(head_dim=96), csa2.ERR_UNSUPPORTED),
    (dict(head_dim=256), csa2.ERR_UNSUPPORTED), (dict(block_table=None, n_blocks=127), csa2.ERR_INVALID_ARG),
    (dict(n_blocks=1 << 24), csa2.ERR_UNSUPPORTED), (dict(max_blocks=1 << 25), csa2.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(lib, kw, code):
    c = ctypes.byref(fake(**kw))
    big = 1 << 40
    assert lib.csa2_kv8_workspace_bytes(c, 1, 32, 16) == 0
    assert lib.csa2_kv8_append(c, 0x1000, 0x2000, csa2.BF16, 512, 512, 1, 0x3000, None, None, None) == code
    assert lib.csa2_kv8_read(c, 0x3000, None, 1, 0x1000, 0x2000, csa2.BF16, None, None) == code
    assert lib.csa2_kv8_attn(c, 0x1000, csa2.BF16, 4096, 4096, 1, 32, None, 0, 0.0, 0x2000, None, 0x8000, big,
                             None) == code
    assert lib.csa2_kv8_select_blocks(c, 0x1000, csa2.BF16, 4096, 4096, 1, 32, None, 16, 1, 1, 0x2000, 0x8000, big,
                                      None) == code
    assert lib.csa2_kv8_block_attn(c, 0x1000, csa2.BF16, 4096, 4096, 1, 32, None, 0x2000, 16, 0.0, 0x3000, None,
                                   0x8000, big, None) == code


def test_null_cache(lib):
    assert lib.csa2_kv8_workspace_bytes(None, 1, 32, 16) == 0
    assert lib.csa2_kv8_append(None, 0x1000, 0x2000, csa2.BF16, 512, 512, 1, 0x3000, None, None, None) == \
        csa2.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(start=None), dict(k=0x1008), dict(v=0x2004), dict(start=0x3001), dict(n=0x3002),
    dict(dt=csa2.E4M3), dict(dt=7), dict(sb=12), dict(st=4), dict(T=-1), dict(T=(1 << 30) + 1), dict(ws=0x8001)])
def test_append_and_read_arguments(lib, kw):
    a = dict(k=0x1000, v=0x2000, dt=csa2.BF16, sb=512, st=512, T=4, start=0x3000, n=None, ws=None)
    a.update(kw)
    c = ctypes.byref(fake())
    assert lib.csa2_kv8_append(c, a["k"], a["v"], a["dt"], a["sb"], a["st"], a["T"], a["start"], a["n"], a["ws"],
                               None) == csa2.ERR_INVALID_ARG
    if not {"sb", "st"} & set(kw):
        assert lib.csa2_kv8_read(c, a["start"], a["n"], a["T"], a["k"], a["v"], a["dt"], a["ws"], None) == \
            csa2.ERR_INVALID_ARG


def test_nothing_to_do_launches_nothing(lib):
    c = ctypes.byref(fake())
    assert lib.csa2_kv8_append(c, 0x1000, 0x2000, csa2.BF16, 512, 512, 0, 0x3000, None, None, None) == csa2.OK
    assert lib.csa2_kv8_read(c, 0x3000, None, 0, 0x1000, 0x2000, csa2.BF16, None, None) == csa2.OK


def test_no_rows_need_no_rows_address(lib):
    # what a tensor without elements has for an address is null
    c = ctypes.byref(fake())
    assert lib.csa2_kv8_append(c, None, None, csa2.BF16, 512, 512, 0, 0x3000, None, None, None) == csa2.OK
    assert lib.csa2_kv8_read(c, 0x3000, None, 0, None, None, csa2.BF16, None, None) == csa2.OK
    assert lib.csa2_kv8_append(ctypes.byref(fake(batch=0)), None, None, csa2.BF16, 512, 512, 0, 0x3000, None, None,
                               None) == csa2.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=0x1008), dict(dt=csa2.F32), dict(dt=csa2.E4M3), dict(sb=4), dict(st=2), dict(T=0), dict(H=0),
    dict(H=30), dict(H=2), dict(n=0x4002), dict(out=None), dict(out=0x2008), dict(lse=0x3002), dict(ws=None),
    dict(ws=0x8008), dict(ws_bytes=4096), dict(window=-1), dict(T=1 << 27)])
def test_attention_arguments(lib, kw):
    a = dict(q=0x1000, dt=csa2.BF16, sb=4096, st=4096, T=1, H=32, n=None, window=0, out=0x2000, lse=0x3000, ws=0x8000,
             ws_bytes=1 << 40)
    a.update(kw)
    c = ctypes.byref(fake())
    assert lib.csa2_kv8_attn(c, a["q"], a["dt"], a["sb"], a["st"], a["T"], a["H"], a["n"], a["window"], 0.0, a["out"],
                             a["lse"], a["ws"], a["ws_bytes"], None) == csa2.ERR_INVALID_ARG
    if "window" not in kw:
        assert lib.csa2_kv8_block_attn(c, a["q"], a["dt"], a["sb"], a["st"], a["T"], a["H"], a["n"], 0x5000, 8, 0.0,
                                       a["out"], a["lse"], a["ws"], a["ws_bytes"], None) == csa2.ERR_INVALID_ARG


@pytest.mark.parametrize("n_sel,first,recent,idx", [(0, 0, 0, 0x5000), (2049, 0, 1, 0x5000), (8, -1, 0, 0x5000),
                                                    (8, 0, -1, 0x5000), (8, 5, 4, 0x5000), (8, 9, 0, 0x5000),
                                                    (8, 1, 1, None), (8, 1, 1, 0x5002)])
def test_selection_arguments(lib, n_sel, first, recent, idx):
    c = ctypes.byref(fake())
    assert lib.csa2_kv8_select_blocks(c, 0x1000, csa2.BF16, 4096, 4096, 1, 32, None, n_sel, first, recent, idx, 0x8000,
                                      1 << 40, None) == csa2.ERR_INVALID_ARG


def test_selection_needs_bounds_and_a_list_needs_entries(lib):
    c = ctypes.byref(fake(k_bounds=None))
    assert lib.csa2_kv8_select_blocks(c, 0x1000, csa2.BF16, 4096, 4096, 1, 32, None, 8, 1, 1, 0x5000, 0x8000, 1 << 40,
                                      None) == csa2.ERR_INVALID_ARG
    c = ctypes.byref(fake())
    for idx, n in ((None, 8), (0x5001, 8), (0x5000, 0)):
        assert lib.csa2_kv8_block_attn(c, 0x1000, csa2.BF16, 4096, 4096, 1, 32, None, idx, n, 0.0, 0x2000, None,
                                       0x8000, 1 << 40, None) == csa2.ERR_INVALID_ARG


def test_row_counts_are_bounded(lib):
    # batch * T * H of 2^31 rows and more are refused
    c = ctypes.byref(fake(batch=2048, n_blocks=1 << 12))
    assert lib.csa2_kv8_workspace_bytes(c, 1 << 15, 32, 0) == 0
    assert lib.csa2_kv8_workspace_bytes(c, 1 << 14, 32, 0) > 0


def test_workspace_grows_with_the_selection(lib):
    c = ctypes.byref(fake())
    plain, chosen = lib.csa2_kv8_workspace_bytes(c, 1, 32, 0), lib.csa2_kv8_workspace_bytes(c, 1, 32, 16)
    assert 0 < plain < chosen and plain % 256 == 0 and chosen - plain >= 2 * 4 * 64 * 4
    need = chosen
    assert lib.csa2_kv8_select_blocks(c, 0x1000, csa2.BF16, 4096, 4096, 1, 32, None, 16, 1, 1, 0x5000, 0x8000,
                                      need - 1, None) == csa2.ERR_INVALID_ARG


def test_status_name(lib):
    assert csa2.status_string(csa2.ERR_NONFINITE) == "CSA2_ERR_NONFINITE"


def test_binding_refuses_what_would_be_misread(lib):
    # a cache of host tensors, a wrong shape, a wrong type: ValueError before any pointer is taken
    with pytest.raises(ValueError):
        csa2.KV8Cache(1, 4, 128, 8, [0], device="cpu")
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)
    k, sc, lens = z(4, 2, 16, 64), z(4, 2, dt=torch.float32), z(1, dt=torch.int32)
    with pytest.raises(ValueError):      # host tensors
        csa2.KV8Cache.wrap(k, k, sc, sc, lens)
    with pytest.raises(ValueError):      # codes of another shape
        csa2.KV8Cache.wrap(k, z(4, 2, 16, 128), sc, sc, lens)
    with pytest.raises(ValueError):      # scales of another type
        csa2.KV8Cache.wrap(k, k, z(4, 2, dt=torch.float64), sc, lens)
    with pytest.raises(ValueError):      # a table that is not [batch, max_blocks]
        csa2.KV8Cache.wrap(k, k, sc, sc, lens, block_table=z(2, 4, dt=torch.int32))


class _Cache:
    """What the binding's argument checks read of a cache, on the host."""
    batch, n_kv_heads, head_dim, device, index = 2, 2, 64, torch.device("cpu"), -1


def test_binding_row_checks():
    c = _Cache()
    rows = torch.zeros(2, 3, 6, 64)
    ptr, sb, st = csa2._kv8_rows(c, rows[:, :, 1:3], 2, "k_new")         # a slice of a fused projection
    assert (sb, st) == (3 * 6 * 64, 6 * 64) and ptr == rows.data_ptr() + 64 * 4
    for bad in (rows[:, :, ::2][:, :, :2], rows[:, :, :2].transpose(1, 2), rows[:1, :, :2], rows[:, :, :3],
                rows[:, :, :2, :32], rows[0, :, :2]):
        with pytest.raises(ValueError):
            csa2._kv8_rows(c, bad, 2, "k_new")
    with pytest.raises(ValueError):
        csa2._kv8_rows(c, torch.zeros(2, 3, 131 * 2)[:, :, :128].unflatten(2, (2, 64)), 2, "k_new")  # stride 262
    for bad in (torch.zeros(2, 3), torch.zeros(2, 2, dtype=torch.int64), torch.zeros(4, 2, dtype=torch.float32)[::2]):
        with pytest.raises(ValueError):
            csa2._kv8_ptr(c, bad, torch.float32, (2, 2), "x")
    c.device, c.index = torch.device("cuda:1"), 1
    with pytest.raises(ValueError):                                      # another device than the cache's
        csa2._kv8_ptr(c, torch.zeros(2, 2), torch.float32, (2, 2), "x")
    with pytest.raises(ValueError):
        csa2._kv8_rows(c, rows[:, :, :2], 2, "q")


class _On:
    """A tensor on a GPU as far as the checks of KV8Cache look at one: type, shape, device, address."""
    is_cuda = True

    def __init__(self, shape, dtype, device=0, addr=0x10000):
        self.shape, self.dtype, self.device, self.addr = torch.Size(shape), dtype, torch.device("cuda", device), addr

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.addr


def parts(**kw):
    """The tensors of a cache of 2 sequences, 8 blocks."""
    d = dict(k_codes=_On((8, 2, 16, 64), torch.uint8), v_codes=_On((8, 2, 16, 64), torch.uint8),
             k_scale=_On((8, 2), torch.float32), v_scale=_On((8, 2), torch.float32), seq_lens=_On((2,), torch.int32),
             k_bounds=_On((8, 2, 2, 64), torch.uint8), block_table=_On((2, 4), torch.int32))
    d.update(kw)
    return d


def test_cache_on_two_devices_is_refused():
    assert csa2.KV8Cache.wrap(**parts()).c.max_blocks == 4
    for name, t in parts().items():
        if name == "k_codes":
            continue
        with pytest.raises(ValueError):
            csa2.KV8Cache.wrap(**parts(**{name: _On(t.shape, t.dtype, device=1)}))


class _Host(torch.Tensor):
    """A host tensor that says it is on the GPU: only its address would be taken."""
    def get_device(self):
        return 0


def test_query_calls_want_a_workspace_and_all_calls_one_with_a_status_word(lib):
    c = csa2.KV8Cache.wrap(**parts())
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt).as_subclass(_Host)
    q, idx, rows, start = z(2, 1, 4, 64), z(2, 1, 2, 3, dt=torch.int32), z(2, 1, 2, 64), z(2, dt=torch.int32)
    calls = [lambda ws: csa2.kv8_attn(c, q, q, ws), lambda ws: csa2.kv8_select_blocks(c, q, idx, ws),
             lambda ws: csa2.kv8_block_attn(c, q, idx, q, ws)]
    for call in calls:
        with pytest.raises(ValueError, match="workspace"):
            call(None)
    calls += [lambda ws: csa2.kv8_append(c, rows, rows, start, ws=ws), lambda ws: csa2.kv8_read(c, start, rows, rows, ws=ws)]
    for call in calls:
        for small in (z(0, dt=torch.uint8), z(3, dt=torch.uint8)):    # a status word is four bytes
            with pytest.raises(ValueError, match="workspace"):
                call(small)


def test_a_tensor_put_in_place_of_a_caches_own_is_the_one_that_calls_use():
    c = csa2.KV8Cache.wrap(**parts())
    lens, table = _On((2,), torch.int32, addr=0x20000), _On((2, 6), torch.int32, addr=0x30000)
    c.seq_lens = lens                                          # as in cache.seq_lens = cache.seq_lens + 1
    assert c.c.seq_lens == 0x20000 and c.seq_lens is lens and c.ref._obj is c.c
    c.block_table = table                                      # a wider table: sequences may grow further
    assert (c.c.block_table, c.c.max_blocks, c.max_blocks) == (0x30000, 6, 6) and c.c.seq_lens == 0x20000
    c.seq_lens = lens                                          # the same again, as += leaves it
    assert c.c.seq_lens == 0x20000
    c.k_bounds = None
    assert c.c.k_bounds is None and c.c.k_codes == 0x10000
    for name, bad in (("seq_lens", _On((2,), torch.int64)), ("seq_lens", _On((2,), torch.int32, device=1)),
                      ("block_table", _On((3, 4), torch.int32)), ("v", _On((8, 2, 16, 128), torch.uint8)),
                      ("seq_lens", torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            setattr(c, name, bad)
        assert c.seq_lens is lens and c.c.seq_lens == 0x20000 and c.block_table is table and c.max_blocks == 6
