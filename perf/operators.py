"""The 8-bit key / value cache and the attention that reads it: what is measured.

The operators (csa2.KV8Cache and the kv8_* calls):

  append   new key and value rows quantised into the cache: E4M3 codes with one
           power-of-two scale per block of tokens and head, and per block, head
           and channel the least and greatest key code (the block's bounds)
  read     cached rows back as the values they stand for
  attn     softmax attention of T query tokens per sequence over the cache,
           causal, grouped heads, optional sliding window
  select   per query token and key head the blocks with the best bound on
           q . k, first and newest blocks always among them
  blocks   attention over the blocks so selected

Where `own` is false every pass is the plain form in elementary torch
operations; where it is true it is the library's calls.
"""
import math
import random

import torch

own = False

KINDS = {"append", "read", "attn", "select", "blocks"}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def case(kind, **kw):
    """A case: `lo` .. `hi` are the shortest and longest sequence of the batch."""
    c = dict(kind=kind, B=1, T=1, lo=1, hi=1, H=32, Hkv=8, D=128, bs=64, dtype="bf16", paged=True, ragged=False,
             window=0, n_sel=0)
    c.update(kw)
    return c


def listed():
    return [
        # one decoded token of each of 32 sequences joins the cache, at any place inside a block
        case("append", name="append-token", B=32, lo=257, hi=4096, Hkv=8),
        # two prompts written in one call, behind a prefix that ends inside a block
        case("append", name="append-prompt", B=2, T=8192, lo=8229, hi=8300, Hkv=8),
        # the newest 128 positions of 32 sequences (a sliding window) read back
        case("read", name="read-window", B=32, T=128, lo=300, hi=4096, Hkv=4),
        # whole sequences read back, as when they leave the cache
        case("read", name="read-sequences", B=8, T=8192, lo=8192, hi=8192, Hkv=8),
        # one short conversation: latency is all
        case("attn", name="attn-short", lo=1000, hi=1000, H=16, Hkv=4, dtype="fp16"),
        # a serving batch with ragged lengths in scattered blocks
        case("attn", name="attn-batch32", B=32, lo=1024, hi=16384, H=64, Hkv=8),
        # one sequence of a million tokens
        case("attn", name="attn-1m", lo=1048576, hi=1048576, H=32, Hkv=4),
        # a chunk of a long prompt over its cached prefix
        case("attn", name="attn-prompt", T=2048, lo=8192, hi=8192, H=32, Hkv=8),
        # block choice over a million tokens, one query token
        case("select", name="select-1m", lo=1048576, hi=1048576, H=64, Hkv=8, n_sel=64),
        # block choice for a serving batch
        case("select", name="select-batch32", B=32, lo=16384, hi=131072, H=32, Hkv=4, n_sel=64),
        # attention over 32 chosen blocks, a serving batch
        case("blocks", name="blocks-batch32", B=32, lo=4096, hi=32768, H=32, Hkv=4, n_sel=32),
        # attention over 64 chosen blocks of one long sequence
        case("blocks", name="blocks-64k", lo=65536, hi=65536, H=16, Hkv=2, dtype="fp16", n_sel=64),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "read", "attn", "attn", "select", "blocks"])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
    c = dict(Hkv=Hkv, H=Hkv * G, D=rng.choice([64, 128, 128]), bs=rng.choice([16, 32, 64, 64, 128]),
             dtype=rng.choice(["bf16", "bf16", "fp16"]), paged=rng.random() < 0.8)
    if kind in ("append", "read"):
        c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
        c["B"] = _spread(rng, 1, 64)
        c["T"] = _spread(rng, 1, max(1, 12000 // c["B"]))
        c["hi"] = c["T"] + rng.randrange(0, 1000)
        c["lo"] = max(1, c["hi"] - rng.randrange(0, 300), c["T"])
        c["ragged"] = rng.random() < 0.3
    elif kind == "attn":
        c["B"] = _spread(rng, 1, 48)
        c["T"] = rng.choice([1, 1, 1, 2, 3, 4, 7, _spread(rng, 8, 600)])
        c["hi"] = _spread(rng, 16, max(64, min(131072, 250000 // c["B"])) if c["T"] < 8 else 4000 // c["B"] + 16)
        c["hi"] = max(c["hi"], c["T"])
        c["lo"] = max(c["T"], _spread(rng, 1, c["hi"]))
        c["window"] = rng.choice([0, 0, 0, 128, 1000])
        c["ragged"] = rng.random() < 0.3
    else:
        c["B"] = _spread(rng, 1, 32)
        c["T"] = rng.choice([1, 1, 1, 2, 4])
        c["hi"] = _spread(rng, 64, min(262144, 1000000 // c["B"]))
        c["lo"] = max(c["T"], _spread(rng, 16, c["hi"]))
        c["n_sel"] = rng.choice([4, 8, 16, 31, 32, 64])
        if kind == "blocks":
            c["hi"] = min(c["hi"], 32768)
            c["lo"] = min(c["lo"], c["hi"])
        c["ragged"] = rng.random() < 0.2
    return case(kind, **c)


def lengths(c):
    """Every sequence's length: the case's alone, so that its work is known."""
    r = random.Random("%(lo)d %(hi)d %(B)d" % c)
    L = [c["hi"], c["lo"]][:c["B"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["B"] - 2)]
    r.shuffle(L)
    return L


def counts(c):
    """How many of the T rows of each sequence the call is for (all, unless the batch is padded)."""
    r = random.Random("%(lo)d %(hi)d %(B)d %(T)d rows" % c)
    return [r.randint(0 if b else 1, c["T"]) if c["ragged"] else c["T"] for b in range(c["B"])]


def _blocks_of(c, visible):
    return min(c["n_sel"], visible)


def work(c):
    L, N, Hkv, H, D, bs, T = lengths(c), counts(c), c["Hkv"], c["H"], c["D"], c["bs"], c["T"]
    e = 4 if c["dtype"] == "fp32" else 2
    rows = sum(N)
    if c["kind"] in ("append", "read"):
        # a row of keys and one of values at the caller's type on one side, one byte a channel on the other
        b = rows * Hkv * D * 2 * (e + 1)
        touched = sum(((l - 1) // bs - (l - n) // bs + 1) for l, n in zip(L, N) if n)
        b += touched * Hkv * (8 + (2 * D if c["kind"] == "append" else 0))
        return {"bytes": b, "flops": rows * Hkv * D * 4}
    io = rows * H * (2 * D * 2 + 4)
    if c["kind"] == "attn":
        seen = pairs = 0
        for l, n in zip(L, N):
            W = c["window"] or l
            if n:
                seen += l - max(0, l - n - W + 1)
            pairs += sum(min(W, l - n + j + 1) for j in range(n))
        return {"bytes": seen * Hkv * 2 * D + seen // bs * Hkv * 8 + io, "flops": 4 * pairs * H * D}
    vis = [[(l - n + j) // bs + 1 for j in range(n)] for l, n in zip(L, N)]
    if c["kind"] == "select":
        read = sum(v[-1] for v in vis if v)
        return {"bytes": read * Hkv * (2 * D + 4) + rows * (H * D * 2 + Hkv * c["n_sel"] * 4),
                "flops": 4 * sum(map(sum, vis)) * H * D}
    sel = sum(_blocks_of(c, x) for v in vis for x in v)
    return {"bytes": sel * Hkv * (bs * 2 * D + 8 + 4) + io, "flops": 4 * sel * bs * H * D}


# ------------------------------------------------------------------ the state
def _rows(g, shape, dtype):
    """Key or value rows as a projection gives them: near normal, some channels wider than others."""
    x = torch.randn(shape, generator=g, device="cuda")
    wide = torch.exp2(torch.randint(-1, 3, shape[-2:], generator=g, device="cuda").float())
    return (x * wide).to(dtype)


def _codes(g, n, Hkv, bs, D):
    """Codes of full blocks: normal values whose greatest lies between 224 and 448, as the scale rule leaves them."""
    out = torch.empty(n, Hkv, bs, D, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (Hkv * bs * D))
    for i in range(0, n, step):
        x = torch.randn(out[i:i + step].shape, generator=g, device="cuda", dtype=torch.float16)
        out[i:i + step] = (x * 75).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, T, Hkv, H, D, bs, kind = c["B"], c["T"], c["Hkv"], c["H"], c["D"], c["bs"], c["kind"]
    dt = DTYPES[c["dtype"]]
    L, N = lengths(c), counts(c)
    max_blocks = (c["hi"] + bs - 1) // bs + 1
    n_blocks = B * max_blocks
    s = dict(c, max_blocks=max_blocks, n_blocks=n_blocks, dt=dt)
    i32 = dict(dtype=torch.int32, device="cuda")
    s["seq_lens"], s["n"] = torch.tensor(L, **i32), torch.tensor(N, **i32)
    s["start"] = s["seq_lens"] - s["n"]
    order = torch.randperm(n_blocks, generator=g, device="cuda") if c["paged"] else torch.arange(n_blocks, device="cuda")
    s["table"] = order.view(B, max_blocks).to(torch.int32).contiguous()
    if kind == "append":
        # what stands in the cache before the call: the partly filled block that the new rows join
        s["k"], s["v"] = (torch.zeros(n_blocks, Hkv, bs, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros(n_blocks, Hkv, device="cuda") for _ in range(2))
        s["kb"] = torch.zeros(n_blocks, Hkv, 2, D, dtype=torch.uint8, device="cuda")
        held = s["start"] // bs * bs
        old = [_rows(g, (B, bs, Hkv, D), dt) for _ in range(2)]
        old = [x * torch.exp2(torch.randint(-2, 1, (B, 1, Hkv, 1), generator=g, device="cuda").float()).to(dt) for x in old]
        _append_plain(s, old[0], old[1], held, s["start"] - held, bs)
        s["new"] = [_rows(g, (B, T, Hkv, D), dt) for _ in range(2)]
        return s
    if kind == "select":
        s["k"], s["v"] = (torch.zeros(n_blocks, Hkv, bs, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        wide = torch.randn(n_blocks, Hkv, 2, D, generator=g, device="cuda") * 30
        mid = torch.randn(n_blocks, Hkv, D, generator=g, device="cuda") * 30
        hi = torch.ceil((mid + 150 + wide[:, :, 0]).clamp(-440, 448))
        lo = torch.floor(torch.minimum(mid - 150 + wide[:, :, 1], hi).clamp(-448, 448))
        s["kb"] = torch.stack([lo, hi], 2).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k"], s["v"] = _codes(g, n_blocks, Hkv, bs, D), _codes(g, n_blocks, Hkv, bs, D)
        s["kb"] = None
    s["ks"], s["vs"] = (torch.exp2(torch.randint(-8, -5, (n_blocks, Hkv), generator=g, device="cuda").float()) for _ in range(2))
    if kind == "read":
        s["out"] = [torch.zeros(B, T, Hkv, D, dtype=dt, device="cuda") for _ in range(2)]
        return s
    # a query row, now and then several times as long as the others
    q = torch.randn(B, T, H, D, generator=g, device="cuda") * torch.exp2(torch.randint(-1, 2, (B, T, H, 1), generator=g, device="cuda").float())
    s["q"] = q.to(dt)
    if kind == "select":
        s["first"], s["recent"] = min(1, c["n_sel"] // 4), min(2, c["n_sel"] // 4)
        s["idx"] = torch.full((B, T, Hkv, c["n_sel"]), -1, **i32)
        return s
    s["out"] = torch.zeros(B, T, H, D, dtype=dt, device="cuda")
    s["lse"] = torch.zeros(B, T, H, device="cuda")
    if kind == "blocks":
        rank = torch.rand(B, T, Hkv, max_blocks, generator=g, device="cuda")
        s["idx"] = _best_blocks(rank, _position(s), bs, c["n_sel"], 1, 1)
    return s


# ------------------------------------------------------------------ plain forms
def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _to_codes(x):
    """Nearest E4M3 code, ties to even, saturating."""
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _position(s):
    """Position of every query token, and -1 for the padding of the batch: [B, T]."""
    j = torch.arange(s["T"], device="cuda")
    p = s["start"][:, None] + j
    return torch.where(j < s["n"][:, None], p, -1)


def _scale(amax):
    """The least power of two 2^e, -120 <= e <= 120, with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(-120, 120)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -120))


def _append_plain(s, k_new, v_new, start, n, T):
    B, Hkv, D, bs = s["B"], s["Hkv"], s["D"], s["bs"]
    nb = min((T + bs - 2) // bs + 1, s["max_blocks"])
    blk = start[:, None] // bs + torch.arange(nb, device="cuda")                      # [B, nb]
    phys = torch.gather(s["table"], 1, blk.clamp(max=s["max_blocks"] - 1).long()).long()
    pos = blk[:, :, None] * bs + torch.arange(bs, device="cuda")                      # [B, nb, bs]
    new = (pos >= start[:, None, None]) & (pos < (start + n)[:, None, None])
    old = (pos < start[:, None, None])
    had = old.any(2)[:, :, None]                                                      # [B, nb, 1]
    touched = new.any(2) & (blk < s["max_blocks"])
    row = (pos - start[:, None, None]).clamp(0, T - 1).long()
    for codes, scales, x_new, bounds in ((s["k"], s["ks"], k_new, s["kb"]), (s["v"], s["vs"], v_new, None)):
        x = torch.gather(x_new.float(), 1, row.view(B, -1, 1, 1).expand(-1, -1, Hkv, D)).view(B, nb, bs, Hkv, D)
        x = torch.where(new[..., None, None], x, 0).transpose(2, 3)                   # [B, nb, Hkv, bs, D]
        was = scales[phys]
        sc = _scale(x.abs().amax((3, 4)))
        sc = torch.where(had, torch.maximum(sc, was), sc)
        before = codes[phys]
        kept = _to_codes(_values(before) * (torch.where(had, was, 1) / sc)[..., None, None])
        fresh = _to_codes(x / sc[..., None, None])
        new_, old_ = new[:, :, None, :, None], old[:, :, None, :, None]
        t = touched[:, :, None]
        if bounds is not None:
            v, b = _values(fresh), _values(bounds[phys]) * (torch.where(had, was, 1) / sc)[..., None, None]
            lo = torch.floor(torch.where(new_, v, 448).amin(3))
            hi = torch.ceil(torch.where(new_, v, -448).amax(3))
            lo = torch.where(had[..., None], torch.minimum(lo, torch.floor(b[:, :, :, 0])), lo)
            hi = torch.where(had[..., None], torch.maximum(hi, torch.ceil(b[:, :, :, 1])), hi)
            bounds[phys] = torch.where(t[..., None, None], _to_codes(torch.stack([lo, hi], 3)), bounds[phys])
        codes[phys] = torch.where(t[..., None, None] & new_, fresh, torch.where(t[..., None, None] & old_, kept, before))
        scales[phys] = torch.where(t, sc, was)


def _cached(s, codes, scales, dim=None):
    """Every sequence's rows as values: [B, Hkv, max_blocks * bs, D]."""
    t = s["table"].long()
    x = _values(codes[t]) * scales[t][..., None, None]                                # [B, nb, Hkv, bs, D]
    return x.transpose(1, 2).reshape(s["B"], s["Hkv"], -1, s["D"])


def _softmax_rows(z, mask):
    z = torch.where(mask, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l == 0, 1, l), (m + torch.log(l))[..., 0]


def _put(s, out, lse):
    """Rows of the padding stay as they were."""
    live = (torch.arange(s["T"], device="cuda") < s["n"][:, None])[:, :, None]
    s["out"] = torch.where(live[..., None], out.to(s["dt"]), s["out"])
    s["lse"] = torch.where(live, lse, s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _best_blocks(score, p, bs, n_sel, first, recent):
    """The n_sel best visible blocks, ascending, -1 last; the first and the newest always, ties to the lowest."""
    nb = score.shape[-1]
    i = torch.arange(nb, device="cuda")
    last = torch.div(p, bs, rounding_mode="floor")[:, :, None, None]                   # block of the query token
    seen = (i <= last) & (p[:, :, None, None] >= 0)
    rank = torch.where(seen, torch.where((i < first) | (i > last - recent), math.inf, score.clamp(min=-3e38)), -math.inf)
    k = min(n_sel, nb)
    top = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :k]
    top = torch.where(torch.gather(seen.expand_as(rank), -1, top), top, nb)
    top = torch.sort(top, dim=-1)[0]
    top = torch.where(top == nb, -1, top)
    return torch.nn.functional.pad(top, (0, n_sel - k), value=-1).to(torch.int32)


def _plain(s):
    B, T, H, Hkv, D, bs, kind = (s[x] for x in ("B", "T", "H", "Hkv", "D", "bs", "kind"))
    if kind == "append":
        _append_plain(s, s["new"][0], s["new"][1], s["start"], s["n"], T)
        return _stored(s)
    p = _position(s)
    if kind == "read":
        phys = torch.gather(s["table"], 1, (p.clamp(min=0) // bs).long()).long()
        off = (p.clamp(min=0) % bs).long()
        live = (p >= 0)[:, :, None, None]
        s["out"] = [torch.where(live, (_values(c[phys, :, off]) * sc[phys][..., None]).to(s["dt"]), o)
                    for c, sc, o in ((s["k"], s["ks"], s["out"][0]), (s["v"], s["vs"], s["out"][1]))]
        return {"k": s["out"][0], "v": s["out"][1]}
    G = H // Hkv
    q = s["q"].float().view(B, T, Hkv, G, D)
    if kind == "attn":
        qg = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
        z = qg @ _cached(s, s["k"], s["ks"]).transpose(2, 3)
        z = z.view(B, Hkv, T, G, -1) / math.sqrt(D)
        t = torch.arange(z.shape[-1], device="cuda")
        seen = t <= p[:, :, None]
        if s["window"]:
            seen = seen & (t > p[:, :, None] - s["window"])
        a, lse = _softmax_rows(z, seen[:, None, :, None])
        out = a.view(B, Hkv, T * G, -1) @ _cached(s, s["v"], s["vs"])
        return _put(s, out.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D),
                    lse.permute(0, 2, 1, 3).reshape(B, T, H))
    if kind == "select":
        m, x = torch.frexp(q.abs().amax(-1, keepdim=True))
        e = torch.where(m <= 127 / 128, x - 7, x - 6)
        qi = torch.round(torch.ldexp(q, -e))                                           # whole numbers, at most 127
        t = s["table"].long()
        b = _values(s["kb"][t]).transpose(1, 2)                                        # [B, Hkv, nb, 2, D]
        both = torch.cat([qi.clamp(max=0), qi.clamp(min=0)], -1).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, 2 * D)
        sc = both @ b.reshape(B, Hkv, -1, 2 * D).transpose(2, 3)                       # whole numbers below 2^24: exact
        sc = sc * s["ks"][t].transpose(1, 2)[:, :, None]
        sc = torch.ldexp(sc.view(B, Hkv, T, G, -1), e.permute(0, 2, 1, 3, 4)).amax(3)
        best = _best_blocks(sc.transpose(1, 2), p, bs, s["n_sel"], s["first"], s["recent"])
        s["idx"] = torch.where((p >= 0)[:, :, None, None], best, s["idx"])
        return {"blocks": s["idx"]}
    i = s["idx"].long()                                                                # [B, T, Hkv, n]
    phys = torch.gather(s["table"].long(), 1, i.clamp(min=0).view(B, -1)).view(i.shape)
    h = torch.arange(Hkv, device="cuda")[:, None]
    k = (_values(s["k"][phys, h]) * s["ks"][phys, h][..., None, None]).flatten(3, 4)   # [B, T, Hkv, n * bs, D]
    z = (q @ k.transpose(3, 4)) / math.sqrt(D)
    pos = i[..., None] * bs + torch.arange(bs, device="cuda")
    seen = ((i >= 0)[..., None] & (pos <= p[:, :, None, None, None])).flatten(3, 4)[:, :, :, None]
    a, lse = _softmax_rows(z, seen)
    v = (_values(s["v"][phys, h]) * s["vs"][phys, h][..., None, None]).flatten(3, 4)
    return _put(s, (a @ v).reshape(B, T, H, D), lse.reshape(B, T, H))


def _stored(s):
    e = torch.float8_e4m3fn
    return {"k": s["k"].view(e), "v": s["v"].view(e), "bounds": s["kb"].view(e), "k_scale": s["ks"], "v_scale": s["vs"]}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import fp4_sparse_attention_csa2_b200 as csa2

    kind = s["kind"]
    if "cache" not in s:
        # the handle and the workspace that a serving program keeps
        s["cache"] = csa2.KV8Cache.wrap(s["k"], s["v"], s["ks"], s["vs"], s["seq_lens"], k_bounds=s["kb"],
                                        block_table=s["table"] if s["paged"] else None, max_blocks=s["max_blocks"])
        s["ws"] = torch.empty(csa2.kv8_workspace_bytes(s["cache"], s["T"], s["H"], s["n_sel"]), dtype=torch.uint8,
                              device="cuda")
        csa2.workspace_init(s["ws"])
        s["rows"] = s["n"] if s["ragged"] else None
    if kind == "append":
        csa2.kv8_append(s["cache"], s["new"][0], s["new"][1], s["start"], n_new=s["rows"], ws=s["ws"])
        return _stored(s)
    if kind == "read":
        csa2.kv8_read(s["cache"], s["start"], s["out"][0], s["out"][1], n_rows=s["rows"], ws=s["ws"])
        return {"k": s["out"][0], "v": s["out"][1]}
    if kind == "attn":
        csa2.kv8_attn(s["cache"], s["q"], s["out"], s["ws"], lse=s["lse"], window=s["window"], n_q=s["rows"])
    elif kind == "select":
        csa2.kv8_select_blocks(s["cache"], s["q"], s["idx"], s["ws"], n_first=s["first"], n_recent=s["recent"],
                               n_q=s["rows"])
        return {"blocks": s["idx"]}
    else:
        csa2.kv8_block_attn(s["cache"], s["q"], s["idx"], s["out"], s["ws"], lse=s["lse"], n_q=s["rows"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4m3_table():
    t = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t.append(-v if c & 128 else v)
    return torch.tensor(t, dtype=torch.float64, device="cuda")


def _round_e4m3(x):
    """x rounded to the grid of E4M3: three bits behind the leading one, steps of 2^-9 below 2^-6, at most 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > x.abs().clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(c, seed):
    if c["kind"] == "select":
        return None  # whole numbers: they have to be equal
    s = prepare(c, seed)
    B, T, H, Hkv, D, bs, kind = (s[x] for x in ("B", "T", "H", "Hkv", "D", "bs", "kind"))
    L, N, G = lengths(c), counts(c), H // Hkv
    value, table = _e4m3_table(), s["table"].tolist() if kind == "append" else s["table"].long()
    if kind == "append":
        if sum(N) * Hkv // bs > 4096:
            return None
        K, V, kb = value[s["k"].int()], value[s["v"].int()], value[s["kb"].int()]
        ks, vs = s["ks"].double(), s["vs"].double()
        for b in range(B):
            at = L[b] - N[b]
            while at < L[b]:
                end, i = min(L[b], (at // bs + 1) * bs), table[b][at // bs]
                r0, r1 = at % bs, at % bs + end - at
                for X, sc, x in ((K, ks, s["new"][0]), (V, vs, s["new"][1])):
                    x = x[b, at - L[b] + N[b]:end - L[b] + N[b]].double().transpose(0, 1)   # [Hkv, rows, D]
                    top = x.abs().amax((1, 2))
                    e = torch.ceil(torch.log2(top / 448)).clamp(-120, 120)
                    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, torch.where(top > 448 * torch.exp2(e), e + 1, e))
                    new = torch.exp2(e.clamp(-120, 120))
                    now = torch.maximum(new, sc[i]) if r0 else new
                    shrink = (sc[i] / now)[:, None, None]
                    if r0:
                        X[i, :, :r0] = _round_e4m3(X[i, :, :r0] * shrink)
                    X[i, :, r0:r1] = _round_e4m3(x / now[:, None, None])
                    if X is K:
                        lo, hi = torch.floor(X[i, :, r0:r1].amin(1)), torch.ceil(X[i, :, r0:r1].amax(1))
                        if r0:
                            lo = torch.minimum(lo, torch.floor(kb[i, :, 0] * shrink[:, 0]))
                            hi = torch.maximum(hi, torch.ceil(kb[i, :, 1] * shrink[:, 0]))
                        kb[i, :, 0], kb[i, :, 1] = lo, hi
                    sc[i] = now
                at = end
        return {"k": K, "v": V, "bounds": kb, "k_scale": ks, "v_scale": vs}

    def rows(codes, scales, b, t0, t1):
        """Rows [t0, t1) of sequence b: [Hkv, t1 - t0, D]."""
        blk = table[b, t0 // bs:(t1 + bs - 1) // bs]
        x = value[codes[blk].int()] * scales[blk].double()[:, :, None, None]
        return x.transpose(0, 1).reshape(Hkv, -1, D)[:, t0 % bs:t0 % bs + t1 - t0]

    if kind == "read":
        out = [o.double() for o in s["out"]]
        for b in range(B):
            if N[b]:
                out[0][b, :N[b]] = rows(s["k"], s["ks"], b, L[b] - N[b], L[b]).transpose(0, 1)
                out[1][b, :N[b]] = rows(s["v"], s["vs"], b, L[b] - N[b], L[b]).transpose(0, 1)
        return {"k": out[0], "v": out[1]}
    out, lse = s["out"].double(), s["lse"].double()
    if kind == "attn":
        for b in range(B):
            if not N[b]:
                continue
            p = torch.arange(L[b] - N[b], L[b], device="cuda")
            t0 = max(0, L[b] - N[b] - s["window"] + 1) // bs * bs if s["window"] else 0
            K, V = rows(s["k"], s["ks"], b, t0, L[b]), rows(s["v"], s["vs"], b, t0, L[b])
            t = torch.arange(t0, L[b], device="cuda")
            seen = (t <= p[:, None]) & ((t > p[:, None] - s["window"]) if s["window"] else (t >= 0))
            for h in range(Hkv):
                z = torch.einsum("jgd,td->gjt", s["q"][b, :N[b], h * G:(h + 1) * G].double(), K[h]) / math.sqrt(D)
                z = z.masked_fill(~seen, -math.inf)
                lse[b, :N[b], h * G:(h + 1) * G] = torch.logsumexp(z, -1).T
                out[b, :N[b], h * G:(h + 1) * G] = torch.einsum("gjt,td->jgd", torch.softmax(z, -1), V[h])
        return {"out": out, "lse": lse}
    chosen = s["idx"].tolist()
    for b in range(B):
        for j in range(N[b]):
            p = L[b] - N[b] + j
            for h in range(Hkv):
                i = torch.tensor([x for x in chosen[b][j][h] if x >= 0], device="cuda")
                t = (i[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)
                keep = t <= p
                blk = table[b, i]
                K = (value[s["k"][blk, h].int()] * s["ks"][blk, h].double()[:, None, None]).reshape(-1, D)[keep]
                V = (value[s["v"][blk, h].int()] * s["vs"][blk, h].double()[:, None, None]).reshape(-1, D)[keep]
                z = s["q"][b, j, h * G:(h + 1) * G].double() @ K.T / math.sqrt(D)
                lse[b, j, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[b, j, h * G:(h + 1) * G] = torch.softmax(z, -1) @ V
    return {"out": out, "lse": lse}
