"""What the 4-bit cache and the windows with sinks are measured on.

Three kinds of cases.  ``decode``: one new query per request over a cache held in 4 bits, or over a window whose first
tokens stay visible (``Cache.append``, ``Cache.decode``).  ``write``: rows quantised to 4 bits as they are written or
handed over from a bf16 cache, and read back (``Cache.append_rows``, ``Cache.copy_from``).  ``prompt``: packed prompts under
a window with sinks (``Cache.prompt``).  ``run`` computes them in elementary torch operations where ``own`` is false and
through the library's entry points where it is true.  Lengths come from the case itself (``shape`` seeds them), values
from the seed.

4 bits: each row of a head in groups of 32 dims with x ~ m + u s, m the group's minimum, s = (max - min) / 15 rounded to
bf16, u = rint((x - m) / s) in 0 .. 15.  Sinks: the query at p sees positions (p - window, p] and [0, sinks).
"""
import math
import random

import torch

own = False
GROUP = 32


def listed():
    return [
        # a step of one short conversation on an idle server: what counts is the latency of the two calls
        dict(name="4-bit step short", kind="decode", quant=True, dtype="bf16", batch=1, hq=32, hkv=8, d=128, lo=777, hi=777,
             window=0, sinks=0, ring=False, paged=False, base=0.0, step=True, shape=1),
        # long documents, whose cache only fits in 4 bits
        dict(name="4-bit decode long", kind="decode", quant=True, dtype="bf16", batch=8, hq=32, hkv=8, d=128, lo=131072,
             hi=131072, window=0, sinks=0, ring=False, paged=False, base=0.0, step=False, shape=2),
        # a server's batch of conversations of all lengths in one pool of pages, under a window with sinks
        dict(name="4-bit step ragged paged sinks", kind="decode", quant=True, dtype="bf16", batch=32, hq=32, hkv=8, d=128, lo=5,
             hi=20000, window=4096, sinks=4, ring=False, paged=True, base=10000.0, step=True, shape=3),
        # a model of many small heads, none of them shared
        dict(name="4-bit decode small heads", kind="decode", quant=True, dtype="bf16", batch=16, hq=32, hkv=32, d=64, lo=1, hi=4096,
             window=0, sinks=0, ring=False, paged=False, base=0.0, step=False, shape=4),
        # rings that have wrapped, eight query heads on each KV head
        dict(name="4-bit decode ring", kind="decode", quant=True, dtype="bf16", batch=4, hq=64, hkv=8, d=128, lo=30000, hi=40000,
             window=32768, sinks=0, ring=True, paged=False, base=0.0, step=False, shape=5),
        # prefills written in 4 bits into a pool of pages, and fetched from it
        dict(name="4-bit write ragged paged", kind="write", copy=False, batch=16, hkv=8, d=128, lo=5, hi=4096, paged=True, shape=6),
        # requests handed over from the cache of their prompts, and back for a next turn
        dict(name="4-bit hand-over and back", kind="write", copy=True, batch=8, hkv=8, d=128, lo=100, hi=16384, paged=False,
             shape=7),
        # one short prefill of small heads
        dict(name="4-bit write short", kind="write", copy=False, batch=1, hkv=4, d=64, lo=77, hi=77, paged=False, shape=8),
        # long conversations under a window with sinks, bf16
        dict(name="sinks decode", kind="decode", quant=False, dtype="bf16", batch=32, hq=32, hkv=8, d=128, lo=4097, hi=8192,
             window=4096, sinks=4, ring=False, paged=False, base=10000.0, step=False, shape=9),
        # a small model of fp32 (parity runs), an odd head size
        dict(name="sinks step fp32", kind="decode", quant=False, dtype="f32", batch=4, hq=8, hkv=2, d=80, lo=30, hi=3000,
             window=500, sinks=7, ring=False, paged=True, base=10000.0, step=True, shape=10),
        # one long document under the window
        dict(name="sinks prompt long", kind="prompt", dtype="bf16", batch=1, hq=32, hkv=8, d=128, lo=16384, hi=16384, prefix=0,
             window=4096, sinks=4, paged=False, base=10000.0, empty=0, shape=11),
        # suffixes behind reused prefixes in a pool of pages, some requests bring no row
        dict(name="sinks prompt ragged paged", kind="prompt", dtype="bf16", batch=12, hq=32, hkv=4, d=64, lo=1, hi=2100,
             prefix=3000, window=1024, sinks=100, paged=True, base=10000.0, empty=4, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode", "decode", "write", "write", "prompt", "prompt"])
    shape = rng.randrange(1 << 20)
    while True:
        if kind == "write":
            hi = _log(rng, 1, 20000)
            c = dict(kind=kind, copy=rng.random() < 0.5, batch=_log(rng, 1, 32), hkv=rng.choice([1, 2, 4, 8, 8, 32]),
                     d=rng.choice([64, 128, 128]), lo=rng.randint(1, hi), hi=hi, paged=rng.random() < 0.5, shape=shape)
        elif kind == "decode":
            quant = rng.random() < 0.65
            f32 = not quant and rng.random() < 0.25
            hq, hkv = rng.choice([(32, 8), (32, 8), (32, 32), (32, 4), (8, 2), (8, 1), (6, 2), (5, 5), (14, 2), (24, 2)])
            hi = _log(rng, 1, 5000 if f32 else 131072)
            window = _log(rng, 1, 32768) if not quant or rng.random() < 0.5 else 0
            ring = quant and window >= 16 and rng.random() < 0.4
            window -= window % 16 if ring else 0
            c = dict(kind=kind, quant=quant, dtype="f32" if f32 else "bf16", batch=_log(rng, 1, 48), hq=hq, hkv=hkv,
                     d=rng.choice([64, 80, 128]) if f32 else rng.choice([64, 128, 128]), lo=rng.randint(1, hi), hi=hi, window=window,
                     sinks=0 if ring or not window else _log(rng, 1, 200), ring=ring, paged=rng.random() < 0.4,
                     base=0.0 if quant else rng.choice([0.0, 10000.0]), step=not ring and rng.random() < 0.3, shape=shape)
        else:
            f32 = rng.random() < 0.15
            hq, hkv = rng.choice([(32, 8), (32, 32), (32, 4), (8, 2), (6, 2), (8, 1), (5, 5)])
            hi = _log(rng, 1, 600 if f32 else 12000)
            c = dict(kind=kind, dtype="f32" if f32 else "bf16", batch=_log(rng, 1, 32), hq=hq, hkv=hkv,
                     d=rng.choice([64, 80, 128]) if f32 else rng.choice([64, 128, 128]), lo=rng.randint(1, hi), hi=hi,
                     prefix=rng.choice([0, _log(rng, 1, 4000)]), window=_log(rng, 1, 4096), sinks=_log(rng, 1, 200),
                     paged=rng.random() < 0.4, base=rng.choice([0.0, 10000.0, 500000.0]), empty=rng.choice([0, 0, 3]), shape=shape)
        w = work(c)
        held = 0 if kind == "prompt" else 4 * c["batch"] * c["hkv"] * c["d"] * c["hi"]
        if w["flops"] <= (2e10 if c.get("dtype") == "f32" else 1e12) and w["bytes"] <= 1.4e9 and held <= 5e9:
            return c


# ---- shapes ----------------------------------------------------------------------------------------------------------
def _type(c):
    return torch.float32 if c.get("dtype") == "f32" else torch.bfloat16


def _elem(c):
    return _type(c).itemsize


def _lengths(c):
    """Rows that each request brings, and rows that it holds before (prompts)."""
    rng = random.Random(c["shape"])
    n = [rng.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]
    if c["kind"] != "prompt":
        return n, [0] * len(n)
    cut = [rng.randint(0, c["prefix"]) for _ in range(c["batch"])]
    if c["empty"]:
        n = [0 if b % c["empty"] == c["empty"] - 1 else x for b, x in enumerate(n)]
    return n, cut


def _visible(p, c):
    """Keys that the query at p sees."""
    first = max(0, p - c["window"] + 1) if c["window"] else 0
    return p + 1 - first + min(c["sinks"], first)


def work(case):
    c = case
    n, cut = _lengths(c)
    t = sum(n)
    if c["kind"] == "write":
        rows = 2 * t * c["hkv"] * c["d"]                    # read as bf16, written in 4 bits; read so, written as bf16
        return {"bytes": int(rows * (2 + 0.625) * 2), "flops": 6 * rows}
    if c["kind"] == "decode":
        # every visible row once, a new row as it comes, the queries and what they get
        keys = sum(_visible(x + c["step"] - 1, c) for x in n)
        row = 2 * c["hkv"] * c["d"] * (0.625 if c["quant"] else _elem(c))
        new = 2 * c["hkv"] * c["d"] * _elem(c) * c["batch"] * c["step"]
        return {"bytes": int(keys * row + new + 2 * c["batch"] * c["hq"] * c["d"] * _elem(c)), "flops": 4 * keys * c["hq"] * c["d"]}
    row = 2 * c["hkv"] * c["d"] * _elem(c)
    reach = sum(_visible(x - 1, c) if x else 0 for x, m in zip(cut, n) if m)
    flops = 0
    for x, m in zip(n, cut):
        grow = max(0, min(x, c["window"] + c["sinks"] - m))  # queries that see every key before them
        flops += grow * m + grow * (grow + 1) // 2 + (x - grow) * (c["window"] + c["sinks"])
    size = 2 * t * c["hq"] * c["d"] * _elem(c) + row * (2 * t + reach)
    if c["paged"]:
        size += 2 * row * sum(x + y for x, y in zip(n, cut))  # the hand-over
    return {"bytes": size, "flops": 4 * c["hq"] * c["d"] * flops}


def _capacity(c):
    n, cut = _lengths(c)
    if c["kind"] == "decode" and c["ring"]:
        return c["window"]
    return -(-(max(x + y for x, y in zip(n, cut)) + 1) // 16) * 16


# ---- inputs ----------------------------------------------------------------------------------------------------------
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _rows(gen, shape, dtype, wide):
    """Rows [requests, heads, n, d]: keys have dims of much larger size and with a mean of their own (wide)."""
    x = torch.empty(shape, device="cuda", dtype=dtype)
    size = torch.exp(torch.randn((1, shape[1], 1, shape[3]), generator=gen, device="cuda") * (0.7 if wide else 0.2))
    mean = torch.randn((1, shape[1], 1, shape[3]), generator=gen, device="cuda") * (1.0 if wide else 0.1)
    for b in range(shape[0]):
        x[b:b + 1] = torch.randn((1,) + tuple(shape[1:]), generator=gen, device="cuda") * size + mean
    return x


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 29)
    t = _type(c)
    n, cut = _lengths(c)
    if c["kind"] == "prompt":
        qkv = _normal(gen, (sum(n), c["hq"] + 2 * c["hkv"], c["d"]), t)          # one projection's output, three views
        q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        shape = (c["batch"], c["hkv"], max(cut), c["d"])
        return dict(q=q, k=k, v=v, pk=_normal(gen, shape, t), pv=_normal(gen, shape, t))
    shape = (c["batch"], c["hkv"], max(n), c["d"])
    x = dict(k=_rows(gen, shape, t, True), v=_rows(gen, shape, t, False))
    if c["kind"] == "decode":
        x["q"] = _normal(gen, (c["batch"], c["hq"], c["d"]), t)
        x["k1"] = _rows(gen, (c["batch"], c["hkv"], 1, c["d"]), t, True)[:, :, 0].contiguous()
        x["v1"] = _rows(gen, (c["batch"], c["hkv"], 1, c["d"]), t, False)[:, :, 0].contiguous()
    return x


def _rotated(x, pos, base):
    """x [..., rows, d] rotated at pos [rows], pairs (2i, 2i + 1); angles in 64 bits, the rest in 32, rounded once."""
    if not base:
        return x
    d = x.shape[-1]
    theta = float(base) ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    angle = pos.double()[:, None] * theta
    cos, sin = angle.cos().float(), angle.sin().float()
    x0, x1 = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack((x0 * cos - x1 * sin, x1 * cos + x0 * sin), -1).flatten(-2).to(x.dtype)


def _quantised(x):
    """Codes (uint8), scales and minima (bf16) of rows [..., d]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((hi - lo) / torch.full_like(lo, 15)).to(torch.bfloat16)          # (by a number, it would be times its reciprocal)
    u = torch.where(s > 0, ((g - lo) / s.float()).round().clamp(0, 15), torch.zeros_like(g))
    return u.to(torch.uint8), s, lo.to(torch.bfloat16)


def _values(u, s, m):
    """The values that the codes stand for, in 32 bits."""
    return (u.float() * s.float() + m.float()).flatten(-2)


def prepare(case, seed):
    c = case
    st = dict(case=c, **_inputs(c, seed))
    st["n"], st["cut"] = _lengths(c)
    cap = _capacity(c)
    if c["kind"] == "prompt":
        st["out"] = torch.empty((sum(st["n"]), c["hq"], c["d"]), dtype=_type(c), device="cuda")
    if own:
        _prepare_own(st, c, cap)
        return st
    shape = (c["batch"], c["hkv"], cap, c["d"])
    if c["kind"] == "write":
        return st
    if c["kind"] == "prompt":
        st["kc"], st["vc"] = (torch.zeros(shape, dtype=_type(c), device="cuda") for _ in "kv")
        for b, m in enumerate(st["cut"]):
            st["kc"][b, :, :m] = _rotated(st["pk"][b, :, :m], torch.arange(m, device="cuda"), c["base"])
            st["vc"][b, :, :m] = st["pv"][b, :, :m]
        return st
    # decode: slot = position, mod the window on a ring; in 4 bits codes, scales and minima of the rows
    for name in ("k", "v"):
        rows = st.pop(name)
        full = torch.zeros(shape, dtype=_type(c), device="cuda")
        for b, x in enumerate(st["n"]):
            pos = torch.arange(max(0, x - cap), x, device="cuda")
            part = rows[b][:, max(0, x - cap):x]
            full[b][:, pos % cap] = _rotated(part, pos, c["base"]) if name == "k" else part
        del rows
        st[name + "c"] = tuple(torch.stack(y) for y in zip(*map(_quantised, full))) if c["quant"] else (full,)
    return st


def _prepare_own(st, c, cap):
    from kv_cache_decode_ring_gb300 import kvc
    n, cut = st["n"], st["cut"]
    pages = sum(-(-min(x + y + 1, cap) // 16) for x, y in zip(n, cut)) if c["paged"] else 0
    cfg = dict(batch=c["batch"], n_kv_heads=c["hkv"], head_dim=c["d"], capacity=cap)
    if c["kind"] == "write":
        plain = dict(cfg, n_q_heads=c["hkv"])
        st["dense"] = kvc.Cache(kvc.make_config(**plain))
        if c["copy"]:
            st["source"] = kvc.Cache(kvc.make_config(**plain))
            st["source"].append_rows(st["k"], st["v"], counts=n)
        st["cache"] = kvc.Cache(kvc.make_config(kv_quant="int4", page_pool=pages, **plain))
        st["rows"] = st["dense"].rows()
        return
    cfg.update(dtype=c["dtype"], n_q_heads=c["hq"], window=c["window"] if c["kind"] == "prompt" or not c["ring"] else 0,
               sinks=c["sinks"], rope_base=c["base"])
    if c["kind"] == "decode":
        st["cache"] = kvc.Cache(kvc.make_config(kv_quant="int4" if c["quant"] else None,
                                                layout="ring" if c["ring"] else "contiguous", page_pool=pages, **cfg))
        st["cache"].append_rows(st.pop("k"), st.pop("v"), counts=n)
        if c["step"]:
            st["cache"].append(st["k1"], st["v1"])
        return
    st["cache"] = kvc.Cache(kvc.make_config(page_pool=pages, **cfg))
    if max(cut):
        st["cache"].append_rows(st["pk"], st["pv"], counts=cut)
    st["dense"] = kvc.Cache(kvc.make_config(**cfg)) if c["paged"] else st["cache"]
    st["rows"] = st["dense"].rows()


# ---- the operators through the library ---------------------------------------------------------------------------------
def _run_own(st):
    c, cache = st["case"], st["cache"]
    every = range(c["batch"])
    if c["kind"] == "decode":
        if c["step"]:
            cache.trim(st["n"])
            cache.append(st["k1"], st["v1"])
        return cache.decode(st["q"])
    if c["kind"] == "write":
        if c["copy"]:
            cache.copy_from(st["source"], every, every)
        else:
            cache.trim(st["cut"])
            cache.append_rows(st["k"], st["v"], counts=st["n"])
        st["dense"].copy_from(cache, every, every)
        return dict(k=st["rows"][0], v=st["rows"][1])
    cache.trim(st["cut"])
    cache.prompt(st["q"], st["k"], st["v"], st["n"], st["out"])
    if c["paged"]:
        st["dense"].copy_from(cache, every, every)
    return dict(out=st["out"], k=st["rows"][0], v=st["rows"][1])


# ---- their plain forms ---------------------------------------------------------------------------------------------------
def _attend(q, k, v, seen):
    """q [n, hq, d] over k, v [hkv, m, d] where seen [n, m]; 32 bits."""
    n, hq, d = q.shape
    hkv = k.shape[0]
    s = q.float().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3) @ k[:, None].float().transpose(-1, -2)
    s = (s / math.sqrt(d)).masked_fill(~seen, -math.inf)
    w = torch.exp(s - s.amax(-1, keepdim=True))
    o = (w @ v[:, None].float()) / w.sum(-1, keepdim=True)
    return o.permute(2, 0, 1, 3).reshape(n, hq, d)


def _plain_decode(st):
    c, q = st["case"], st["q"]
    cap = _capacity(c)
    out = torch.empty_like(q)
    for b, x in enumerate(st["n"]):
        if c["step"]:
            at = torch.tensor([x], device=q.device)
            for held, row in ((st["kc"], _rotated(st["k1"][b][:, None], at, c["base"])), (st["vc"], st["v1"][b][:, None])):
                for full, part in zip(held, _quantised(row) if c["quant"] else (row,)):
                    full[b][:, x % cap] = part[:, 0]
            x += 1
        if c["ring"]:
            slots = torch.arange(min(x, cap), device=q.device)
        else:
            first = max(0, x - c["window"]) if c["window"] else 0
            slots = torch.cat((torch.arange(min(c["sinks"], first), device=q.device), torch.arange(first, x, device=q.device)))
        kv = [_values(*(full[b][:, slots] for full in held)) if c["quant"] else held[0][b][:, slots] for held in (st["kc"], st["vc"])]
        qb = _rotated(q[b].float(), torch.tensor([x - 1], device=q.device), c["base"])
        out[b] = _attend(qb[None], kv[0], kv[1], torch.ones((1, len(slots)), dtype=torch.bool, device=q.device))[0].to(out.dtype)
    return out


def _plain_write(st):
    c = st["case"]
    held = []
    for rows in (st["k"], st["v"]):
        dense = torch.zeros((c["batch"], c["hkv"], _capacity(c), c["d"]), dtype=torch.bfloat16, device="cuda")
        for b, x in enumerate(st["n"]):
            dense[b, :, :x] = _values(*_quantised(rows[b, :, :x])).to(torch.bfloat16)
        held.append(dense)
    return dict(k=held[0], v=held[1])


def run(state):
    st, c = state, state["case"]
    if own:
        return _run_own(st)
    if c["kind"] == "decode":
        return _plain_decode(st)
    if c["kind"] == "write":
        return _plain_write(st)
    kc, vc, at = st["kc"], st["vc"], 0
    for b, (n, cut) in enumerate(zip(st["n"], st["cut"])):
        if n == 0:
            continue
        pos = torch.arange(cut, cut + n, device="cuda")
        q, k, v = (st[x][at:at + n].transpose(0, 1) for x in "qkv")
        q, k = _rotated(q, pos, c["base"]).transpose(0, 1), _rotated(k, pos, c["base"])
        kc[b, :, cut:cut + n], vc[b, :, cut:cut + n] = k, v
        step = max(1, (1 << 29) // (c["hq"] * (c["window"] + c["sinks"] + 512)))          # rows whose scores fit memory
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            first = max(0, cut + i0 - c["window"] + 1)
            j = torch.cat((torch.arange(min(c["sinks"], first), device="cuda"), torch.arange(first, cut + i1, device="cuda")))
            p = pos[i0:i1, None]
            seen = (j <= p) & ((j > p - c["window"]) | (j < c["sinks"]))
            st["out"][at + i0:at + i1] = _attend(q[i0:i1], kc[b][:, j], vc[b][:, j], seen).to(_type(c))
        at += n
    return dict(out=st["out"], k=kc, v=vc)


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------------
def _turn(x, pos, base):
    """Complex rotation of the pairs (2i, 2i + 1) of x [..., rows, d] at pos [rows], in 64 bits."""
    if not base:
        return x.double()
    d = x.shape[-1]
    spectrum = torch.tensor([base ** (-2 * i / d) for i in range(d // 2)], device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None] * spectrum
    z = torch.view_as_complex(x.double().contiguous().unflatten(-1, (-1, 2))) * torch.polar(torch.ones_like(angle), angle)
    return torch.view_as_real(z).flatten(-2)


def _held4(x):
    """What 4 bits hold of rows [..., d] (bf16 values), in 64 bits."""
    y = x.double()
    g = y.reshape(*y.shape[:-1], y.shape[-1] // GROUP, GROUP)
    low = g.min(-1, keepdim=True).values
    scale = ((g.max(-1, keepdim=True).values - low) / torch.full_like(low, 15.0)).to(torch.bfloat16).double()
    code = torch.nan_to_num((g - low) / scale, nan=0.0, posinf=0.0).round().clamp(0.0, 15.0)
    return (low + code * scale).reshape(y.shape)


def exact(case, seed):
    c = case
    x = _inputs(c, seed)
    n, cut = _lengths(c)
    cap = _capacity(c)
    t = _type(c)
    if c["kind"] == "write":
        out = {}
        for name in "kv":
            dense = torch.zeros((c["batch"], c["hkv"], cap, c["d"]), device="cuda", dtype=torch.float64)
            for b in range(c["batch"]):
                dense[b, :, :n[b]] = _held4(x[name][b, :, :n[b]])
            out[name] = dense
        return out
    group = c["hq"] // c["hkv"]
    if c["kind"] == "decode":
        out = torch.zeros((c["batch"], c["hq"], c["d"]), device="cuda", dtype=torch.float64)
        for b in range(c["batch"]):
            kb, vb, end = x["k"][b, :, :n[b]], x["v"][b, :, :n[b]], n[b]
            if c["step"]:
                kb, vb, end = torch.cat((kb, x["k1"][b][:, None]), 1), torch.cat((vb, x["v1"][b][:, None]), 1), end + 1
            pos = torch.arange(end, device="cuda")
            seen = (pos >= 0) if not c["window"] else (pos >= end - c["window"]) | (pos < c["sinks"])
            pos, kb, vb = pos[seen], kb[:, seen], vb[:, seen]
            for h in range(c["hkv"]):
                # keys enter the products as the cache holds them, the query as it is
                kh, vh = _turn(kb[h], pos, c["base"]).to(t), vb[h]
                kh, vh = (_held4(kh), _held4(vh)) if c["quant"] else (kh.double(), vh.double())
                qh = _turn(x["q"][b, h * group:(h + 1) * group], torch.full((1,), end - 1, device="cuda"), c["base"])
                out[b, h * group:(h + 1) * group] = (qh @ kh.T / math.sqrt(c["d"])).softmax(-1) @ vh
        return out
    if 4 * c["hq"] * c["d"] * sum(a * (a + b) for a, b in zip(n, cut)) > 6e12:
        return None
    k = torch.zeros((c["batch"], c["hkv"], cap, c["d"]), device="cuda", dtype=torch.float64)
    v = torch.zeros_like(k)
    out = torch.zeros((sum(n), c["hq"], c["d"]), device="cuda", dtype=torch.float64)
    at = 0
    for b in range(c["batch"]):
        end = cut[b] + n[b]
        pos = torch.arange(end, device="cuda")
        k[b, :, :end] = _turn(torch.cat((x["pk"][b, :, :cut[b]], x["k"][at:at + n[b]].transpose(0, 1)), 1), pos, c["base"])
        v[b, :, :end] = torch.cat((x["pv"][b, :, :cut[b]], x["v"][at:at + n[b]].transpose(0, 1)), 1).double()
        for h in range(c["hq"] if n[b] else 0):
            # queries and keys enter the products as the cache's type holds them
            kh = k[b, h // group, :end].to(t).double()
            qh = _turn(x["q"][at:at + n[b], h], pos[cut[b]:], c["base"]).to(t).double()
            for i0 in range(0, n[b], 4096):
                i1 = min(n[b], i0 + 4096)
                s = qh[i0:i1] @ kh[:cut[b] + i1].T / math.sqrt(c["d"])
                away = pos[cut[b] + i0:cut[b] + i1, None] - pos[:cut[b] + i1]
                s[(away < 0) | ((away >= c["window"]) & (pos[:cut[b] + i1] >= c["sinks"]))] = -math.inf
                out[at + i0:at + i1, h] = s.softmax(-1) @ v[b, h // group, :cut[b] + i1]
        at += n[b]
    return dict(out=out, k=k, v=v)
