"""What the prompt, page and multi-axis rotary operators are measured on.

Three kinds of cases.  ``prompt``: packed prompts of different lengths, appended to a cache and attended causally
(``Cache.prompt``).  ``pages``: requests of a cache forked into branches, copied into another cache, freed and compacted
(``Cache.fork``, ``copy_from``, ``free``, ``compact``).  ``rope``: rotary positions with several axes
(``kvc_rope_axes``).  ``run`` computes them in elementary torch operations where ``own`` is false and through the
library's entry points where it is true.  Lengths come from the case itself (``shape`` seeds them), values from the seed.
"""
import math
import random

import torch

own = False


def listed():
    return [
        # one short question to an idle server: what counts is the latency of a call
        dict(name="prompt short", kind="prompt", dtype="bf16", batch=1, hq=32, hkv=8, d=128, lo=37, hi=37, prefix=0,
             window=0, paged=False, base=10000.0, empty=0, shape=1),
        # sixteen requests arrive together in a paged pool and are handed over to the decode cache
        dict(name="prompt ragged paged", kind="prompt", dtype="bf16", batch=16, hq=32, hkv=8, d=128, lo=5, hi=1500, prefix=0,
             window=0, paged=True, base=10000.0, empty=0, shape=2),
        # one long document
        dict(name="prompt long", kind="prompt", dtype="bf16", batch=1, hq=32, hkv=8, d=128, lo=16384, hi=16384, prefix=0,
             window=0, paged=False, base=10000.0, empty=0, shape=3),
        # a sliding-window model with small heads: suffixes behind reused prefixes, some requests bring no row
        dict(name="prompt window prefix", kind="prompt", dtype="bf16", batch=12, hq=32, hkv=4, d=64, lo=1, hi=2100, prefix=3000,
             window=1024, paged=False, base=10000.0, empty=4, shape=4),
        # a small fp32 cache (parity runs of a model)
        dict(name="prompt fp32", kind="prompt", dtype="f32", batch=4, hq=8, hkv=2, d=128, lo=30, hi=300, prefix=100,
             window=0, paged=False, base=10000.0, empty=0, shape=5),
        # one prompt into sixteen samples, each with rows of its own
        dict(name="fork rows", kind="pages", op="fork", dtype="bf16", sources=1, branches=16, hkv=8, d=128, lo=4096, hi=4096,
             shape=6),
        # a step of parallel sampling on shared pages, handed over to a decode cache
        dict(name="fork pages, append, copy", kind="pages", op="branch", dtype="bf16", sources=8, branches=7, hkv=8, d=128,
             lo=100, hi=1000, shape=7),
        # requests leave, the pool is compacted, new ones come, the whole is handed over
        dict(name="free, compact, refill", kind="pages", op="compact", dtype="bf16", sources=24, branches=0, hkv=8, d=128,
             lo=17, hi=3000, shape=8),
        # a decode step's queries and keys in one projection output: latency counts
        dict(name="rope step", kind="rope", dtype="bf16", rows=64, heads=40, cols=48, d=128, sections="16,24,24", halves=False,
             per_axis=False, base=10000.0, far=100000),
        # the tokens of a long video: a spectrum for each of time, height and width
        dict(name="rope video", kind="rope", dtype="bf16", rows=32760, heads=24, cols=24, d=128, sections="22,21,21", halves=True,
             per_axis=True, base=10000.0, far=500),
        # fp32, two axes over a part of each head
        dict(name="rope image fp32", kind="rope", dtype="f32", rows=4097, heads=13, cols=13, d=80, sections="16,16", halves=True,
             per_axis=False, base=500.0, far=70),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "prompt", "pages", "pages", "rope"])
    shape = rng.randrange(1 << 20)
    while True:
        if kind == "prompt":
            f32 = rng.random() < 0.15
            hq, hkv = rng.choice([(32, 8), (32, 32), (32, 4), (8, 2), (6, 2), (8, 1), (5, 5)])
            hi = _log(rng, 1, 600 if f32 else 12000)
            c = dict(kind=kind, dtype="f32" if f32 else "bf16", batch=_log(rng, 1, 32), hq=hq, hkv=hkv,
                     d=rng.choice([64, 80, 128]) if f32 else rng.choice([64, 128, 128]), lo=rng.randint(1, hi), hi=hi,
                     prefix=rng.choice([0, _log(rng, 1, 4000)]), window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                     paged=rng.random() < 0.4, base=rng.choice([0.0, 10000.0, 500000.0]), empty=rng.choice([0, 0, 3]), shape=shape)
        elif kind == "pages":
            op = rng.choice(["fork", "branch", "compact"])
            hi = _log(rng, 1, 6000)
            c = dict(kind=kind, op=op, dtype=rng.choice(["bf16", "bf16", "f32"]),
                     sources=rng.randint(2, 32) if op == "compact" else rng.randint(1, 8),
                     branches=0 if op == "compact" else _log(rng, 1, 24), hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 80, 128]),
                     lo=rng.randint(1, hi), hi=hi, shape=shape)
        else:
            d = rng.choice([64, 80, 96, 128])
            axes = rng.choice([1, 2, 3])
            left, sections = d // 2 - rng.choice([0, 0, 8]), []
            for a in range(axes - 1):
                sections.append(rng.randint(1, left - (axes - 1 - a)))
                left -= sections[-1]
            sections.append(left)
            heads = rng.randint(1, 48)
            c = dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=_log(rng, 1, 30000), heads=heads,
                     cols=heads + rng.choice([0, 0, 8]), d=d, sections=",".join(map(str, sections)), halves=rng.random() < 0.5,
                     per_axis=rng.random() < 0.5, base=rng.choice([100.0, 10000.0, 1000000.0]), far=_log(rng, 10, 2000000))
        w = work(c)
        if w["flops"] <= (2e10 if c["dtype"] == "f32" else 2.2e12) and w["bytes"] <= 4e8:
            return c


# ---- shapes ----------------------------------------------------------------------------------------------------------
def _elem(c):
    return 2 if c["dtype"] == "bf16" else 4


def _type(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _lengths(c):
    """Prompt rows and cached prefix rows of each request."""
    rng = random.Random(c["shape"])
    n = [rng.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]
    cut = [rng.randint(0, c["prefix"]) for _ in range(c["batch"])]
    if c["empty"]:
        n = [0 if b % c["empty"] == c["empty"] - 1 else x for b, x in enumerate(n)]
    return n, cut


def _held(c):
    """Rows of each source request (pages cases)."""
    rng = random.Random(c["shape"])
    return [rng.randint(c["lo"], c["hi"]) for _ in range(c["sources"])]


def _branches(c):
    """The source of every slot: sources first, then their branches in turn."""
    m = c["sources"]
    return list(range(m)) + [i % m for i in range(m * c["branches"])]


def _keys(n, cut, window):
    """Visible keys of all queries at cut .. cut + n - 1."""
    if not window:
        return n * cut + n * (n + 1) // 2
    grow = max(0, min(n, window - cut))          # queries that still see everything
    return grow * cut + grow * (grow + 1) // 2 + (n - grow) * window


def work(case):
    c = case
    if c["kind"] == "rope":
        n = c["rows"] * c["heads"] * c["d"]
        axes = len(c["sections"].split(","))
        return {"bytes": 2 * n * _elem(c) + 4 * axes * c["rows"], "flops": 3 * n}
    row = 2 * c["hkv"] * c["d"] * _elem(c)                                   # a key and its value, every head
    if c["kind"] == "pages":
        held = _held(c)
        if c["op"] == "fork":                                                # each source read once, each branch written once
            return {"bytes": row * sum(held) * (1 + c["branches"]), "flops": 0}
        if c["op"] == "branch":                                              # prompts and new rows read, the dense copy written
            slots = [held[s] for s in _branches(c)]
            return {"bytes": row * (sum(held) + len(slots) + sum(x + 1 for x in slots)), "flops": 0}
        moved = sum(-(-x // 16) * 16 for x in held)                          # each half moves down once
        return {"bytes": row * (2 * sum(held) + 2 * moved + 2 * sum(held)), "flops": 0}
    n, cut = _lengths(c)
    t = sum(n)
    reach = sum(x - max(0, x - c["window"] + 1) if c["window"] else x for x, m in zip(cut, n) if m)
    size = 2 * t * c["hq"] * c["d"] * _elem(c) + row * (2 * t + reach)
    if c["paged"]:
        size += 2 * row * sum(x + y for x, y in zip(n, cut))                # the hand-over
    return {"bytes": size, "flops": 4 * c["hq"] * c["d"] * sum(_keys(x, y, c["window"]) for x, y in zip(n, cut))}


# ---- inputs ----------------------------------------------------------------------------------------------------------
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    t = _type(c)
    if c["kind"] == "rope":
        axes = len(c["sections"].split(","))
        x = _normal(gen, (c["rows"], c["cols"], c["d"]), t)
        pos = torch.randint(0, c["far"], (axes, c["rows"]), generator=gen, device="cuda", dtype=torch.int32)
        return dict(x=x[:, :c["heads"]], pos=pos)
    if c["kind"] == "pages":
        held = _held(c)
        m, s = c["sources"], max(held)
        new = m * (1 + c["branches"])
        return dict(k=_normal(gen, (m, c["hkv"], s, c["d"]), t), v=_normal(gen, (m, c["hkv"], s, c["d"]), t),
                    k1=_normal(gen, (new, c["hkv"], c["d"]), t), v1=_normal(gen, (new, c["hkv"], c["d"]), t))
    n, cut = _lengths(c)
    qkv = _normal(gen, (sum(n), c["hq"] + 2 * c["hkv"], c["d"]), t)          # one projection's output, three views
    q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
    shape = (c["batch"], c["hkv"], max(cut), c["d"])
    return dict(q=q, k=k, v=v, pk=_normal(gen, shape, t), pv=_normal(gen, shape, t))


def _capacity(c):
    if c["kind"] == "prompt":
        s = max(x + y for x, y in zip(*_lengths(c)))
        return -(-s // 16) * 16 if c["paged"] else max(s, 1)
    return -(-(max(_held(c)) + 1) // 16) * 16


def prepare(case, seed):
    c = case
    st = dict(case=c, **_inputs(c, seed))
    if c["kind"] == "rope":
        st["sections"] = [int(x) for x in c["sections"].split(",")]
        st["out"] = torch.empty((c["rows"], c["heads"], c["d"]), dtype=_type(c), device="cuda")
        return st
    cap = _capacity(c)
    if c["kind"] == "pages":
        st["held"], st["source"] = _held(c), _branches(c)
        slots = len(st["source"])
        st["cut"] = st["held"] + [0] * (slots - len(st["held"]))
    else:
        st["n"], st["cut"] = _lengths(c)
        slots = c["batch"]
        st["out"] = torch.empty((sum(st["n"]), c["hq"], c["d"]), dtype=_type(c), device="cuda")
    if own:
        _prepare_own(st, c, cap, slots)
        return st
    st["kc"] = torch.zeros((slots, c["hkv"], cap, c["d"]), dtype=_type(c), device="cuda")
    st["vc"] = torch.zeros_like(st["kc"])
    k, v = (st["k"], st["v"]) if c["kind"] == "pages" else (st["pk"], st["pv"])
    for b, m in enumerate(st["cut"]):
        if m:
            kb = k[b, :, :m]
            if c["kind"] == "prompt" and c["base"]:
                kb = _rotated(kb.transpose(0, 1), torch.arange(m, device="cuda"), c["base"]).transpose(0, 1)
            st["kc"][b, :, :m] = kb
            st["vc"][b, :, :m] = v[b, :, :m]
    if c["kind"] == "pages" and c["op"] == "branch":
        st["last"] = torch.tensor([st["held"][s] for s in st["source"]], device="cuda")
    return st


def _prepare_own(st, c, cap, slots):
    from kv_cache_decode_ring_gb300 import kvc
    pad = lambda x: torch.cat((x, x.new_zeros((slots - x.shape[0],) + tuple(x.shape[1:]))))  # noqa: E731
    if c["kind"] == "prompt":
        pages = sum(-(-(x + y) // 16) for x, y in zip(st["n"], st["cut"])) if c["paged"] else 0
        cfg = dict(dtype=c["dtype"], batch=slots, n_q_heads=c["hq"], n_kv_heads=c["hkv"], head_dim=c["d"], capacity=cap,
                   window=c["window"] if c["window"] < cap else 0, rope_base=c["base"])
        k, v, paged = st["pk"], st["pv"], c["paged"]
    else:
        pages = 0 if c["op"] == "fork" else sum(-(-x // 16) for x in st["held"]) + 2 * slots
        cfg = dict(dtype=c["dtype"], batch=slots, n_q_heads=c["hkv"], n_kv_heads=c["hkv"], head_dim=c["d"], capacity=cap)
        k, v, paged = pad(st["k"]), pad(st["v"]), c["op"] != "fork"
    st["cache"] = kvc.Cache(kvc.make_config(page_pool=pages, **cfg))
    if max(st["cut"]):
        st["cache"].append_rows(k.contiguous(), v.contiguous(), counts=st["cut"])
    st["dense"] = kvc.Cache(kvc.make_config(**cfg)) if paged else st["cache"]
    st["rows"] = st["dense"].rows()


# ---- the operators through the library ---------------------------------------------------------------------------------
def _run_own(st):
    c = st["case"]
    if c["kind"] == "rope":
        from kv_cache_decode_ring_gb300 import kvc
        return kvc.kvc_rope_axes(st["x"], st["pos"], st["sections"], c["base"], st["out"], halves=c["halves"], per_axis=c["per_axis"])
    cache, (kd, vd) = st["cache"], st["rows"]
    if c["kind"] == "prompt":
        cache.trim(st["cut"])
        cache.prompt(st["q"], st["k"], st["v"], st["n"], st["out"])
        if c["paged"]:
            every = range(c["batch"])
            st["dense"].copy_from(cache, every, every)
        return dict(out=st["out"], k=kd, v=vd)
    m, slots = c["sources"], len(st["source"])
    if c["op"] == "fork":
        cache.fork(st["source"][m:], range(m, slots))
        return dict(k=kd, v=vd)
    every = range(slots)
    if c["op"] == "branch":
        cache.fork(st["source"][m:], range(m, slots))
        cache.append(st["k1"], st["v1"])
        st["dense"].copy_from(cache, every, every)
        cache.free(range(m, slots))
        cache.trim(st["cut"])
        return dict(k=kd, v=vd)
    used = []
    for odd in (1, 0):
        cache.free(range(odd, slots, 2))
        used.append(cache.compact())
        cache.append_rows(st["k"], st["v"], counts=[x if b % 2 == odd else 0 for b, x in enumerate(st["held"])])
    st["dense"].copy_from(cache, every, every)
    return dict(k=kd, v=vd, used=used)


# ---- their plain forms ---------------------------------------------------------------------------------------------------
def _rotated(x, pos, base):
    """x [rows, heads, d] rotated at pos [rows], pairs (2i, 2i + 1); angles in 64 bits, the rest in 32, rounded once."""
    d = x.shape[-1]
    theta = float(base) ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    angle = pos.double()[:, None] * theta
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x0, x1 = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack((x0 * cos - x1 * sin, x1 * cos + x0 * sin), -1).flatten(-2).to(x.dtype)


def _attend(q, k, v, cut, window, out):
    """q [n, hq, d] at positions cut .. cut + n - 1 over k, v [hkv, cut + n, d], in blocks of rows that fit memory."""
    n, hq, d = q.shape
    hkv = k.shape[0]
    step = max(1, (1 << 29) // (hq * k.shape[1]))
    for i0 in range(0, n, step):
        i1 = min(n, i0 + step)
        lo, hi = max(0, cut + i0 - window + 1) if window else 0, cut + i1
        p = torch.arange(cut + i0, cut + i1, device=q.device)[:, None]
        j = torch.arange(lo, hi, device=q.device)
        seen = (j <= p) & ((j > p - window) if window else (j >= 0))
        s = q[i0:i1].float().view(i1 - i0, hkv, hq // hkv, d).permute(1, 2, 0, 3) @ k[:, None, lo:hi].float().transpose(-1, -2)
        s = (s / math.sqrt(d)).masked_fill(~seen, -math.inf)
        w = torch.exp(s - s.amax(-1, keepdim=True))
        o = (w @ v[:, None, lo:hi].float()) / w.sum(-1, keepdim=True)
        out[i0:i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, hq, d).to(out.dtype)


def run(state):
    st, c = state, state["case"]
    if own:
        return _run_own(st)
    if c["kind"] == "rope":
        return _rope_plain(st)
    kc, vc = st["kc"], st["vc"]
    if c["kind"] == "prompt":
        at = 0
        for b, (n, cut) in enumerate(zip(st["n"], st["cut"])):
            if n == 0:
                continue
            q, k, v = (st[x][at:at + n] for x in "qkv")
            if c["base"]:
                pos = torch.arange(cut, cut + n, device=q.device)
                q, k = _rotated(q, pos, c["base"]), _rotated(k, pos, c["base"])
            kc[b, :, cut:cut + n] = k.transpose(0, 1)
            vc[b, :, cut:cut + n] = v.transpose(0, 1)
            _attend(q, kc[b, :, :cut + n], vc[b, :, :cut + n], cut, c["window"], st["out"][at:at + n])
            at += n
        return dict(out=st["out"], k=kc, v=vc)
    m = c["sources"]
    if c["op"] == "compact":
        for b, n in enumerate(st["held"]):
            kc[b, :, :n] = st["k"][b, :, :n]
            vc[b, :, :n] = st["v"][b, :, :n]
        pages = [-(-x // 16) for x in st["held"]]
        return dict(k=kc, v=vc, used=[sum(pages[0::2]), sum(pages[1::2])])
    for slot in range(m, len(st["source"])):
        src = st["source"][slot]
        n = st["held"][src]
        kc[slot, :, :n] = kc[src, :, :n]
        vc[slot, :, :n] = vc[src, :, :n]
    if c["op"] == "branch":
        each = torch.arange(len(st["source"]), device=kc.device)
        kc[each, :, st["last"]] = st["k1"]
        vc[each, :, st["last"]] = st["v1"]
    return dict(k=kc, v=vc)


def _pairs(c, sections):
    """Exponents (of the base) and axes of the rotated pairs."""
    total = sum(sections)
    axis = [a for a, s in enumerate(sections) for _ in range(s)]
    if c["per_axis"]:
        return [-j / s for s in sections for j in range(s)], axis
    return [-i / total for i in range(total)], axis


def _rope_plain(st):
    c, x, out = st["case"], st["x"], st["out"]
    exps, axis = _pairs(c, st["sections"])
    p = len(axis)
    theta = torch.tensor([c["base"] ** e for e in exps], device=x.device, dtype=torch.float64)
    angle = st["pos"].double()[torch.tensor(axis, device=x.device)].T * theta                        # [rows, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    first, second = (slice(0, p), slice(p, 2 * p)) if c["halves"] else (slice(0, 2 * p, 2), slice(1, 2 * p, 2))
    x0, x1 = x[..., first].float(), x[..., second].float()
    out[..., first] = (x0 * cos - x1 * sin).to(out.dtype)
    out[..., second] = (x1 * cos + x0 * sin).to(out.dtype)
    out[..., 2 * p:] = x[..., 2 * p:]
    return out


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------------
def _turn(x, angle, first, second):
    """Complex rotation of the pairs (first, second) of x [..., d] by angle, in 64 bits."""
    y = x.double().clone()
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    x = _inputs(c, seed)
    if c["kind"] == "rope":
        sections = [int(s) for s in c["sections"].split(",")]
        exps, axis = _pairs(c, sections)
        p = len(axis)
        first, second = (slice(0, p), slice(p, 2 * p)) if c["halves"] else (slice(0, 2 * p, 2), slice(1, 2 * p, 2))
        theta = torch.tensor([math.exp(e * math.log(c["base"])) for e in exps], device="cuda", dtype=torch.float64)
        angle = torch.stack([x["pos"][a].double() for a in axis], -1) * theta
        return _turn(x["x"], angle[:, None], first, second)
    cap = _capacity(c)
    if c["kind"] == "pages":
        held, source = _held(c), _branches(c)
        k = torch.zeros((len(source), c["hkv"], cap, c["d"]), device="cuda", dtype=torch.float64)
        v = torch.zeros_like(k)
        for slot, s in enumerate(source):
            for full, rows, new in ((k, x["k"], x["k1"]), (v, x["v"], x["v1"])):
                full[slot, :, :held[s]] = rows[s, :, :held[s]].double()
                if c["op"] == "branch":
                    full[slot, :, held[s]] = new[slot].double()
        if c["op"] == "compact":
            need = [math.ceil(n / 16) for n in held]
            return dict(k=k, v=v, used=[sum(need[0::2]), sum(need[1::2])])
        return dict(k=k, v=v)
    n, cut = _lengths(c)
    if 4 * c["hq"] * c["d"] * sum(a * (a + b) for a, b in zip(n, cut)) > 6e12:
        return None
    t = _type(c)
    k = torch.zeros((c["batch"], c["hkv"], cap, c["d"]), device="cuda", dtype=torch.float64)
    v = torch.zeros_like(k)
    out = torch.zeros((sum(n), c["hq"], c["d"]), device="cuda", dtype=torch.float64)
    spectrum = torch.tensor([c["base"] ** (-2 * i / c["d"]) if c["base"] else 0.0 for i in range(c["d"] // 2)],
                            device="cuda", dtype=torch.float64)
    at = 0
    for b in range(c["batch"]):
        end = cut[b] + n[b]
        pos = torch.arange(end, device="cuda").double()
        rows = torch.cat((x["pk"][b, :, :cut[b]], x["k"][at:at + n[b]].transpose(0, 1)), 1)
        angle = pos[:, None] * spectrum
        k[b, :, :end] = _turn(rows, angle, slice(0, None, 2), slice(1, None, 2))
        v[b, :, :end] = torch.cat((x["pv"][b, :, :cut[b]], x["v"][at:at + n[b]].transpose(0, 1)), 1).double()
        for h in range(c["hq"] if n[b] else 0):
            # queries and keys enter the products as the cache's type holds them
            kh = k[b, h * c["hkv"] // c["hq"], :end].to(t).double()
            qh = _turn(x["q"][at:at + n[b], h], angle[cut[b]:], slice(0, None, 2), slice(1, None, 2)).to(t).double()
            for i0 in range(0, n[b], 4096):
                i1 = min(n[b], i0 + 4096)
                s = qh[i0:i1] @ kh[:cut[b] + i1].T / math.sqrt(c["d"])
                away = pos[cut[b] + i0:cut[b] + i1, None] - pos[:cut[b] + i1]
                s[(away < 0) | (away >= (c["window"] or end + 1))] = -math.inf
                out[at + i0:at + i1, h] = s.softmax(-1) @ v[b, h * c["hkv"] // c["hq"], :cut[b] + i1]
        at += n[b]
    return dict(out=out, k=k, v=v)
