"""The 4-bit tier on the GPU: rows bit for bit against the plain quantiser, decode attention and its windows against 64 bits,
conversion from and to bf16 caches, and what else a cache does (trim, pages, rings, store, graphs, streams)."""
import math

import numpy as np
import pytest
import torch

import _int4 as i4
from kv_cache_decode_ring_gb300 import kvc

pytestmark = pytest.mark.gpu


def make(layout="contiguous", **kw):
    cfg = dict(kv_quant="int4", batch=3, n_q_heads=8, n_kv_heads=2, head_dim=128, capacity=512, layout=layout, out_dtype="f32")
    cfg.update(kw)
    if layout == "ring":
        cfg.setdefault("max_position", 4096)
    return kvc.Cache(kvc.make_config(**cfg))


def rows(seed, B, H, n, d, wide=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, H, n, d), generator=g)
    if wide:
        x = x * torch.exp(torch.randn((1, H, 1, d), generator=g) * 0.7) + torch.randn((1, H, 1, d), generator=g)
    return x.bfloat16().cuda()


class Model:
    """Every row that was appended, in order, and what is visible of it."""

    def __init__(self, cache, base=0.0, window=0, sinks=0):
        self.c, self.base, self.window, self.sinks = cache, base, window, sinks
        self.k, self.v = ([torch.zeros((cache.Hkv, 0, cache.d), dtype=torch.bfloat16, device="cuda") for _ in range(cache.B)] for _ in "kv")

    def append(self, k, v, counts):
        for b, n in enumerate(counts):
            self.k[b] = torch.cat((self.k[b], k[b, :, :n]), 1)
            self.v[b] = torch.cat((self.v[b], v[b, :, :n]), 1)

    def trim(self, cuts):
        for b, n in enumerate(cuts):
            self.k[b], self.v[b] = self.k[b][:, :n], self.v[b][:, :n]

    def keys(self, b):
        return i4.rotated(self.k[b], torch.arange(self.k[b].shape[1]), self.base)

    def check_rows(self):
        ring, S = self.c.cfg.layout == kvc.KVC_RING, self.c.S
        got = [torch.from_numpy(self.c.export(w)) for w in (kvc.KVC_EXPORT_K4, kvc.KVC_EXPORT_V4)]
        pos = self.c.export(kvc.KVC_EXPORT_POSITIONS)
        for b in range(self.c.B):
            n = self.k[b].shape[1]
            p = torch.arange(max(0, n - S) if ring else 0, n)
            slots = p % S
            want = np.full(S, -1, np.int32)
            want[slots.numpy()] = p.numpy()
            assert np.array_equal(pos[b], want)
            for x, y, value in ((self.keys(b), got[0], False), (self.v[b], got[1], True)):
                assert torch.equal(i4.row_bytes(x[:, p], value).cpu(), y[b][:, slots]), (b, value)
        assert np.array_equal(self.c.next_positions(), [k.shape[1] for k in self.k])

    def check_decode(self, q, out, what=""):
        for b in range(self.c.B):
            n = self.k[b].shape[1]
            p = torch.arange(n, device="cuda")
            seen = (p >= n - self.window) | (p < self.sinks) if self.window else p >= 0
            kp, vp = (tuple(y for y in i4.quantise(x[:, seen])) for x in (self.keys(b), self.v[b]))
            qb = i4.turned(q[b], n - 1, self.base)
            ref, w = i4.attend(qb, i4.values(*kp), i4.values(*vp))
            bound = i4.decode_bound(qb, kp, vp, w)
            if out.dtype == torch.bfloat16:
                bound = bound + ref.abs() * 2.0 ** -8
            err = (out[b].double() - ref).abs()
            assert (err <= bound).all(), "%s request %d: %.3g against %.3g" % (what, b, err.max(), bound.max())
            assert err.mean() <= 0.1 * bound.mean() or out.dtype == torch.bfloat16


SHAPES = [("contiguous", 0), ("contiguous", 90), ("ring", 0)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("base", [0.0, 10000.0])
@pytest.mark.parametrize("layout,pool", SHAPES + [("ring", 60)])
def test_rows_bit_for_bit(d, base, layout, pool):
    cap = 128 if layout == "ring" else 512
    c = make(layout, head_dim=d, rope_base=base, page_pool=pool, capacity=cap)
    m = Model(c, base)
    for step, counts in enumerate([(5, 0, 170), (1, 33, 16), (0, 0, 0), (200, 1, 7)]):
        k, v = (rows(10 * step + i, 3, 2, max(counts) or 1, d) for i in range(2))
        c.append_rows(k, v, counts=counts)
        m.append(k, v, counts)
        m.check_rows()
    for step in range(3):
        k, v = (rows(100 + 10 * step + i, 3, 2, 1, d) for i in range(2))
        c.append(k[:, :, 0].contiguous(), v[:, :, 0].contiguous())
        m.append(k, v, (1, 1, 1))
    m.check_rows()
    assert c.device_status() == 0


def test_rows_of_special_values():
    # ties of the quotient, equal values, ranges without a scale, infinities, NaN, both zeros, the largest values
    d = 128
    x = rows(1, 1, 2, 40, d)
    x[0, 0, 0, :32] = 3.25
    x[0, 0, 1, :32] = torch.arange(32).bfloat16() / 2                    # s = 31/30 rounded; quotients of all kinds
    x[0, 0, 2, :32] = torch.arange(32).clamp(max=30).bfloat16()          # s = 2: odd values are ties
    x[0, 0, 3, :32] = 0
    x[0, 0, 3, 1] = 1e-40
    x[0, 0, 4, 7] = math.inf
    x[0, 0, 5, 40] = -math.inf
    x[0, 0, 6, 100] = math.nan
    x[0, 0, 7, 3], x[0, 0, 7, 4] = 3e38, -3e38                           # a range past fp32
    x[0, 0, 8, 3], x[0, 0, 8, 4] = 3e38, 0.0                             # a scale past 2^100
    x[0, 0, 9, :32] = torch.linspace(-1, 1, 32).bfloat16() * 2.0 ** -110
    x[0, 0, 10, :32] = torch.linspace(0, 1, 32).bfloat16() * 2.0 ** -130
    c = make(batch=1)
    c.append_rows(x, x.flip(2).contiguous())
    for which, y, value in ((kvc.KVC_EXPORT_K4, x, False), (kvc.KVC_EXPORT_V4, x.flip(2), True)):
        got, want = torch.from_numpy(c.export(which))[0, :, :40], i4.row_bytes(y[0], value).cpu()
        assert torch.equal(got[..., :d // 2], want[..., :d // 2])
        a, b = (z[..., d // 2:].contiguous().view(torch.bfloat16).float() for z in (got, want))
        assert torch.equal(a.nan_to_num(77.0), b.nan_to_num(77.0)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (6, 2), (8, 1), (5, 1), (24, 2), (9, 1), (48, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_heads(hq, hkv, d):
    c = make(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, rope_base=10000.0)
    m = Model(c, 10000.0)
    counts = (1, 300, 47)
    k, v = rows(1, 3, hkv, 300, d), rows(2, 3, hkv, 300, d, False)
    c.append_rows(k, v, counts=counts)
    m.append(k, v, counts)
    q = rows(3, 3, hq, 1, d, False)[:, :, 0].contiguous()
    m.check_decode(q, c.decode(q))
    assert c.device_status() == 0


@pytest.mark.parametrize("layout,pool", SHAPES + [("ring", 100)])
@pytest.mark.parametrize("window", [0, 1, 17, 200])
def test_decode_lengths(layout, pool, window):
    if layout == "ring":
        window = 16 * (window // 16 or 1)
    c = make(layout, page_pool=pool, capacity=window if layout == "ring" else 512, window=0 if layout == "ring" else window,
             rope_base=10000.0)
    m = Model(c, 10000.0, window)
    for step, counts in enumerate([(1, 2, 15), (15, 14, 1), (1, 1, 1), (15, 111, 128), (1, 1, 1), (100, 3, 96)]):
        k, v = rows(10 * step, 3, 2, max(counts), 128), rows(10 * step + 1, 3, 2, max(counts), 128, False)
        if max(counts) == 1:
            c.append(k[:, :, 0].contiguous(), v[:, :, 0].contiguous())
        else:
            c.append_rows(k, v, counts=counts)
        m.append(k, v, counts)
        q = rows(10 * step + 2, 3, 8, 1, 128, False)[:, :, 0].contiguous()
        m.check_decode(q, c.decode(q), "step %d" % step)
    assert c.device_status() == 0


@pytest.mark.parametrize("n", [2047, 2048, 20011])
@pytest.mark.parametrize("hq", [4, 8])
def test_decode_long(n, hq):
    # several splits, keys of very different size, bf16 outputs too
    for out in ("f32", "bf16"):
        c = make(batch=1, n_q_heads=hq, n_kv_heads=1, capacity=20480, out_dtype=out)
        m = Model(c)
        k, v = rows(1, 1, 1, n, 128), rows(2, 1, 1, n, 128, False)
        k[:, :, n // 2:] *= 3
        c.append_rows(k, v)
        m.append(k, v, (n,))
        q = rows(3, 1, hq, 1, 128, False)[:, :, 0].contiguous()
        cmax, tanh = (torch.ones((1, hq), device="cuda") for _ in range(2))
        m.check_decode(q, c.decode(q, cmax=cmax, tanh=tanh))
        assert not cmax.any() and not tanh.any()


def test_masked_rows_may_hold_anything():
    # rows before the window and rows that a trim dropped, in the same tiles as visible ones
    c = make(batch=1, window=40)
    m = Model(c, 0.0, 40)
    k, v = rows(1, 1, 2, 100, 128), rows(2, 1, 2, 100, 128)
    for x in (k, v):
        x[0, :, 50:60] = math.nan
        x[0, :, 96:] = math.inf
    c.append_rows(k, v)
    c.trim([95])
    m.append(k[:, :, :95], v[:, :, :95], (95,))
    k1, v1 = rows(3, 1, 2, 5, 128), rows(4, 1, 2, 5, 128)
    c.append_rows(k1, v1, counts=[5])
    m.append(k1, v1, (5,))
    q = rows(5, 1, 8, 1, 128, False)[:, :, 0].contiguous()
    m.check_decode(q, c.decode(q))
    k1[:] = v1[:] = math.nan
    c.append_rows(k1, v1, counts=[3])
    c.trim([100])                      # rows 100 .. 102 were NaN
    m.check_decode(q, c.decode(q))


def test_visible_rows_that_are_not_finite_spoil_what_sees_them():
    c = make(batch=2, n_q_heads=2, n_kv_heads=2)
    k, v = rows(1, 2, 2, 70, 128), rows(2, 2, 2, 70, 128)
    v[0, 1, 33, 40] = math.inf                       # group 1 of head 1
    k[1, 0, 5, 3] = math.nan
    c.append_rows(k, v)
    out = c.decode(rows(3, 2, 2, 1, 128, False)[:, :, 0].contiguous())
    assert out[0, 0].isfinite().all() and out[1, 1].isfinite().all()
    assert out[0, 1, 32:64].isnan().all() and out[0, 1, :32].isfinite().all() and out[0, 1, 64:].isfinite().all()
    assert out[1, 0].isnan().all()


@pytest.mark.parametrize("hq,d", [(4, 128), (8, 128), (3, 64)])
@pytest.mark.parametrize("what", ["large", "small", "groups", "outlier", "growing", "sharp", "query"])
def test_decode_of_values_of_all_sizes(hq, d, what):
    """Weights times scales stay within fp16's range, whatever the rows hold, and what is small next to them keeps its bits."""
    n = 700
    c = make(batch=1, n_q_heads=hq, n_kv_heads=1, head_dim=d, capacity=1024)
    m = Model(c)
    k, v = rows(1, 1, 1, n, d), rows(2, 1, 1, n, d, False)
    q = rows(3, 1, hq, 1, d, False)[:, :, 0].contiguous()
    if what == "large":
        v *= 2.0 ** 110
    elif what == "small":
        v *= 2.0 ** -95
    elif what == "groups":                           # a group of dims 2^30 times as large as the next
        v[..., :32] *= 2.0 ** 30
    elif what == "outlier":                          # a row of large values that hardly anything weighs
        v[0, 0, 300] *= 2.0 ** 20
        k[0, 0, 300] = -q[0, :1].float().sign().bfloat16() * 6
    elif what == "growing":                          # ever larger values, and scores
        v *= (2.0 ** torch.linspace(-20, 40, n, device="cuda"))[:, None].bfloat16()
        k *= torch.linspace(0.1, 4, n, device="cuda")[:, None].bfloat16()
    elif what == "sharp":
        k *= 40
    else:
        q[0, :, ::7] *= 2.0 ** 12                    # a few dims decide
        k *= 2.0 ** -8
    c.append_rows(k, v)
    m.append(k, v, (n,))
    m.check_decode(q, c.decode(q), what)


@pytest.mark.parametrize("hq,d", [(4, 128), (8, 128), (3, 64)])
def test_decode_of_values_near_the_end_of_the_range(hq, d):
    # scales of 2^113: the norm of their weights is below 2^-104, its inverse times a code's unit past fp32
    n = 700
    c = make(batch=1, n_q_heads=hq, n_kv_heads=1, head_dim=d, capacity=1024)
    m = Model(c)
    k, v = rows(1, 1, 1, n, d), rows(2, 1, 1, n, d, False) * 2.0 ** 115
    c.append_rows(k, v)
    m.append(k, v, (n,))
    q = rows(3, 1, hq, 1, d, False)[:, :, 0].contiguous()
    m.check_decode(q, c.decode(q))


@pytest.mark.parametrize("hq,d", [(4, 128), (8, 64)])
@pytest.mark.parametrize("n,spoilt", [(1, 1), (300, 300), (5000, 5000), (5000, 4096)])
def test_keys_that_are_all_nan_spoil_the_answer(hq, d, n, spoilt):
    # (whole splits of them too: those have no largest score)
    c = make(batch=1, n_q_heads=hq, n_kv_heads=1, head_dim=d, capacity=5008)
    k, v = rows(1, 1, 1, n, d), rows(2, 1, 1, n, d)
    k[:, :, :spoilt] = math.nan
    c.append_rows(k, v)
    assert c.decode(rows(3, 1, hq, 1, d, False)[:, :, 0].contiguous()).isnan().all()


def dense(like, **kw):
    cfg = dict(batch=like.B, n_q_heads=like.Hq, n_kv_heads=like.Hkv, head_dim=like.d, capacity=like.S,
               layout="ring" if like.cfg.layout == kvc.KVC_RING else "contiguous", rope_base=like.cfg.rope_base,
               max_position=like.cfg.max_position)
    return kvc.Cache(kvc.make_config(**dict(cfg, **kw)))


@pytest.mark.parametrize("layout", ["contiguous", "ring"])
@pytest.mark.parametrize("pool4,pool16", [(0, 0), (120, 0), (0, 120)])
@pytest.mark.parametrize("d", [64, 128])
def test_conversion(layout, pool4, pool16, d):
    """bf16 -> 4 bits -> bf16: codes as appends write them, values m + u s rounded to bf16; one source, several destinations."""
    cap = 160 if layout == "ring" else 512
    c = make(layout, head_dim=d, capacity=cap, page_pool=pool4, rope_base=10000.0)
    a = dense(c, page_pool=pool16)
    m = Model(c, 10000.0)
    counts = (500 if layout == "ring" else 399, 0, 131)
    k, v = rows(1, 3, 2, max(counts), d), rows(2, 3, 2, max(counts), d)
    a.append_rows(k, v, counts=counts)
    m.append(k, v, counts)
    c.copy_from(a, [0, 1, 2], [0, 1, 2])
    m.check_rows()
    k1, v1 = (rows(7 + i, 3, 2, 1, d) for i in range(2))                   # and it goes on
    c.append(k1[:, :, 0].contiguous(), v1[:, :, 0].contiguous())
    m.append(k1, v1, (1, 1, 1))
    m.check_rows()
    back = dense(c, page_pool=pool16)
    back.copy_from(c, [2, 0, 2], [0, 1, 2])
    got = [torch.from_numpy(back.export(w)).view(torch.bfloat16) for w in (kvc.KVC_EXPORT_K, kvc.KVC_EXPORT_V)]
    for dst, src in enumerate((2, 0, 2)):
        n = m.k[src].shape[1]
        p = torch.arange(max(0, n - cap), n)
        for x, y in ((m.keys(src), got[0]), (m.v[src], got[1])):
            want = i4.held(x[:, p]).float().bfloat16().cpu()                  # (rounded to fp32 on the way, as by the kernel)
            assert torch.equal(want, y[dst][:, p % cap])
    assert list(back.next_positions()) == [m.k[s].shape[1] for s in (2, 0, 2)]


def test_conversion_refuses_other_types():
    c = make()
    with pytest.raises(kvc.KvcError) as e:
        c.copy_from(dense(c, dtype="f32"), [0], [0])
    assert e.value.code == kvc.KVC_ERR_ARG
    with pytest.raises(kvc.KvcError) as e:
        c.copy_from(dense(c, kv_quant="int8"), [0], [0])
    assert e.value.code == kvc.KVC_ERR_ARG


def test_fork_trim_and_compact_share_pages():
    c = make(page_pool=40, capacity=256)
    m = Model(c)
    k, v = rows(1, 3, 2, 100, 128), rows(2, 3, 2, 100, 128)
    c.append_rows(k, v, counts=[100, 0, 0])
    m.append(k, v, (100, 0, 0))
    c.fork([0, 0], [1, 2])
    for b in (1, 2):
        m.k[b], m.v[b] = m.k[0], m.v[0]
    assert c.page_counts() == (33, 7)
    k1, v1 = rows(3, 3, 2, 30, 128), rows(4, 3, 2, 30, 128)
    c.append_rows(k1, v1, counts=[1, 30, 0])                    # copies of the shared last page
    m.append(k1, v1, (1, 30, 0))
    m.check_rows()
    c.trim([33, 130, 50])
    m.trim((33, 130, 50))
    used = c.compact()
    assert used == 40 - c.page_counts()[0]
    m.check_rows()
    q = rows(5, 3, 8, 1, 128, False)[:, :, 0].contiguous()
    m.check_decode(q, c.decode(q))


def test_ring_trim_rules():
    c = make("ring", batch=1, capacity=64)
    k, v = rows(1, 1, 2, 100, 128), rows(2, 1, 2, 100, 128)
    c.append_rows(k, v)
    with pytest.raises(kvc.KvcError) as e:
        c.trim([50])
    assert e.value.code == kvc.KVC_ERR_EVICTED


@pytest.mark.parametrize("d", [64, 128])
def test_store(d):
    c = make(store_slots=2, capacity=256, head_dim=d)
    m = Model(c)
    k, v = rows(1, 3, 2, 90, d), rows(2, 3, 2, 90, d)
    c.append_rows(k, v, counts=[90, 3, 0])
    m.append(k, v, (90, 3, 0))
    c.store_save(1, 0, 90)
    c.store_load(1, 2, 77)
    m.k[2], m.v[2] = m.k[0][:, :77], m.v[0][:, :77]
    m.check_rows()


def test_captured_steps():
    """A graph of append and decode replayed twice, on a stream of its own, and past the capacity."""
    c = make(batch=2, capacity=32, rope_base=10000.0)
    m = Model(c, 10000.0)
    k, v = rows(1, 2, 2, 20, 128), rows(2, 2, 2, 20, 128, False)
    q = rows(3, 2, 8, 1, 128, False)[:, :, 0].contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.append_rows(k, v, counts=[20, 9])
        k1, v1 = k[:, :, 0].contiguous(), v[:, :, 0].contiguous()
        out = c.decode(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.append(k1, v1)
            c.decode(q, out)
    m.append(k, v, (20, 9))
    for _ in range(2):
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        m.append(k[:, :, :1], v[:, :, :1], (1, 1))
        m.check_decode(q, out)
    with torch.cuda.stream(s):
        for _ in range(12):
            graph.replay()
    s.synchronize()
    assert c.device_status() & 1                     # request 0 ran past its 32 slots: nothing is written there
    got = torch.from_numpy(c.export(kvc.KVC_EXPORT_K4))
    want = torch.cat((k[0], k[0, :, :1].expand(-1, 12, -1)), 1)
    assert torch.equal(got[0], i4.row_bytes(i4.rotated(want, torch.arange(32), 10000.0), False).cpu())


def test_refusals():
    c = make(max_chunk=16)
    k, v = rows(1, 3, 2, 4, 128), rows(2, 3, 2, 4, 128)
    q = rows(3, 3, 8, 4, 128)
    with pytest.raises(kvc.KvcError) as e:
        c.decode(q[:, :, 0].contiguous())            # nothing cached
    assert e.value.code == kvc.KVC_ERR_ARG
    c.append_rows(k, v)
    flat = lambda x, n: x.transpose(1, 2).reshape(12, n, 128).contiguous()  # noqa: E731
    with pytest.raises(kvc.KvcError) as e:
        c.prompt(flat(q, 8), flat(k, 2), flat(v, 2), [4, 4, 4])
    assert e.value.code == kvc.KVC_ERR_UNSUPPORTED
    with pytest.raises(kvc.KvcError) as e:
        c.chunk(q.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous())
    assert e.value.code == kvc.KVC_ERR_UNSUPPORTED
    q1 = q[:, :, 0].contiguous()
    with pytest.raises(kvc.KvcError) as e:
        kvc.kvc_decode_attn_noalloc(c.h, q1, torch.empty_like(q1, dtype=torch.float32))
    assert e.value.code == kvc.KVC_ERR_UNSUPPORTED
    with pytest.raises(kvc.KvcError) as e:
        c.decode(q1, ct=torch.zeros((3, 8, 512), device="cuda"))
    assert e.value.code == kvc.KVC_ERR_ARG
    with pytest.raises(kvc.KvcError) as e:
        c.export(kvc.KVC_EXPORT_K)
    assert e.value.code == kvc.KVC_ERR_ARG
    with pytest.raises(kvc.KvcError) as e:
        c.append_rows(*(rows(9 + i, 3, 2, 509, 128) for i in range(2)))
    assert e.value.code == kvc.KVC_ERR_CAPACITY
    assert c.rows()[0].shape == (3, 2, 512, 80) and c.rows()[0].dtype == torch.uint8


@pytest.mark.parametrize("hq,d", [(4, 128), (8, 64)])
def test_decode_of_lengths_that_the_host_does_not_know(hq, d):
    # replayed appends move the lengths on the device: a decode launched for the host's lengths still covers them
    c = make(batch=2, n_q_heads=hq, n_kv_heads=1, head_dim=d, capacity=2048, window=1500, sinks=5, rope_base=10000.0)
    m = Model(c, 10000.0, 1500, 5)
    k, v = rows(1, 2, 1, 1, d), rows(2, 2, 1, 1, d, False)
    k0, v0 = rows(3, 2, 1, 9, d), rows(4, 2, 1, 9, d, False)
    c.append_rows(k0, v0, counts=[9, 2])
    m.append(k0, v0, (9, 2))
    k1, v1 = k[:, :, 0].contiguous(), v[:, :, 0].contiguous()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.append(k1, v1)
    for _ in range(1800):
        graph.replay()
    torch.cuda.synchronize()
    for x, y, z in ((m.k, k, 0), (m.v, v, 0)):
        for b in range(2):
            x[b] = torch.cat((x[b], y[b].expand(-1, 1800, -1)), 1)
    q = rows(5, 2, hq, 1, d, False)[:, :, 0].contiguous()
    m.check_decode(q, c.decode(q))
    assert c.device_status() == 0


@pytest.mark.parametrize("hkv,d", [(1, 64), (1, 128), (3, 64), (40, 128)])
def test_token_appends_of_any_number_of_heads(hkv, d):
    c = make(n_q_heads=hkv, n_kv_heads=hkv, head_dim=d, capacity=32, rope_base=500.0)
    m = Model(c, 500.0)
    for step in range(18):
        k, v = (rows(10 * step + i, 3, hkv, 1, d) for i in range(2))
        c.append(k[:, :, 0].contiguous(), v[:, :, 0].contiguous())
        m.append(k, v, (1, 1, 1))
    m.check_rows()


@pytest.mark.parametrize("layout", ["contiguous", "ring"])
@pytest.mark.parametrize("d", [64, 128])
def test_copies_between_4_bit_caches(layout, d):
    cap = 96 if layout == "ring" else 256
    a, b = make(layout, head_dim=d, capacity=cap, page_pool=60), make(layout, head_dim=d, capacity=cap, batch=2)
    m = Model(b)
    k, v = rows(1, 3, 2, 200, d), rows(2, 3, 2, 200, d)
    a.append_rows(k, v, counts=[200, 0, 77])
    b.copy_from(a, [2, 0], [0, 1])
    m.append(k[[2, 0]], v[[2, 0]], (77, 200))
    m.check_rows()
    a.copy_from(b, [1, 1], [1, 2])
    m = Model(a)
    m.append(k[[0, 0, 0]], v[[0, 0, 0]], (200, 200, 200))
    m.check_rows()


@pytest.mark.parametrize("B", [70, 1100])
def test_many_requests(B):
    # more than a sample of lengths, and than one launch of appends
    c = make(batch=B, n_q_heads=4, n_kv_heads=1, head_dim=64, capacity=64, window=20, sinks=3)
    k, v, q = rows(1, B, 1, 33, 64), rows(2, B, 1, 33, 64, False), rows(3, B, 4, 1, 64, False)[:, :, 0].contiguous()
    counts = [1 + i * 7 % 33 for i in range(B)]
    c.append_rows(k, v, counts=counts)
    out = c.decode(q)
    for b in range(0, B, 23 if B > 100 else 3):
        n = counts[b]
        p = torch.arange(n, device="cuda")
        seen = (p >= n - 20) | (p < 3)
        kp, vp = i4.quantise(k[b, :, :n][:, seen]), i4.quantise(v[b, :, :n][:, seen])
        ref, w = i4.attend(q[b].double(), i4.values(*kp), i4.values(*vp))
        assert ((out[b].double() - ref).abs() <= i4.decode_bound(q[b].double(), kp, vp, w)).all(), b


def test_offsets_past_32_bits():
    # rows of the last requests lie past 4 GB of K
    c = make(batch=5, n_q_heads=16, n_kv_heads=16, capacity=1 << 20)
    m = Model(c)
    k, v = rows(1, 5, 16, 40, 128), rows(2, 5, 16, 40, 128)
    c.append_rows(k, v, counts=[0, 40, 1, 3, 39])
    k1, v1 = rows(3, 5, 16, 1, 128), rows(4, 5, 16, 1, 128)
    c.append(k1[:, :, 0].contiguous(), v1[:, :, 0].contiguous())
    m.append(k, v, (0, 40, 1, 3, 39))
    m.append(k1, v1, (1,) * 5)
    kr, vr = (x[:, :, :64] for x in c.rows())
    for b in range(5):
        n = m.k[b].shape[1]
        assert torch.equal(kr[b, :, :n], i4.row_bytes(m.k[b], False)) and torch.equal(vr[b, :, :n], i4.row_bytes(m.v[b], True))
    q = rows(5, 5, 16, 1, 128, False)[:, :, 0].contiguous()
    m.check_decode(q, c.decode(q))
    other = kvc.Cache(kvc.make_config(batch=5, n_q_heads=16, n_kv_heads=16, capacity=64))
    other.copy_from(c, [4], [4])
    got = other.rows()[0][4, :, :40]
    assert torch.equal(got, i4.held(m.k[4]).float().bfloat16())


def test_replayed_appends_past_the_mapped_pages_write_nothing():
    c = make(batch=2, capacity=64, page_pool=8)
    m = Model(c)
    k, v = rows(1, 2, 2, 30, 128), rows(2, 2, 2, 30, 128)
    c.append_rows(k, v, counts=[30, 14])
    m.append(k, v, (30, 14))
    k1, v1 = k[:, :, 0].contiguous(), v[:, :, 0].contiguous()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.append(k1, v1)
    before = [x.clone() for x in c.rows()]
    for _ in range(4):
        graph.replay()                                # both requests have room for two rows in the pages of the capture
    torch.cuda.synchronize()
    assert c.device_status() & 1
    table = c.export(kvc.KVC_EXPORT_PAGE_TABLE)
    for x, y, rows_, value in ((before[0], c.rows()[0], k1, False), (before[1], c.rows()[1], v1, True)):
        for b, n in enumerate((30, 14)):
            page = table[b][n // 16]
            x[page, :, n % 16:] = i4.row_bytes(rows_[b], value)[:, None]
        assert torch.equal(x, y)
