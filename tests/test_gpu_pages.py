"""Whole requests forked, copied and freed, pages shared, copied on write and compacted
([LOOP] §八 Q1; [LEAN] §6.1: the logical view equals the interpretation of the pages).

A model keeps, per request, the list of tokens that it has appended.  After every few random calls
the cache is held to a fresh unpaged cache that appended the same lists in one go: every live row,
code, scale and witness bit for bit, positions, lengths, and the books of the pool (each page free,
or held as often as block-table entries name it).
"""
import random

import numpy as np
import pytest
import torch

from kv_cache_decode_ring_gb300 import kvc
from kv_cache_decode_ring_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

VOCAB = 64


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_decode_ring_gb300 import build
    build.build()


class Model:
    """A cache beside the token lists of its requests."""

    def __init__(self, B=6, Hkv=2, d=64, cap=96, layout="contiguous", quant=None, dtype="bf16", pages=0, rope=10000.0, key=(3, 9), g=2):
        self.B, self.Hkv, self.d, self.cap, self.layout, self.quant, self.pages, self.g = B, Hkv, d, cap, layout, quant, pages, g
        self.kw = dict(dtype=dtype, layout=layout, kv_quant=quant, n_q_heads=g * Hkv, n_kv_heads=Hkv, head_dim=d, capacity=cap,
                       rope_base=rope, max_position=4000, layer_index=3 if quant == "int8-dither" else 0,
                       dither_key=key if quant == "int8-dither" else (0, 0), max_chunk=64 if not quant else 0)
        self.cache = kvc.Cache(kvc.make_config(batch=B, page_pool=pages, **self.kw))
        self.ids = [[] for _ in range(B)]
        self.req = list(range(B))
        self.table = [wl.normal((VOCAB, Hkv, d), 1, n, "cuda", self.cache.torch_dtype) for n in "kv"]
        self.rng = random.Random(0)

    def rows(self, ids):
        t = torch.tensor(ids, device="cuda", dtype=torch.long)
        return [x[t] for x in self.table]

    def append(self):
        new = [self.rng.randrange(VOCAB) for _ in range(self.B)]
        k, v = self.rows(new)
        self.cache.append(k.contiguous(), v.contiguous())
        for ids, t in zip(self.ids, new):
            ids.append(t)

    def append_rows(self, counts, prompt=False):
        new = [[self.rng.randrange(VOCAB) for _ in range(n)] for n in counts]
        if prompt:
            k, v = self.rows(sum(new, []))
            q = torch.zeros(sum(counts), self.g * self.Hkv, self.d, dtype=k.dtype, device="cuda")
            self.cache.prompt(q, k, v, counts)
        else:
            n = max(max(counts), 1)
            k, v = (x.transpose(1, 2).contiguous() for x in
                    (torch.stack(y) for y in zip(*(self.rows(t + [0] * (n - len(t))) for t in new))))
            self.cache.append_rows(k, v, counts=counts)
        for ids, t in zip(self.ids, new):
            ids += t

    def fork(self, src, dst):
        self.cache.fork(src, dst)
        for s, t in zip(src, dst):
            self.ids[t], self.req[t] = list(self.ids[s]), self.req[s]

    def copy_from(self, other, src, dst):
        self.cache.copy_from(other.cache, src, dst)
        for s, t in zip(src, dst):
            self.ids[t], self.req[t] = list(other.ids[s]), other.req[s]

    def free(self, reqs):
        self.cache.free(reqs)
        for b in reqs:
            self.ids[b] = []

    def trim(self, cuts):
        self.cache.trim(cuts)
        self.ids = [ids[:c] for ids, c in zip(self.ids, cuts)]

    def check(self, decode=True):
        c = self.cache
        assert c.device_status() == 0
        lengths = [len(x) for x in self.ids]
        assert list(c.next_positions()) == lengths and list(c.export(kvc.KVC_EXPORT_NEXT_POSITION)) == lengths
        fresh = kvc.Cache(kvc.make_config(batch=self.B, **self.kw))
        if self.quant == "int8-dither":
            for b, r in enumerate(self.req):
                fresh.set_request_id(b, r)
        n = max(lengths)
        if n:
            k, v = (x.transpose(1, 2).contiguous() for x in
                    (torch.stack(y) for y in zip(*(self.rows(t + [0] * (n - len(t))) for t in self.ids))))
            fresh.append_rows(k, v, counts=lengths)
        mine, want = c.export(kvc.KVC_EXPORT_POSITIONS), fresh.export(kvc.KVC_EXPORT_POSITIONS)
        assert np.array_equal(mine, want)
        live = want >= 0
        if not self.quant:
            for which in (kvc.KVC_EXPORT_K, kvc.KVC_EXPORT_V):
                a, b = (x.export(which).transpose(0, 2, 1, 3)[live] for x in (c, fresh))
                assert np.array_equal(a, b), which
        else:
            for b, m in enumerate(lengths):
                nb = min(m // 16, self.cap // 16)
                for which, per in ((kvc.KVC_EXPORT_KQ, 16), (kvc.KVC_EXPORT_VQ, 16), (kvc.KVC_EXPORT_SK, 1), (kvc.KVC_EXPORT_SV, 1),
                                   (kvc.KVC_EXPORT_WITNESS, 16)):
                    if which == kvc.KVC_EXPORT_WITNESS and self.quant == "int8-dither":
                        continue
                    assert np.array_equal(c.export(which)[b][:, :nb * per], fresh.export(which)[b][:, :nb * per]), (which, b)
                for which in (kvc.KVC_EXPORT_KTAIL, kvc.KVC_EXPORT_VTAIL):
                    assert np.array_equal(c.export(which)[b][:, :m % 16], fresh.export(which)[b][:, :m % 16]), (which, b)
        if self.pages:
            table = c.export(kvc.KVC_EXPORT_PAGE_TABLE)
            held = np.bincount(table[table >= 0], minlength=self.pages)
            assert c.page_counts() == (int((held == 0).sum()), int((held > 1).sum()))
            for b, m in enumerate(lengths):
                want = min(-(-m // 16), self.cap // 16)
                assert (table[b, :want] >= 0).all()
                if self.layout != "ring":
                    assert (table[b, want:] < 0).all()
        if decode and min(lengths) > 0 and not (self.layout == "ring" and self.trimmed):
            q = wl.normal((self.B, self.g * self.Hkv, self.d), 2, "q", "cuda", c.torch_dtype)
            a, b = c.decode(q).float(), fresh.decode(q).float()
            # the same rows; splits of a paged cache may differ in order
            assert (a - b).abs().max() <= 4e-3 * 2

    trimmed = False


KINDS = [
    dict(),
    dict(pages=40),
    dict(dtype="f32", d=6, pages=40),
    dict(dtype="f32", cap=90, Hkv=3),
    dict(layout="ring", cap=48, pages=22),
    dict(layout="ring", cap=50),
    dict(quant="int8", pages=40),
    dict(quant="int8"),
    dict(quant="int8", layout="ring", cap=48, pages=22),
    dict(quant="int8-dither", pages=40, d=128),
    dict(quant="int8-dither", layout="ring", cap=32),
]


@pytest.mark.parametrize("seed", range(2))
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join("%s=%s" % kv for kv in k.items()) or "rows")
def test_random_calls(kind, seed):
    m = Model(**kind)
    m.rng = rng = random.Random(100 + seed)
    ring = m.layout == "ring"
    limit = 3000 if ring else m.cap
    for step in range(70):
        op = rng.choice(["append", "append", "rows", "prompt", "fork", "fork", "free", "trim", "compact", "copy"])
        before = (m.cache.page_counts() if m.pages else None, [list(x) for x in m.ids])
        try:
            if op == "append" and max(map(len, m.ids)) + 1 <= limit:
                m.append()
            elif op in ("rows", "prompt"):
                if op == "prompt" and (m.quant or (ring and (m.cap % 16 or m.kw["dtype"] == "f32"))):
                    continue
                m.append_rows([min(rng.choice([0, 0, 1, 5, 16, 40]), limit - len(x)) for x in m.ids], op == "prompt")
            elif op in ("fork", "copy"):
                order = list(range(m.B))
                rng.shuffle(order)
                n = rng.randint(1, m.B - 1)
                src = [rng.choice(order[n:]) for _ in range(n)]
                (m.fork if op == "fork" else lambda s, t: m.copy_from(m, s, t))(src, order[:n])
            elif op == "free":
                m.free(rng.sample(range(m.B), rng.randint(0, 3)))
            elif op == "trim" and not ring:
                m.trim([len(x) if rng.random() < 0.5 else max(0, len(x) // 16 - 1) * 16 if m.quant else rng.randint(0, len(x))
                        for x in m.ids])
            elif op == "compact" and m.pages:
                used = m.cache.compact()
                table = m.cache.export(kvc.KVC_EXPORT_PAGE_TABLE)
                assert used == len(np.unique(table[table >= 0])) and table.max() < used
        except kvc.KvcError as e:
            # a full pool refuses and changes nothing
            assert e.code == kvc.KVC_ERR_CAPACITY and m.pages, (op, e)
            assert m.cache.page_counts() == before[0] and m.ids == before[1]
            m.free([max(range(m.B), key=lambda b: len(m.ids[b]))])
        if step % 7 == 6:
            m.check()
    m.check()


def test_branches_share_until_they_write():
    m = Model(B=5, cap=64, pages=12)
    m.append_rows([37, 0, 0, 0, 0])
    assert m.cache.page_counts() == (9, 0)
    m.fork([0] * 4, [1, 2, 3, 4])
    assert m.cache.page_counts() == (9, 3)               # nothing copied
    m.check()
    m.append()                                            # four of the five holders copy the last page; the fifth keeps it
    assert m.cache.page_counts() == (5, 2)
    m.check()
    m.free([1, 2])
    assert m.cache.page_counts() == (7, 2)
    m.free([0, 3])                                        # one holder left
    assert m.cache.page_counts() == (9, 0)
    m.check()
    m.fork([4, 4], [0, 4 - 1])
    m.trim([32, 0, 0, 5, 38])                             # page 1 of request 3, page 2 of request 0 given up
    assert m.cache.page_counts() == (9, 2)
    m.append_rows([1, 0, 0, 1, 0])                        # request 0 starts page 2 anew, request 3 copies page 0
    assert m.cache.page_counts() == (7, 2)
    m.check()


def test_a_full_pool_refuses_the_write_not_the_fork():
    m = Model(B=3, cap=64, pages=3)
    m.append_rows([40, 0, 0])
    m.fork([0, 0], [1, 2])
    with pytest.raises(kvc.KvcError) as e:
        m.append()
    assert e.value.code == kvc.KVC_ERR_CAPACITY
    m.check()
    m.free([2])
    with pytest.raises(kvc.KvcError):
        m.append()
    m.free([1])
    m.append_rows([1, 0, 0])
    m.check()


def test_store_slots_and_shared_pages():
    # a save reads shared pages, a load gives them up
    cfg = kvc.make_config("f32", "contiguous", None, 3, 2, 2, 16, 64, page_pool=9, store_slots=1)
    c = kvc.Cache(cfg)
    k = torch.randn(3, 2, 40, 16, device="cuda")
    c.append_rows(k, k, counts=[40, 0, 0])
    c.fork([0, 0], [1, 2])
    c.store_save(0, 1, 40)
    c.append(k[:, :, 0].contiguous(), k[:, :, 1].contiguous())
    assert c.page_counts() == (4, 2)
    c.store_load_batch([0, 0], [0, 2], [33, 17])
    assert list(c.next_positions()) == [33, 41, 17] and c.page_counts() == (1, 0)
    K = c.export(kvc.KVC_EXPORT_K)
    assert np.array_equal(K[0][:, :33], k[0].cpu().numpy()[:, :33]) and np.array_equal(K[2][:, :17], k[0].cpu().numpy()[:, :17])
    assert np.array_equal(K[1][:, :40], k[0].cpu().numpy())


def test_chunk_after_a_fork():
    w = wl.small("fork-chunk", B=3, Hq=4, Hkv=2, d=128, capacity=128, rope_base=10000.0, seed=3)
    a, b = (kvc.Cache.from_workload(w, max_chunk=32, page_pool=p, out_dtype="f32") for p in (24, 0))
    k, v = (x.cuda() for x in w.prefill_chunk(0, 41))
    a.append_rows(k, v, counts=[41, 0, 0])
    a.fork([0, 0], [1, 2])
    same = [x[:1].expand(3, -1, -1, -1).contiguous() for x in (k, v)]
    b.append_rows(*same)
    q, k2, v2 = (w.queries((3, 32, 4, 128), "s").cuda(), w.keys((3, 32, 2, 128), "s").cuda(), w.values((3, 32, 2, 128), "s").cuda())
    assert torch.equal(a.chunk(q, k2, v2), b.chunk(q, k2, v2))
    assert a.page_counts()[1] == 2


@pytest.mark.parametrize("layout,pa,pb", [("contiguous", 30, 0), ("contiguous", 0, 30), ("contiguous", 30, 30), ("contiguous", 0, 0),
                                          ("ring", 14, 0), ("ring", 0, 14)])
@pytest.mark.parametrize("quant", [None, "int8", "int8-dither"])
def test_copies_between_caches(layout, pa, pb, quant):
    cap = 64
    a = Model(B=4, cap=cap, layout=layout, pages=pa, quant=quant)
    b = Model(B=6, cap=cap if layout == "ring" else 96, layout=layout, pages=pb, quant=quant, g=4)
    a.append_rows([40, 3, 0, 64])
    b.append_rows([0, 17, 1, 40, 2, 0])
    b.copy_from(a, [0, 3, 0, 2], [1, 5, 0, 3])
    a.check()
    b.check()
    b.append()
    b.check()
    a.append_rows([1, 1, 1, 0])
    a.check()
    b.check()


def test_copy_needs_pages_before_it_gives_any_up():
    a, b = Model(B=2, cap=96), Model(B=2, cap=96, pages=6)
    a.append_rows([96, 30])
    b.append_rows([64, 5])
    with pytest.raises(kvc.KvcError) as e:
        b.copy_from(a, [0, 0], [0, 1])
    assert e.value.code == kvc.KVC_ERR_CAPACITY
    b.check()
    b.copy_from(a, [1, 1], [0, 1])
    b.check()
    assert b.cache.page_counts() == (2, 0)


def test_many_requests_and_many_sources():
    # more destinations and more sources than one launch holds
    B = 700
    m = Model(B=B, Hkv=1, d=64, cap=32, pages=1500)
    m.append_rows([b % 20 if b < 100 else 0 for b in range(B)])
    m.fork([b % 100 for b in range(100, B)], list(range(100, B)))
    m.check(decode=False)
    r = Model(B=B, Hkv=1, d=64, cap=48)
    r.copy_from(m, list(range(B)), list(reversed(range(B))))
    r.check(decode=False)
    m.free(list(range(0, B, 2)))
    m.cache.compact()
    m.check(decode=False)


def test_region_views():
    m = Model(B=2, cap=32, pages=8, dtype="f32")
    m.append_rows([20, 7])
    K, V = m.cache.rows()
    table = m.cache.export(kvc.KVC_EXPORT_PAGE_TABLE)
    want = m.cache.export(kvc.KVC_EXPORT_K)
    assert np.array_equal(K[int(table[0, 1]), :, :4].cpu().numpy(), want[0][:, 16:20])
    m.free([0])
    used = m.cache.compact()
    assert used == 1
    assert np.array_equal(m.cache.rows()[1][0, :, :7].cpu().numpy(), m.cache.export(kvc.KVC_EXPORT_V)[1][:, :7])


def test_refusals():
    m = Model(B=3, cap=32, pages=6)
    m.append_rows([20, 1, 1])

    def refused(code, f, *a):
        with pytest.raises(kvc.KvcError) as e:
            f(*a)
        assert e.value.code == code

    c = m.cache
    for src, dst in (([0], [0]), ([0, 1], [1, 2]), ([0, 0], [1, 1]), ([3], [0]), ([0], [3]), ([-1], [0]), ([0], [-1])):
        refused(kvc.KVC_ERR_ARG, c.fork, src, dst)
        if src[0] != 3:
            refused(kvc.KVC_ERR_ARG, c.copy_from, c, src, dst)
    for reqs in ([0, 0], [3], [-1]):
        refused(kvc.KVC_ERR_ARG, c.free, reqs)
    with pytest.raises(ValueError):
        c.fork([0, 1], [2])
    c.fork([], [])
    c.free([])
    m.check()
    for kw in (dict(dtype="f32"), dict(d=128), dict(Hkv=1), dict(rope=0.0), dict(layout="ring"), dict(quant="int8")):
        refused(kvc.KVC_ERR_ARG, Model(**{"B": 3, "cap": 32, **kw}).cache.copy_from, c, [0], [0])
    refused(kvc.KVC_ERR_CAPACITY, Model(B=3, cap=16).cache.copy_from, c, [0], [0])
    refused(kvc.KVC_ERR_ARG, Model(B=3, quant="int8-dither", key=(1, 1)).cache.copy_from, Model(B=3, quant="int8-dither").cache, [0], [0])
    plain = Model(B=3, cap=32)
    refused(kvc.KVC_ERR_UNSUPPORTED, plain.cache.compact)
    refused(kvc.KVC_ERR_UNSUPPORTED, plain.cache.page_counts)
    # under capture: nothing enqueued, nothing changed; a write into a shared page likewise
    m.fork([0], [1])
    k, v = (x.contiguous() for x in m.rows([0, 1, 2]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for f, a in ((c.fork, ([0], [2])), (c.free, ([0],)), (c.compact, ()), (c.copy_from, (plain.cache, [0], [0])), (c.append, (k, v))):
            refused(kvc.KVC_ERR_UNSUPPORTED, f, *a)
        torch.zeros(1, device="cuda")
    m.check()
    # restored blocks do not follow a request; a destination's return to the pool
    gate = kvc.Cache(kvc.make_config("bf16", "contiguous", "int8", 2, 4, 2, 64, 64, int8_exact_blocks=4))
    k = torch.randn(2, 2, 40, 64, device="cuda").bfloat16()
    gate.append_rows(k, k)
    full = torch.zeros(2, 2, 64, 64, dtype=torch.bfloat16, device="cuda")
    gate.restore([(0, 0, 1), (0, 1, 0)], full, full)
    refused(kvc.KVC_ERR_UNSUPPORTED, gate.fork, [0], [1])
    gate.fork([1], [0])
    gate.restore([(1, 0, 0), (1, 1, 0), (0, 0, 0), (0, 1, 1)], full, full)               # all four entries are free again
    gate.free([0, 1])
    assert (gate.export(kvc.KVC_EXPORT_XMAP) == -1).all()


def test_prompt_fork_decode_free_together():
    """Rotated by three axes, prompted into a paged cache, forked, decoded in branches, freed and compacted:
    every step's output against the same run in an unpaged cache that was filled row by row."""
    B, Hq, Hkv, d, n = 6, 8, 2, 128, 53
    cfg = dict(dtype="bf16", batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d, capacity=128, out_dtype="f32")
    paged, plain = kvc.Cache(kvc.make_config(page_pool=20, **cfg)), kvc.Cache(kvc.make_config(**cfg))
    qkv = torch.randn(2 * n, Hq + 2 * Hkv, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    pos = torch.randint(0, 60, (3, 2 * n), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    kvc.kvc_rope_axes(qkv[:, :Hq + Hkv], pos, [16, 24, 24], 10000.0, qkv[:, :Hq + Hkv])          # queries and keys, in place
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    out = paged.prompt(q, k, v, [n, n, 0, 0, 0, 0])
    paged.fork([0, 0, 1, 1], [2, 3, 4, 5])
    source = [0, 1, 0, 0, 1, 1]
    rows = [torch.stack([x[s * n:(s + 1) * n] for s in source]).transpose(1, 2).contiguous() for x in (k, v)]
    plain.append_rows(*rows)
    # the prompt's last row is what a decode at that position gives; |o| <= max |v| < 5
    last = plain.decode(torch.stack([q[s * n + n - 1] for s in source]).contiguous())
    assert (out[[n - 1, 2 * n - 1]] - last[:2]).abs().max() <= 2.2 * 2.0 ** -8 * 10
    for step in range(20):
        g = torch.Generator().manual_seed(10 + step)
        x = torch.randn(B, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
        p = torch.full((3, B), 60 + step, dtype=torch.int32, device="cuda")
        kvc.kvc_rope_axes(x[:, :Hq + Hkv], p, [16, 24, 24], 10000.0, x[:, :Hq + Hkv])
        q1, k1, v1 = (t.contiguous() for t in x.split([Hq, Hkv, Hkv], 1))
        got = []
        for c in (paged, plain):
            c.append(k1, v1)
            got.append(c.decode(q1))
        assert (got[0] - got[1]).abs().max() <= 4e-3 * 6
        if step == 9:
            paged.free([1, 4])
            paged.compact()
            paged.fork([5, 2], [1, 4])
            plain.fork([5, 2], [1, 4])
    assert paged.device_status() == 0 and plain.device_status() == 0


def ring_after_a_fork():
    """A wrapped paged ring forked, one row appended to every request: one page of four is each branch's own."""
    m = Model(B=3, d=128, cap=64, layout="ring", pages=16)
    m.append_rows([70, 0, 5])
    m.fork([0], [1])
    m.append()
    assert m.cache.page_counts()[1] == 3
    return m


def test_captured_writes_into_a_ring_need_every_page_to_be_private():
    # replays go round the ring: a page that is shared would be written by them sooner or later, although
    # the captured call itself stays in a page of its own
    m = ring_after_a_fork()
    c = m.cache
    x = [torch.zeros(*s, 128, dtype=torch.bfloat16, device="cuda") for s in ((3, 2), (3, 2, 1), (2, 4), (2, 2), (3, 1, 4), (3, 1, 2))]
    step, rows, q, kv, cq, ckv = x
    free = c.page_counts()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for f, a in ((c.append, (step, step)), (c.append_rows, (rows, rows)), (c.append_rows, (rows, rows, [0, 1, 0])),
                     (c.prompt, (q, kv, kv, [1, 0, 1])), (c.chunk, (cq, ckv, ckv))):
            with pytest.raises(kvc.KvcError) as e:
                f(*a)
            assert e.value.code == kvc.KVC_ERR_UNSUPPORTED
        torch.zeros(1, device="cuda")
    assert c.page_counts() == free
    m.check()
    # a request whose pages are its own may be captured beside them
    g = torch.cuda.CUDAGraph()
    tok = m.rows([7])
    with torch.cuda.graph(g):
        c.append_rows(*(t[:, :, None].expand(3, -1, 1, -1).contiguous() for t in tok), counts=[0, 0, 1])
    g.replay()
    m.ids[2].append(7)
    m.check()


@pytest.mark.parametrize("call", ["append_rows", "prompt"])
def test_replays_round_a_private_ring_leave_its_branches_alone(call):
    m = ring_after_a_fork()
    c = m.cache
    m.append_rows([64, 0, 0])                                   # request 0 has written all of its pages
    assert c.page_counts()[1] == 0
    m.check()
    others = {w: c.export(w)[1:] for w in (kvc.KVC_EXPORT_K, kvc.KVC_EXPORT_V, kvc.KVC_EXPORT_POSITIONS)}
    tok = m.rows([9])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        if call == "prompt":
            c.prompt(torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda"), *tok, [1, 0, 0])
        else:
            c.append_rows(*(t[:, :, None].expand(3, -1, 1, -1).contiguous() for t in tok), counts=[1, 0, 0])
    for _ in range(80):
        g.replay()
    assert c.device_status() == 0
    for w, want in others.items():
        assert np.array_equal(c.export(w)[1:], want)
    assert list(c.export(kvc.KVC_EXPORT_NEXT_POSITION)) == [70 + 1 + 64 + 80, 71, 6]


@pytest.mark.parametrize("call", ["append", "append_rows"])
@pytest.mark.parametrize("kind", [dict(d=128), dict(d=6), dict(dtype="f32"), dict(quant="int8"), dict(quant="int8-dither", d=128)],
                         ids=lambda k: "-".join("%s=%s" % kv for kv in k.items()))
def test_replayed_appends_past_the_mapped_pages_are_reported(kind, call):
    # a captured call maps the pages of its own rows; replays that leave them write nothing, wherever the
    # pool's pages lie (page 0 holds live rows here), and set the device error
    m = Model(B=2, cap=64, pages=8, **kind)
    m.append_rows([40, 24])
    assert m.cache.compact() == 5
    tok = [t.expand(2, -1, -1).contiguous() for t in m.rows([5])]
    rows = [t[:, :, None].contiguous() for t in tok]
    m.cache.append(*tok)                                            # (loads the kernels before the capture)
    m.ids = [x + [5] for x in m.ids]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.cache.append(*tok) if call == "append" else m.cache.append_rows(*rows)
    for _ in range(7):                                              # up to slots 47 and 31, the last of their pages
        g.replay()
    m.ids = [x + [5] * 7 for x in m.ids]
    c = m.cache
    assert c.device_status() == 0 and list(c.export(kvc.KVC_EXPORT_NEXT_POSITION)) == [48, 32]
    fresh = Model(B=2, cap=64, pages=0, **kind)
    names = [kvc.KVC_EXPORT_K, kvc.KVC_EXPORT_V] if not m.quant else [kvc.KVC_EXPORT_KQ, kvc.KVC_EXPORT_VQ, kvc.KVC_EXPORT_SK, kvc.KVC_EXPORT_SV,
                                                                    kvc.KVC_EXPORT_KTAIL, kvc.KVC_EXPORT_VTAIL]
    names += [kvc.KVC_EXPORT_WITNESS] if m.quant == "int8" else []
    stored = [c.state[off:off + n] for off, n in (kvc.kvc_region(c.h, w) for w in names)]
    before, positions = [x.clone() for x in stored], c.export(kvc.KVC_EXPORT_POSITIONS)
    for _ in range(20):
        g.replay()
    assert c.device_status() == 1 and c.device_status() == 0        # read and cleared
    for w, x, y in zip(names, stored, before):
        assert torch.equal(x, y), w
    assert np.array_equal(c.export(kvc.KVC_EXPORT_POSITIONS), positions)
    assert list(c.export(kvc.KVC_EXPORT_NEXT_POSITION)) == ([48, 32] if call == "append" else [68, 52])
    # what the valid rows hold is what one call after another would have written
    k, v = (torch.stack(x).transpose(1, 2).contiguous()
            for x in zip(*(fresh.rows((ids + [0] * 48)[:48]) for ids in m.ids)))
    fresh.cache.append_rows(k, v, counts=[48, 32])
    for b, n in enumerate((48, 32)):
        for w in names:
            if w in (kvc.KVC_EXPORT_KTAIL, kvc.KVC_EXPORT_VTAIL):
                continue
            per = n if w in (kvc.KVC_EXPORT_K, kvc.KVC_EXPORT_V, kvc.KVC_EXPORT_KQ, kvc.KVC_EXPORT_VQ, kvc.KVC_EXPORT_WITNESS) else n // 16
            assert np.array_equal(c.export(w)[b][:, :per], fresh.cache.export(w)[b][:, :per]), (w, b)


def test_a_trimmed_ring_waits_for_a_row_of_every_request_that_lost_one():
    # a wrapped ring has overwritten the first key of the window of the row at cut - 1: until the request
    # appends, its decode would lack that key.  Rows of other requests do not lift the guard
    for rows in ("append_rows", "prompt"):
        m = Model(B=3, d=64, cap=48, layout="ring")
        m.append_rows([100, 20, 130])
        m.trim([99, 20, 130])
        q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")

        def decodes():
            calls = [m.cache.decode, lambda q: kvc.kvc_decode_attn_noalloc(m.cache.h, q, torch.empty_like(q))]
            answers = set()
            for f in calls:
                try:
                    f(q)
                    answers.add(True)
                except kvc.KvcError as e:
                    assert e.code == kvc.KVC_ERR_ARG
                    answers.add(False)
            assert len(answers) == 1
            return answers.pop()

        assert not decodes()
        m.append_rows([0, 3, 1], rows == "prompt")
        assert not decodes(), rows
        m.fork([0], [1])                                          # the branch lacks the same key
        m.append_rows([1, 0, 0], rows == "prompt")
        assert not decodes()
        m.append_rows([0, 1, 0], rows == "prompt")
        assert decodes()
        m.check()
        m.trim([len(x) - (b == 2) for b, x in enumerate(m.ids)])
        m.free([2])
        m.append_rows([0, 0, 1], rows == "prompt")               # an empty request lacks nothing
        m.check()


def test_a_ring_trimmed_before_it_wrapped_decodes():
    # every key of the window is still there, as it is where the trim dropped nothing
    m = Model(B=2, d=64, cap=48, layout="ring")
    m.append_rows([40, 100])
    m.trim([31, 100])
    m.check()


def test_copies_carry_the_ring_guard_of_the_request():
    a, b = (Model(B=2, d=64, cap=48, layout="ring") for _ in range(2))
    a.append_rows([100, 60])
    b.append_rows([7, 60])
    a.trim([99, 60])
    b.copy_from(a, [1], [0])                                      # a request that lacks nothing
    b.check()
    b.copy_from(a, [0], [1])
    with pytest.raises(kvc.KvcError) as e:
        b.cache.decode(torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"))
    assert e.value.code == kvc.KVC_ERR_ARG
    b.append_rows([0, 1])
    b.check()


def test_a_loaded_ring_waits_for_a_row_too():
    cfg = kvc.make_config("f32", "ring", None, 2, 2, 2, 16, 16, max_position=200, store_slots=1)
    c = kvc.Cache(cfg)
    k = torch.randn(2, 2, 40, 16, device="cuda")
    q = torch.randn(2, 2, 16, device="cuda")
    c.append_rows(k, k)
    want = c.decode(q)
    c.store_save(0, 0, 40)
    c.store_load(0, 1, 39)
    row = k[:, :, 39:].contiguous()
    c.append_rows(row, row, counts=[1, 0])
    with pytest.raises(kvc.KvcError) as e:
        c.decode(q)
    assert e.value.code == kvc.KVC_ERR_ARG
    c.append_rows(k[:1, :, 39:].expand(2, -1, -1, -1).contiguous(), k[:1, :, 39:].expand(2, -1, -1, -1).contiguous(), counts=[0, 1])
    assert torch.equal(c.decode(q[:1].expand(2, -1, -1).contiguous())[1], want[0])
    c.store_load(0, 1, 40)                                        # whole: nothing is missing
    assert torch.equal(c.decode(q[:1].expand(2, -1, -1).contiguous())[1], want[0])


def test_what_trimmed_rows_overwrote_stays_lost():
    # one step back at a time goes no further than one step: position 39 overwrote 23, which 38 attends to
    cfg = kvc.make_config("f32", "ring", None, 1, 2, 2, 16, 16, max_position=200, store_slots=1)
    c = kvc.Cache(cfg)
    k = torch.randn(1, 2, 40, 16, device="cuda")
    c.append_rows(k, k)
    c.trim([39])
    c.trim([39])
    c.store_save(0, 0, 39)
    for f in (lambda: c.trim([38]), lambda: c.store_load(0, 0, 38)):
        with pytest.raises(kvc.KvcError) as e:
            f()
        assert e.value.code == kvc.KVC_ERR_EVICTED
    c.store_load(0, 0, 39)
    with pytest.raises(kvc.KvcError):
        c.decode(k[:, :, 0].contiguous())
    row = k[:, :, 39:].contiguous()
    c.append_rows(row, row)
    fresh = kvc.Cache(cfg)
    fresh.append_rows(k, k)
    q = torch.randn(1, 2, 16, device="cuda")
    assert torch.equal(c.decode(q), fresh.decode(q))
    c.trim([0])                                                   # from nothing, everything is possible again
    c.append_rows(k[:, :, :3].contiguous(), k[:, :, :3].contiguous())
    c.decode(q)
    c.trim([1])
    c.decode(q)


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("pages", [0, 16], ids=["rows", "pages"])
def test_random_ring_trims(pages, seed):
    # what a ring may be trimmed to, loaded at and decoded from, against slots that are simulated one by one
    W, B = 32, 3
    m = Model(B=B, d=64, cap=W, layout="ring", pages=pages)
    cfg = kvc.make_config(batch=B, page_pool=pages, store_slots=2, **m.kw)
    m.cache = c = kvc.Cache(cfg)
    m.rng = rng = random.Random(seed)
    slots = [{} for _ in range(B)]                                # slot -> position
    store = [None, None]                                          # (slots, tokens)
    q = wl.normal((B, 4, 64), 3, "q", "cuda", c.torch_dtype)

    def held(s, lo, hi):
        return all(s.get(p % W) == p for p in range(max(0, lo), hi))

    def put(b, lo):
        for p in range(lo, len(m.ids[b])):
            slots[b][p % W] = p

    def accepted(f):
        try:
            f()
            return True
        except kvc.KvcError as e:
            assert e.code in (kvc.KVC_ERR_EVICTED, kvc.KVC_ERR_ARG)
            return False

    for step in range(120):
        n = [len(x) for x in m.ids]
        op = rng.choice(["rows", "rows", "append", "prompt", "trim", "trim", "fork", "free", "save", "load", "copy"])
        if op in ("rows", "prompt"):
            m.append_rows([rng.choice([0, 0, 1, 2, 20, 60]) for _ in range(B)], op == "prompt")
        elif op == "append":
            m.append()
        elif op == "trim":
            cuts = [rng.choice([x, x, max(0, x - 1), max(0, x - 2), rng.randint(0, x)]) for x in n]
            want = all(held(s, cut - W + 1, cut) for s, cut in zip(slots, cuts))
            assert accepted(lambda: c.trim(cuts)) == want, (step, n, cuts)
            if want:
                m.ids = [ids[:cut] for ids, cut in zip(m.ids, cuts)]
                slots = [{k: p for k, p in s.items() if p < cut} for s, cut in zip(slots, cuts)]
        elif op in ("fork", "copy"):
            a, b = rng.sample(range(B), 2)
            m.fork([a], [b]) if op == "fork" else m.copy_from(m, [a], [b])
            slots[b] = dict(slots[a])
        elif op == "free":
            b = rng.randrange(B)
            m.free([b])
            slots[b] = {}
        elif op == "save" and max(n):
            b, i = rng.choice([b for b in range(B) if n[b]]), rng.randrange(2)
            c.store_save(i, b, n[b])
            store[i] = (dict(slots[b]), list(m.ids[b]))
        elif op == "load" and store[0] and store[1]:
            b, i = rng.randrange(B), rng.randrange(2)
            s, ids = store[i]
            cut = rng.choice([len(ids), max(0, len(ids) - 1), max(0, len(ids) - 2)])
            want = held(s, cut - W + 1, cut)
            assert accepted(lambda: c.store_load(i, b, cut)) == want, (step, len(ids), cut)
            if want:
                m.ids[b], slots[b] = ids[:cut], {k: p for k, p in s.items() if p < cut}
        for b in range(B):
            if len(m.ids[b]) > n[b] and op in ("rows", "prompt", "append"):
                put(b, n[b])
        whole = [held(s, len(x) - W, len(x)) for s, x in zip(slots, m.ids)]
        if min(len(x) for x in m.ids):
            assert accepted(lambda: c.decode(q)) == all(whole), (step, op, whole)
            if all(whole) and step % 5 == 0:
                m.check()


@pytest.mark.parametrize("quant", ["int8", "int8-dither"])
def test_a_trimmed_int8_ring_still_holds_its_window(quant):
    # an INT8 ring overwrites a block when a newer one completes, and a wrapped one is trimmed within its exact
    # tail only: blocks and tail hold every key, before the next append and beside rows of other requests
    def cache(counts):
        m = Model(B=2, d=64, cap=48, layout="ring", quant=quant)
        m.rng = random.Random(7)
        m.append_rows(counts)
        return m

    q = wl.normal((2, 4, 64), 3, "q", "cuda", torch.bfloat16)
    m = cache([105, 70])
    for cut in (104, 103):
        m.trim([cut, 70])
        fresh = kvc.Cache(kvc.make_config(batch=2, **m.kw))
        k, v = (torch.stack([t[:105] for t in x]).transpose(1, 2).contiguous() for x in zip(*(m.rows((ids + [0] * 105)[:105]) for ids in m.ids)))
        fresh.append_rows(k, v, counts=[cut, 70])
        assert torch.equal(m.cache.decode(q), fresh.decode(q)), cut
    m.append_rows([0, 3])
    assert torch.equal(m.cache.decode(q)[0], fresh.decode(q)[0])
    with pytest.raises(kvc.KvcError) as e:
        m.trim([100, 73])                                         # one row back at a time
    assert e.value.code == kvc.KVC_ERR_EVICTED
