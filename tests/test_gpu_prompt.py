"""Packed prompts (kvc_prompt_attn): rows of every request appended and attended, each request
with a cut and a count of its own, against attention in 64 bits over the rows the cache holds.

Tolerances.  With weights p_j in fp32 (fp32 caches, head sizes other than 64 and 128) the bound is
that of the other attention calls (1e-5 or 2e-3, absolute and relative, plus a bf16 output's
half step).  On the tensor cores each weight is rounded to bf16, p_j (1 + e_j) with |e_j| <= 2^-8,
so the result moves by at most sum p_j |e_j| |v_j| <= 2^-8 sum p_j |v_j|; fp32 accumulation of the scores (128 products) and ex2 add relative errors below 2^-13 to a weight.
The bound taken is 1.1 * 2^-8 (sum p_j |v_j| + |o|) plus the output's half step.
"""
import math

import numpy as np
import pytest
import torch

from kv_cache_decode_ring_gb300 import kvc
from kv_cache_decode_ring_gb300 import workloads as wl
from oracle import numerics as nm

from _parity import TOL, bf16_half_ulp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_decode_ring_gb300 import build
    build.build()


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def rotate(x, pos, base, dtype):
    """x [n, heads, d] (cache dtype) rotated at pos in fp32 and rounded to the cache dtype."""
    if base == 0.0 or x.shape[0] == 0:
        return x
    n, heads, d = x.shape
    y = np.stack([nm.rope_rotate(np.ascontiguousarray(x[:, h].float().numpy()), np.asarray(pos), base) for h in range(heads)], 1)
    return rounded(y, dtype)


def attend(q, K, V, cut, window):
    """out and sum p |v| of queries q [n, Hq, d] at cut + i over K, V [L, Hkv, d], all rows, in 64 bits."""
    n, Hq, d = q.shape
    L, Hkv = K.shape[:2]
    qd, Kd, Vd = (x.double().transpose(0, 1) for x in (q, K, V))
    p = torch.arange(cut, cut + n)[:, None]
    j = torch.arange(L)
    seen = (j <= p) & ((j > p - window) if window else (j >= 0))
    out, mag = torch.empty(Hq, n, d, dtype=torch.float64), torch.empty(Hq, n, d, dtype=torch.float64)
    for h in range(Hq):
        k, v = Kd[h * Hkv // Hq], Vd[h * Hkv // Hq]
        w = torch.softmax((qd[h] @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf), -1)
        if torch.isfinite(v).all():
            out[h], mag[h] = w @ v, w @ v.abs()
        else:                                               # keys that are not seen add nothing, whatever they hold
            for i in range(n):
                out[h, i], mag[h, i] = w[i, seen[i]] @ v[seen[i]], w[i, seen[i]] @ v[seen[i]].abs()
    return out.transpose(0, 1).numpy(), mag.transpose(0, 1).numpy()


class Twin:
    """A cache and the rows that it should hold: per request K, V [len, Hkv, d] in the cache dtype."""

    def __init__(self, dtype="bf16", B=2, Hq=8, Hkv=2, d=128, cap=512, layout="contiguous", window=0, pages=0, base=10000.0,
                 out="f32", max_chunk=0, max_position=0):
        self.dtype, self.B, self.Hq, self.Hkv, self.d, self.base = dtype, B, Hq, Hkv, d, base
        self.window = cap if layout == "ring" else window
        self.layout, self.cap = layout, cap
        self.cache = kvc.Cache(kvc.make_config(dtype, layout, None, B, Hq, Hkv, d, cap, window, max_position, base, max_chunk, out,
                                               page_pool=pages))
        self.K = [torch.empty(0, Hkv, d, dtype=self.cache.torch_dtype) for _ in range(B)]
        self.V = [torch.empty(0, Hkv, d, dtype=self.cache.torch_dtype) for _ in range(B)]
        self.drawn = 0

    def draw(self, n, heads):
        self.drawn += 1
        return wl.normal((n, heads, self.d), 5, "prompt%d" % self.drawn, dtype=self.cache.torch_dtype)

    def take(self, counts, k, v):
        at = 0
        for b, n in enumerate(counts):
            pos = np.arange(len(self.K[b]), len(self.K[b]) + n)
            self.K[b] = torch.cat((self.K[b], rotate(k[at:at + n], pos, self.base, self.dtype)))
            self.V[b] = torch.cat((self.V[b], v[at:at + n]))
            at += n

    def prefill(self, lengths):
        n = max(lengths)
        if n == 0:
            return
        k, v = self.draw(self.B * n, self.Hkv), self.draw(self.B * n, self.Hkv)
        kb, vb = (x.view(self.B, n, self.Hkv, self.d).transpose(1, 2).contiguous().cuda() for x in (k, v))
        self.cache.append_rows(kb, vb, counts=lengths)
        pick = torch.cat([torch.arange(b * n, b * n + m) for b, m in enumerate(lengths)])
        self.take(lengths, k[pick], v[pick])

    def trim(self, cuts):
        self.cache.trim(cuts)
        self.K = [x[:c] for x, c in zip(self.K, cuts)]
        self.V = [x[:c] for x, c in zip(self.V, cuts)]

    def prompt(self, counts, fused=True, spare=0, qkv=None, **kw):
        """One call, checked against the reference; returns the output (host) and the inputs."""
        T = sum(counts)
        if qkv is None:
            qkv = self.draw(T + spare, self.Hq + 2 * self.Hkv)
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], 1)
        dev = qkv.cuda()
        dq, dk, dv = dev.split([self.Hq, self.Hkv, self.Hkv], 1)
        if not fused:
            dq, dk, dv = (x.contiguous() for x in (dq, dk, dv))
        out = torch.full((T + spare, self.Hq, self.d), 7.5, dtype=self.cache.out_dtype, device="cuda")
        self.cache.prompt(dq, dk, dv, counts, out, **kw)
        cuts = [len(x) for x in self.K]
        self.take(counts, k[:T], v[:T])
        got = out.cpu()
        assert (got[T:] == 7.5).all(), "rows behind the last request written"
        at = 0
        for b, n in enumerate(counts):
            if n:
                qr = rotate(q[at:at + n], np.arange(cuts[b], cuts[b] + n), self.base, self.dtype)
                ref, mag = attend(qr, self.K[b], self.V[b], cuts[b], self.window)
                self.compare(got[at:at + n], ref, mag, (b, cuts[b], n))
            at += n
        return got, qkv

    def compare(self, got, ref, mag, what):
        if self.dtype == "bf16" and self.d in (64, 128):
            bound = 1.1 * 2.0 ** -8 * (mag + np.abs(ref))
        else:
            bound = TOL[self.dtype] * (1 + np.abs(ref))
        if got.dtype == torch.bfloat16:
            bound = bound + bf16_half_ulp(ref)
        excess = np.abs(got.double().numpy() - ref) - bound
        assert np.isfinite(excess).all() and excess.max() <= 0, (what, excess.max(), np.unravel_index(excess.argmax(), excess.shape))

    def check_state(self):
        assert self.cache.device_status() == 0
        want = [len(x) for x in self.K]
        assert list(self.cache.next_positions()) == want
        assert list(self.cache.export(kvc.KVC_EXPORT_NEXT_POSITION)) == want
        pos = self.cache.export(kvc.KVC_EXPORT_POSITIONS)
        for which, rows in ((kvc.KVC_EXPORT_K, self.K), (kvc.KVC_EXPORT_V, self.V)):
            held = self.cache.export(which)
            for b, x in enumerate(rows):
                p = np.arange(max(0, len(x) - self.cap), len(x))
                assert np.array_equal(pos[b][p % self.cap], p)
                assert (np.delete(pos[b], p % self.cap) == -1).all()
                raw = x.view(torch.int16 if self.dtype == "bf16" else torch.int32).numpy()[p]
                mine = held[b].view(np.int16 if self.dtype == "bf16" else np.int32)[:, p % self.cap].transpose(1, 0, 2)
                assert np.array_equal(mine, raw), (which, b)


SHAPES = [
    # dtype, Hq, Hkv, d, window, base, output
    ("bf16", 8, 2, 128, 0, 10000.0, "f32"),
    ("bf16", 8, 2, 128, 0, 0.0, None),
    ("bf16", 3, 3, 128, 0, 10000.0, None),
    ("bf16", 8, 1, 64, 0, 10000.0, "f32"),
    ("bf16", 5, 1, 64, 37, 10000.0, None),
    ("bf16", 6, 2, 128, 100, 10000.0, "f32"),
    ("bf16", 4, 2, 128, 1, 10000.0, "f32"),
    ("bf16", 4, 2, 80, 0, 10000.0, "f32"),
    ("bf16", 2, 1, 256, 50, 10000.0, None),
    ("f32", 4, 2, 128, 0, 10000.0, None),
    ("f32", 3, 1, 6, 9, 10000.0, "bf16"),
    ("f32", 2, 2, 64, 0, 0.0, None),
]


@pytest.mark.parametrize("paged", [False, True], ids=["rows", "pages"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_prompts_match_reference(shape, paged):
    dtype, Hq, Hkv, d, window, base, out = shape
    # (views of a 6-dim projection are not 16-byte aligned: fused rows from 64 dims on)
    counts = [[130, 0, 1, 67], [1, 1, 1, 1], [3, 128, 40, 0]]
    t = Twin(dtype, 4, Hq, Hkv, d, 384, window=window, pages=4 * 24 if paged else 0, base=base, out=out)
    t.prefill([0, 17, 131, 16])
    for c in counts:
        t.prompt(c, fused=d != 6, spare=3)
    t.check_state()


@pytest.mark.parametrize("g", [1, 2, 3, 4, 8, 16])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 300])
def test_lengths_around_the_tiles(n, g):
    t = Twin("bf16", 1, g, 1, 128, 700, base=0.0, out="f32")
    t.prefill([n % 5 * 33])
    t.prompt([n], fused=False)
    t.check_state()


@pytest.mark.parametrize("cut", [0, 1, 15, 16, 127, 128, 129, 200])
@pytest.mark.parametrize("window", [0, 2, 128, 130, 500])
def test_cuts_and_windows(cut, window):
    t = Twin("bf16", 2, 4, 1, 64, 500, window=window, out="f32")
    t.prefill([cut, 3])
    t.prompt([70, 200])
    t.check_state()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("W,paged", [(16, False), (64, True), (144, False), (256, True)])
def test_rings(W, paged, d):
    # suffixes longer than the ring, cuts inside a block, a trim, requests without rows
    t = Twin("bf16", 3, 4, 2, d, W, "ring", pages=3 * (W // 16) if paged else 0, max_chunk=300, max_position=1000, out="f32")
    t.prefill([5, W + 7, 0])
    t.prompt([300, 1, 40], spare=2)
    t.check_state()
    t.prompt([9, 0, W], fused=False)
    lengths = [len(x) for x in t.K]
    t.trim([x - 1 if x > W else x for x in lengths] if W > 16 else lengths)
    t.prompt([33, 17, 1])
    t.check_state()


def test_after_a_trim():
    t = Twin("bf16", 2, 4, 2, 128, 512, out="f32")
    t.prefill([300, 129])
    t.trim([257, 0])
    t.prompt([100, 130])
    t.check_state()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_masked_rows_do_not_reach_the_result(dtype, d, bad):
    # stale rows behind the cut, rows before the window, and a later row of the same tile hold
    # values that are not finite: queries that do not see them stay right
    t = Twin(dtype, 1, 4, 2, d, 512, window=50, out="f32")
    k = torch.full((1, 2, 300, d), bad, dtype=t.cache.torch_dtype, device="cuda")
    t.cache.append_rows(k, k)
    t.cache.trim([0])
    t.prefill([40])
    qkv = t.draw(200, 8)
    clean, _ = t.prompt([200], qkv=qkv.clone())
    # the same prompt with one value row and one key row spoilt: only the 50 queries from it on change
    for head, at in ((6, 60), (4, 130)):
        t.trim([40])
        spoilt = qkv.clone()
        spoilt[at, head] = bad
        q, kk, vv = spoilt.cuda().split([4, 2, 2], 1)
        got = t.cache.prompt(q, kk, vv, [200]).cpu()
        kv = (head - 4) % 2
        seen = torch.zeros(200, 4, dtype=torch.bool)
        seen[at:at + 50, 2 * kv:2 * kv + 2] = True
        same = torch.isfinite(got) & ((got - clean).abs() <= 2.0 ** -7 * (1 + clean.abs()))
        assert same[~seen].all()
        # what sees it follows the definition in 64 bits: not finite exactly where that is not
        K, V = torch.cat((t.K[0][:40], rotate(spoilt[:, 4:6], np.arange(40, 240), t.base, dtype))), torch.cat((t.V[0][:40], spoilt[:, 6:8]))
        ref, _ = attend(rotate(spoilt[:, :4], np.arange(40, 240), t.base, dtype), K, V, 40, 50)
        assert torch.equal(torch.isnan(got), torch.from_numpy(np.isnan(ref)))
        assert torch.equal(torch.isinf(got), torch.from_numpy(np.isinf(ref)))
        t.K[0], t.V[0] = torch.cat((t.K[0][:40], K[40:])), torch.cat((t.V[0][:40], V[40:]))
    t.trim([40])


def test_large_scores_and_equal_rows():
    # scores of +-several hundred (one key takes all the weight), then all keys equal (a mean)
    t = Twin("bf16", 1, 2, 1, 128, 300, base=0.0, out="f32")
    qkv = t.draw(200, 4)
    qkv[:, :3] *= 16
    t.prompt([200], qkv=qkv)
    t = Twin("bf16", 1, 2, 1, 64, 300, base=0.0, out="f32")
    qkv = t.draw(200, 4)
    qkv[:, 2] = 1.0
    t.prompt([200], qkv=qkv)


def test_rows_equal_one_token_decodes():
    a = Twin("bf16", 2, 8, 2, 128, 300, base=0.0, out="f32")
    b = Twin("bf16", 2, 8, 2, 128, 300, base=0.0, out="f32")
    for t in (a, b):
        t.prefill([100, 3])
    out, qkv = a.prompt([20, 20])
    q, k, v = (x.cuda() for x in qkv.split([8, 2, 2], 1))
    for i in range(20):
        pick = torch.tensor([i, 20 + i], device="cuda")
        b.cache.append(k[pick].contiguous(), v[pick].contiguous())
        one = b.cache.decode(q[pick].contiguous()).cpu()
        # both within 1.1 * 2^-8 (sum p |v| + |o|), sum p |v| <= max |v| < 5 for these draws
        assert (one - out[[i, 20 + i]]).abs().max() <= 2.2 * 2.0 ** -8 * 10


def test_captured_call_replays_from_the_device_positions():
    a, b = (Twin("bf16", 3, 8, 2, 128, 600, out="f32") for _ in range(2))
    for t in (a, b):
        t.prefill([10, 0, 77])
    counts = [5, 130, 1]
    qkv = a.draw(136, 12).cuda()
    q, k, v = qkv.split([8, 2, 2], 1)
    warm = Twin("bf16", 3, 8, 2, 128, 600, out="f32")
    warm.cache.prompt(q, k, v, counts)
    out = torch.empty(136, 8, 128, device="cuda")
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        a.cache.prompt(q, k, v, counts, out)
    for step in range(3):
        qkv.copy_(a.draw(136, 12))
        g.replay()
        want = b.cache.prompt(q, k, v, counts)
        torch.cuda.synchronize()
        assert torch.equal(out, want), step
    for which in (kvc.KVC_EXPORT_K, kvc.KVC_EXPORT_V, kvc.KVC_EXPORT_POSITIONS, kvc.KVC_EXPORT_NEXT_POSITION):
        assert np.array_equal(a.cache.export(which), b.cache.export(which))


@pytest.mark.parametrize("dtype,d,paged", [("bf16", 128, False), ("bf16", 64, True), ("bf16", 96, True), ("f32", 64, False), ("f32", 64, True)])
def test_replays_past_the_capacity_are_reported(dtype, d, paged):
    # the host counts a captured call once; replays that run out of rows or of mapped pages
    # write nothing there, leave the other requests' rows alone and set the device error
    t = Twin(dtype, 2, 4, 2, d, 64, pages=8 if paged else 0)
    t.prefill([40, 20])
    qkv = t.draw(12, 8).cuda()
    q, k, v = qkv.split([4, 2, 2], 1)
    out = torch.empty(12, 4, d, dtype=t.cache.out_dtype, device="cuda")
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        t.cache.prompt(q, k, v, [0, 12], out)          # request 1: rows 20 .. 31, pages up to slot 31 mapped
    g.replay()
    assert t.cache.device_status() == 0
    before = [x.clone() for x in t.cache.rows()]
    replays = 4                                        # 32 .. 79: past the mapped pages, past the capacity
    for _ in range(replays):
        g.replay()
    assert t.cache.device_status() == 1
    assert t.cache.device_status() == 0            # read and cleared
    if paged:
        for x, y in zip(t.cache.rows(), before):
            assert torch.equal(x, y)
    else:
        for x, y in zip(t.cache.rows(), before):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1, :, :32], y[1, :, :32])
    assert list(t.cache.export(kvc.KVC_EXPORT_NEXT_POSITION)) == [40, 32 + 12 * replays]


def test_two_handles_on_two_streams():
    ts = [Twin("bf16", 2, 8, 2, 128, 1200, out="f32") for _ in range(2)]
    qkvs = [t.draw(1500, 12).cuda() for t in ts]
    qkvs[1].mul_(0.5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    outs = []
    for t, x, s in zip(ts, qkvs, streams):
        outs.append(t.cache.prompt(*x.split([8, 2, 2], 1), [1100, 400], torch.empty(1500, 8, 128, device="cuda"), stream=s))
    torch.cuda.synchronize()
    for t, x, o in zip(ts, qkvs, outs):
        t.trim([0, 0])
        again = t.cache.prompt(*x.split([8, 2, 2], 1), [1100, 400])
        assert torch.equal(o, again)


@pytest.mark.parametrize("Hq,Hkv,d,window,paged", [(8, 2, 128, 0, True), (2, 2, 128, 0, False), (8, 1, 64, 40, False), (12, 4, 64, 0, True)])
def test_many_short_units(Hq, Hkv, d, window, paged):
    # several units of work for every SM, most of one to three tiles, ragged, some requests empty
    rng = np.random.default_rng(3)
    B = 150
    counts = [int(x) for x in rng.choice([0, 1, 5, 40, 64, 65, 130, 260], B)]
    cuts = [int(x) for x in rng.integers(0, 100, B)]
    t = Twin("bf16", B, Hq, Hkv, d, 368, window=window, pages=B * 23 if paged else 0, out="f32")
    t.prefill(cuts)
    t.prompt(counts)
    t.prompt([1] * B)
    t.check_state()


@pytest.mark.parametrize("layout,window,paged", [("contiguous", 0, False), ("contiguous", 0, True), ("contiguous", 1500, False), ("ring", 0, True)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 128), (2, 2, 64), (8, 1, 64)])
def test_few_rows_behind_long_prefixes(Hq, Hkv, d, layout, window, paged):
    # few rows and many keys: the keys are split over CTAs and joined
    cap = 2048 if layout == "ring" else 3300
    cap -= cap % 16 if paged else 0
    t = Twin("bf16", 2, Hq, Hkv, d, cap, layout, window=window, pages=2 * cap // 16 if paged else 0, max_chunk=64, max_position=4000)
    t.prefill([3000, 700])
    for counts in ([1, 1], [0, 1], [3, 0], [20, 9]):
        t.prompt(counts)
    t.check_state()


@pytest.mark.parametrize("dtype,d", [("f32", 128), ("f32", 6), ("f32", 80), ("f32", 256), ("bf16", 96), ("bf16", 250)])
@pytest.mark.parametrize("window,paged", [(0, False), (0, True), (900, False)])
def test_few_rows_behind_long_prefixes_on_the_cuda_cores(dtype, d, window, paged):
    # as above, and calls of many rows, whose keys are not split
    cap = 1504
    t = Twin(dtype, 3, 4, 1, d, cap, window=window, pages=3 * cap // 16 if paged else 0, max_position=4000)
    t.prefill([1300, 0, 257])
    for counts in ([1, 1, 1], [0, 1, 0], [9, 0, 3], [90, 64, 1], [1, 0, 40]):
        t.prompt(counts)
    t.check_state()


def test_more_requests_than_one_launch_holds():
    B = 1100
    t = Twin("bf16", B, 2, 1, 64, 16, base=0.0, out="f32")
    t.prompt([b % 4 for b in range(B)])
    t.prompt([3 - b % 4 for b in range(B)])
    t.check_state()


def test_refusals():
    t = Twin("bf16", 2, 4, 2, 128, 64)
    c = t.cache
    q, k, v = (torch.zeros(40, h, 128, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
    for counts in ([1], [20, 21], [1, 2, 3]):
        with pytest.raises(ValueError):
            c.prompt(q, k, v, counts)
    for x in ((q.float(), k, v), (q[:, :3], k, v), (q, k.cpu(), v), (q.transpose(0, 1).contiguous().transpose(0, 1), k, v), (q, k[:30], v)):
        with pytest.raises(ValueError):
            c.prompt(*x, [1, 2])
    with pytest.raises(ValueError):
        c.prompt(q, torch.zeros(40, 3, 128, dtype=torch.bfloat16, device="cuda")[:, :2], v, [1, 2])     # k and v rows apart

    def refused(code, f):
        with pytest.raises(kvc.KvcError) as e:
            f()
        assert e.value.code == code

    refused(kvc.KVC_ERR_ARG, lambda: c.prompt(q, k, v, [-1, 2]))
    big = torch.zeros(70, 8, 128, dtype=torch.bfloat16, device="cuda")
    refused(kvc.KVC_ERR_CAPACITY, lambda: c.prompt(*big.split([4, 2, 2], 1), [65, 1]))
    assert list(c.next_positions()) == [0, 0] and (c.export(kvc.KVC_EXPORT_POSITIONS) == -1).all()
    odd = torch.zeros(40 * 8 * 128 + 8, dtype=torch.bfloat16, device="cuda")[1:1 + 40 * 8 * 128].view(40, 8, 128)
    refused(kvc.KVC_ERR_ARG, lambda: c.prompt(*odd.split([4, 2, 2], 1), [1, 1]))                        # 2-byte aligned
    same = Twin("bf16", 2, 4, 2, 128, 64, out="bf16").cache
    buf = torch.zeros(40, 12, 128, dtype=torch.bfloat16, device="cuda")
    spare = torch.zeros(80, 4, 128, dtype=torch.bfloat16, device="cuda")
    for x, out in ((buf[:, :8].split([4, 2, 2], 1), buf.view(-1)[8 * 128:][:40 * 4 * 128].view(40, 4, 128)),   # between its rows
                   ((q, k, v), q), ((q, spare.view(160, 2, 128)[2:42], v), spare[:40])):
        refused(kvc.KVC_ERR_ARG, lambda: same.prompt(*x, [2, 3], out))
    one = kvc._ints([1, 0])
    refused(kvc.KVC_ERR_ARG, lambda: kvc._check(kvc.lib().kvc_prompt_attn(
        c.h, q.data_ptr(), 1 << 38, k.data_ptr(), v.data_ptr(), 0, kvc._at(one), buf.data_ptr(), 0), "stride"))
    wide = kvc.Cache(kvc.make_config("f32", "contiguous", None, 1, 70000, 70000, 2, 16))
    refused(kvc.KVC_ERR_UNSUPPORTED, lambda: wide.prompt(*(torch.zeros(1, 70000, 2, device="cuda") for _ in range(3)), [1]))
    refused(kvc.KVC_ERR_UNSUPPORTED, lambda: wide.free([0]))
    c.prompt(q, k, v, [0, 0])                                                                            # nothing to do
    int8 = kvc.Cache(kvc.make_config("bf16", "contiguous", "int8", 2, 4, 2, 128, 64))
    refused(kvc.KVC_ERR_UNSUPPORTED, lambda: int8.prompt(q, k, v, [1, 1]))
    ring = kvc.Cache(kvc.make_config("bf16", "ring", None, 2, 4, 2, 128, 40, max_chunk=8))
    refused(kvc.KVC_ERR_UNSUPPORTED, lambda: ring.prompt(q, k, v, [1, 1]))
    ring = kvc.Cache(kvc.make_config("bf16", "ring", None, 2, 4, 2, 128, 48, max_chunk=8))
    refused(kvc.KVC_ERR_ARG, lambda: ring.prompt(q, k, v, [9, 1]))
    paged = kvc.Cache(kvc.make_config("bf16", "contiguous", None, 2, 4, 2, 128, 64, page_pool=2))
    refused(kvc.KVC_ERR_CAPACITY, lambda: paged.prompt(q, k, v, [17, 1]))
    assert paged.page_counts() == (2, 0)
    paged.prompt(q, k, v, [16, 1])
    assert paged.page_counts() == (0, 0)


@pytest.mark.parametrize("d,Hq,Hkv,window", [(128, 8, 2, 0), (64, 8, 1, 0), (128, 4, 4, 1500), (64, 4, 1, 1500)])
@pytest.mark.parametrize("cut,n", [(2750, 250), (2990, 10), (0, 3000)])
def test_long_rows_by_their_root_mean_square(d, Hq, Hkv, window, cut, n):
    # The bound above has every weight rounded the same way; over many keys one lost key would hide in it.
    # Roundings of p_j to bf16 do not depend on one another: |e_j| <= 2^-8, so an output's error has a root
    # mean square of at most 2^-8 sqrt(sum p_j^2 v_j^2).  Scores of 128 products, 2^x and sums over 3000 keys
    # in fp32 stay below 2^-13 sqrt(sum p_j^2 v_j^2) + 2^-16 |o| beside it.  The mean over thousands of
    # outputs is held to that plus a tenth; a key left out of 3000 equal ones would read 5 times as much.
    t = Twin("bf16", 1, Hq, Hkv, d, 3008, window=window, base=0.0, out="f32")
    t.prefill([cut])
    qkv = t.draw(n, Hq + 2 * Hkv)
    qkv[:, :Hq] *= 0.25                                              # weights spread over the keys
    got, _ = t.prompt([n], qkv=qkv)
    rows = [i for i in range(n) if cut + i >= 1000][-300:]
    q, K, V = qkv[rows, :Hq].double(), t.K[0].double(), t.V[0].double()
    p = torch.tensor([cut + i for i in rows])[:, None]
    j = torch.arange(cut + n)
    seen = (j <= p) & ((j > p - window) if window else (j >= 0))
    err, allowed = 0.0, 0.0
    for h in range(Hq):
        k, v = K[:, h * Hkv // Hq], V[:, h * Hkv // Hq]
        w = torch.softmax((q[:, h] @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf), -1)
        err += (got[rows, h].double() - w @ v).square().sum().item()
        allowed += (2.0 ** -8 + 2.0 ** -13) ** 2 * (w.square() @ v.square()).sum().item() + (2.0 ** -16) ** 2 * (w @ v).square().sum().item()
    assert err <= 1.1 ** 2 * allowed, math.sqrt(err / allowed)


@pytest.mark.parametrize("d,n,cut", [(128, 130, 2800), (64, 130, 2800), (128, 2, 2990), (64, 2, 2990), (128, 1000, 0)])
def test_equal_keys_lose_none(d, n, cut):
    # equal scores: every weight is the same and rounds to 1 in bf16, so an output is the mean of the values
    # to fp32 accumulation: at most 3000 / 16 + 32 sums, each off by 2^-22 of the largest partial sum (of any
    # run of keys: twice the largest of those from the first one).  The weights' fp32 sum is off by the
    # rounding of the scaled maximum, below 32: 2^-20 ln 2, and the quotient by 2^-22
    t = Twin("bf16", 1, 4, 1, d, 3008, base=0.0, out="f32")
    k = torch.ones(1, 1, cut, d, dtype=torch.bfloat16)
    v = wl.normal((cut + n, 1, d), 9, "equal%d" % d, dtype=torch.bfloat16)
    if cut:
        t.cache.append_rows(k.cuda(), v[:cut].transpose(0, 1)[None].contiguous().cuda())
    q = torch.ones(n, 4, d, dtype=torch.bfloat16, device="cuda")
    out = t.cache.prompt(q, torch.ones(n, 1, d, dtype=torch.bfloat16, device="cuda"), v[cut:].cuda(), [n]).cpu().double()
    sums = v[:, 0].double().cumsum(0)
    count = torch.arange(1, cut + n + 1, dtype=torch.float64)[:, None]
    mean = (sums / count)[cut:]
    bound = (220 * 2.0 ** -22 * 2 * sums.abs().cummax(0).values / count)[cut:] + 2.0 ** -19 * mean.abs()
    assert ((out - mean[:, None]).abs() <= bound[:, None]).all(), ((out - mean[:, None]).abs() / bound[:, None]).max()
