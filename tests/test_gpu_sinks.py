"""Windows whose first positions stay visible: decode (every kernel that serves it) and packed prompts against 64 bits."""
import math

import pytest
import torch

import _int4 as i4
from kv_cache_decode_ring_gb300 import kvc

pytestmark = pytest.mark.gpu


def draw(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


class Twin:
    """A cache and the rows that it should hold: per request K (rotated) and V [Hkv, len, d]."""

    def __init__(self, dtype="bf16", quant=None, B=3, hq=8, hkv=2, d=128, cap=512, window=100, sinks=4, pages=0, base=10000.0, **kw):
        self.window, self.sinks, self.base, self.seed = window, sinks, base, 0
        self.quant = quant
        self.c = kvc.Cache(kvc.make_config(dtype, "contiguous", quant, B, hq, hkv, d, cap, window, rope_base=base, sinks=sinks,
                                           page_pool=pages, out_dtype="f32", **kw))
        self.dtype = self.c.torch_dtype
        self.K, self.V = ([torch.zeros((hkv, 0, d), dtype=self.dtype, device="cuda") for _ in range(B)] for _ in "kv")

    def draw(self, *shape):
        self.seed += 1
        return draw(self.seed, shape, self.dtype)

    def take(self, b, k, v):
        n = self.K[b].shape[1]
        self.K[b] = torch.cat((self.K[b], i4.rotated(k, torch.arange(n, n + k.shape[1]), self.base)), 1)
        self.V[b] = torch.cat((self.V[b], v), 1)

    def append(self, counts, k=None, v=None):
        n = max(counts)
        if n == 0:
            return
        c = self.c
        k = self.draw(c.B, c.Hkv, n, c.d) if k is None else k
        v = self.draw(c.B, c.Hkv, n, c.d) if v is None else v
        c.append_rows(k, v, counts=counts)
        for b, m in enumerate(counts):
            self.take(b, k[b, :, :m], v[b, :, :m])

    def trim(self, cuts):
        self.c.trim(cuts)
        for b, n in enumerate(cuts):
            self.K[b], self.V[b] = self.K[b][:, :n], self.V[b][:, :n]

    def seen(self, p, n):
        j = torch.arange(n, device="cuda")
        return (j <= p[:, None]) & ((j > p[:, None] - self.window) | (j < self.sinks))

    def decode(self, what=""):
        c = self.c
        q = self.draw(c.B, c.Hq, c.d)
        out = c.decode(q)
        for b in range(c.B):
            n = self.K[b].shape[1]
            seen = self.seen(torch.tensor([n - 1], device="cuda"), n)[0]
            k, v, qb = self.K[b][:, seen], self.V[b][:, seen], i4.turned(q[b], n - 1, self.base)
            if self.quant:
                kp, vp = i4.quantise(k), i4.quantise(v)
                ref, w = i4.attend(qb, i4.values(*kp), i4.values(*vp))
                bound = i4.decode_bound(qb, kp, vp, w)
            else:
                k, v = k.double(), v.double()
                ref, w = i4.attend(qb, k, v)
                r = c.Hq // c.Hkv
                # query and weights in two bf16 parts (2^-17) or fp32; fp32 sums of d products (2^-23 each at most), and of up
                # to 64 keys a chain; 2^x off by 2^-22; scores weigh twice, in a weight and in the sum of all
                size = torch.einsum("hd,hnd->hn", qb.abs(), k.repeat_interleave(r, 0).abs()).amax(-1) / math.sqrt(c.d)
                score = size * (2.0 ** -17 + 2.0 ** -22 + c.d * 2.0 ** -23) + 2.0 ** -22
                mag = torch.einsum("hn,hnd->hd", w, v.repeat_interleave(r, 0).abs())
                bound = (2 * score[:, None] + 2.0 ** -17 + 100 * 2.0 ** -23) * mag
            err = (out[b].double() - ref).abs()
            assert (err <= bound).all(), (what, b, n, float(err.max()), float(bound.max()))
        return q, out

    def prompt(self, counts, spare=0, qkv=None):
        c, T = self.c, sum(counts)
        if qkv is None:
            qkv = self.draw(T + spare, c.Hq + 2 * c.Hkv, c.d)
        q, k, v = qkv.split([c.Hq, c.Hkv, c.Hkv], 1)
        if c.d * q.element_size() % 16:
            q, k, v = (x.contiguous() for x in (q, k, v))
        out = torch.full((T + spare, c.Hq, c.d), 7.5, device="cuda")
        c.prompt(q, k, v, counts, out)
        assert (out[T:] == 7.5).all()
        at = 0
        for b, n in enumerate(counts):
            cut = self.K[b].shape[1]
            self.take(b, k[at:at + n].transpose(0, 1), v[at:at + n].transpose(0, 1))
            if n:
                self.compare(out[at:at + n].double(), q[at:at + n], b, cut)
            at += n
        return out

    def compare(self, out, q, b, cut):
        n, r = q.shape[0], self.c.Hq // self.c.Hkv
        p = torch.arange(cut, cut + n, device="cuda")
        q = i4.rotated(q.transpose(0, 1), p, self.base).double()                      # rounded to the cache's type, as keys are
        seen = self.seen(p, cut + n)
        for h in range(self.c.Hq):
            k, v = self.K[b][h // r].double(), self.V[b][h // r].double()
            s = (q[h] @ k.nan_to_num(0, 0, 0).T / math.sqrt(self.c.d)).masked_fill(~seen, -math.inf)
            w = s.softmax(-1)
            clean = v.nan_to_num(0, 0, 0)
            ref, mag = w @ clean, w @ clean.abs()
            # tensor cores: weights rounded to bf16, 2^-8 of them in the numerator (their sum is fp32); else fp32 throughout
            rough = self.dtype == torch.bfloat16 and self.c.d in (64, 128)
            bound = 1.1 * 2.0 ** -8 * (mag + ref.abs()) if rough else 1e-5 * (1 + mag)
            mine = out[:, h]
            if not v.isfinite().all():
                spoilt = (seen.double() @ (~v.isfinite()).double()) > 0               # what a row sees that is not finite
                assert not mine[spoilt].isfinite().any()
                mine = torch.where(spoilt, ref, mine)
            err = (mine - ref).abs()
            assert (err <= bound).all(), (b, h, cut, n, float(err.max()))


KERNELS = [("bf16", None, 8, 2, 128), ("bf16", None, 8, 1, 64), ("bf16", None, 2, 2, 128), ("bf16", None, 4, 2, 64),
           ("bf16", None, 9, 1, 64), ("bf16", None, 2, 2, 80), ("f32", None, 4, 2, 80), ("f32", None, 3, 1, 6),
           ("bf16", "int4", 8, 2, 128), ("bf16", "int4", 8, 1, 64)]


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("pages", [0, 120])
@pytest.mark.parametrize("window,sinks", [(1, 1), (17, 4), (200, 100), (33, 16), (16, 17), (100, 10000)])
def test_decode(kernel, pages, window, sinks):
    dtype, quant, hq, hkv, d = kernel
    t = Twin(dtype, quant, 3, hq, hkv, d, 512, window, sinks, pages)
    for step, counts in enumerate([(1, 16, 17), (1, 1, 1), (15, 0, 190), (1, 1, 1), (480, 100, 1)]):
        t.append(counts)
        t.decode("step %d" % step)
    assert t.c.device_status() == 0


@pytest.mark.parametrize("kernel", [("bf16", None, 4, 1, 128), ("bf16", None, 1, 1, 64), ("bf16", "int4", 8, 1, 128), ("f32", None, 2, 1, 64)],
                         ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("sinks", [5, 1500, 3000])
def test_decode_of_many_sinks(kernel, sinks):
    # sinks over several splits, up to the window and past it
    dtype, quant, hq, hkv, d = kernel
    t = Twin(dtype, quant, 2, hq, hkv, d, 8192, 2000, sinks)
    for counts in [(1990, 2600), (500, 1), (2000, 5000)]:
        t.append(counts)
        t.decode()


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("pages", [0, 60])
def test_decode_masked_rows_may_hold_anything(kernel, pages):
    dtype, quant, hq, hkv, d = kernel
    t = Twin(dtype, quant, 1, hq, hkv, d, 512, 40, 5, pages)
    k, v = t.draw(1, hkv, 200, d), t.draw(1, hkv, 200, d)
    for x, bad in ((k, math.nan), (v, math.inf), (v, math.nan)):
        x[:, :, 5:160:2] = bad                    # rows behind the sinks, up to the window (160 .. 199)
        x[:, :, 195:] = bad
    t.append([200], k, v)
    t.trim([195])
    t.append([5])
    assert torch.isfinite(t.decode()[1]).all()


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("n", [1, 300])
def test_decode_of_keys_that_are_all_nan(kernel, n):
    dtype, quant, hq, hkv, d = kernel
    c = Twin(dtype, quant, 1, hq, hkv, d, 512, 100, 20, base=0.0).c
    k = draw(1, (1, hkv, n, d), c.torch_dtype) * math.nan
    c.append_rows(k, draw(2, k.shape, c.torch_dtype))
    assert c.decode(draw(3, (1, hq, d), c.torch_dtype)).isnan().all()


@pytest.mark.parametrize("d", [64, 80])
def test_splits_of_sinks_that_are_all_nan_spoil_the_answer(d):
    # 1 split of the window and 24 of the sinks, 64 keys each, joined by 8 warps: all that the third one takes
    c = Twin("f32", None, 1, 2, 1, d, 2048, 17, 1500, base=0.0).c
    k = draw(1, (1, 1, 2000, d), torch.float32)
    for i in (1, 9, 17):
        k[:, :, 64 * i:64 * i + 64] = math.nan
    c.append_rows(k, draw(2, k.shape, torch.float32))
    assert c.decode(draw(3, (1, 2, d), torch.float32)).isnan().all()


def test_decode_as_a_graph_and_without_allocation():
    """Replays move the window past the sinks on the device; the fixed-scratch variant agrees."""
    t = Twin("bf16", None, 2, 8, 2, 128, 256, 20, 3)
    t.append((21, 2))
    k, v, q = t.draw(2, 2, 128), t.draw(2, 2, 128), t.draw(2, 8, 128)
    out = t.c.decode(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        t.c.append(k, v)
        t.c.decode(q, out)
    for _ in range(30):
        graph.replay()
    torch.cuda.synchronize()
    for b in range(2):
        for _ in range(30):
            t.take(b, k[b][:, None], v[b][:, None])
        n = t.K[b].shape[1]
        seen = t.seen(torch.tensor([n - 1], device="cuda"), n)[0]
        ref, _ = i4.attend(i4.turned(q[b], n - 1, t.base), t.K[b][:, seen].double(), t.V[b][:, seen].double())
        assert (out[b].double() - ref).abs().max() < 1e-3
    again = torch.empty_like(out)
    kvc.kvc_decode_attn_noalloc(t.c.h, q, again)
    assert torch.equal(out, again)


PROMPTS = [("bf16", 8, 2, 128), ("bf16", 5, 1, 64), ("bf16", 6, 2, 128), ("bf16", 4, 2, 80), ("f32", 4, 2, 128), ("f32", 3, 1, 6),
           ("f32", 2, 1, 256)]


@pytest.mark.parametrize("kernel", PROMPTS, ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("pages", [0, 200])
@pytest.mark.parametrize("window,sinks", [(1, 1), (17, 4), (130, 100), (33, 16), (16, 170), (100, 10000)])
def test_prompts(kernel, pages, window, sinks):
    dtype, hq, hkv, d = kernel
    t = Twin(dtype, None, 4, hq, hkv, d, 512, window, sinks, pages)
    t.append((0, 17, 131, 16))
    for counts in [(130, 0, 1, 67), (1, 1, 1, 1), (3, 200, 40, 0), (300, 20, 111, 129)]:
        t.prompt(counts, spare=2)
    t.decode()
    assert t.c.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pages", [0, 700])
@pytest.mark.parametrize("cut", [0, 79, 80, 1000, 2601])
def test_prompt_long(d, pages, cut):
    # many tiles: sinks of their own tiles and of the window's; a part of each where few rows stand behind a long prefix
    t = Twin("bf16", None, 2, 4, 1, d, 5008, 1024, 100, pages)
    t.append((cut, 0))
    t.prompt((2003, 5))
    t.prompt((3, 1300))
    t.prompt((1, 1))


def test_prompt_split_keys():
    # few rows behind a long window with many sinks: their keys go to several CTAs, some of sinks only
    for dtype, d in (("bf16", 128), ("bf16", 64), ("f32", 64)):
        t = Twin(dtype, None, 1, 4, 1, d, 8192, 3000, 1500)
        t.append((7000,))
        t.prompt((9,))
        t.prompt((200,))


@pytest.mark.parametrize("kernel", [("bf16", 8, 2, 128), ("bf16", 8, 2, 64), ("f32", 4, 2, 64)], ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("pages", [0, 60])
def test_prompt_rows_that_are_not_finite(kernel, pages):
    dtype, hq, hkv, d = kernel
    # masked for every row: nothing of them may show
    t = Twin(dtype, None, 1, hq, hkv, d, 512, 40, 5, pages)
    k, v = t.draw(1, hkv, 200, d), t.draw(1, hkv, 200, d)
    k[:, :, 5:161], v[:, :, 5:161:2], v[:, :, 6:161:2] = math.nan, math.inf, math.nan
    t.append([200], k, v)
    out = t.prompt([70])
    assert out.isfinite().all()
    # values of a sink, of a sink that the first rows' windows hold too, and of a row in the window: their dims, in rows that see them
    t = Twin(dtype, None, 2, hq, hkv, d, 512, 40, 5, pages)
    k, v = t.draw(2, hkv, 100, d), t.draw(2, hkv, 100, d)
    v[0, 0, 3, 1], v[0, 0, 70, 2], v[0, 0, 30, 3] = math.inf, -math.inf, math.nan
    v[1, 1, 2, 4] = math.nan
    t.append((100, 20), k, v)
    t.prompt((60, 90))


def test_refusals():
    t = Twin(cap=512, max_chunk=16)
    x = t.draw(3, 4, 8, 128)
    with pytest.raises(kvc.KvcError) as e:
        t.c.chunk(x, x[:, :, :2].contiguous(), x[:, :, :2].contiguous())
    assert e.value.code == kvc.KVC_ERR_UNSUPPORTED


def test_prompt_as_a_graph():
    # a captured prompt replayed: its window leaves the sinks behind on the device
    t = Twin("bf16", None, 1, 8, 2, 128, 512, 40, 5)
    t.append((30,))
    qkv = t.draw(50, 12, 128)
    q, k, v = qkv.split([8, 2, 2], 1)
    out = torch.empty((50, 8, 128), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.c.prompt(q, k, v, [50], out)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        cut = t.K[0].shape[1]
        t.take(0, k.transpose(0, 1), v.transpose(0, 1))
        t.compare(out.double(), q, 0, cut)
    assert t.c.device_status() == 0
