"""Decode over 4-bit rows keeps 21 bits of queries and weights, whatever the number of heads: fp32 outputs within bounds some
hundred times below what dropping a few keys would change."""
import pytest
import torch

import _int4 as i4
from _int4_bounds import decode_bound
from test_gpu_int4 import SHAPES, Model, make, rows

pytestmark = pytest.mark.gpu


class Exact(Model):
    def check_decode(self, q, out, what=""):
        for b in range(self.c.B):
            n = self.k[b].shape[1]
            p = torch.arange(n, device="cuda")
            seen = (p >= n - self.window) | (p < self.sinks) if self.window else p >= 0
            kp, vp = (i4.quantise(x[:, seen]) for x in (self.keys(b), self.v[b]))
            qb = i4.turned(q[b], n - 1, self.base)
            ref, w = i4.attend(qb, i4.values(*kp), i4.values(*vp))
            bound = decode_bound(qb, kp, vp, w, query=2.0 ** -21, weight=2.0 ** -21, turned=bool(self.base))
            err = (out[b].double() - ref).abs()
            assert (err <= bound).all(), "%s request %d: %.3g times the bound" % (what, b, (err / bound).nan_to_num(1e30).max())


@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (6, 2), (8, 1), (5, 1), (24, 2), (9, 1), (48, 3), (16, 1), (7, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("base", [0.0, 10000.0])
def test_heads(hq, hkv, d, base):
    c = make(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, rope_base=base)
    m = Exact(c, base)
    counts = (1, 300, 47)
    k, v = rows(1, 3, hkv, 300, d), rows(2, 3, hkv, 300, d, False)
    c.append_rows(k, v, counts=counts)
    m.append(k, v, counts)
    q = rows(3, 3, hq, 1, d, False)[:, :, 0].contiguous()
    m.check_decode(q, c.decode(q))


@pytest.mark.parametrize("layout,pool", SHAPES + [("ring", 100)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 7), (17, 1), (200, 150)])
@pytest.mark.parametrize("hq", [4, 16])
def test_lengths(layout, pool, window, sinks, hq):
    if layout == "ring":
        window, sinks = 16 * (window // 16 or 1), 0
    c = make(layout, n_q_heads=hq, page_pool=pool, capacity=window if layout == "ring" else 512, window=0 if layout == "ring" else window,
             sinks=sinks, rope_base=10000.0)
    m = Exact(c, 10000.0, window, sinks)
    for step, counts in enumerate([(1, 2, 15), (15, 14, 1), (1, 1, 1), (15, 111, 128), (1, 1, 1), (100, 3, 96)]):
        k, v = rows(10 * step, 3, 2, max(counts), 128), rows(10 * step + 1, 3, 2, max(counts), 128, False)
        c.append_rows(k, v, counts=counts)
        m.append(k, v, counts)
        q = rows(10 * step + 2, 3, hq, 1, 128, False)[:, :, 0].contiguous()
        m.check_decode(q, c.decode(q), "step %d" % step)


@pytest.mark.parametrize("n", [2047, 2048, 20011])
@pytest.mark.parametrize("hq,d", [(4, 128), (8, 128), (8, 64)])
@pytest.mark.parametrize("sharp", [1, 10, 40])
def test_long(n, hq, d, sharp):
    c = make(batch=1, n_q_heads=hq, n_kv_heads=1, head_dim=d, capacity=20480)
    m = Exact(c)
    k, v = rows(1, 1, 1, n, d) * sharp, rows(2, 1, 1, n, d, False)
    k[:, :, n // 2:] *= 3
    c.append_rows(k, v)
    m.append(k, v, (n,))
    q = rows(3, 1, hq, 1, d, False)[:, :, 0].contiguous()
    m.check_decode(q, c.decode(q))


def test_answers_do_not_depend_on_the_order_of_requests():
    # 128 requests, 32 of them long: where those stand in the batch changes neither the splits nor, with them, any bit
    B, hkv, hq, d, long_, short = 128, 4, 16, 128, 6000, 90
    g = torch.Generator().manual_seed(1)
    lens = [long_ - 7 * b if b % 4 == 3 else 1 + (short + b) % 100 for b in range(B)]
    k, v = rows(1, 1, hkv, long_, d), rows(2, 1, hkv, long_, d, False)
    q = rows(3, B, hq, 1, d, False)[:, :, 0].contiguous()
    outs = []
    for order in (list(range(B)), sorted(range(B), key=lambda b: lens[b]), torch.randperm(B, generator=g).tolist()):
        c = make(batch=B, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, capacity=6000)
        c.append_rows(k.expand(B, -1, -1, -1).contiguous(), v.expand(B, -1, -1, -1).contiguous(), counts=[lens[b] for b in order])
        out = c.decode(q[order].contiguous())
        outs.append(torch.empty_like(out).index_copy_(0, torch.tensor(order, device="cuda"), out))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
