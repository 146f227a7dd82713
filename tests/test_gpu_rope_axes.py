"""Rotary positions with several axes (kvc_rope_axes) against rotation in 64 bits.

Tolerance, for a pair of inputs of magnitudes |x0|, |x1|: the angle is off by the rounding of the
fixed-point turn to fp32 (2^-25 half turns: 9.4e-8 rad) and by the frequency's own double rounding
(position * theta * 2^-52), the sine and cosine by 2 units of 2^-24 at most, the two products and the
sum by 2^-24 each, and the result is rounded to the output type (half a step).
"""
import math

import numpy as np
import pytest
import torch

from kv_cache_decode_ring_gb300 import build as kbuild
from kv_cache_decode_ring_gb300 import kvc


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


def reference(x, pos, sections, base, halves, per_axis):
    """64-bit rotation and the bound on the error before output rounding."""
    x = x.double().cpu().numpy()
    pos = pos.cpu().numpy().astype(np.float64)
    P = sum(sections)
    y, bound = x.copy(), np.zeros_like(x)
    p = 0
    for a, s in enumerate(sections):
        for j in range(s):
            theta = base ** (-(j / s) if per_axis else -(p / P))
            i0, i1 = (p, P + p) if halves else (2 * p, 2 * p + 1)
            ang = pos[a] * theta
            c, sn = np.cos(ang)[:, None], np.sin(ang)[:, None]
            y[..., i0] = x[..., i0] * c - x[..., i1] * sn
            y[..., i1] = x[..., i1] * c + x[..., i0] * sn
            size = np.abs(x[..., i0]) + np.abs(x[..., i1])
            err = 9.4e-8 + np.abs(ang) * 2.0 ** -51 + 4 * 2.0 ** -24
            bound[..., i0] = bound[..., i1] = size * err[:, None]
            p += 1
    return y, bound


def check(x, pos, sections, base, out, halves, per_axis):
    ref, bound = reference(x, pos, sections, base, halves, per_axis)
    half = torch.finfo(x.dtype).eps / 2
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= bound + half * (np.abs(ref) + bound)).all(), (err - bound - half * np.abs(ref)).max()
    P = 2 * sum(sections)
    assert torch.equal(out[..., P:], x[..., P:])


CASES = [
    # rows, heads, cols, d, sections, halves, per_axis, base, positions below
    (1, 1, 1, 2, [1], False, False, 10000.0, 100),
    (1, 40, 48, 128, [16, 24, 24], False, False, 10000.0, 100000),
    (5, 3, 3, 128, [64], True, False, 10000.0, 2 ** 31 - 1),
    (130, 7, 9, 64, [8, 12, 12], True, False, 1000000.0, 5000),
    (33, 2, 2, 80, [16, 16], True, False, 500.0, 70),
    (33, 2, 2, 80, [7, 10, 3], False, True, 500.0, 70),           # 40 rotated dims pass the rest through
    (257, 5, 6, 96, [11, 13], True, True, 10000.0, 3000),         # halves of 24 pairs
    (9, 3, 3, 14, [3, 2], True, False, 10000.0, 300),             # nothing a multiple of 16 bytes
    (9, 3, 4, 256, [16] * 8, False, True, 0.5, 300),              # frequencies above one turn's
    (1000, 1, 1, 128, [1, 63], True, False, 10000.0, 40000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:4])))
def test_matches_reference(case, dtype):
    rows, heads, cols, d, sections, halves, per_axis, base, far = case
    g = torch.Generator().manual_seed(11)
    full = torch.randn(rows, cols, d, generator=g).to(dtype).cuda()
    x = full[:, :heads]
    pos = torch.randint(-far, far, (len(sections), rows), generator=g, dtype=torch.int64).to(torch.int32).cuda()
    out = kvc.kvc_rope_axes(x, pos, sections, base, halves=halves, per_axis=per_axis)
    check(x, pos, sections, base, out, halves, per_axis)
    # in place, the heads beside it and the dims behind the sections untouched
    inplace = full.clone()
    y = inplace[:, :heads]
    assert kvc.kvc_rope_axes(y, pos, sections, base, y, halves=halves, per_axis=per_axis) is y
    assert torch.equal(y, out) and torch.equal(inplace[:, heads:], full[:, heads:])
    # into rows of another stride, the gap untouched
    wide = torch.full((rows, heads + 2, d), 3.0, dtype=dtype, device="cuda")
    kvc.kvc_rope_axes(x, pos, sections, base, wide[:, :heads], halves=halves, per_axis=per_axis)
    assert torch.equal(wide[:, :heads], out) and (wide[:, heads:] == 3.0).all()


@pytest.mark.gpu
def test_one_axis_equals_the_caches_rotation():
    # keys rotated here and stored as they are = keys that the cache rotates itself, to the rounding
    # of the table's cosines: at most one step of bf16, and seldom
    B, n, Hkv, d = 2, 200, 2, 128
    k = torch.randn(B * n, Hkv, d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B)[None].contiguous()
    turned = kvc.kvc_rope_axes(k, pos, [d // 2], 10000.0)
    own, plain = (kvc.Cache(kvc.make_config("bf16", "contiguous", None, B, 2, Hkv, d, 256, rope_base=r)) for r in (10000.0, 0.0))
    for cache, x in ((own, k), (plain, turned)):
        rows = x.view(B, n, Hkv, d).transpose(1, 2).contiguous()
        cache.append_rows(rows, rows)
    a, b = own.rows()[0][:, :, :n].float(), plain.rows()[0][:, :, :n].float()
    assert (a != b).float().mean() < 1e-3
    assert ((a - b).abs() <= 2.0 ** -7 * a.abs() + 1e-6).all()


@pytest.mark.gpu
def test_on_a_stream_and_captured():
    x = torch.randn(64, 8, 128, device="cuda").bfloat16()
    pos = torch.randint(0, 999, (3, 64), dtype=torch.int32, device="cuda")
    want = kvc.kvc_rope_axes(x, pos, [16, 24, 24])
    torch.cuda.synchronize()
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.kvc_rope_axes(x, pos, [16, 24, 24], 10000.0, out)
    x2 = torch.randn_like(x)
    x.copy_(x2)
    g.replay()
    assert torch.equal(out, kvc.kvc_rope_axes(x, pos, [16, 24, 24])) and not torch.equal(out, want)


def _raw(**kw):
    """The C entry point with host-checked arguments only: every call here is refused before the GPU is touched."""
    import ctypes
    a = dict(x=4096, xs=0, y=1 << 20, ys=0, dtype=kvc.KVC_BF16, rows=4, heads=2, d=64, pos=8192, axes=2, sections=(8, 8), base=1e4, flags=0)
    a.update(kw)
    s = (ctypes.c_int32 * max(1, len(a["sections"])))(*a["sections"]) if a["sections"] is not None else None
    return kvc.lib().kvc_rope_axes(a["x"], a["xs"], a["y"], a["ys"], a["dtype"], a["rows"], a["heads"], a["d"], a["pos"], a["axes"], s,
                                   a["base"], a["flags"], None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(y=None), dict(pos=None), dict(sections=None), dict(dtype=2), dict(rows=-1), dict(heads=0), dict(d=63),
    dict(d=0), dict(d=258), dict(axes=0), dict(axes=9, sections=(1,) * 9), dict(sections=(0, 8)), dict(sections=(16, 17)),
    dict(sections=(2 ** 31 - 1, 2 ** 31 - 1)), dict(base=0.0), dict(base=-1.0), dict(base=math.inf), dict(base=math.nan),
    dict(flags=4), dict(xs=127), dict(ys=1), dict(x=4097), dict(pos=8193), dict(y=4096 + 256), dict(y=4096, ys=256),
    dict(heads=1 << 20), dict(rows=1 << 40),
], ids=lambda b: "-".join("%s=%s" % kv for kv in b.items()))
def test_refusals(bad):
    assert _raw(**bad) == kvc.KVC_ERR_ARG


def test_no_rows_is_no_work():
    assert _raw(rows=0) == kvc.KVC_OK


@pytest.mark.gpu
@pytest.mark.parametrize("heads,d,rows", [(600000, 8, 2), (65536 * 8 + 1, 16, 1)])
def test_few_rows_of_very_many_heads(heads, d, rows):
    x = torch.randn(rows, heads, d, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    pos = torch.tensor([[5, 1000][:rows]], dtype=torch.int32, device="cuda")
    out = kvc.kvc_rope_axes(x, pos, [d // 2], 10000.0)
    check(x, pos, [d // 2], 10000.0, out, False, False)


@pytest.mark.parametrize("bad", [dict(base=5e-324, sections=(16, 16)), dict(base=5e-324, sections=(31, 1), flags=2)], ids=["all", "axis"])
def test_refuses_frequencies_beyond_a_doubles_range(bad):
    assert _raw(**bad) == kvc.KVC_ERR_ARG
