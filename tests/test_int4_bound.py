"""The bound of the decode over 4-bit rows, on the CPU: it holds for an evaluation with the kernel's roundings, and no answer with
keys left out stays within it."""
import math

import pytest
import torch

import _int4 as i4
from _int4_bounds import decode_bound

BITS = dict(query=2.0 ** -21, weight=2.0 ** -21)
SHAPES = [(4, 1, 128, 300), (8, 1, 128, 300), (5, 1, 64, 47), (9, 1, 128, 300), (16, 1, 64, 300), (8, 1, 128, 20011), (48, 3, 64, 300)]


def rows(seed, H, n, d, wide=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((H, n, d), generator=g)
    if wide:
        x = x * torch.exp(torch.randn((H, 1, d), generator=g) * 0.7) + torch.randn((H, 1, d), generator=g)
    return x.bfloat16()


def case(hq, hkv, d, n, wide):
    k, v = rows(1, hkv, n, d, wide), rows(2, hkv, n, d, False)
    return rows(3, hq, 1, d, False)[:, 0].double(), i4.quantise(k), i4.quantise(v)


def kept(parts, keep):
    return tuple(x[:, keep] for x in parts)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hkv,d,n", SHAPES)
def test_wrong_answers_pass_the_bound(hq, hkv, d, n, wide):
    q, kp, vp = case(hq, hkv, d, n, wide)
    ref, w = i4.attend(q, i4.values(*kp), i4.values(*vp))
    bound = decode_bound(q, kp, vp, w, **BITS)
    past = lambda y: ((y - ref).abs() > bound).any(-1)  # noqa: E731
    assert past(torch.zeros_like(ref)).all()
    i = torch.arange(n)
    for keep in (i >= 5, i // 32 % 4 != 1, i < n - 1):                       # the first keys, a warp's tiles, the newest key
        wrong, _ = i4.attend(q, i4.values(*kept(kp, keep)), i4.values(*kept(vp, keep)))
        # (heads that give what is left out less than a thousandth of their weight do not count)
        weighs = w[:, ~keep].sum(-1) > 1e-3
        assert weighs.any() or n > 10000
        assert past(wrong)[weighs].all()
    wrong, _ = i4.attend(q, i4.values(*kp), i4.values(vp[0], vp[1], vp[2] * 0))
    assert past(wrong).all()


@pytest.mark.parametrize("hq,hkv,d,n", SHAPES)
@pytest.mark.parametrize("sharp", [1, 10, 40])
def test_the_roundings_of_the_kernel_stay_within_it(hq, hkv, d, n, sharp):
    # query and weights in two fp16 parts, the reference a whole number, fp32 elsewhere
    q, kp, vp = case(hq, hkv, d, n, True)
    kp = (kp[0], kp[1] * sharp, kp[2] * sharp)
    r, G = hq // hkv, d // 32
    ref, w = i4.attend(q, i4.values(*kp), i4.values(*vp))
    bound = decode_bound(q, kp, vp, w, **BITS)
    two = lambda x: (lambda h: h.float() + (x - h.float()).half().float())(x.half())  # noqa: E731
    each = lambda x: x.float().repeat_interleave(r, 0)  # noqa: E731
    qs = q.float() * (math.log2(math.e) / math.sqrt(d))
    up = 2.0 ** (14 - qs.abs().amax(-1, keepdim=True).log2().floor())
    qh = (two(qs * up) / up).unflatten(-1, (G, 32))
    ku, vu = (each(x[0]).unflatten(-1, (G, 32)) for x in (kp, vp))
    s = (torch.einsum("hgx,hngx->hng", qh, ku) * each(kp[1]) + qs.unflatten(-1, (G, 32)).sum(-1)[:, None] * each(kp[2])).sum(-1)
    p = torch.exp2(s - s.amax(-1, keepdim=True).ceil())
    ps = p[..., None] * each(vp[1])
    norm = 2.0 ** (9 - ps.amax(1, keepdim=True).log2().floor())
    o = torch.einsum("hng,hngx->hgx", two(ps * norm) / norm, vu) + (p[..., None] * each(vp[2])).sum(1)[..., None]
    err = (o.flatten(1) / p.sum(-1, keepdim=True)).double() - ref
    assert (err.abs() <= bound).all()
