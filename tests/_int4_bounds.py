"""How far the decode over 4-bit rows may be off, from its roundings one by one."""
import math

import torch

import _int4 as i4


def decode_bound(q, kparts, vparts, p, query=2.0 ** -11, weight=2.0 ** -11, turned=False):
    """q [hq, d] the query at its position and p [hq, n] the weights, in 64 bits; kparts, vparts: codes, scales and minima of the
    n visible rows of each KV head.  Outputs in fp32.

    A query's dim enters the products with codes off by `query` relative (1.01 2^-39 of its head's largest dim where that is
    below fp16's normal numbers), and exactly as fp32 holds it the sums of the minima's terms; 2^-22 for the
    product with log2(e)/sqrt(d).  Rotated in fp32 by cosines of fp32 (`turned`): three roundings of 2^-24 of |x_i| + |x_j|, which is at most
    sqrt(2) times the sum of the pair's magnitudes afterwards: 2^-21 of that sum.  A score sums d products of codes and G = d / 32 terms of minima: 32 products
    in two accumulations of the matrix unit, whose adds truncate (2^-23 of the sum of magnitudes each, aligned to the largest), G
    fused multiply-adds of scales, 5 + G of a group's query sum and the minima, 3 joins.  Its product with the softmax's unit is one rounding, and
    2^x is off by 2^-22, its argument (the score's distance from the softmax's reference, at most 5 from the largest) by 2^-24 of itself.
    A weight is an fp32 number, 1 for a score at the reference: one of 2^-126 or less may be held as 0 (the largest is 2^5 at most,
    and a warp's reference lies below the largest score of all by what its partial sums are scaled with, in fp32 too).
    Scores off by e change weights by 2 e relative at most (numerator and sum).
    A weight times its scale enters off by `weight`, or by 2^-25 where fp16's subnormal numbers hold it, the largest of its
    group being 2^7 at least, or its power of two the largest (2^120).  A weight passes min(n, 4096) / 32 + 64 additions at most on its way to the output (of a split: a chain per warp, four warps; splits)."""
    d, r, n = q.shape[-1], q.shape[0] // kparts[1].shape[0], p.shape[-1]
    G = d // i4.GROUP
    each = lambda x: x.double().abs().repeat_interleave(r, 0)  # noqa: E731
    ks, km, vs, vm = each(kparts[1]), each(kparts[2]), each(vparts[1]), each(vparts[2])       # [hq, n, G]
    ku, vu = (x[0].double().repeat_interleave(r, 0) for x in (kparts, vparts))                # [hq, n, d]
    spread = lambda x: x.repeat_interleave(i4.GROUP, -1)  # noqa: E731
    qa = q.abs()
    codes = torch.einsum("hd,hnd->hn", qa, ku * spread(ks)) / math.sqrt(d)
    minima = torch.einsum("hd,hnd->hn", qa, spread(km)) / math.sqrt(d)
    floor = 1.01 * 2.0 ** -39 * qa.amax(-1)[:, None] * (ku * spread(ks)).sum(-1) / math.sqrt(d)
    size = codes + minima
    turn = 0.0
    if turned:
        pair = qa.unflatten(-1, (-1, 2)).sum(-1).repeat_interleave(2, -1)
        turn = 2.0 ** -21 * torch.einsum("hd,hnd->hn", pair, ku * spread(ks) + spread(km)) / math.sqrt(d)
    err = turn + codes * query + floor + size * (2.0 ** -22 + (4 + G + 5 + G + 3 + 1) * 2.0 ** -23)
    far = (p.amax(-1, keepdim=True) / p.clamp(min=2.0 ** -1000)).log2() + 5
    err = err + 2.0 ** -22 + 2.0 ** -24 * far
    # a weight's own change, and the sum's: that of all weights at once
    rel = err + (p * err).sum(-1, keepdim=True) + (min(n, 4096) / 32 + 64) * 2.0 ** -23
    terms = torch.einsum("hn,hnd->hd", p * rel, vu * spread(vs) + spread(vm))
    gone = torch.einsum("hn,hnd->hd", p * (p < 2.0 ** -120 * p.amax(-1, keepdim=True)), vu * spread(vs) + spread(vm))
    held = weight * torch.einsum("hn,hnd->hd", p, vu * spread(vs))
    top = (p[..., None] * vs).amax(1)                                                         # [hq, G]
    small = (2.0 ** -32 * spread(top) + 2.0 ** -145) * vu.sum(1)
    return terms + held + gone + small + 2.0 ** -148
