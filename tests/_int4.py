"""4-bit rows written out plainly: groups of 32 dims, x ~ m + u s with m = min x, s = bf16((max x - min x) / 15),
u = rint((x - m) / s) in 0 .. 15; and attention over rows and masks in 64 bits."""
import math

import torch

GROUP = 32


def quantise(x: torch.Tensor):
    """Codes (uint8), scales and minima (bf16, one per group) of bf16 rows [..., d]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((hi - lo) / torch.full_like(lo, 15.0)).bfloat16()
    s = torch.where(s.float().isfinite(), s, torch.full_like(s, math.nan))
    u = ((g - lo) / s.float()).round().clamp(0, 15)
    u = torch.where(s.float() > 0, u, torch.zeros_like(u))
    return u.flatten(-2).to(torch.uint8), s.squeeze(-1), lo.squeeze(-1).bfloat16()


def values(u, s, m) -> torch.Tensor:
    """What the codes stand for, in 64 bits."""
    return (u.double().unflatten(-1, (-1, GROUP)) * s.double()[..., None] + m.double()[..., None]).flatten(-2)


def held(x):
    return values(*quantise(x))


def order(d: int, value: bool) -> list:
    """Dims of the nibbles of a row's codes, from the lowest on."""
    G = d // GROUP
    if value:
        return [GROUP * (h % G) + 4 * (h // G) + i for h in range(d // 4) for i in range(4)]
    return [GROUP * (w % G) + 8 * (w // G) + j for w in range(d // 8) for j in range(8)]


def row_bytes(x, value: bool) -> torch.Tensor:
    """The bytes of rows [..., d] as the cache stores them: [..., 5 d / 8] uint8."""
    u, s, m = quantise(x)
    n = u[..., order(x.shape[-1], value)]
    codes = n[..., 0::2] | n[..., 1::2] << 4
    pairs = torch.stack((s, m), -1).flatten(-2).contiguous().view(torch.uint8)
    return torch.cat((codes, pairs), -1)


def rotated(x, pos, base):
    """bf16 rows [..., n, d] rotated at pos [n] as a cache stores keys: pairs (2i, 2i + 1), fp32, rounded once."""
    if not base:
        return x
    d = x.shape[-1]
    theta = torch.tensor([base ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=x.device)
    a = pos.to(x.device).double()[:, None] * theta
    c, s = a.cos().float(), a.sin().float()
    x0, x1 = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack((x0 * c - x1 * s, x1 * c + x0 * s), -1).flatten(-2).to(x.dtype)


def turned(x, pos, base):
    """Rows [..., d] rotated at one position in 64 bits."""
    x = x.double()
    if not base:
        return x
    d = x.shape[-1]
    a = torch.tensor([pos * base ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=x.device)
    y = torch.empty_like(x)
    y[..., 0::2] = x[..., 0::2] * a.cos() - x[..., 1::2] * a.sin()
    y[..., 1::2] = x[..., 1::2] * a.cos() + x[..., 0::2] * a.sin()
    return y


def attend(q, k, v):
    """q [hq, d], k and v [hkv, n, d] in 64 bits: outputs [hq, d] and weights [hq, n]."""
    r = q.shape[0] // k.shape[0]
    k, v = k.repeat_interleave(r, 0), v.repeat_interleave(r, 0)
    p = (torch.einsum("hd,hnd->hn", q, k) / math.sqrt(q.shape[-1])).softmax(-1)
    return torch.einsum("hn,hnd->hd", p, v), p


def decode_bound(q, kparts, vparts, p, steps=2048):
    """How far the kernel's fp32 result may be off, from its roundings (kparts, vparts: u, s, m of the visible rows).

    The query enters as fp16 (2^-11 relative; up to 4 heads a KV head as two parts, 2^-21), times log2(e)/sqrt(d) in fp32 and
    rotated in fp32 from fp32 cosines (2^-22 of |q_i| + |q_j|); the weights of codes as fp16 (2^-11).  Products are summed
    in fp32 as codes of at most 15 s and a term m, with at most d/16 + 8 roundings of 2^-23 (the matrix unit's
    adds truncate) a score and `steps` / 32 + 24 for an output's chain of adds.  2^x is off by 2^-22.  A score off by e
    changes weights by 2 e relative at most (numerator and sum)."""
    d, r = q.shape[-1], q.shape[0] // kparts[1].shape[0]
    wide = lambda parts: (15 * parts[1].double().abs() + parts[2].double().abs()).repeat_interleave(r, 0)  # noqa: E731
    qg = q.abs().unflatten(-1, (-1, GROUP)).sum(-1)                                           # [hq, G]
    size = (wide(kparts) * qg[:, None]).sum(-1).amax(-1) / math.sqrt(d)                       # [hq]
    score = size * ((2.0 ** -21 if r <= 4 else 2.0 ** -11) + 2.0 ** -21 + (d / 16 + 8) * 2.0 ** -23) + 2.0 ** -22
    rel = 2 * score[:, None] + 2.0 ** -11 + (steps / 32 + 24) * 2.0 ** -23
    wv = wide(vparts).repeat_interleave(GROUP, -1)
    return rel * torch.einsum("hn,hnd->hd", p, wv)
