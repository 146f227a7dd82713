"""Groups whose scale is a subnormal bf16 number, or none: off by the group's range at most (CPU only)."""
import torch

import _int4 as i4


def test_tiny_ranges():
    g = torch.Generator().manual_seed(1)
    x = torch.rand((4000, 64), generator=g) * 2.0 ** (-134 + 16 * torch.rand((4000, 1), generator=g))
    x[0, :32] = torch.linspace(0, 1.49 * 15 * 2.0 ** -133, 32)               # a scale that loses a third of its size
    x = x.bfloat16()
    u, s, m = i4.quantise(x)
    group = x.double().unflatten(-1, (-1, 32))
    err = (i4.values(u, s, m) - x.double()).abs().unflatten(-1, (-1, 32)).amax(-1)
    spread = group.amax(-1) - group.amin(-1)
    normal = s.double() >= 2.0 ** -126
    assert (err <= torch.where(normal, s.double() / 2 * (1 + 2.0 ** -20), spread)).all()
    assert normal.any() and (s == 0).any() and (err[0, 0] > 3 * s[0, 0].double())
