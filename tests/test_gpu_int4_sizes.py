"""Decode over 4-bit rows whose values and scores change in size along a split, against 64 bits."""
import pytest
import torch

import _int4 as i4
from _int4_bounds import decode_bound
from test_gpu_int4 import Model, make, rows

pytestmark = pytest.mark.gpu


def check(m, q, out, requests, **kw):
    """Requests of a Model without a window or rotary positions: outputs in fp32 within the bound of their roundings."""
    worst = 0.0
    for b in requests:
        kp, vp = i4.quantise(m.k[b]), i4.quantise(m.v[b])
        ref, w = i4.attend(q[b].double(), i4.values(*kp), i4.values(*vp))
        bound, err = decode_bound(q[b].double(), kp, vp, w, **kw), (out[b].double() - ref).abs()
        assert (err <= bound).all(), "request %d: %d of %d past the bound, %.3g times" % (
            b, (~(err <= bound)).sum(), err.numel(), (err / bound).nan_to_num(1e30).max())
        worst = max(worst, (err / bound).max().item())
    return worst


def scores_rise(hq, hkv, d, B, n, early):
    """Keys that answer the queries of their KV head with scores of about -50, and from `early` on ordinary ones."""
    g = torch.Generator().manual_seed(5)
    sign = torch.randint(0, 2, (B, hkv, 1, d), generator=g).float() * 2 - 1
    q = torch.randn((B, hkv, hq // hkv, d), generator=g).abs() * sign
    k = torch.randn((B, hkv, n, d), generator=g)
    k[:, :, :early] = -6 * sign + 0.5 * k[:, :, :early]
    return q.reshape(B, hq, d).bfloat16().cuda(), k.bfloat16().cuda()


# (32 requests of 16 KV heads fill the SMs, so that splits are several steps of 128 keys long)
SHAPES = [(16, 128), (64, 128), (128, 128), (48, 64)]


@pytest.mark.parametrize("hq,d", SHAPES)
@pytest.mark.parametrize("fall", [24, 28, 32, 60, 200])
def test_values_that_fall_while_scores_rise(hq, d, fall):
    # early values 2^fall as large as the late ones, of weights below 2^-70: late weights keep their bits
    B, hkv, n = 32, 16, 512
    c = make(batch=B, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, capacity=n)
    m = Model(c)
    q, k = scores_rise(hq, hkv, d, B, n, 128)
    v = rows(2, B, hkv, n, d, False)
    v[:, :, :128] *= 2.0 ** (fall // 2)
    v[:, :, 128:] *= 2.0 ** -(fall - fall // 2)
    if fall > 100:                                   # (what weighs nothing at all)
        k[:, :, :128] *= 4
    c.append_rows(k, v)
    m.append(k, v, (n,) * B)
    check(m, q, c.decode(q), (0, 7, B - 1))


@pytest.mark.parametrize("hq,d", SHAPES)
def test_values_that_fall_step_by_step(hq, d):
    # every step of 128 keys 2^25 smaller than the one before, and of scores 30 higher; the last ones rise again
    B, hkv, n = 32, 16, 640
    c = make(batch=B, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, capacity=n)
    m = Model(c)
    q, k = scores_rise(hq, hkv, d, B, n, 0)
    sign = q.float().view(B, hkv, hq // hkv, d)[:, :, :1].sign()
    v = rows(2, B, hkv, n, d, False)
    for step, (size, score) in enumerate([(2.0 ** 50, -7), (2.0 ** 25, -4), (1.0, -1), (2.0 ** -25, 2), (2.0 ** -10, 2)]):
        at = slice(128 * step, 128 * step + 128)
        k[:, :, at] = (0.5 * k[:, :, at].float() + score * sign).bfloat16()
        v[:, :, at] *= size
    c.append_rows(k, v)
    m.append(k, v, (n,) * B)
    check(m, q, c.decode(q), (0, 9, B - 1))


@pytest.mark.parametrize("hq,d", SHAPES)
@pytest.mark.parametrize("size", [-108, -115, -120])
def test_tiny_values_keep_their_bits(hq, d, size):
    # (scales of 2^-122 at the last size, normal numbers of bf16)
    B, hkv, n = 2, 16, 300
    c = make(batch=B, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, capacity=304)
    m = Model(c)
    q, k = scores_rise(hq, hkv, d, B, n, 100)
    v = rows(2, B, hkv, n, d, False) * 2.0 ** size
    c.append_rows(k, v)
    m.append(k, v, (n,) * B)
    check(m, q, c.decode(q), range(B))


@pytest.mark.parametrize("hq,d", SHAPES)
@pytest.mark.parametrize("size", [-124, -100, 100, 118, 122, 127])
def test_queries_of_all_sizes(hq, d, size):
    # keys as small as the queries are large, or as large as they are small; a head's largest dim up to the end of bf16's range
    B, hkv, n = 2, 16, 300
    c = make(batch=B, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, capacity=304)
    m = Model(c)
    g = torch.Generator().manual_seed(7)
    q = (torch.rand((B, hq, d), generator=g) * 0.99).bfloat16().cuda() * 2.0 ** size
    k, v = rows(1, B, hkv, n, d, False) * 2.0 ** min(-size, 120), rows(2, B, hkv, n, d, False)
    k[:, :, ::3] *= 4
    c.append_rows(k, v)
    m.append(k, v, (n,) * B)
    check(m, q, c.decode(q), range(B))
