"""The decode of fp32 caches and other head sizes, with its rows copied to shared memory and without: the same answers, and
times in proportion to the bytes."""
import pytest
import torch

from kv_cache_decode_ring_gb300 import kvc

pytestmark = pytest.mark.gpu


def filled(dtype, B, hq, hkv, d, n, seed=0):
    c = kvc.Cache(kvc.make_config(dtype=dtype, batch=B, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, capacity=n))
    g = torch.Generator("cuda").manual_seed(seed)
    one = lambda *s: torch.randn(s, generator=g, device="cuda").to(c.torch_dtype)  # noqa: E731
    k, v, q = one(1, hkv, n, d), one(1, hkv, n, d), one(1, hq, d)
    c.append_rows(k.expand(B, -1, -1, -1).contiguous(), v.expand(B, -1, -1, -1).contiguous())
    return c, q.expand(B, -1, -1).contiguous(), (k, v, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 80), (4, 4, 256), (8, 2, 96), (12, 1, 160), (3, 3, 10), (5, 1, 256)])
def test_the_same_answers_in_small_and_large_batches(dtype, hq, hkv, d):
    n = 333
    small, q1, (k, v, q) = filled(dtype, 1, hq, hkv, d, n)
    large, q2, _ = filled(dtype, 50, hq, hkv, d, n)
    a, b = small.decode(q1), large.decode(q2)
    assert torch.equal(a.expand_as(b), b)
    kk, vv = (x[0].double().repeat_interleave(hq // hkv, 0) for x in (k, v))
    w = (torch.einsum("hd,hnd->hn", q[0].double(), kk) / d ** 0.5).softmax(-1)
    ref = torch.einsum("hn,hnd->hd", w, vv)
    # bf16 outputs are rounded once (2^-9 relative).  fp32: scores as sums of d products, weights that change twice as much
    # (numerator and sum), n additions
    score = (torch.einsum("hd,hnd->hn", q[0].double().abs(), kk.abs()) / d ** 0.5).amax(-1) * (d + 4) * 2.0 ** -24 + 2.0 ** -21
    bound = (2 * score[:, None] + (n + 8) * 2.0 ** -24) * torch.einsum("hn,hnd->hd", w, vv.abs())
    bound = bound + (ref.abs() * 2.0 ** -8 if dtype == "bf16" else 0.0)
    assert ((a[0].double() - ref).abs() <= bound).all()


def time_of(dtype, B, hq, hkv, d, n):
    c, q, _ = filled(dtype, B, hq, hkv, d, n)
    out, best = c.decode(q), 1e9
    for _ in range(12):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        c.decode(q, out)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    c.close()
    return best


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 80), (8, 8, 256), (32, 8, 256), (16, 8, 160)])
def test_half_the_bytes_take_no_longer(hq, hkv, d):
    # (1.8 to 2.9 times as long where bf16 rows were converted as they came)
    assert time_of("bf16", 32, hq, hkv, d, 2048) <= 1.3 * time_of("f32", 32, hq, hkv, d, 2048)


def test_twice_the_bytes_take_little_more_than_twice_as_long():
    # (4.2 times where rows of 256 dims left one CTA on an SM)
    assert time_of("f32", 32, 8, 8, 256, 2048) <= 3.5 * time_of("f32", 32, 8, 8, 128, 2048)
