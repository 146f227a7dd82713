"""The 4-bit row format and what a configuration of the tier may be (CPU only)."""
import math

import pytest
import torch

import _int4 as i4
from kv_cache_decode_ring_gb300 import build as kbuild
from kv_cache_decode_ring_gb300 import kvc


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


@pytest.mark.parametrize("d", [64, 128])
def test_every_dim_has_one_nibble(d):
    for value in (False, True):
        assert sorted(i4.order(d, value)) == list(range(d))


def test_half_a_step_at_most():
    # s is off by 2^-8 relative at most, so the largest quotient stays below 15.06 and no code is clamped by more than
    # 0.06 of a step: every value is within half a step of what it is held as (plus the quotient's own 2^-24)
    torch.manual_seed(3)
    x = (torch.randn(400, 128) * torch.exp(2 * torch.randn(400, 1)) + torch.randn(400, 1)).bfloat16()
    u, s, m = i4.quantise(x)
    err = (i4.values(u, s, m) - x.double()).abs().unflatten(-1, (-1, 32))
    assert (err <= s.double()[..., None] * (0.5 + 15 * 2.0 ** -23)).all()


def test_equal_values_and_values_that_are_not_finite():
    x = torch.full((3, 64), 1.5).bfloat16()
    x[1, 5], x[2, 40] = math.inf, math.nan
    y = i4.held(x)
    assert (y[0] == 1.5).all()
    assert y[1, :32].isnan().all() and (y[1, 32:] == 1.5).all()
    assert y[2, 32:].isnan().all() and (y[2, :32] == 1.5).all()


def config(**kw):
    return kvc.make_config(**dict(dict(kv_quant="int4", batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, capacity=64), **kw))


def test_rows_take_five_bits_an_element():
    # K and V rows of 80 bytes against 256: 2 x 176 a key and KV head.  The splits' workspace takes back 520 bytes for each of
    # 4 query heads every 128 keys, 16.3 a key (the other arrays are the same): 335 are left
    small = kvc.kvc_state_bytes(config(capacity=1 << 16))
    large = kvc.kvc_state_bytes(config(capacity=1 << 16, kv_quant=None))
    assert large - small > 2 * 2 * (1 << 16) * 335


@pytest.mark.parametrize("bad", [dict(dtype="f32"), dict(head_dim=96), dict(head_dim=256), dict(capacity=72), dict(int8_split=1024),
                                 dict(int8_exact_blocks=4), dict(layout="ring", capacity=40, max_position=64),
                                 dict(layout="ring", window=32), dict(page_pool=-1), dict(store_slots=-1)])
def test_refused_configurations(bad):
    with pytest.raises(kvc.KvcError) as e:
        kvc.kvc_state_bytes(config(**bad))
    assert e.value.code == kvc.KVC_ERR_ARG


@pytest.mark.parametrize("good", [dict(), dict(head_dim=64), dict(n_q_heads=24), dict(window=33), dict(layout="ring"), dict(page_pool=5),
                                  dict(store_slots=2), dict(out_dtype="f32"), dict(max_chunk=16), dict(layout="ring", page_pool=9)])
def test_accepted_configurations(good):
    assert kvc.kvc_state_bytes(config(**good)) > 0


@pytest.mark.parametrize("bad", [dict(sinks=4), dict(sinks=-1, window=16), dict(sinks=4, layout="ring"),
                                 dict(sinks=4, window=16, kv_quant="int8"), dict(sinks=4, window=16, kv_quant="int8-dither")])
def test_refused_sinks(bad):
    with pytest.raises(kvc.KvcError) as e:
        kvc.kvc_state_bytes(config(**bad))
    assert e.value.code == kvc.KVC_ERR_ARG


@pytest.mark.parametrize("quant", [None, "int4"])
def test_accepted_sinks(quant):
    for sinks in (1, 48, 1 << 30):
        assert kvc.kvc_state_bytes(config(kv_quant=quant, window=16, sinks=sinks)) > 0
