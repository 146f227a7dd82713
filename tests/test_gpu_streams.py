"""Outputs that a call makes for itself are memory of the stream that writes them: memory of the caller's
current stream may still be read there by work that was enqueued before its last owner let go of it."""
import pytest
import torch

from kv_cache_decode_ring_gb300 import kvc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_decode_ring_gb300 import build
    build.build()


def calls(B=64, n=64, Hq=64, Hkv=8, d=128):
    """(what, call taking a stream, shape and type of its output); outputs of a few MB each."""
    bf16 = torch.bfloat16
    cache = kvc.Cache(kvc.make_config("bf16", "contiguous", None, B, Hq, Hkv, d, 512, max_chunk=n))
    q, k = (torch.randn(B, n, h, d, device="cuda").to(bf16) for h in (Hq, Hkv))
    one = [x[:, 0].contiguous() for x in (q, k)]
    cache.append(one[1], one[1])
    pos = torch.zeros(1, B * n, dtype=torch.int32, device="cuda")
    gate = kvc.Cache(kvc.make_config("bf16", "contiguous", "int8", 8, 64, 64, 128, 8192))
    ct = torch.rand(8, 64, 8192, device="cuda")
    return [
        ("decode", lambda s: cache.decode(one[0], stream=s), (B, Hq, d), bf16),
        ("chunk", lambda s: cache.chunk(q, k, k, stream=s), (B, n, Hq, d), bf16),
        ("prompt", lambda s: cache.prompt(q.view(-1, Hq, d), k.view(-1, Hkv, d), k.view(-1, Hkv, d), [n] * B, stream=s),
         (B * n, Hq, d), bf16),
        ("rotary", lambda s: kvc.kvc_rope_axes(q.view(-1, Hq, d), pos, [d // 2], stream=s), (B * n, Hq, d), bf16),
        ("risk", lambda s: gate.block_risk(ct, stream=s), (8, 64, 512), torch.float32),
    ]


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_outputs_belong_to_the_stream_that_writes_them(raw):
    s = torch.cuda.Stream()
    for what, call, shape, dtype in calls():
        want = call(None)
        torch.cuda.synchronize()
        # a block that the current stream has just given up: the next allocation there takes it
        held = torch.empty(shape, dtype=dtype, device="cuda")
        at = held.data_ptr()
        del held
        again = torch.empty(shape, dtype=dtype, device="cuda")
        assert again.data_ptr() == at
        del again
        out = call(s.cuda_stream if raw else s)
        torch.cuda.synchronize()
        assert out.shape == want.shape and out.dtype == want.dtype
        assert out.data_ptr() != at, what
        if what in ("rotary", "risk"):
            assert torch.equal(out, want)


def test_the_current_stream_by_its_handle():
    # the default stream's handle and the current stream's are no other streams
    x = torch.randn(4096, 64, 128, device="cuda")
    pos = torch.zeros(1, 4096, dtype=torch.int32, device="cuda")
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            want = kvc.kvc_rope_axes(x, pos, [64])
            for handle in (s, s.cuda_stream):
                held = torch.empty_like(x)
                at = held.data_ptr()
                del held
                out = kvc.kvc_rope_axes(x, pos, [64], stream=handle)
                assert out.data_ptr() == at and torch.equal(out, want)
                del out
        torch.cuda.synchronize()


def test_the_state_belongs_to_the_stream_that_clears_it():
    cfg = kvc.make_config("bf16", "contiguous", None, 8, 8, 8, 128, 512)
    n = kvc.kvc_state_bytes(cfg)
    held = torch.empty(n, dtype=torch.uint8, device="cuda")
    at = held.data_ptr()
    del held
    assert kvc.Cache(cfg, stream=torch.cuda.Stream()).state.data_ptr() != at


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_outputs_outlive_the_current_streams_work(raw):
    # an output let go of while the current stream still has to read it is not handed to the next call
    s = torch.cuda.Stream()
    on = s.cuda_stream if raw else s
    x = torch.randn(4096, 64, 128, device="cuda")
    pos, zero = (torch.full((1, 4096), p, dtype=torch.int32, device="cuda") for p in (1, 0))
    want, copy = kvc.kvc_rope_axes(x, pos, [64]), torch.empty_like(x)
    torch.cuda.synchronize()
    out = kvc.kvc_rope_axes(x, pos, [64], stream=on)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(200_000_000)
    copy.copy_(out)
    at = out.data_ptr()
    del out
    again = kvc.kvc_rope_axes(x, zero, [64], stream=on)
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and torch.equal(again, x)
