"""Trims that give up few pages, more than a launch carries, and more than are listed: the device's table follows."""
import numpy as np
import pytest
import torch

from kv_cache_decode_ring_gb300 import kvc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("capacity", [2048, 65536])
@pytest.mark.parametrize("cuts", [[2000] * 3 + [2047] * 37, [1600] * 40, [0, 2048] * 20, [1024] * 40, [0] * 40, [7] * 40])
def test_tables_and_answers_after_a_trim(capacity, cuts):
    B, n, d = 40, 2048, 64
    c = kvc.Cache(kvc.make_config(batch=B, n_q_heads=1, n_kv_heads=1, head_dim=d, capacity=capacity, page_pool=B * n // 16 + 100, out_dtype="f32"))
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn((B, 1, n, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    c.append_rows(k, v)
    c.trim(cuts)
    held = [(x + 15) // 16 for x in cuts]
    table = c.export(kvc.KVC_EXPORT_PAGE_TABLE)
    assert [(row >= 0).sum() for row in table] == held and all((row[:m] >= 0).all() for row, m in zip(table, held))
    assert c.page_counts()[0] == B * n // 16 + 100 - sum(held)
    used = table[table >= 0]
    assert len(np.unique(used)) == len(used)
    k1, v1 = (torch.randn((B, 1, 40, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    counts = [min(40, 2048 + 20 - x) for x in cuts] if capacity > n else [min(40, n - x) for x in cuts]
    c.append_rows(k1, v1, counts=counts)
    lens = [x + m for x, m in zip(cuts, counts)]
    if min(lens) > 0:
        q = torch.randn((B, 1, d), generator=g, device="cuda").bfloat16()
        out = c.decode(q)
        for b in (0, 1, 17, B - 1):
            kk, vv = (torch.cat((x[b, 0, :cuts[b]], y[b, 0, :counts[b]])).double() for x, y in ((k, k1), (v, v1)))
            w = (kk @ q[b, 0].double() / d ** 0.5).softmax(0)
            # two bf16 parts of query and weights, fp32 sums: far below the rows' own size
            assert ((out[b, 0].double() - w @ vv).abs() <= 2e-3 * (w @ vv.abs())).all()
    assert c.device_status() == 0


def test_captured_trims_give_up_the_pages_of_their_capture():
    # 1280 pages, more than a launch carries: what the host's table becomes later does not reach a replay
    B, n, d = 40, 2048, 64
    c = kvc.Cache(kvc.make_config(batch=B, n_q_heads=1, n_kv_heads=1, head_dim=d, capacity=n, page_pool=B * n // 16))
    k = torch.randn((B, 1, n, d), device="cuda").bfloat16()
    c.append_rows(k, k)
    torch.cuda.synchronize()
    before = c.export(kvc.KVC_EXPORT_PAGE_TABLE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.trim([1536] * B)
    assert np.array_equal(c.export(kvc.KVC_EXPORT_PAGE_TABLE), before)             # nothing has run yet
    graph.replay()
    torch.cuda.synchronize()
    after = c.export(kvc.KVC_EXPORT_PAGE_TABLE)
    assert np.array_equal(after[:, :96], before[:, :96]) and (after[:, 96:] == -1).all()
    c.append_rows(k[:, :, :512].contiguous(), k[:, :, :512].contiguous())
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(c.export(kvc.KVC_EXPORT_PAGE_TABLE), after)
