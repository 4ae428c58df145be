"""The cache calls in CUDA graphs, as a decode loop uses them, and their results from call to call."""
import pytest
import torch

from tests._cache import build_cache, cu_of, queries

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new,old,window", [([1, 1], [70, 2000], 100), ([3, 2], [40, 3000], 2 ** 31 - 1),
                                            ([90, 40], [300, 0], 64), ([40], [3000], 2 ** 31 - 1)])
def test_a_step_replayed_from_a_graph(kda, new, old, window, dtype):
    """Append, attention, trim, fork and compaction captured once and replayed over other inputs in the same buffers:
    bit for bit the calls made one by one.  (One token, a few over CTA clusters, a prefill, a short step behind a
    long row; the fp32 kernel over clusters.)"""
    page, heads, group, total = 32, 2, 4, sum(new)
    c = build_cache([a + b for a, b in zip(new, old)], page, heads, dtype, seed=61, spare_pages=8)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    free = [r for r in range(c["table"].shape[0]) if r not in c["slot"].tolist()]
    rope, cu = kda.rope_table(4096, 64), cu_of(new)
    pos = torch.cat([torch.arange(o, o + n) for n, o in zip(new, old)]).to("cuda", torch.int32)
    x = queries(total, heads * group + 2 * heads, dtype, 61)
    parent, child, rows = c["slot"][:1].contiguous(), i32(free[:1]), c["slot"].contiguous()
    live = i32([0])

    def step(x, pool, table, kv_len):
        q, k, v = x.split([heads * group, heads, heads], dim=1)
        qn = kda.kda_qk_norm_rope_append(q, k, v, rope, pos, pool, table, c["slot"], cu, kv_len)
        o = kda.kda_window_attention(qn, pool, table, c["slot"], cu, kv_len, window, 4, max_tokens=max(new))
        kda.kda_pages_release(table, kv_len, rows, page, window, 4)
        kda.kda_pages_fork(pool[None], table, kv_len, parent, child, page)
        kda.kda_pages_compact(pool[None], table, num_live=live)
        return o

    start = c["pool"], c["table"], c["kv_len"]
    buffers = [x.clone()] + [t.clone() for t in start]
    step(*[b.clone() for b in buffers])  # the library is loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(*buffers)
    for seed in (1, 2):
        other = queries(total, x.shape[1], dtype, 61 + seed)
        want_buffers = [other] + [t.clone() for t in start]
        want = step(*want_buffers)
        for b, t in zip(buffers, [other, *start]):
            b.copy_(t)
        o.fill_(-7.0)
        graph.replay()
        assert torch.equal(o, want)
        assert all(torch.equal(b, t) for b, t in zip(buffers, want_buffers))
    assert kda.kda_get_device_status()[0] == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new,old,group", [([1], [3000], 8), ([1, 1, 1], [9000, 10, 4000], 12), ([4, 2], [5000, 700], 8),
                                           ([16], [6000], 4), ([40], [6000], 4), ([300, 7], [900, 4000], 2)])
def test_calls_over_clusters_repeat_bit_for_bit(kda, new, old, group, dtype):
    """Rows whose keys are shared by several CTAs: the order of the joins goes by the sizes alone."""
    c = build_cache([a + b for a, b in zip(new, old)], 64, 1, dtype, seed=67)
    q, cu = queries(sum(new), group, dtype, 67), cu_of(new)
    ask = lambda: kda.kda_window_attention(q, c["pool"], c["table"], c["slot"], cu, c["kv_len"], None, 0,
                                           max_tokens=max(new))
    want = ask()
    busy = torch.randn((2048, 2048), device="cuda")
    for i in range(20):
        if i % 2:
            torch.mm(busy, busy)  # the GPU in another state
        assert torch.equal(ask(), want)
    assert kda.kda_get_device_status()[0] == 0
