"""Calls that are given a stream of their own: what they allocate belongs to that stream."""
import contextlib
import types

import numpy as np
import pytest
import torch

from tests._cache import build_cache, compact64, cu_of, fork64, queries, rope64
from tests._parity import TOL_FP32, assert_close, to64


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


# ---- without a GPU: where each tensor that a call makes is allocated ----
def _calls(kda):
    """(name, call) of every entry point that allocates, on CPU tensors."""
    H, T, N = 2, 5, 1
    bf, f32 = lambda *s: torch.zeros(s, dtype=torch.bfloat16), lambda *s: torch.zeros(s)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    x, cu = bf(T, H, 128), torch.tensor([0, T], dtype=torch.int32)
    rec = (x, x, x, f32(T, H, 128), f32(T, H), cu)
    layer = (x, x, x, f32(3, 4, H, 128), x, f32(H), f32(H, 128), bf(T, H), x, cu)
    front = layer[:8] + (cu,)
    pools = (i32(T), f32(4, H, 128, 128), bf(4, 3, 3, H, 128))
    pool, table, kv = f32(6, 2, H, 16, 128), i32(3, 4), i32(3)
    cache = (pool, table, i32(1), cu, kv)
    q = f32(T, H, 128)
    return {
        "kda_prefill": lambda s: kda.kda_prefill(*rec, stream=s),
        "kda_prefill_with_checkpoints": lambda s: kda.kda_prefill_with_checkpoints(*rec, 32, stream=s),
        "kda_prefill_head_decay": lambda s: kda.kda_prefill_head_decay(*rec, stream=s),
        "kda_decode_step": lambda s: kda.kda_decode_step(x, x, x, f32(T, H, 128), f32(T, H), f32(T, H, 128, 128), stream=s),
        "kda_frontend": lambda s: kda.kda_frontend(*front, stream=s),
        "kda_output_gate": lambda s: kda.kda_output_gate(x, x, stream=s),
        "kda_layer_core": lambda s: kda.kda_layer_core(*layer, stream=s),
        "kda_layer_core_fused": lambda s: kda.kda_layer_core_fused(*layer, stream=s),
        "kda_layer_core_fused_with_checkpoints":
            lambda s: kda.kda_layer_core_fused_with_checkpoints(*layer, 32, stream=s),
        "kda_decode_layer": lambda s: kda.kda_decode_layer(*layer[:9], *pools, stream=s),
        "kda_decode_tokens": lambda s: kda.kda_decode_tokens(*rec, i32(N), f32(4, H, 128, 128), True, stream=s),
        "kda_decode_layer_tokens":
            lambda s: kda.kda_decode_layer_tokens(*layer[:9], cu, i32(N), *pools[1:], True, stream=s),
        "kda_qk_norm_rope": lambda s: kda.kda_qk_norm_rope(q, q, None, None, stream=s),
        "kda_qk_norm_rope_append": lambda s: kda.kda_qk_norm_rope_append(q, q, q, None, None, *cache, stream=s),
        "kda_window_attention": lambda s: kda.kda_window_attention(q, *cache, 8, stream=s),
        "kda_pages_fork": lambda s: kda.kda_pages_fork(pool[None], table, kv, i32(1), i32(1), 16, stream=s),
        "kda_pages_compact": lambda s: kda.kda_pages_compact(pool[None], table, stream=s),
    }


ALLOCATING = ("kda_prefill kda_prefill_with_checkpoints kda_prefill_head_decay kda_decode_step kda_frontend "
              "kda_output_gate kda_layer_core kda_layer_core_fused kda_layer_core_fused_with_checkpoints "
              "kda_decode_layer kda_decode_tokens kda_decode_layer_tokens kda_qk_norm_rope kda_qk_norm_rope_append "
              "kda_window_attention kda_pages_fork kda_pages_compact").split()


@pytest.mark.parametrize("name", ALLOCATING)
def test_what_a_call_allocates_belongs_to_its_stream(kda, name, monkeypatch):
    """With the library's launches and torch's stream switch replaced: every torch.empty of a call that is given a
    stream happens while that stream is the current one."""
    current, made, launched = [None], [], []

    @contextlib.contextmanager
    def switch(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def record(empty):
        def f(*a, **kw):
            made.append(current[0])
            return empty(*a, **kw)
        return f

    real = kda.library()

    class Lib:
        def __getattr__(self, entry):
            if entry.endswith("workspace_size"):
                return getattr(real, entry)
            return lambda *a: launched.append(getattr(a[-1], "value", a[-1])) or 0

    calls = _calls(kda)  # before torch.empty is watched
    assert set(calls) == set(ALLOCATING)
    monkeypatch.setattr(kda, "_lib", Lib())
    monkeypatch.setattr(kda, "_launch", lambda s, dev: s.cuda_stream)  # (it refuses CPU tensors)
    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch, "empty", record(torch.empty))
    monkeypatch.setattr(torch, "empty_like", record(torch.empty_like))
    stream = types.SimpleNamespace(cuda_stream=0x1230)
    calls[name](stream)
    assert launched == [0x1230]
    assert made and all(s is stream for s in made)


# ---- on the GPU ----
@pytest.mark.gpu
def test_page_calls_on_a_side_stream_keep_their_workspace(kda):
    """While the current stream allocates and fills blocks of the workspace's size, a side stream forks and compacts:
    the result is that of the plain form each time."""
    R, M, P, page, layers = 40, 33, 1500, 16, 2
    rng = np.random.RandomState(5)
    table, kv_len = np.full((R, M), -1, np.int32), np.zeros(R, np.int32)
    names = list(rng.permutation(P))
    for r in range(R // 2):
        kv_len[r] = n = int(rng.randint(1, M * page))
        for i in range(-(-n // page)):
            table[r, i] = names.pop()
    parent, child = np.arange(10), np.arange(20, 30)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    start = torch.randint(-2 ** 31, 2 ** 31 - 1, (layers, P, 2048), dtype=torch.int32, device="cuda")
    t, n, moves = fork64(table, kv_len, P, page, parent, child)
    want = start.clone()
    for s, d in moves:
        want[:, d] = want[:, s].clone()
    t, live, moves = compact64(t, P)
    src, dst = i32([s for s, _ in moves]).long(), i32([d for _, d in moves]).long()
    want[:, dst] = want[:, src]
    side, need = torch.cuda.Stream(), kda.kda_pages_workspace_size(P, R)
    p, c = i32(parent), i32(child)
    busy = torch.randn((4096, 4096), device="cuda")
    for _ in range(50):
        pool, dt, dn = start.clone(), i32(table), i32(kv_len)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mm(busy, busy)  # the page kernels come after this
        kda.kda_pages_fork(pool, dt, dn, p, c, page, stream=side)
        blocks = [torch.full((need,), 1, dtype=torch.uint8, device="cuda") for _ in range(4)]
        _, count = kda.kda_pages_compact(pool, dt, stream=side)
        blocks += [torch.full((need,), 1, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
        assert np.array_equal(dt.cpu().numpy(), t) and np.array_equal(dn.cpu().numpy(), n) and count.item() == live
        assert torch.equal(pool, want)
    assert kda.kda_get_device_status()[0] == 0


@pytest.mark.gpu
def test_append_and_rotation_on_a_side_stream(kda):
    """Outputs that a call on a side stream makes, dropped and made again while the current stream fills blocks of
    their size."""
    new, page = [3, 40], 16
    c = build_cache([n + 9 for n in new], page, 2, torch.float32, seed=7)
    x = queries(sum(new), 8, torch.float32, 7)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    table = kda.rope_table(100)
    pos = torch.arange(sum(new), dtype=torch.int32, device="cuda")
    ref_q, ref_k = (rope64(t, None, table, pos, 128, False, True) for t in (q, k))
    side, cu, clean = torch.cuda.Stream(), cu_of(new), c["pool"].clone()
    busy = torch.randn((4096, 4096), device="cuda")
    rows, slot = c["table"].tolist(), c["slot"].tolist()
    for _ in range(10):
        c["pool"].copy_(clean)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mm(busy, busy)
        kda.kda_qk_norm_rope(q, k, table, pos, stream=side)  # dropped at once
        blocks = [torch.full((sum(new), h, 128), 3.0, device="cuda") for h in (4, 2)]
        out = kda.kda_qk_norm_rope_append(q, k, v, table, pos, c["pool"], c["table"], c["slot"], cu, c["kv_len"],
                                          stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(bool((b == 3.0).all()) for b in blocks)
        assert_close(to64(out), ref_q, TOL_FP32, "q")
        t = 0
        for b, n in enumerate(new):
            for i in range(n):
                at = c["pool"][rows[slot[b]][(9 + i) // page], :, :, (9 + i) % page]
                assert_close(to64(at[0]), ref_k[t], TOL_FP32, "k")
                assert torch.equal(at[1], v[t])
                t += 1
    assert kda.kda_get_device_status()[0] == 0
