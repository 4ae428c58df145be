"""Norm + rotation of q and k, and the append to the cache, against a 64-bit plain implementation.

fp32 arithmetic rounded once: max-abs over rms 1e-5 (a 128-term sum of squares, a square root and
four products leave about 1e-6), plus half an ulp of the value where the output is bf16."""
import numpy as np
import pytest
import torch

from tests._cache import build_cache, cu_of, rope64
from tests._parity import TOL_FP32, assert_close, to64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def inputs(T, Hq, Hkv, dtype, seed, positions=500, weights=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn((T, Hq + 2 * Hkv, 128), generator=g, device="cuda", dtype=dtype)
    pos = torch.randint(0, positions, (T,), generator=g, device="cuda", dtype=torch.int32)
    w = [1 + 0.3 * torch.randn(128, generator=g, device="cuda") if weights else None for _ in range(2)]
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, w


def near(got, ref, what):
    assert_close(to64(got), ref, TOL_FP32, what, got.dtype == BF16)


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (3, 5, 2), (257, 12, 1), (64, 96, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 48, 64, 96, 128])
def test_rotation_and_norm(kda, T, Hq, Hkv, interleaved, rotary):
    for din, dout, norm, weights in ((BF16, BF16, True, True), (FP32, FP32, True, False),
                                     (FP32, BF16, False, False), (BF16, FP32, True, True)):
        q, k, _, pos, w = inputs(T, Hq, Hkv, din, T + rotary, weights=weights)
        table = kda.rope_table(500, rotary) if rotary else None
        qo, ko = kda.kda_qk_norm_rope(q, k, table, pos, w[0], w[1], 1e-6, norm=norm, interleaved=interleaved,
                                      out_dtype=dout)
        assert qo.dtype == dout and kda.kda_get_device_status()[0] == 0
        t64 = table if rotary else torch.zeros((500, 0, 2))
        near(qo, rope64(q, w[0], t64, pos, rotary, interleaved, norm), "q")
        near(ko, rope64(k, w[1], t64, pos, rotary, interleaved, norm), "k")


def test_in_place_and_strides(kda):
    """A dense q may be its own output; a padded token stride is read as such."""
    q, k, _, pos, w = inputs(37, 4, 2, FP32, 5)
    table = kda.rope_table(500)
    want = kda.kda_qk_norm_rope(q, k, table, pos, w[0], w[1])
    qd, kd = q.contiguous(), k.contiguous()
    got = kda.kda_qk_norm_rope(qd, kd, table, pos, w[0], w[1], q_out=qd, k_out=kd)
    assert got[0] is qd and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_norm_of_zero_and_large_rows(kda):
    """mean(x^2) of zeros is eps alone; 1e18 squared is within fp32."""
    q = torch.zeros((2, 1, 128), device="cuda")
    q[1] = 1e18
    qo, _ = kda.kda_qk_norm_rope(q, q.clone(), None, None, norm=True, eps=1e-6)
    assert bool((qo[0] == 0).all()) and bool(((qo[1] - 1).abs() < 1e-6).all())


def test_rope_table_at_far_positions(kda):
    """2^20 positions: the angles are formed in 64 bits, so that the last ones are as good as the first."""
    t = kda.rope_table(1 << 20, 64, base=500000.0, magnitude=1.25)
    i = np.arange(32)
    ang = ((1 << 20) - 1) * 500000.0 ** (-2 * i / 64)
    assert np.abs(to64(t[-1]) - 1.25 * np.stack([np.cos(ang), np.sin(ang)], -1)).max() < 2e-7


def test_rope_table_with_own_frequencies(kda):
    inv = torch.linspace(1.0, 0.01, 8, dtype=torch.float64, device="cuda")
    t = kda.rope_table(50, 16, inv_freq=inv)
    ang = np.arange(50)[:, None] * inv.cpu().numpy()
    assert np.abs(to64(t)[..., 0] - np.cos(ang)).max() < 1e-7


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("din,dout", [(BF16, BF16), (FP32, FP32), (FP32, BF16)])
def test_append_writes_the_pages(kda, page, din, dout):
    new, old = [1, 40, 0, 3, 130], [0, 100, 7, 2 * page - 1, page]
    c = build_cache([a + b for a, b in zip(new, old)], page, 2, dout, seed=page)
    q, k, v, pos, w = inputs(sum(new), 6, 2, din, page)
    table = kda.rope_table(500, 64)
    before = c["pool"].clone()
    qo = kda.kda_qk_norm_rope_append(q, k, v, table, pos, c["pool"], c["table"], c["slot"], cu_of(new),
                                     c["kv_len"], w[0], w[1])
    assert kda.kda_get_device_status()[0] == 0
    near(qo, rope64(q, w[0], table, pos, 64, False, True), "q")
    k64 = rope64(k, w[1], table, pos, 64, False, True)
    rows, slot, t = c["table"].tolist(), c["slot"].tolist(), 0
    written = torch.zeros(before.shape[:1] + before.shape[3:4], dtype=torch.bool, device="cuda")
    for b, n in enumerate(new):
        for i in range(n):
            j = old[b] + i
            where = rows[slot[b]][j // page], j % page
            written[where] = True
            near(c["pool"][where[0], 0, :, where[1]], k64[t], "k in its page")
            assert torch.equal(c["pool"][where[0], 1, :, where[1]], v[t].to(dout))
            t += 1
    untouched = ~written[:, None, None, :, None].expand_as(before)
    assert torch.equal(c["pool"][untouched], before[untouched])


def test_append_refuses_tokens_without_a_place(kda):
    """A missing page, a row shorter than the step, a bad slot: those k and v are not written."""
    for what in ("page", "short", "slot", "kv_len"):
        c = build_cache([20, 20], 16, 1, FP32, seed=3)
        q, k, v, pos, w = inputs(6, 2, 1, FP32, 3)
        slot = c["slot"].tolist()
        if what == "page":
            c["table"][slot[1], 1] = c["pool"].shape[0]
        elif what == "short":
            c["kv_len"][slot[1]] = 2
        elif what == "slot":
            c["slot"][1] = -1
        else:
            c["kv_len"][slot[1]] = -4
        before = c["pool"].clone()
        qo = kda.kda_qk_norm_rope_append(q, k, v, kda.rope_table(500), pos, c["pool"], c["table"], c["slot"],
                                         cu_of([3, 3]), c["kv_len"], w[0], w[1])
        code, detail = kda.kda_get_device_status()
        assert code == 6 and detail in (3, 4, 5), what
        near(qo, rope64(q, w[0], kda.rope_table(500), pos, 128, False, True), "q")
        changed = (c["pool"] != before).flatten(1).any(1).nonzero().view(-1).tolist()
        mine = {int(c["table"][slot[0], 1])}
        assert set(changed) <= mine | ({int(c["table"][slot[1], 0])} if what == "short" else set()), what


def test_position_out_of_the_table_is_refused(kda):
    q, k, _, pos, w = inputs(4, 2, 1, FP32, 7)
    pos[2] = 500
    out = torch.full((4, 2, 128), -7.0, device="cuda"), torch.full((4, 1, 128), -7.0, device="cuda")
    kda.kda_qk_norm_rope(q, k, kda.rope_table(500), pos, w[0], w[1], q_out=out[0], k_out=out[1])
    assert kda.kda_get_device_status() == (6, 2)
    assert bool((out[0][2] == -7).all()) and bool((out[1][2] == -7).all())
    assert not bool((out[0][[0, 1, 3]] == -7).any())


def test_no_tokens(kda):
    q = torch.empty((0, 2, 128), device="cuda")
    qo, ko = kda.kda_qk_norm_rope(q, q, None, None)
    assert qo.shape == ko.shape == (0, 2, 128)


def test_norm_rope_then_attention(kda):
    """The two as a layer uses them: a prefill of 90 tokens, then single tokens, equals attention over
    keys normed and rotated in 64 bits."""
    from tests._cache import attention64
    page, Hq, Hkv, total, first = 16, 4, 2, 96, 90
    c = build_cache([total], page, Hkv, FP32, seed=51)
    q, k, v, _, w = inputs(total, Hq, Hkv, FP32, 51)
    table, row = kda.rope_table(200, 64), c["slot"].item()
    pos = torch.arange(total, dtype=torch.int32, device="cuda")
    outs, done = [], 0
    for n in [first] + [1] * (total - first):
        c["kv_len"][row] = done + n
        t = slice(done, done + n)
        qn = kda.kda_qk_norm_rope_append(q[t], k[t], v[t], table, pos[t].contiguous(), c["pool"], c["table"],
                                         c["slot"], cu_of([n]), c["kv_len"], w[0], w[1])
        outs.append(kda.kda_window_attention(qn, c["pool"], c["table"], c["slot"], cu_of([n]), c["kv_len"], 30, 4,
                                             max_tokens=n))
        done += n
    assert kda.kda_get_device_status()[0] == 0
    k64, q64 = rope64(k, w[1], table, pos, 64, False, True), rope64(q, w[0], table, pos, 64, False, True)
    exact = torch.zeros((c["pool"].shape[0], 2, Hkv, page, 128), dtype=torch.float64, device="cuda")
    for j in range(total):
        p = int(c["table"][row, j // page])
        exact[p, 0, :, j % page] = torch.from_numpy(k64[j]).cuda()
        exact[p, 1, :, j % page] = v[j].double()
    ref, _ = attention64(torch.from_numpy(q64), {**c, "pool": exact}, [total], 30, 4)
    assert_close(to64(torch.cat(outs)), ref, TOL_FP32, "o")
