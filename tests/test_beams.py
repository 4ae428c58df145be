"""Beam selection and reordering against plain implementations.

Selection compares totals in 64 bits, formed from sums of fp32 exponentials.  Each exponential of a term
d below the maximum is off by at most about (d + 2) 2^-23 of itself, and the terms of a row, weighted with
themselves, have d e^-d <= 1: the log-sum-exp is off by less than 2^-20 in all, the fp32 score by that and its
rounding.  Orders are compared where the totals differ by more; equal ones have to be equal by
construction (the same logits and scores), and then go by beam, logit and token.
"""
import numpy as np
import pytest
import torch

from tests._branches import beam_reorder64, beam_slots64, select64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def make(B, K, V, dtype, seed, pad=0, spread=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn((B, K, V + pad), generator=g, device="cuda") * spread).to(dtype)[..., :V]
    return x, torch.empty((B, K), device="cuda").uniform_(-9, 0, generator=g)


def check(kda, logits, scores, choices, ended=None, end_token=-1, **kw):
    got = kda.kda_beam_select(logits, scores, choices, ended=ended, end_token=end_token, **kw)
    torch.cuda.synchronize()
    want = select64(logits, scores, choices, ended, end_token)
    for name, x, y in zip(("parent", "token", "ended"), (got[0], got[1], got[3]), (want[0], want[1], want[3])):
        assert np.array_equal(x.cpu().numpy(), y), name
    s = got[2].double().cpu().numpy()
    assert np.array_equal(np.isinf(s), np.isinf(want[2]) | (np.abs(want[2]) > 3.5e38))
    fine = np.isfinite(s)
    assert (np.abs(s[fine] - want[2][fine]) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(want[2][fine]) * 1.001).all()
    return got


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B,K,V,N,pad", [
    (1, 1, 1, 1, 0), (1, 1, 1, 5, 0), (1, 4, 3, 12, 0), (2, 3, 7, 8, 2), (1, 4, 32768, 4, 0), (3, 5, 1000, 10, 1),
    (2, 8, 4095, 16, 0), (2, 2, 8191, 64, 3), (1, 64, 513, 64, 0), (5, 3, 50001, 7, 5), (1, 2, 100003, 33, 61),
    (70, 2, 300, 4, 0), (2, 1, 262144, 1, 0), (1, 1, 2097152, 9, 0)])
def test_against_64_bits(kda, B, K, V, N, pad, dtype):
    logits, scores = make(B, K, V, dtype, seed=V + N, pad=pad)
    check(kda, logits, scores, N)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [20, 700, 5000, 40000])
def test_ties_go_to_the_lowest_index(kda, V, dtype):
    """Few distinct logits, equal beams: every place of the order is decided by beam and token."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    for values in (1, 2, 5):
        one = torch.randint(values, (1, 1, V), generator=g, device="cuda").to(dtype)
        check(kda, one.expand(2, 3, V).contiguous(), torch.full((2, 3), -1.5, device="cuda"), 12)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B,K,V,N", [(2, 32, 60000, 64), (1, 64, 20001, 64), (3, 24, 33000, 40)])
@pytest.mark.parametrize("apart", [0.0, 0.5, 3.0, 40.0])
def test_some_beams_ahead(kda, B, K, V, N, apart, dtype):
    """Many choices of many beams, the lower ones better by more and more: all of the best come from a few of them."""
    logits, scores = make(B, K, V, dtype, seed=K + N)
    check(kda, logits, scores / 9 - apart * torch.arange(K, device="cuda"), N)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [37, 3000, 70000])
def test_masked_tokens(kda, V, dtype):
    """-inf, the type's lowest value, NaN and +inf among the logits; rows of nothing else; beams that do not exist."""
    low = torch.finfo(dtype).min
    logits, scores = make(6, 3, V, dtype, seed=V)
    logits = logits.clone()
    logits[0, :, 5:] = -INF                     # five tokens left
    logits[1, :, 3:] = low                      # three, and the rest as low as can be
    logits[2, 0], logits[2, 2] = -INF, low      # nothing; nothing but the lowest
    logits[3, 1, ::3] = float("nan")
    logits[4, 0, V // 2] = INF
    logits[4, 1, :] = INF
    scores[4, 2] = float("nan")
    scores[5] = torch.tensor([-2.0, -INF, -INF])  # the first step: one beam
    logits[5, 0, : V // 2] = -INF
    for N in (1, 3, 20):
        check(kda, logits, scores, N)
    logits[:] = -INF
    parent, token, score, over = check(kda, logits, scores, 4, end_token=1)
    assert bool((parent == -1).all() and (token == -1).all() and (score == -INF).all() and (over == False).all())  # noqa: E712


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N", [3, 64])
def test_the_best_come_late(kda, N, dtype):
    """Logits that rise along the vocabulary, or whose first tokens are masked: what a segment's beginning says about its
    best is of no use."""
    V = 150000
    logits, scores = make(3, 2, V, dtype, seed=N)
    logits = logits.clone()
    logits[0] += torch.linspace(0, 40, V, device="cuda").to(dtype)
    logits[1, :, :140000] = -INF
    logits[2, 0, ::2] = torch.finfo(dtype).min
    logits[2, 1, : V // 2] = torch.finfo(dtype).min
    check(kda, logits, scores, N)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_ended_beams(kda, dtype):
    logits, scores = make(8, 4, 900, dtype, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ended = torch.rand((8, 4), generator=g, device="cuda") < 0.5
    ended[0], ended[1] = True, False
    scores[2] = -3.25  # ended beams of one score: the lower beam first
    scores[3, 0] = -INF
    logits = logits.clone()
    logits[ended] = float("nan")  # not read
    logits[:, :, 7] += 6  # the end token is likely
    logits[ended] = float("nan")
    for N in (2, 4, 9):
        check(kda, logits, scores, N, ended, 7)
    check(kda, logits, scores, 4, ended.to(torch.uint8), 899)


def test_ordering_of_logits(kda):
    """Signs, zeros of both signs, denormals and the largest numbers, in a row of their own each."""
    v = [0.0, -0.0, 1e-40, -1e-40, 3.4e38, -3.4e38, 1.0, -1.0, 1.0, 0.0, -0.0, 2e-38]
    logits = torch.tensor([v, v[::-1], v[3:] + v[:3]], device="cuda")[None]
    check(kda, logits, torch.tensor([[-1.0, -1.0, -1.0]], device="cuda"), 30)


def test_rows_that_start_anywhere(kda):
    """Vocabularies of odd size, rows and first elements off any boundary."""
    for dtype in (BF16, FP32):
        for V, first, width in ((33, 1, 40), (4001, 3, 4007), (8185, 7, 8200), (12289, 5, 12301)):
            g = torch.Generator(device="cuda")
            g.manual_seed(V)
            whole = torch.randn((2, 3, width), generator=g, device="cuda").to(dtype)
            whole[..., :first] = 100
            whole[..., first + V:] = 100
            scores = torch.zeros((2, 3), device="cuda")
            check(kda, whole[..., first: first + V], scores, 5)


def test_select_in_a_graph_on_a_stream_and_again(kda):
    logits, scores = make(4, 5, 60000, BF16, seed=5)
    want = [t.clone() for t in check(kda, logits, scores, 8)]
    busy = torch.randn((2048, 2048), device="cuda")
    for i in range(10):
        if i % 2:
            torch.mm(busy, busy)
        assert all(torch.equal(x, y) for x, y in zip(kda.kda_beam_select(logits, scores, 8), want))
    x, s = logits.clone(), scores.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.kda_beam_select(x, s, 8)
    for seed in (6, 7):
        other, t = make(4, 5, 60000, BF16, seed=seed)
        x.copy_(other)
        s.copy_(t)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, kda.kda_beam_select(other, t, 8)))
    side, need = torch.cuda.Stream(), kda.kda_beam_select_workspace_size(4, 5, 60000, 8)
    for _ in range(10):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mm(busy, busy)
        out = kda.kda_beam_select(logits, scores, 8, stream=side)
        blocks = [torch.full((need,), 1, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        del blocks


# --------------------------------------------------------------------------------------
# Reordering
# --------------------------------------------------------------------------------------
def state(B, K, page, seed, layers=2, spare_rows=3, spare_pages=None, words=512):
    rng = np.random.RandomState(seed)
    R, M = B * K + spare_rows, 9
    kv_len = rng.randint(0, M * page + 1, R).astype(np.int32)
    counts = -(-kv_len // page)
    pages = int(counts.sum()) + (B * K if spare_pages is None else spare_pages)
    names = list(rng.permutation(pages))
    table = np.full((R, M), -1, np.int32)
    for r in range(R):
        for i in range(counts[r]):
            table[r, i] = names.pop()
    slot = rng.permutation(R)[: B * K].reshape(B, K).astype(np.int32)
    pool = torch.randint(-2 ** 31, 2 ** 31 - 1, (layers, pages, words), dtype=torch.int32, device="cuda")
    return rng, table, kv_len, slot, pool, pages


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def reorder(kda, parent, slot, table, kv_len, pool, pages, page, refused=()):
    want = beam_reorder64(parent, slot, table, kv_len, pages, page)
    assert list(want[3]) == sorted({d for d in refused})
    expect = pool.clone()
    for s, d in want[6]:
        expect[:, d] = pool[:, s]
    t, n, sl = i32(table), i32(kv_len), i32(slot)
    src, dst = kda.kda_beam_reorder(i32(parent), sl, pool, t, n, page)
    torch.cuda.synchronize()
    for name, x, y in (("slot", sl, want[0]), ("src", src, want[1]), ("dst", dst, want[2]), ("table", t, want[4]),
                       ("kv_len", n, want[5])):
        assert np.array_equal(x.cpu().numpy(), y), name
    assert torch.equal(pool, expect)
    sl = i32(slot)  # without a cache: the same rows
    src, dst = kda.kda_beam_reorder(i32(parent), sl, num_rows=table.shape[0])
    assert np.array_equal(sl.cpu().numpy(), want[0]) and np.array_equal(src.cpu().numpy(), want[1])
    assert np.array_equal(dst.cpu().numpy(), want[2])


@pytest.mark.parametrize("B,K,page", [(1, 1, 16), (1, 2, 64), (1, 4, 16), (3, 5, 32), (40, 4, 16), (2, 32, 64), (2, 33, 16),
                                      (3, 64, 128), (1100, 2, 16)])
def test_reorder(kda, B, K, page):
    rng, table, kv_len, slot, pool, pages = state(B, K, page, seed=B * 100 + K)
    for kind in range(4):
        parent = (rng.randint(0, K, (B, K)) if kind == 0 else np.zeros((B, K), int) if kind == 1
                  else np.stack([rng.permutation(K) for _ in range(B)]) if kind == 2
                  else rng.randint(-1, K + 1, (B, K)))  # some without a parent
        reorder(kda, parent, slot, table, kv_len, pool.clone(), pages, page)
        assert kda.kda_get_device_status()[0] == 0


def test_reorder_refuses_slots_that_do_not_exist_or_repeat(kda):
    """The prompts that hold them stay as they were; the others go on."""
    rng, table, kv_len, slot, pool, pages = state(5, 4, 16, seed=9)
    parent = rng.randint(0, 4, (5, 4))
    R = table.shape[0]
    for change, refused in [((1, 2, R), [1]), ((3, 0, -1), [3]), ((2, 1, int(slot[2, 3])), [2]),
                            ((0, 0, int(slot[4, 2])), [0, 4])]:
        bad = slot.copy()
        bad[change[0], change[1]] = change[2]
        reorder(kda, parent, bad, table, kv_len, pool.clone(), pages, 16, refused)
        status, detail = kda.kda_get_device_status()
        assert status == 6 and detail in refused


def test_reorder_without_a_page_left(kda):
    """As a fork: the branches that find none are left empty, in order."""
    rng, table, kv_len, slot, pool, pages = state(2, 4, 16, seed=11, spare_pages=0)
    kv_len[:] = np.where(kv_len % 16 == 0, np.maximum(kv_len - 3, 0), kv_len)
    table[:] = np.where(np.arange(9)[None] < -(-kv_len // 16)[:, None], table, -1)
    # every page stays named: rows of no beam hold those of the beams that leave
    keep = [r for r in range(table.shape[0]) if r not in slot.reshape(-1)]
    free = [p for p in range(pages) if p not in table.reshape(-1)]
    gone = [int(x) for r in slot.reshape(-1) for x in table[r] if x >= 0]
    named = (free + gone)[: len(keep) * 9]
    for i, p in enumerate(named):
        table[keep[i // 9], i % 9] = p
    parent = np.zeros((2, 4), int)
    want = beam_reorder64(parent, slot, table, kv_len, pages, 16)
    reorder(kda, parent, slot, table, kv_len, pool.clone(), pages, 16)
    if any(s >= 0 and want[5][d] == 0 and kv_len[s] > 0 for s, d in zip(want[1], want[2]) if d >= 0):
        assert kda.kda_get_device_status()[0] == 6


def test_states_follow_their_beams(kda):
    """With kda_pages_copy, every beam has what its parent had, in all pools."""
    rng, table, kv_len, slot, pool, pages = state(6, 4, 16, seed=13)
    R = table.shape[0]
    S = torch.randn((2, R, 3, 128), device="cuda")
    conv = torch.randn((1, R, 2, 128), device="cuda").to(BF16)
    for step in range(5):
        parent = rng.randint(0, 4, (6, 4))
        rows = np.take_along_axis(slot, parent, 1).reshape(-1)
        want_s, want_c, want_n = S[:, rows].clone(), conv[:, rows].clone(), kv_len[rows]
        sl = i32(slot)
        t, n = i32(table), i32(kv_len)
        src, dst = kda.kda_beam_reorder(i32(parent), sl, pool, t, n, 16)
        kda.kda_pages_copy(S, src, dst)
        kda.kda_pages_copy(conv, src, dst)
        slot, table, kv_len = sl.cpu().numpy(), t.cpu().numpy(), n.cpu().numpy()
        now = slot.reshape(-1)
        assert torch.equal(S[:, now], want_s) and torch.equal(conv[:, now], want_c) and np.array_equal(kv_len[now], want_n)
        assert len(set(now.tolist())) == now.size
    assert kda.kda_get_device_status()[0] == 0


def test_reorder_in_a_graph(kda):
    rng, table, kv_len, slot, pool, pages = state(4, 4, 16, seed=15)
    parent = i32(rng.randint(0, 4, (4, 4)))
    start = [pool, i32(table), i32(kv_len), i32(slot)]
    buffers = [x.clone() for x in start]

    def step(parent, pool, t, n, sl):
        return kda.kda_beam_reorder(parent, sl, pool, t, n, 16)

    step(parent, *[x.clone() for x in start])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        src, dst = step(parent, *buffers)
    for _ in range(2):
        parent.copy_(i32(rng.randint(0, 4, (4, 4))))
        for b, x in zip(buffers, start):
            b.copy_(x)
        want = [x.clone() for x in start]
        s, d = step(parent, *want)
        graph.replay()
        assert torch.equal(s, src) and torch.equal(d, dst) and all(torch.equal(x, y) for x, y in zip(buffers, want))
    assert kda.kda_get_device_status()[0] == 0


@pytest.mark.parametrize("pages,rows", [(1 << 20, 300), (500, 1 << 18)])
def test_reorder_at_the_limits_of_the_table(kda, pages, rows):
    """As many pages and rows as the call takes: the plan's shared memory."""
    rng = np.random.RandomState(17)
    table, kv_len = np.full((rows, 2), -1, np.int32), np.zeros(rows, np.int32)
    slot = rng.permutation(rows)[:8].reshape(2, 4).astype(np.int32)
    names = rng.permutation(pages)[:16]
    for i, r in enumerate(slot.reshape(-1)):
        table[r], kv_len[r] = names[2 * i: 2 * i + 2], 17 + i
    pool = torch.randint(-99, 99, (1, pages, 4), dtype=torch.int32, device="cuda")
    reorder(kda, rng.randint(0, 4, (2, 4)), slot, table, kv_len, pool, pages, 16)
    assert kda.kda_get_device_status()[0] == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_one_beam_of_rows_of_any_stride(kda, dtype):
    """One beam a prompt out of a padded output, and one of several beams: dense rows, evenly spaced."""
    logits, scores = make(5, 3, 4001, dtype, seed=23, pad=6)
    check(kda, logits[:, 0].unsqueeze(1), scores[:, :1].contiguous(), 7)
    check(kda, logits[:, 1:2], scores[:, 1:2].contiguous(), 7)
    check(kda, logits.transpose(0, 1)[2].unsqueeze(1), scores[:, 2:].contiguous(), 7)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [130, 5000, 70000])
def test_infinities_tie_with_the_largest_number(kda, V, dtype):
    """A logit of +inf counts as the largest fp32 number: among those and fp32 logits that are it the lower token goes first,
    whichever of the two it is and wherever in the row they lie."""
    most = torch.finfo(dtype).max
    logits, scores = make(8, 2, V, dtype, seed=V)
    logits = logits.clone()
    logits[0, :, 3], logits[0, :, 100] = most, INF
    logits[1, :, 100], logits[1, :, 3] = most, INF
    logits[2, :, V // 2], logits[2, :, V - 1] = most, INF            # in other chunks, other segments
    logits[3, :, V // 2], logits[3, :, V - 1] = INF, most
    logits[4, :, 1::2], logits[4, :, 0] = INF, most                  # more than can be ranked by counting
    logits[5], logits[5, 0, : V // 3] = most, INF
    logits[6, 0, ::7], logits[6, 1, V // 4:] = most, INF
    logits[7, :, 90:], logits[7, :, 64:90] = INF, most
    for N in (1, 2, 5, 40):
        check(kda, logits, scores, N)


def crowded(left, seed=19):
    """Two prompts of four beams in two pages each, the last one part-filled; two further rows name every page but `left`
    that no row has, so that the beams that leave free none."""
    rng = np.random.RandomState(seed)
    R, M, page, pages = 11, 12, 16, 16 + left
    names, slot = rng.permutation(pages), rng.permutation(R)[:8].reshape(2, 4).astype(np.int32)
    table, kv_len = np.full((R, M), -1, np.int32), np.zeros(R, np.int32)
    for i, r in enumerate(slot.reshape(-1)):
        table[r, :2], kv_len[r] = names[2 * i: 2 * i + 2], 17 + i
    keep = [r for r in range(R) if r not in slot]
    table[keep[0], :8], table[keep[2], :8] = names[:8], names[8:16]
    kv_len[keep[0]] = kv_len[keep[2]] = 128
    pool = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, pages, 64), dtype=torch.int32, device="cuda" if torch.cuda.is_available() else "cpu")
    return table, kv_len, slot, pool, pages, page


# parents: all of the first beam; some of none (they need no page)
CROWDED = [([[0, 0, 0, 0], [0, 0, 0, 0]], [1, 2, 3, 5, 6, 7]), ([[2, 2, 1, 1], [3, -1, 3, 3]], [1, 3, 6, 7]),
           ([[-1, 4, 0, 0], [1, 1, 2, 0]], [3, 5])]


@pytest.mark.parametrize("left", [0, 1, 2, 5])
@pytest.mark.parametrize("parent,branches", CROWDED)
def test_reorder_where_pages_run_out(kda, parent, branches, left):
    """The branches get the pages that are left, in order; the others' rows are left empty, and said."""
    table, kv_len, slot, pool, pages, page = crowded(left)
    parent = np.array(parent)
    want = beam_reorder64(parent, slot, table, kv_len, pages, page)
    dst = want[2].tolist()
    for n, i in enumerate(branches):  # (what the plain implementation says, spelled out)
        row = want[4][dst[i]].tolist()
        if n < left:
            assert want[5][dst[i]] == kv_len[want[1][i]] and row[1] >= 0 and row[2:] == [-1] * 10
        else:
            assert want[5][dst[i]] == 0 and row == [-1] * 12
    assert len(want[6]) == min(left, len(branches))
    kda.kda_get_device_status()
    reorder(kda, parent, slot, table, kv_len, pool, pages, page)
    lost = branches[left:]
    status, detail = kda.kda_get_device_status()
    assert (status == 6 and detail in lost) if lost else status == 0
