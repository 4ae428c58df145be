"""Attention over a shared prefix against a 64-bit plain implementation.

Tolerances, elementwise, as for the windowed attention.  bf16: a probability rounded to bf16 is off by
at most 2^-8 of itself and so is the rounded output; the fp32 parts (128-term scores, exponentials,
sums, the join of the parts) stay below 2^-12 of it.  With a = sum_j softmax_j |v_j| that is
|o - ref| <= 2^-8 (a + |ref|) + 2^-12 a.  fp32: max-abs over rms 1e-5, the bound of every fp32 path here.
"""
import ctypes
import time

import numpy as np
import pytest
import torch

from tests._branches import build_branches, prefix64
from tests._cache import cu_of, queries
from tests._parity import TOL_FP32, assert_close, to64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def call(kda, q, c, new, **kw):
    kw.setdefault("max_tokens", max(list(new) + [1]))
    o = kda.kda_prefix_attention(q, c["pool"], c["table"], c["slot"], cu_of(new), c["kv_len"], c["cu_groups"],
                                 c["prefix_len"], **kw)
    torch.cuda.synchronize()
    return o


def check(o, q, c, new, scale=128 ** -0.5):
    ref, a = prefix64(q, c, new, scale)
    o64 = to64(o)
    if o.dtype == FP32:
        return assert_close(o64, ref, TOL_FP32, "o")
    assert np.isfinite(o64).all()
    over = np.abs(o64 - ref) - (2.0 ** -8 * (a + np.abs(ref)) + 2.0 ** -12 * a)
    assert over.max(initial=-1.0) <= 1e-30, f"{over.max():.3e} over the bound at {np.unravel_index(over.argmax(), over.shape)}"


# (prefix of each group, [own tokens of each branch] of each group, tokens of the step of each branch, kv heads, group, page)
SHAPES = [
    ([0], [[1]], [1], 1, 1, 16),                                             # one token that sees itself
    ([1], [[1]], [1], 1, 1, 16),
    ([64], [[1, 1]], [1, 1], 2, 4, 64),                                      # a tile, and nothing of its own before
    ([500], [[1, 9, 30]], [1, 1, 1], 2, 12, 64),                             # beams, a prefix that ends inside a page
    ([127, 128, 129, 0], [[3], [1, 2], [4, 4, 4], [5, 70]], [1] * 8, 1, 8, 32),   # tile edges, a group without a prefix
    ([1000, 37], [[20, 300], [5]], [2, 3, 5], 2, 3, 16),                     # drafts
    ([300], [[6] * 33], [1] * 33, 1, 16, 128),                               # 528 rows: more than two row tiles
    ([700, 1300], [[4] * 20, [130] * 3], [1] * 23, 1, 6, 64),
    ([77], [[40, 2, 9], []], [0, 2, 7], 1, 5, 16),                           # a request without tokens, a group without requests
    ([260], [[400]], [300], 1, 2, 32),                                           # many tokens of one request
    ([90], [[70, 90]], [64, 33], 2, 4, 16),
    ([150], [[20] * 3], [9, 1, 20], 1, 33, 64),                              # odd heads a kv head
    ([140], [[9, 3]], [2, 1], 1, 128, 32),                                   # one kv head of 128 query heads
    ([5000], [[3, 70]], [1, 1], 1, 2, 128),                                  # one item over many CTAs
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_64_bits(kda, shape, dtype):
    prefix, mine, new, heads, group, page = shape
    c = build_branches(prefix + [0] * (len(mine) - len(prefix)), mine, page, heads, dtype, seed=len(new) * 31 + page)
    q = queries(sum(new), heads * group, dtype, 3)
    o = call(kda, q, c, new)
    assert kda.kda_get_device_status()[0] == 0
    check(o, q, c, new)


def test_many_groups(kda):
    """More groups than a CTA has threads, of all kinds of lengths, some without requests."""
    rng = np.random.RandomState(5)
    prefix = [int(rng.choice([0, 3, 16, 40, 129])) for _ in range(900)]
    mine = [[int(rng.randint(1, 20)) for _ in range(rng.randint(0, 3))] for _ in prefix]
    new = [1] * sum(len(m) for m in mine)
    for dtype in (BF16, FP32):
        c = build_branches(prefix, mine, 16, 1, dtype, seed=3)
        q = queries(len(new), 2, dtype, 3)
        o = call(kda, q, c, new)
        assert kda.kda_get_device_status()[0] == 0
        check(o, q, c, new)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", [(7, 8, 4, 64, 4), (70, 8, 5, 16, 3), (43, 40, 1, 32, 16), (330, 1, 16, 128, 1),
                                   (90, 4, 6, 16, 4), (90, 4, 8, 64, 7), (330, 8, 4, 32, 2), (330, 8, 5, 32, 7)])
def test_many_requests(kda, shape, dtype):
    """More (request, kv head) pairs than CTAs fit on the GPU: requests of all lengths and numbers of tokens (also
    none), one of them refused, and values that are not finite in the step's own tokens and where nothing is."""
    B, heads, group, page, most = shape
    rng = np.random.RandomState(B)
    sizes = [B // 2, 0, B - B // 2 - 1, 1]
    new = [int(rng.randint(1, most + 1)) if i % 5 else min(most, i) for i in range(B)]
    mine = [[new[sum(sizes[:g]) + i] + int(rng.randint(0, 260)) * (i % 3) for i in range(n)] for g, n in enumerate(sizes)]
    c = build_branches([300, 7, 0, 40], mine, page, heads, dtype, seed=B)
    table, kv_len, slot = (c[k].cpu().numpy() for k in ("table", "kv_len", "slot"))
    clean = {**c, "pool": c["pool"].clone()}
    for b in range(0, B, 3):  # behind the last token of its page
        n = int(kv_len[slot[b]])
        if n % page:
            c["pool"][table[slot[b], n // page], :, :, n % page:] = float("nan")
    late = max(range(B), key=lambda b: new[b] * (b % 3 != 0))  # a value that only the last token sees
    if new[late] > 1:
        j = int(kv_len[slot[late]]) - 1
        c["pool"][table[slot[late], j // page], 1, :, j % page, 5] = float("inf")
    q = queries(sum(new), heads * group, dtype, B)
    cu = cu_of(new).tolist()
    refused = next(b for b in range(B // 2, B) if new[b] and b != late)
    gone = torch.full_like(q, 7.0)
    call(kda, q, {**c, "slot": c["slot"].clone().index_fill_(0, torch.tensor([refused], device="cuda"), -1)}, new, o=gone)
    # (where it is the first of its group, the prefix is read through its row: then the group is refused)
    ends = np.cumsum(sizes)
    g = int(np.searchsorted(ends, refused, side="right"))
    group_of = range(int(ends[g]) - sizes[g], int(ends[g]))
    lost = list(group_of) if refused == group_of[0] else [refused]
    status, detail = kda.kda_get_device_status()
    assert status == 6 and detail in lost
    o = call(kda, q, c, new)
    assert kda.kda_get_device_status()[0] == 0
    same = torch.ones(len(q), dtype=torch.bool, device="cuda")
    for b in lost:
        same[cu[b]:cu[b + 1]] = False
    assert torch.equal(torch.nan_to_num(gone[same].float()), torch.nan_to_num(o[same].float()))
    assert bool((gone[~same] == 7.0).all())
    if new[late] > 1:
        last = cu[late + 1] - 1
        assert not torch.isfinite(o[last, :, 5]).any()
        o[last] = call(kda, q, clean, new)[last]
    check(o, q, clean, new)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("group,heads,most", [(6, 2, 40), (6, 2, 100000), (5, 16, 40), (13, 2, 40)])
def test_a_few_long_requests_among_many(kda, group, heads, most, dtype):
    """Single tokens for the most part, and some requests that bring many row blocks, with short and long own keys.

    fp32: 1e-5 of the root mean square is a typical error's bound, and too little for the largest of 4 million
    elements (1.04e-5 was seen).  What holds for each: a score is 128 fused steps and a multiplication, off by at most
    129 half steps of A = scale sum_i |q_i| |k_ji|; less the maximum (a difference of at most 2 A) by 2 more; its
    exponential (two units) by 2^-22 of itself.  So a weight is off by a factor within e^(+-D), D = 131 * 2^-24 A + 2^-22;
    sums of n < 512 of them, weighted or not, by n half steps each; their ratio rounds twice (1 / l, and the product).
    |o - ref| <= (e^(2 D + 2 n 2^-24 + 2^-22) - 1) a with a = sum_j softmax_j |v_j|.
    """
    B = 300
    new = [1] * B
    for b, n in ((0, 13), (7, 40), (150, 3), (151, 0), (299, 29)):
        new[b] = n
    mine = [[n + (b * 37) % (90 if b % 4 else 9) for b, n in enumerate(new)]]
    c = build_branches([70], mine, 32, heads, dtype, seed=most % 97)
    q = queries(sum(new), heads * group, dtype, 71)
    o = call(kda, q, c, new, max_tokens=most)
    assert kda.kda_get_device_status()[0] == 0
    if dtype == BF16:
        return check(o, q, c, new)
    ref, a = prefix64(q, c, new)
    k = c["pool"][:, 0].transpose(0, 1).reshape(heads, -1, 128).abs()
    most_a = torch.stack([(x.abs() @ k[h].T).amax(-1) for h, x in enumerate(q.reshape(len(q), heads, group, 128).unbind(1))], 1)
    d = 131 * 2.0 ** -24 * 128 ** -0.5 * to64(most_a).reshape(len(q), heads * group, 1) + 2.0 ** -22
    assert (np.abs(to64(o) - ref) <= np.expm1(2 * d + 2 * 512 * 2.0 ** -24 + 2.0 ** -22) * a).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_same_as_window_attention_without_a_window(kda, dtype):
    """Rows that share their prefix: the two calls differ by roundings alone."""
    new = [1, 2, 1, 4]
    c = build_branches([333, 64], [[7, 40], [1, 90]], 32, 2, dtype, seed=7)
    q = queries(sum(new), 16, dtype, 7)
    o = call(kda, q, c, new)
    w = kda.kda_window_attention(q, c["pool"], c["table"], c["slot"], cu_of(new), c["kv_len"], None, max_tokens=4)
    ref, a = prefix64(q, c, new)
    if dtype == FP32:
        assert_close(to64(o), to64(w), 2 * TOL_FP32, "o")
    else:
        assert (np.abs(to64(o) - to64(w)) <= 2 * (2.0 ** -8 * (a + np.abs(ref)) + 2.0 ** -12 * a)).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_the_prefix_is_read_through_the_first_request_s_row(kda, dtype):
    """What the other rows name below the prefix's length is not read: they may name nothing."""
    new = [1, 1, 1]
    c = build_branches([200], [[30, 5, 70]], 16, 2, dtype, seed=11)
    q = queries(3, 8, dtype, 11)
    want = call(kda, q, c, new)
    slot = c["slot"].tolist()
    c["table"][slot[1], : 200 // 16] = -1
    c["table"][slot[2], : 200 // 16] = c["pool"].shape[0] + 5
    assert torch.equal(call(kda, q, c, new), want)
    check(want, q, c, new)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new", [[1, 1], [3, 2], [40, 2]])
def test_unmapped_pages_hold_no_keys(kda, new, dtype):
    """Pages missing from the prefix and from a request's own keys; a request that has none left at all gives 0."""
    c = build_branches([150, 90], [[60], [50]], 16, 2, dtype, seed=13)
    slot = c["slot"].tolist()
    c["table"][slot[0], 2] = -1
    c["table"][slot[0], 150 // 16 + 1] = c["pool"].shape[0]
    c["table"][slot[1], :] = -7
    q = queries(sum(new), 6, dtype, 13)
    o = call(kda, q, c, new)
    assert kda.kda_get_device_status()[0] == 0
    assert bool((o[new[0]:] == 0).all())
    check(o, q, c, new)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("new", [[1, 1], [3, 5], [50, 2]])
def test_what_no_token_sees_does_not_reach_the_output(kda, new, value, dtype):
    """Behind the rows' last tokens, in pages that no row names, and in the pages of the prefix behind its end as the
    other branches have them."""
    page, lp, mine = 32, 149, [60, 71]
    c = build_branches([lp], [mine], page, 2, dtype, seed=17)
    slot, table = c["slot"].tolist(), c["table"].tolist()
    named = {x for r in slot for x in table[r]} - {-1}
    for p in range(c["pool"].shape[0]):
        if p not in named:
            c["pool"][p] = value
    for r, n in zip(slot, mine):
        if (lp + n) % page:
            c["pool"][table[r][(lp + n) // page], :, :, (lp + n) % page:] = value
    # the second branch's copy of the prefix's last part-filled page: its part below the prefix's end is not read
    c["pool"][table[slot[1]][lp // page], :, :, : lp % page] = value
    clean = {**c, "pool": torch.nan_to_num(c["pool"].float(), 0.0, 0.0, 0.0).to(dtype)}
    q = queries(sum(new), 8, dtype, 17)
    o = call(kda, q, c, new)
    check(o, q, clean, new)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n", [4, 30])
def test_a_later_token_s_nan_stays_its_own(kda, n, value, dtype):
    """A value of the step itself that is not finite: tokens before it and the other branch are untouched."""
    new, lp, bad = [n, 2], 70, n // 2
    c = build_branches([lp], [[20 + n, 9]], 16, 1, dtype, seed=19)
    row = c["table"][c["slot"][0].item()].tolist()
    j = lp + 20 + bad
    clean = {**c, "pool": c["pool"].clone()}
    c["pool"][row[j // 16], 1, :, j % 16, 3] = value
    q = queries(sum(new), 4, dtype, 19)
    o, ref = call(kda, q, c, new), call(kda, q, clean, new)
    assert torch.isfinite(o[:bad]).all() and torch.isfinite(o[n:]).all()
    assert not torch.isfinite(o[bad:n, :, 3]).any()
    check(torch.cat([o[:bad], ref[bad:n], o[n:]]), q, clean, new)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-3])
def test_scales(kda, scale, dtype):
    new = [1, 2]
    c = build_branches([100], [[20, 33]], 32, 1, dtype, seed=23)
    q = queries(3, 4, dtype, 23)
    check(call(kda, q, c, new, scale=scale), q, c, new, scale)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_scores_of_any_size(kda, dtype):
    """Scores of the prefix far above and far below those of the own keys: the join keeps what counts.  fp32: a score
    is a sum of 128 rounded products, off by up to d = 128 2^-24 scale sum_i |q_i k_i|, which moves a weight by
    e^(2 d) and the output by (e^(2 d) - 1) (a + |ref|); with scores of some hundreds that is above the usual bound."""
    new = [1, 1, 1]
    for factor in (30.0, 0.01):
        c = build_branches([300], [[9, 40, 100]], 32, 1, dtype, seed=29)
        names = c["table"][c["slot"][0].item(), : 300 // 32].long()
        c["pool"][names, 0] *= factor
        q = queries(3, 8, dtype, 29) * 4
        o = call(kda, q, c, new)
        if dtype == BF16:
            check(o, q, c, new)
            continue
        ref, a = prefix64(q, c, new)
        keys = c["pool"][:, 0].double().abs().reshape(-1, 128)
        d = 128 * 2.0 ** -24 * 128 ** -0.5 * (q.double().abs() @ keys.T).amax(-1).cpu().numpy()[..., None]
        bound = np.expm1(2 * d) * (a + np.abs(ref)) + TOL_FP32 * np.sqrt((ref ** 2).mean())
        assert (np.abs(to64(o) - ref) <= bound).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_refused_requests_leave_their_rows(kda, dtype):
    """Slots, lengths, token ranges and prefixes out of range are refused one by one; the others are computed."""
    new, lp = [1, 2, 1, 1], [100, 40]
    c = build_branches(lp, [[20, 30], [9, 5]], 16, 1, dtype, seed=31)
    q = queries(5, 4, dtype, 31)
    good = call(kda, q, c, new)
    check(good, q, c, new)
    first = [0, 1, 3, 4, 5]

    def run(refused, detail, max_tokens=2, **change):
        o = torch.full_like(q, 7.0)
        d = {**{k: v.clone() for k, v in c.items()}, **change}
        call(kda, q, d, new, o=o, max_tokens=max_tokens)
        assert kda.kda_get_device_status() == (6, detail)
        for b in range(4):
            part = slice(first[b], first[b + 1])
            assert torch.equal(o[part], torch.full_like(o[part], 7.0) if b in refused else good[part]), b

    def put(name, i, x):
        t = c[name].clone()
        t[i] = x
        return {name: t}

    rows = c["table"].shape[0]
    run({1}, 1, **put("slot", 1, rows))
    run({1}, 1, **put("slot", 1, -1))
    run({3}, 3, **put("kv_len", c["slot"][3].item(), -1))
    run({3}, 3, **put("kv_len", c["slot"][3].item(), c["table"].shape[1] * 16 + 1))
    run({1}, 1, **put("kv_len", c["slot"][1].item(), 101))     # two tokens, one of them inside the prefix
    run({1}, 1, max_tokens=1)
    # a group without a row or with a prefix out of range: all its requests
    for change in (put("slot", 2, rows), put("prefix_len", 1, -1), put("prefix_len", 1, c["table"].shape[1] * 16 + 1)):
        d = {**{k: v.clone() for k, v in c.items()}, **change}
        o = torch.full_like(q, 7.0)
        call(kda, q, d, new, o=o)
        status, detail = kda.kda_get_device_status()
        assert status == 6 and detail in (2, 3)
        assert torch.equal(o[:3], good[:3]) and bool((o[3:] == 7.0).all())


def test_requests_outside_any_group_and_groups_that_overlap(kda):
    new = [1] * 4
    for dtype in (BF16, FP32):
        c = build_branches([100, 40], [[20, 30], [9, 5]], 16, 1, dtype, seed=37)
        q = queries(4, 4, dtype, 37)
        good = call(kda, q, c, new)
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
        for cu, done in [(i32(0, 2, 3), (0, 1, 2)), (i32(1, 2, 4), (2, 3)), (i32(0, 2, 9), (0, 1)), (i32(-3, 2, 4), (2, 3))]:
            o = torch.full_like(q, 7.0)
            call(kda, q, {**c, "cu_groups": cu}, new, o=o)
            assert kda.kda_get_device_status()[0] == 6
            for b in range(4):
                if b in done:
                    assert torch.equal(o[b], good[b])
        # the same requests in five hundred groups: more work than the workspace holds is not begun
        c = build_branches([40], [[3] * 100], 16, 1, dtype, seed=38)
        q = queries(100, 16, dtype, 38)
        o = torch.full_like(q, 7.0)
        call(kda, q, {**c, "cu_groups": i32(*[100 * (g % 2) for g in range(1001)]), "prefix_len": i32(*[40] * 1000)},
             [1] * 100, o=o)
        assert kda.kda_get_device_status()[0] == 6
        assert bool((o == 7.0).all())


def test_no_tokens(kda):
    c = build_branches([40], [[3, 4]], 16, 1, BF16, seed=41)
    q = queries(0, 4, BF16, 41)
    assert call(kda, q, c, [0, 0]).shape == (0, 4, 128)
    assert kda.kda_get_device_status()[0] == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_loose_max_tokens(kda, dtype):
    new = [1, 3, 2]
    c = build_branches([200], [[9, 30, 100]], 32, 2, dtype, seed=43)
    q = queries(sum(new), 8, dtype, 43)
    for most in (3, 17, 100000):
        check(call(kda, q, c, new, max_tokens=most), q, c, new)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", [([3000, 500], [[40] * 9, [7] * 2], [1] * 11, 2, 8, 64),
                                   ([9000], [[3, 700]], [2, 1], 1, 4, 32),
                                   ([300, 64], [[9, 50] * 60, [130] * 60], [1, 3] * 90, 2, 6, 32)])
def test_replayed_from_a_graph_and_repeated_bit_for_bit(kda, shape, dtype):
    """One capture over buffers whose contents, lengths and prefixes change between replays."""
    prefix, mine, new, heads, group, page = shape
    c = build_branches(prefix, mine, page, heads, dtype, seed=47)
    q, cu = queries(sum(new), heads * group, dtype, 47), cu_of(new)
    ask = lambda q, c: kda.kda_prefix_attention(q, c["pool"], c["table"], c["slot"], cu, c["kv_len"], c["cu_groups"],
                                                c["prefix_len"], max_tokens=max(new))
    want = ask(q, c)
    busy = torch.randn((2048, 2048), device="cuda")
    for i in range(10):
        if i % 2:
            torch.mm(busy, busy)  # the GPU in another state
        assert torch.equal(ask(q, c), want)
    buffers = {k: v.clone() for k, v in c.items()}
    x = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = ask(x, buffers)
    for shorter in (0, 37):  # the same rows with another cut between shared and own keys
        other = {**c, "prefix_len": (c["prefix_len"] - shorter).contiguous()}
        x.copy_(queries(sum(new), heads * group, dtype, 48 + shorter))
        buffers["prefix_len"].copy_(other["prefix_len"])
        graph.replay()
        assert torch.equal(o, ask(x, other))
        check(o, x, other, new)
    assert kda.kda_get_device_status()[0] == 0


def test_on_a_side_stream(kda):
    """What the call allocates belongs to its stream, while the current stream allocates blocks of that size."""
    new = [1, 2]
    c = build_branches([500], [[9, 30]], 32, 2, BF16, seed=53)
    q = queries(3, 16, BF16, 53)
    want, cu = call(kda, q, c, new), cu_of(new)
    side, busy = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    need = kda.kda_prefix_attention_workspace_size(BF16, 2, 3, 1, 16, 2)
    for _ in range(10):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mm(busy, busy)
        o = kda.kda_prefix_attention(q, c["pool"], c["table"], c["slot"], cu, c["kv_len"], c["cu_groups"],
                                     c["prefix_len"], max_tokens=2, stream=side)
        blocks = [torch.full((need,), 1, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, want)
        del blocks


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_two_calls_at_once(kda, dtype):
    """Two streams, each with a workspace of its own, give what one after the other does."""
    inputs = []
    for seed, (prefix, mine, new) in enumerate([([3000, 40], [[9] * 40, [300] * 40], [1] * 80), ([700], [[50] * 200], [1] * 200)]):
        c = build_branches(prefix, mine, 32, 2, dtype, seed=67 + seed)
        inputs.append((queries(len(new), 16, dtype, 67 + seed), c, new))
    want = [call(kda, *x) for x in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    cu = [cu_of(new) for _, _, new in inputs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (q, c, new) in enumerate(inputs):
            got[i].append(kda.kda_prefix_attention(q, c["pool"], c["table"], c["slot"], cu[i], c["kv_len"], c["cu_groups"],
                                                   c["prefix_len"], max_tokens=1, stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])
    assert kda.kda_get_device_status()[0] == 0


# prefixes, own keys and new tokens: one of each kind of kernel over the own keys (single rows of a cluster, two blocks
# of rows, many requests), with prefixes and without
GIVING_UP = [([300], [[9, 30]], [1, 1]), ([700], [[9, 30]], [7, 5]), ([300], [[20] * 160], [1] * 160),
             ([0], [[9, 30]], [1, 1]), ([0], [[20] * 160], [1] * 160)]


@pytest.mark.parametrize("shape", GIVING_UP)
def test_waits_that_run_out_are_reported(kda, shape):
    """The debug library arms one call whose load warps fetch nothing and whose waits give up after 1 ms: the call ends
    soon, with the status and with o as it was, and the next one through the same workspace is right."""
    from gated_delta_rule_kda_gb300 import build
    prefix, mine, new = shape
    c = build_branches(prefix, mine, 32, 2, BF16, seed=61)
    q, cu, T, B = queries(sum(new), 8, BF16, 61), cu_of(new), sum(new), len(new)
    want = call(kda, q, c, new)
    check(want, q, c, new)
    lib = ctypes.CDLL(build.build(debug=True))
    lib.kda_prefix_attention.argtypes = kda.library().kda_prefix_attention.argtypes
    lib.kda_get_device_status.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    stream, detail, o = torch.cuda.current_stream().cuda_stream, ctypes.c_uint32(0), torch.full_like(q, -7.0)
    size = kda.kda_prefix_attention_workspace_size(BF16, B, T, 1, 8, 2)
    workspace = torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    def attend():
        R, M = c["table"].shape
        P = c["pool"].shape[0]
        assert lib.kda_prefix_attention(0, B, T, max(new), 8, 2, P, 32, R, M, 1, q.data_ptr(), c["pool"].data_ptr(),
                                        c["table"].data_ptr(), c["slot"].data_ptr(), cu.data_ptr(), c["kv_len"].data_ptr(),
                                        c["cu_groups"].data_ptr(), c["prefix_len"].data_ptr(), 128 ** -0.5, o.data_ptr(),
                                        workspace.data_ptr(), size, stream) == 0
        return lib.kda_get_device_status(stream, ctypes.byref(detail))

    assert lib.kda_debug_inject_prefix_timeout() == 0
    t0 = time.perf_counter()
    assert attend() == 5 and detail.value >= 128
    assert time.perf_counter() - t0 < 0.5
    assert bool((o == -7.0).all())
    assert attend() == 0 and torch.equal(o, want)


# One of each kind of kernel over the own keys: single rows of a cluster, two blocks of rows, many requests head by head,
# several heads at once (with own keys in one tile and in many), and with two blocks of rows.  No request brings more rows
# than most.
OWN_KERNELS = [
    ([300, 0], [[9, 70], [33]], [1, 1, 1], 2, 4, 32),
    ([300], [[20, 300]], [7, 7], 2, 4, 32),
    ([100], [[3 + 40 * (i % 5) for i in range(160)]], [1] * 160, 2, 4, 32),
    ([90], [[3 + 50 * (i % 3) for i in range(330)]], [1] * 330, 8, 2, 16),
    ([90], [[3 + 50 * (i % 3) for i in range(100)]], [3] * 100, 2, 8, 64),
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["q", "k"])
@pytest.mark.parametrize("shape", OWN_KERNELS)
def test_scores_that_are_not_finite_give_nan(kda, shape, where, value, dtype):
    """A NaN or infinity in a query, or in an own key that some tokens see: their rows are what the definition gives (NaN
    where a score is NaN or +inf), not what o held before, and all others are untouched by it.

    fp32: the bound of test_a_few_long_requests_among_many with what the join adds to a weight, a difference of maxima (at
    most 2 A), its product with log2 e (rounded itself) and an approximate 2^x: 6 A half steps and 2^-22 more."""
    prefix, mine, new, heads, group, page = shape
    c = build_branches(prefix, mine, page, heads, dtype, seed=73)
    q = queries(sum(new), heads * group, dtype, 73)
    slot, kv_len, table, cu = c["slot"].tolist(), c["kv_len"].tolist(), c["table"].tolist(), cu_of(new).tolist()
    hit = sorted({0, 1, len(new) - 1})
    clean_q, clean_k = q.clone(), c["pool"][:, 0].clone()
    for b in hit:
        if where == "q":
            q[cu[b + 1] - 1, (3 * b) % (heads * group), 7] = value
        else:
            j = kv_len[slot[b]] - 1 - new[b] // 2  # seen by the later ones of its tokens
            c["pool"][table[slot[b]][j // page], 0, b % heads, j % page, 7] = value
    o = torch.full_like(q, 7.0)
    call(kda, q, c, new, o=o)
    assert kda.kda_get_device_status()[0] == 0
    with np.errstate(invalid="ignore"):
        ref, a = prefix64(q, c, new)
    o64, lost = to64(o), np.isnan(ref).any(-1)
    assert lost.any() and not lost.all()
    assert np.isnan(ref[lost]).all() and np.isnan(o64[lost]).all()
    o64, ref, a = o64[~lost], ref[~lost], a[~lost]
    if dtype == BF16:
        bound = 2.0 ** -8 * (a + np.abs(ref)) + 2.0 ** -12 * a
    else:
        size = torch.einsum("thgd,hkd->thgk", clean_q.double().abs().reshape(len(q), heads, group, 128),
                            clean_k.double().abs().transpose(0, 1).reshape(heads, -1, 128)).amax(-1)
        d = 137 * 2.0 ** -24 * 128 ** -0.5 * to64(size).reshape(len(q), heads * group, 1)[~lost] + 2.0 ** -21
        bound = np.expm1(2 * d + 2 * max(kv_len) * 2.0 ** -24 + 2.0 ** -22) * a
    assert (np.abs(o64 - ref) <= bound).all()


@pytest.mark.parametrize("mine,new,heads,group,page", [
    ([1100, 300, 9, 40], [100, 1, 1, 1], 1, 4, 32),                       # two turns of 32 rows, clusters of four
    ([1500, 20, 3, 1, 70, 5, 9, 600], [200] + [1] * 7, 2, 4, 64),         # four turns, a CTA each
    ([900] + [30] * 9, [100] + [1] * 9, 2, 1, 16),                        # four turns of 16 rows
    ([2000, 2000], [300, 1], 1, 3, 128),                                  # clusters of eight
])
def test_a_request_of_many_turns(kda, mine, new, heads, group, page):
    """Few requests, of which one brings far more rows than the others: its CTAs go over its own keys once a block of rows,
    each turn's tiles where the last turn's partial outputs were."""
    c = build_branches([150], [mine], page, heads, BF16, seed=79)
    q, cu = queries(sum(new), heads * group, BF16, 79), cu_of(new)
    o = call(kda, q, c, new)
    assert kda.kda_get_device_status()[0] == 0
    check(o, q, c, new)
    busy = torch.randn((2048, 2048), device="cuda")
    for i in range(30):
        if i % 2:
            torch.mm(busy, busy)
        again = kda.kda_prefix_attention(q, c["pool"], c["table"], c["slot"], cu, c["kv_len"], c["cu_groups"],
                                         c["prefix_len"], max_tokens=max(new))
        assert torch.equal(again, o)


def test_rows_that_take_longer_than_a_wait(kda):
    """A value that the last token alone sees is not finite, in a request of so many own keys that its rows, computed one by
    one, take longer than the kernels wait for anything (2 s).  The CTA has further requests to go on with: its warps that
    wait meanwhile do not give up.  (The first token's row: fp32 sums of 380,000 terms, one after the other, off by at most
    2^-24 of the sum of the sizes each, above and below.)"""
    B, heads, page, keys, late = 3000, 16, 128, 380000, 7
    new = [2] * B
    c = build_branches([64], [[5] * late + [keys] + [5] * (B - late - 1)], page, 1, BF16, seed=83)
    q = queries(2 * B, heads, BF16, 83)
    want = call(kda, q, c, new)
    row, j = c["slot"][late].item(), 64 + keys - 1
    c["pool"][c["table"][row, j // page].item(), 1, 0, j % page, 5] = float("inf")
    o = call(kda, q, c, new)
    assert kda.kda_get_device_status() == (0, 0)
    first = 2 * late
    assert torch.equal(o[:first], want[:first]) and torch.equal(o[first + 2:], want[first + 2:])
    assert bool((o[first + 1, :, 5] == float("inf")).all())
    at = torch.arange(j, device="cuda")
    kv = c["pool"][c["table"][row].long()[at // page], :, 0, at % page].double()
    p = torch.softmax(q[first].double() @ kv[:, 0].T * 128 ** -0.5, -1)
    ref, a = p @ kv[:, 1], p @ kv[:, 1].abs()
    assert ((o[first].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2 * keys * 2.0 ** -24 + 2.0 ** -12) * a).all()


def test_called_over_and_over(kda):
    """Thirty thousand calls over prefixes of all lengths, single row tiles of few rows: whatever the CTA's warps run into,
    none is left behind by the others (a wait that runs out takes 2 s, and is reported)."""
    rng = np.random.RandomState(89)
    prefix = [int(n) for n in rng.randint(500, 8192, 16)]
    mine = [[int(n) for n in rng.randint(1, 300, 4)] for _ in prefix]
    new = [1] * 64
    c = build_branches(prefix, mine, 64, 8, BF16, seed=89)
    q, cu = queries(64, 96, BF16, 89), cu_of(new)
    want = call(kda, q, c, new)
    o, workspace = torch.empty_like(q), torch.empty(kda.kda_prefix_attention_workspace_size(BF16, 64, 64, 16, 96, 8),
                                                    dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(100):
            kda.kda_prefix_attention(q, c["pool"], c["table"], c["slot"], cu, c["kv_len"], c["cu_groups"], c["prefix_len"],
                                     max_tokens=1, o=o, workspace=workspace)
    for i in range(300):
        graph.replay()
        if i % 20 == 19:  # (the first lost call ends the test)
            assert kda.kda_get_device_status() == (0, 0)
            assert torch.equal(o, want)
            o.fill_(7.0)
