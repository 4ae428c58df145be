"""Sliding-window attention over the paged cache against a 64-bit plain implementation.

Tolerances, elementwise.  bf16: a probability rounded to bf16 is off by at most 2^-8 of itself and
so is the rounded output; the fp32 parts (128-term scores, exponentials, sums) stay below 2^-12 of
it.  With a = sum_j softmax_j |v_j| that is |o - ref| <= 2^-8 (a + |ref|) + 2^-12 a.
fp32: max-abs over rms 1e-5, the bound of every fp32 path here.
"""
import numpy as np
import pytest
import torch

from tests._cache import attention64, build_cache, cu_of, queries
from tests._parity import TOL_FP32, assert_close, to64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def call(kda, q, c, new, window, sinks, **kw):
    kw.setdefault("max_tokens", max(list(new) + [1]))
    o = kda.kda_window_attention(q, c["pool"], c["table"], c["slot"], cu_of(new), c["kv_len"], window, sinks, **kw)
    torch.cuda.synchronize()
    return o


def check(o, q, c, new, window, sinks, scale=128 ** -0.5):
    ref, a = attention64(q, c, new, 2 ** 31 if window is None else window, sinks, scale)
    o64 = to64(o)
    if o.dtype == FP32:
        return assert_close(o64, ref, TOL_FP32, "o")
    assert np.isfinite(o64).all()
    over = np.abs(o64 - ref) - (2.0 ** -8 * (a + np.abs(ref)) + 2.0 ** -12 * a)
    assert over.max(initial=-1.0) <= 1e-30, f"{over.max():.3e} over the bound at {np.unravel_index(over.argmax(), over.shape)}"


# (tokens of each request, tokens before them, kv heads, group, page, window, sinks)
SHAPES = [
    ([1], [0], 1, 1, 16, 1, 0),                                   # one token that sees itself
    ([1], [499], 2, 12, 64, 100, 4),                              # decode, window and sinks
    ([1] * 5, [0, 15, 16, 17, 300], 2, 8, 16, 33, 5),             # page edges
    ([1, 1, 1], [1000, 63, 700], 1, 16, 128, 5000, 0),            # nothing out of the window
    ([4, 4, 1, 0, 3], [40, 0, 700, 9, 128], 2, 3, 32, 129, 1),    # a few tokens each, one none
    ([2, 7], [900, 333], 1, 8, 64, 200, 70),                      # sinks over a page
    ([16], [1500], 1, 4, 64, 1024, 4),                            # 64 rows a kv head
    ([17, 3], [130, 5], 2, 5, 16, 50, 3),
    ([64, 1, 33], [0, 200, 7], 1, 2, 32, 64, 0),
    ([300], [0], 2, 4, 64, 2 ** 31 - 1, 0),                       # plain causal
    ([130, 259], [300, 0], 1, 1, 128, 77, 2),
    ([200], [513], 1, 12, 16, 128, 9),
    ([150], [0], 1, 6, 64, 1, 0),                                 # every token sees itself only
    ([140], [260], 1, 7, 32, 60, 150),                            # more sinks than window
    ([9], [20], 1, 128, 32, 12, 2),                               # one kv head of 128 query heads
    ([40], [90], 1, 33, 64, 50, 0),
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_64_bits(kda, shape, dtype):
    new, old, heads, group, page, window, sinks = shape
    c = build_cache([a + b for a, b in zip(new, old)], page, heads, dtype, seed=len(new) * 31 + page)
    q = queries(sum(new), heads * group, dtype, 3)
    o = call(kda, q, c, new, window, sinks)
    assert kda.kda_get_device_status()[0] == 0
    check(o, q, c, new, window, sinks)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new,old,group", [([1, 1], [70, 200], 8), ([6], [100], 8), ([260], [40], 4)])
def test_large_max_tokens_gives_the_same_answer(kda, new, old, group, dtype):
    """max_tokens is a promise, not a size: a loose one may take another kernel, not another answer."""
    c = build_cache([a + b for a, b in zip(new, old)], 32, 2, dtype, seed=5)
    q = queries(sum(new), 2 * group, dtype, 5)
    for most in (max(new), 300, 100000):
        check(call(kda, q, c, new, 90, 3, max_tokens=most), q, c, new, 90, 3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new,length", [([3], 1), ([5], 0), ([1], 0), ([300], 20), ([200], 0)])
def test_tokens_before_the_row_see_nothing_and_give_zero(kda, new, length, dtype):
    """A row shorter than the step's tokens: the first ones have a negative index."""
    c = build_cache([length], 16, 1, dtype, seed=9)
    q = queries(sum(new), 4, dtype, 9)
    o = call(kda, q, c, new, 7, 2)
    assert bool((o[: new[0] - length] == 0).all())
    check(o, q, c, new, 7, 2)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new,old", [([1, 2], [300, 431]), ([90, 140], [300, 431])])
def test_unmapped_pages_hold_no_keys(kda, new, old, dtype):
    """Entries of -1 or past the pool inside, before and at the end of the visible range; the second
    request has none left."""
    lens = [a + b for a, b in zip(new, old)]
    c = build_cache(lens, 32, 2, dtype, seed=11)
    table, slot = c["table"], c["slot"].tolist()
    table[slot[0], 3] = -1
    table[slot[0], (lens[0] - 1) // 32] = c["pool"].shape[0]
    table[slot[1], :] = -7
    q = queries(sum(new), 6, dtype, 11)
    o = call(kda, q, c, new, 250, 40)
    assert kda.kda_get_device_status()[0] == 0
    assert bool((o[new[0]:] == 0).all())
    check(o, q, c, new, 250, 40)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("new,old,group", [([1], [200], 8), ([3], [200], 4), ([70], [200], 2), ([150], [0], 12)])
def test_values_outside_the_visible_keys_do_not_reach_the_output(kda, new, old, group, value, dtype):
    """Everything that no token of the step sees (before the window, behind the row's last token, other
    pages) is set to NaN, an infinity, or the largest values: the output is finite and right."""
    length, page, window, sinks = new[0] + old[0], 32, 40, 5
    c = build_cache([length], page, 2, dtype, seed=13)
    q = queries(new[0], 2 * group, dtype, 13)
    row = c["table"][c["slot"][0].item()].tolist()
    named = set(row) - {-1}
    for p in range(c["pool"].shape[0]):
        if p not in named:
            c["pool"][p] = value
    for j in range((length + page - 1) // page * page):
        if j >= length or not (j > old[0] - window or j < sinks):
            c["pool"][row[j // page], :, :, j % page] = value
    clean = {**c, "pool": torch.nan_to_num(c["pool"].float(), 0.0, 0.0, 0.0).to(dtype)}
    o = call(kda, q, c, new, window, sinks)
    check(o, q, clean, new, window, sinks)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("new,group", [([6], 2), ([100], 3), ([400], 2)])
def test_a_later_or_earlier_token_s_nan_stays_its_own(kda, new, group, value, dtype):
    """One key/value of the step itself is not finite: tokens that see it give non-finite rows, tokens
    before it and those whose window has passed it are untouched."""
    n, window = new[0], 50
    bad = n // 2
    c = build_cache([n + 30], 16, 1, dtype, seed=17)
    row = c["table"][c["slot"][0].item()].tolist()
    j = 30 + bad
    clean = {**c, "pool": c["pool"].clone()}
    c["pool"][row[j // 16], 1, :, j % 16, 3] = value
    q = queries(n, group, dtype, 17)
    o = call(kda, q, c, new, window, 0)
    sees = [bad <= i < bad + window for i in range(n)]
    assert not bool(torch.isfinite(o[sees][:, :, 3].float()).any())
    keep = [not s for s in sees]
    ref, a = attention64(q, clean, new, window, 0)
    got = to64(o)
    if dtype == FP32:
        assert_close(got[keep], ref[keep], TOL_FP32, "unseeing rows")
    else:
        assert (np.abs(got - ref) <= 2.0 ** -8 * (a + np.abs(ref)) + 2.0 ** -12 * a + 1e-30)[keep].all()


@pytest.mark.parametrize("new,old", [([1, 1], [100, 100]), ([80, 80], [50, 50])])
def test_rows_may_be_shared_and_calls_repeat_bit_for_bit(kda, new, old):
    c = build_cache([new[0] + old[0]], 64, 2, BF16, seed=19)
    c["slot"] = c["slot"][[0, 0]].contiguous()
    q = queries(sum(new), 16, BF16, 19)
    q[new[0]:] = q[: new[0]]
    o = call(kda, q, c, new, 64, 4)
    assert torch.equal(o[: new[0]], o[new[0]:])
    assert torch.equal(o, call(kda, q, c, new, 64, 4))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new", [[2, 1, 2], [70, 1, 90]])
def test_refused_requests_leave_their_rows(kda, new, dtype):
    c = build_cache([n + 20 for n in new], 16, 1, dtype, seed=23)
    q = queries(sum(new), 4, dtype, 23)
    good = c["slot"].clone(), c["kv_len"].clone()
    want = call(kda, q, c, new, 30, 0)
    for what in ("slot", "kv_len", "max_tokens"):
        c["slot"], c["kv_len"] = good[0].clone(), good[1].clone()
        kw = {}
        if what == "slot":
            c["slot"][1] = c["table"].shape[0]
            refused = 1
        elif what == "kv_len":
            c["kv_len"][c["slot"][1].item()] = c["table"].shape[1] * 16 + 1
            refused = 1
        else:
            kw["max_tokens"] = new[2] - 1
            refused = 2 if new[0] < new[2] else 0
        o = torch.full_like(q, -7.0)
        call(kda, q, c, new, 30, 0, o=o, **kw)
        code, detail = kda.kda_get_device_status()
        assert code == 6 and detail in ({refused} if what != "max_tokens" else {0, 2})
        at = np.concatenate([[0], np.cumsum(new)])
        for b, n in enumerate(new):
            rows = o[at[b]:at[b + 1]]
            if (b == 1 and what != "max_tokens") or (what == "max_tokens" and n > kw["max_tokens"]):
                assert bool((rows == -7.0).all()), (what, b)
            else:
                assert_same(rows, want[at[b]:at[b + 1]])


def assert_same(x, y):
    # a request's rows, whatever kernel or split took them: within one rounding of the type
    tol = 2.0 ** -6 if x.dtype == BF16 else 1e-5
    assert bool(((x.float() - y.float()).abs() <= tol * (1 + y.float().abs())).all())


@pytest.mark.parametrize("new", [[1, 1], [33, 40]])
def test_pages_past_32_bits(kda, new):
    """A pool of more than 2^32 elements; the rows' pages are its last ones."""
    heads, page = 8, 64
    pages = 2 ** 32 // (2 * heads * page * 128) + 40
    pool = torch.empty((pages, 2, heads, page, 128), dtype=BF16, device="cuda")
    small = build_cache([n + 200 for n in new], page, heads, BF16, seed=29)
    n = small["pool"].shape[0]
    pool[pages - n:] = small["pool"]
    c = {**small, "pool": pool, "table": torch.where(small["table"] >= 0, small["table"] + (pages - n), -1).to(torch.int32)}
    q = queries(sum(new), heads, BF16, 29)
    assert torch.equal(call(kda, q, c, new, 150, 4), call(kda, q, small, new, 150, 4))
    check(call(kda, q, small, new, 150, 4), q, small, new, 150, 4)


@pytest.mark.parametrize("new", [[1, 1], [100, 30]])
def test_another_stream_and_scale(kda, new):
    c = build_cache([n + 60 for n in new], 32, 2, BF16, seed=31)
    q = queries(sum(new), 4, BF16, 31)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cu = cu_of(new)
    torch.cuda.synchronize()
    o = kda.kda_window_attention(q, c["pool"], c["table"], c["slot"], cu, c["kv_len"], 50, 2, 0.03,
                                 max_tokens=max(new), stream=s)
    s.synchronize()
    check(o, q, c, new, 50, 2, 0.03)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-30, 2.0])
@pytest.mark.parametrize("new", [[1, 1], [100, 30]])
def test_any_scale(kda, new, scale, dtype):
    """A negative scale turns the order of the keys round; zero weighs the visible ones alike."""
    c = build_cache([n + 60 for n in new], 32, 2, dtype, seed=33)
    q = queries(sum(new), 4, dtype, 33)
    if scale == 2.0:
        q = q * 0.25
    check(call(kda, q, c, new, 50, 2, scale=scale), q, c, new, 50, 2, scale)


def test_no_tokens_and_many_requests(kda):
    c = build_cache([3] * 100, 16, 1, BF16, seed=37)
    q = queries(0, 4, BF16, 37)
    assert call(kda, q, c, [0] * 100, 5, 0, max_tokens=1).shape == (0, 4, 128)
    new = [(i * 7) % 3 for i in range(100)]
    q = queries(sum(new), 4, BF16, 37)
    for most in (2, 1000):
        check(call(kda, q, c, new, 5, 0, max_tokens=most), q, c, new, 5, 0)


def test_decode_of_ragged_lengths_over_many_splits(kda):
    """Long rows beside short ones in one step, at sizes where a row is read by several CTAs."""
    lens = [5000, 1, 129, 3000, 64, 65]
    for group, n in ((8, 1), (3, 5)):
        new = [min(n, x) for x in lens]
        c = build_cache(lens, 64, 1, BF16, seed=41)
        q = queries(sum(new), group, BF16, 41)
        for window, sinks in ((None, 0), (2048, 100)):
            check(call(kda, q, c, new, window, sinks), q, c, new, window, sinks)


@pytest.mark.parametrize("new,group", [([40], 4), ([9, 33, 0], 5), ([70], 1), ([2], 33)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (1500, 70)])
@pytest.mark.parametrize("bad", [False, True])
def test_short_steps_behind_long_rows(kda, new, group, window, sinks, bad):
    """Few rows over many keys: CTAs share an item's keys and join their results.  With `bad`, a value of the
    first request's first token is NaN: its other tokens see it too, the other requests do not."""
    c = build_cache([n + 3000 + 100 * i for i, n in enumerate(new)], 32, 2, BF16, seed=47)
    q = queries(sum(new), 2 * group, BF16, 47)
    clean = {**c, "pool": c["pool"].clone()}
    if bad:
        j = 3000
        c["pool"][int(c["table"][int(c["slot"][0]), j // 32]), 1, 0, j % 32, 7] = float("nan")
    o = call(kda, q, c, new, window, sinks)
    assert torch.equal(torch.isnan(o), torch.isnan(call(kda, q, c, new, window, sinks)))
    if bad:
        seen = torch.zeros_like(o, dtype=torch.bool)
        seen[: new[0], :group, 7] = True
        assert torch.equal(torch.isnan(o), seen)
        o = torch.where(seen, call(kda, q, clean, new, window, sinks), o)
    check(o, q, clean, new, window, sinks)


def test_large_scores(kda):
    """Scores of some hundreds, growing and falling along the row: the running maximum keeps every
    exponential in range.  q and k are scaled so that products are exact in bf16."""
    n, length = 40, 700
    c = build_cache([length], 64, 1, BF16, seed=43)
    row = c["table"][c["slot"][0].item()].tolist()
    for j in range(length):
        c["pool"][row[j // 64], 0, :, j % 64] *= 0.25 * (1 + j // 64 % 5)
    q = 8 * queries(n, 4, BF16, 43)
    for new in ([n], [2]):
        check_large(call(kda, q[: new[0]].contiguous(), c, new, 600, 3), q[: new[0]], c, new)


def check_large(o, q, c, new):
    # scores up to S carry an absolute error of about 128 2^-24 S, the same relative error on e^s
    ref, a = attention64(q, c, new, 600, 3)
    err = np.abs(to64(o) - ref)
    assert (err <= 2.0 ** -8 * (a + np.abs(ref)) + 2.0 ** -8 * a).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new", [1, 3, 70])
@pytest.mark.parametrize("page,behind", [(64, 64), (16, 16), (16, 100)])
def test_rows_up_to_the_last_index_that_is_accepted(kda, page, behind, new, dtype):
    """A row that ends within 128 tokens of 2^31, with pages for its first tokens and for those near its end: the answer
    of a short row that holds the same keys at the same places."""
    far, near, window, sinks = 2 ** 31 - behind, 1024 - behind, 90, 5
    small = build_cache([near], page, 2, dtype, seed=53)
    q = queries(new, 6, dtype, 53)
    width = (2 ** 31 - 1) // page
    row = small["table"][small["slot"][0].item()]
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = row[0]
    last = -(-near // page)
    first = (near - new - window) // page
    shift = (2 ** 31 - 1024) // page  # the end of the one row on the other's
    table[0, first + shift: last + shift] = row[first:last]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = dict(pool=small["pool"], table=table, slot=zero, kv_len=zero + far)
    o = call(kda, q, c, [new], window, sinks)
    assert kda.kda_get_device_status()[0] == 0
    check(o, q, small, [new], window, sinks)
