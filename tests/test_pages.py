"""Copy, fork, release and compaction of cache pages: whole numbers and bytes, all exact."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests._cache import compact64, fork64, release64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make(R, M, P, page, seed, layers=2, fill=0.5, share=True, shape=(2, 1, 128)):
    """Rows of random lengths over distinct pages (some shared with an earlier row)."""
    rng = np.random.RandomState(seed)
    table, kv_len = np.full((R, M), -1, np.int32), np.zeros(R, np.int32)
    names = list(rng.permutation(P))
    for r in range(R):
        n = int(rng.randint(0, M * page + 1) * fill)
        c = -(-n // page)
        if c > len(names):
            break
        table[r, :c] = [names.pop() for _ in range(c)]
        kv_len[r] = n
        if share and r and rng.rand() < 0.3 and c:
            k = rng.randint(1, c + 1)
            table[r, :k] = table[r - 1, :k]
    pool = torch.arange(layers * P * int(np.prod(shape)), device="cuda", dtype=torch.int32).view(layers, P, *shape)
    return pool, table, kv_len


def apply(pool, moves):
    want = pool.clone()
    for s, d in moves:
        want[:, d] = pool[:, s]
    return want


@pytest.mark.parametrize("shape", [(4,), (12,), (2, 1, 4096), (3, 1000)])
@pytest.mark.parametrize("layers", [1, 3])
def test_copy(kda, shape, layers):
    P = 40
    pool = torch.arange(layers * P * int(np.prod(shape)), device="cuda", dtype=torch.int32).view(layers, P, *shape)
    src, dst = [3, 39, 7, -1, 9, 40], [0, 1, 2, 5, -3, 6]
    want = apply(pool, list(zip(src, dst))[:3])
    kda.kda_pages_copy(pool, i32(src), i32(dst))
    assert torch.equal(pool, want)
    kda.kda_pages_copy(pool, i32([]), i32([]))
    assert torch.equal(pool, want)


def test_copy_of_recurrent_state_rows(kda):
    """A row of a KDA state pool is a page: a request takes a read-only snapshot into its own row."""
    pool = torch.randn((1, 6, 2, 128, 128), device="cuda")
    want = pool[0, 4].clone()
    kda.kda_pages_copy(pool, i32([4]), i32([1]))
    assert torch.equal(pool[0, 1], want)


@pytest.mark.parametrize("R,M,P,page", [(2, 1, 4, 16), (5, 7, 31, 16), (40, 33, 700, 64), (300, 9, 3000, 128), (9, 4, 5000, 16)])
@pytest.mark.parametrize("forks", [1, 2, "third"])
def test_fork(kda, R, M, P, page, forks):
    pool, table, kv_len = make(R, M, P, page, seed=R + P)
    F = max(1, R // 3) if forks == "third" else min(forks, R - 1)
    rng = np.random.RandomState(F)
    rows = rng.permutation(R)
    child, parent = rows[:F], rng.choice(rows[F:], F)
    t, n, moves = fork64(table, kv_len, P, page, parent, child)
    dt, dn, got = i32(table), i32(kv_len), pool.clone()
    for _ in range(2):  # what the children named is released, so a second call changes nothing
        kda.kda_pages_fork(got, dt, dn, i32(parent), i32(child), page)
        assert np.array_equal(dt.cpu().numpy(), t) and np.array_equal(dn.cpu().numpy(), n)
        assert torch.equal(got, apply(pool, moves))
    assert kda.kda_get_device_status()[0] == 0


def test_fork_more_than_a_thousand(kda):
    R, M, P, page = 2500, 2, 6000, 16
    pool, table, kv_len = make(R, M, P, page, seed=1, share=False)
    child, parent = np.arange(1250, 2500), np.arange(1250)
    t, n, moves = fork64(table, kv_len, P, page, parent, child)
    dt, dn = i32(table), i32(kv_len)
    want = apply(pool, moves)
    kda.kda_pages_fork(pool, dt, dn, i32(parent), i32(child), page)
    assert np.array_equal(dt.cpu().numpy(), t) and np.array_equal(dn.cpu().numpy(), n)
    assert torch.equal(pool, want)


def test_fork_without_pages_or_rows_is_refused(kda):
    """Three part-filled forks and one free page; a parent and a child out of range; a row forked to itself."""
    table = np.array([[0, 1], [2, 3], [4, -1], [-1, -1], [-1, -1], [-1, -1], [-1, -1]], np.int32)
    kv_len = np.array([20, 32, 5, 0, 0, 9, 0], np.int32)
    pool = torch.arange(6 * 128, device="cuda", dtype=torch.int32).view(1, 6, 128)
    parent, child = np.array([0, 0, 2, 9, 1, 1, 1]), np.array([3, 4, 5, 6, -2, 1, 7])
    t, n, moves = fork64(table, kv_len, 6, 16, parent, child)
    assert moves == [(1, 5)]
    dt, dn = i32(table), i32(kv_len)
    want = apply(pool, moves)
    kda.kda_pages_fork(pool, dt, dn, i32(parent), i32(child), 16)
    code, detail = kda.kda_get_device_status()
    assert code == 6 and detail in (1, 2, 3, 4, 5, 6)
    assert np.array_equal(dt.cpu().numpy(), t) and np.array_equal(dn.cpu().numpy(), n)
    assert torch.equal(pool, want)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 4), (50, 100), (10 ** 6, 0), (2 ** 31 - 1, 2 ** 31 - 1), (17, 16)])
def test_release(kda, window, sinks):
    R, M, page = 23, 40, 16
    _, table, kv_len = make(R, M, 900, page, seed=window % 97)
    rows = [0, 5, 22, 5, 7]
    t, n = release64(table, kv_len, rows, page, window, sinks)
    dt, dn = i32(table), i32(kv_len)
    kda.kda_pages_release(dt, dn, i32(rows), page, window, sinks)
    assert kda.kda_get_device_status()[0] == 0
    assert np.array_equal(dt.cpu().numpy(), t) and np.array_equal(dn.cpu().numpy(), n)
    kda.kda_pages_release(dt, dn, i32([R, 3]), page)
    assert kda.kda_get_device_status() == (6, 0)
    t, n = release64(t, n, [3], page, 0, 0)
    assert np.array_equal(dt.cpu().numpy(), t) and np.array_equal(dn.cpu().numpy(), n)


@pytest.mark.parametrize("R,M,P", [(1, 1, 1), (3, 5, 33), (40, 33, 900), (7, 3, 64), (200, 20, 100000)])
@pytest.mark.parametrize("fill", [0.0, 0.2, 1.0])
def test_compact(kda, R, M, P, fill):
    pool, table, kv_len = make(R, M, P, 16, seed=P, fill=fill, shape=(8,))
    if fill == 0.2:
        table[R // 2, 0] = P + 3  # names no page: kept as it is
    t, L, moves = compact64(table, P)
    want = apply(pool, moves)
    for place in (False, True):
        dt, got = i32(table), pool.clone()
        out, live = kda.kda_pages_compact(got, dt, table_out=None if place else torch.empty_like(dt))
        assert live.item() == L and np.array_equal(out.cpu().numpy(), t) and torch.equal(got, want)
        assert place or np.array_equal(dt.cpu().numpy(), table)
        again, live = kda.kda_pages_compact(got, out)
        assert np.array_equal(again.cpu().numpy(), t) and torch.equal(got, want)


def test_pages_at_the_limit_and_past_32_bits(kda):
    """2^20 pages, and a pool of more than 4 GB: offsets are 64-bit."""
    P = 1 << 20
    pool = torch.empty((1, P, 1056), dtype=torch.int32, device="cuda")  # 4.4 GB
    table = np.array([[P - 1, P - 2, 5, 0]], np.int32)
    for p in (P - 1, P - 2, 5, 0):
        pool[0, p] = p
    dt = i32(table)
    _, live = kda.kda_pages_compact(pool, dt)
    t, L, moves = compact64(table, P)
    assert live.item() == L == 4 and np.array_equal(dt.cpu().numpy(), t)
    for s, d in moves:
        assert bool((pool[0, d] == s).all())


def test_fork_then_attention_sees_the_same_row(kda):
    """A branch answers as its parent until it appends; its append does not reach the parent."""
    from tests._cache import build_cache, cu_of, queries
    c = build_cache([100], 16, 1, torch.bfloat16, seed=3, spare_rows=2, spare_pages=4)
    parent = c["slot"].item()
    child = [r for r in range(3) if r != parent][0]
    q = queries(1, 8, torch.bfloat16, 3)
    ask = lambda row: kda.kda_window_attention(q, c["pool"], c["table"], i32([row]), cu_of([1]), c["kv_len"], 64, 4, max_tokens=1)
    kda.kda_pages_fork(c["pool"][None], c["table"], c["kv_len"], i32([parent]), i32([child]), 16)
    want = ask(parent)
    assert torch.equal(ask(child), want)
    c["kv_len"][child] += 1
    k = queries(1, 1, torch.bfloat16, 5)
    kda.kda_qk_norm_rope_append(q, k, k, None, None, c["pool"], c["table"], i32([child]), cu_of([1]), c["kv_len"])
    assert torch.equal(ask(parent), want) and not torch.equal(ask(child), want)
    kda.kda_pages_release(c["table"], c["kv_len"], i32([child]), 16)
    kda.kda_pages_compact(c["pool"][None], c["table"])
    assert torch.equal(ask(parent), want)
    assert kda.kda_get_device_status()[0] == 0


BOUNDARY = """
import torch
from gated_delta_rule_kda_gb300 import kda
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
# the fork's plan holds a bit a page and a bit a row, the compaction's a bit a page, both 128 bytes beside them
for P, R in ((392128, 33), (392160, 33), (392161, 33), (393152, 33), (393153, 33)):
    pool = torch.zeros((1, P, 4), dtype=torch.int32, device="cuda")
    pool[0, 7], table, kv_len = 9, torch.full((R, 1), -1, dtype=torch.int32, device="cuda"), i32([0] * R)
    table[2, 0], kv_len[2] = 7, 5
    kda.kda_pages_fork(pool, table, kv_len, i32([2]), i32([4]), 16)
    assert table[4, 0].item() == 0 and kv_len[4].item() == 5 and bool((pool[0, 0] == 9).all()), P
for P in (392192, 392193, 393216, 393217):
    pool = torch.zeros((1, P, 4), dtype=torch.int32, device="cuda")
    pool[0, P - 1] = 9
    table, live = kda.kda_pages_compact(pool, i32([[P - 1]]))
    assert live.item() == 1 and table.item() == 0 and bool((pool[0, 0] == 9).all()), P
assert kda.kda_get_device_status()[0] == 0
"""


def test_plans_around_the_default_shared_memory_limit(kda):
    """Pools whose bitmap and the plan's few static bytes lie below, at and above 48 KB together, in a process
    that has made no larger call before."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", BOUNDARY], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("length,shared", [(32, 2), (20, 1), (0, 0), (1, 0), (64, 4), (63, 3)])
def test_fork_takes_no_page_past_the_parent_s_tokens(kda, length, shared):
    """A parent with pages mapped past its tokens (reserved ahead, or left when its length was lowered): the child
    shares those that are full and has a page of its own for a part-filled one; the rest stays the parent's."""
    page, names = 16, [6, 1, 8, 3]
    table = np.array([names, [-1] * 4, [2, 9, 9, -1]], np.int32)
    pool = torch.arange(10 * 64, device="cuda", dtype=torch.int32).view(1, 10, 64)
    want_row, want = [-1] * 4, pool.clone()
    want_row[:shared] = names[:shared]
    if length % page:
        want_row[shared] = 0  # the lowest page that no row names
        want[:, 0] = pool[:, names[shared]]
    dt, dn = i32(table), i32([length, 7, 20])
    kda.kda_pages_fork(pool, dt, dn, i32([0]), i32([1]), page)
    assert dt.tolist() == [names, want_row, table[2].tolist()] and dn.tolist() == [length, length, 20]
    assert torch.equal(pool, want)
    assert kda.kda_get_device_status()[0] == 0


@pytest.mark.parametrize("length", [32, 20])
def test_branches_of_a_row_with_pages_ahead_append_apart(kda, length):
    """Both rows grow across the page edge: each finds its own keys and values, and a branch that has not been given
    a page yet is refused instead of writing the parent's."""
    page, steps = 16, 20
    g = torch.Generator(device="cuda")
    g.manual_seed(length)
    pool = torch.randn((1, 12, 2, 1, page, 128), generator=g, device="cuda")
    table, kv_len = i32([[3, 4, 5, 6], [-1] * 4]), i32([length, 0])
    kda.kda_pages_fork(pool, table, kv_len, i32([0]), i32([1]), page)
    x = torch.randn((2, steps, 2, 1, 128), generator=g, device="cuda")  # row, step, key / value

    def append(t, rows):
        n = len(rows)
        kda.kda_qk_norm_rope_append(x[rows, t, 0], x[rows, t, 0], x[rows, t, 1], None, None, pool[0], table, i32(rows),
                                    i32(list(range(n + 1))), kv_len, norm=False)

    spare = iter([10, 11])
    for t in range(steps):
        j = length + t
        kv_len[:] = j + 1
        if table[1, j // page].item() < 0:
            before = pool.clone()
            append(t, [1])
            assert kda.kda_get_device_status()[0] == 6 and torch.equal(pool, before)
            table[1, j // page] = next(spare)
        append(t, [0, 1])
    assert kda.kda_get_device_status()[0] == 0
    for r in range(2):
        for t in range(steps):
            j = length + t
            assert torch.equal(pool[0, table[r, j // page].item(), :, :, j % page], x[r, t])
