"""A beam search as a user's program runs it, step after step: keys and values appended, attention over the prompt and
the beams' own tokens, the best continuations, rows and states reordered.  After each step everything is compared with
what the beams' histories (lists of tokens) say in 64 bits; the tolerances are those of the operators' own tests.
"""
import numpy as np
import pytest
import torch

from tests._branches import select64
from tests._parity import TOL_FP32, assert_close, to64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
VOCAB, HEADS, GROUP, D = 997, 2, 4, 128


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def give_pages(table, kv_len, rows, page, pages):
    """The caller's allocator: rows that grew into a page that they do not have get the lowest that no row names."""
    t, n = table.cpu().numpy(), kv_len.cpu().numpy()
    for r in rows:
        last = (int(n[r]) - 1) // page
        if t[r, last] < 0:
            t[r, last] = min(set(range(pages)) - set(t[t >= 0].tolist()))
    table.copy_(torch.from_numpy(t))


@pytest.mark.parametrize("dtype,page,prompts,steps", [(BF16, 16, [37, 64, 5], 24), (FP32, 32, [50, 1], 20), (BF16, 64, [600], 10)])
def test_beam_search(kda, dtype, page, prompts, steps):
    B, K, rng = len(prompts), 4, np.random.RandomState(sum(prompts))
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(prompts))
    draw = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    wq, wk, wv = draw(VOCAB, HEADS * GROUP, D).to(dtype), draw(VOCAB, HEADS, D).to(dtype), draw(VOCAB, HEADS, D).to(dtype)
    head, state_of = draw(HEADS * GROUP * D, VOCAB) / 8, draw(VOCAB, 64)
    rows, width, pages, end = B * K + 3, max(prompts) // page + steps // page + 3, 400, 7
    pool = torch.full((1, pages, 2, HEADS, page, D), float("nan"), device="cuda", dtype=dtype)  # never written: NaN
    table, kv_len = torch.full((rows, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    state = torch.full((1, rows, 64), float("nan"), device="cuda")

    # the prompts, each in the row of its first beam, and then in all of them
    slot = i32(rng.permutation(rows)[:B * K].reshape(B, K))
    seen = [[int(x) for x in rng.randint(0, VOCAB, n)] for n in prompts]
    first = slot[:, 0].contiguous()
    for b in range(B):
        for j in range(0, prompts[b], page):
            n = min(page, prompts[b] - j)
            kv_len[first[b]] += n
            give_pages(table, kv_len, [int(first[b])], page, pages)
    tokens = i32(sum(seen, []))
    cu = i32(np.concatenate([[0], np.cumsum(prompts)]))
    kda.kda_qk_norm_rope_append(wq[tokens.long()], wk[tokens.long()], wv[tokens.long()], None, None, pool[0], table, first, cu,
                                kv_len, norm=False)
    kda.kda_pages_fork(pool, table, kv_len, first.repeat_interleave(K - 1), slot[:, 1:].reshape(-1).contiguous(), page)
    for b in range(B):
        state[0, slot[b].long()] = state_of[torch.tensor(seen[b], device="cuda")].sum(0)
    assert kda.kda_get_device_status()[0] == 0

    history = [[list(seen[b]) for _ in range(K)] for b in range(B)]
    # (beams that are one and the same to begin with: all but one are marked as not there)
    scores = torch.full((B, K), -float("inf"), device="cuda")
    scores[:, 0] = 0
    ended = torch.zeros((B, K), dtype=torch.uint8, device="cuda")
    token = i32(rng.randint(0, VOCAB, (B, 1)).repeat(K, 1))
    cu_groups, prefix_len = i32(np.arange(B + 1) * K), i32(prompts)
    for step in range(steps):
        over = ended.bool().cpu().numpy()
        new = [0 if x else 1 for x in over.reshape(-1)]
        live = [(b, k) for b in range(B) for k in range(K) if not over[b, k]]
        x = torch.cat([token[b, k:k + 1] for b, k in live]).long() if live else torch.zeros(0, dtype=torch.long, device="cuda")
        at = torch.tensor([int(slot[b, k]) for b, k in live], dtype=torch.long, device="cuda")
        kv_len[at] += 1
        give_pages(table, kv_len, at.tolist(), page, pages)
        state[0, at] += state_of[x]
        for (b, k), t in zip(live, x.tolist()):
            history[b][k].append(t)
        cu = i32(np.concatenate([[0], np.cumsum(new)]))
        flat = slot.reshape(-1)
        q = kda.kda_qk_norm_rope_append(wq[x], wk[x], wv[x], None, None, pool[0], table, flat, cu, kv_len, norm=False)
        o = kda.kda_prefix_attention(q, pool[0], table, flat, cu, kv_len, cu_groups, prefix_len)
        alone = kda.kda_window_attention(q, pool[0], table, flat, cu, kv_len, 2 ** 31 - 1)
        logits = torch.zeros((B * K, VOCAB), device="cuda")
        if live:
            logits[torch.tensor(new, device="cuda").bool()] = o.reshape(len(live), -1).float() @ head
        logits = logits.reshape(B, K, VOCAB)
        parent, token, score, done = kda.kda_beam_select(logits, scores, ended=ended, end_token=end)
        want = select64(logits, scores, K, ended, end)
        src, dst = kda.kda_beam_reorder(parent, slot, pool, table, kv_len, page)
        kda.kda_pages_copy(state, src, dst)
        scores, ended = score, done
        assert kda.kda_get_device_status()[0] == 0

        # attention: from the histories
        for i, (b, k) in enumerate(live):
            h = torch.tensor(history[b][k], device="cuda")
            qs, ks, vs = to64(wq[x[i]]).reshape(HEADS, GROUP, D), to64(wk[h]), to64(wv[h])
            s = np.einsum("hgd,jhd->hgj", qs, ks) * D ** -0.5
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            ref = np.einsum("hgj,jhd->hgd", p, vs).reshape(-1, D)
            for got in (to64(o[i]), to64(alone[i])):
                if dtype is FP32:
                    assert_close(got, ref, TOL_FP32, "o")
                else:
                    a = np.einsum("hgj,jhd->hgd", p, np.abs(vs)).reshape(-1, D)
                    assert (np.abs(got - ref) <= 2.0 ** -8 * (a + np.abs(ref)) + 2.0 ** -12 * a).all()
        # selection, and the histories go with the beams
        np.testing.assert_array_equal(parent.cpu().numpy(), want[0])
        np.testing.assert_array_equal(token.cpu().numpy(), want[1])
        np.testing.assert_array_equal(done.bool().cpu().numpy(), want[3])
        np.testing.assert_allclose(to64(score), want[2], rtol=0, atol=2.0 ** -19 + 2.0 ** -23 * 40 * steps)
        history = [[list(history[b][int(k)]) for k in want[0][b]] for b in range(B)]
        # the cache: whatever rows the beams have, they hold these histories; so do their states
        names, lens = table.cpu().numpy(), kv_len.cpu().numpy()
        assert len(set(flat.tolist())) == B * K
        for b in range(B):
            for k in range(K):
                r, h = int(slot[b, k]), torch.tensor(history[b][k], device="cuda")
                assert lens[r] == len(history[b][k])
                j = np.arange(len(history[b][k]))
                page_of, inside = torch.tensor(names[r][j // page], device="cuda").long(), torch.tensor(j % page, device="cuda")
                assert torch.equal(pool[0][page_of, 0, :, inside], wk[h]) and torch.equal(pool[0][page_of, 1, :, inside], wv[h])
                # (sums of the same terms, in fp32 one by one and at once: half a step of the sum's size a term)
                size = float(state_of[h].abs().sum(0).max())
                assert float((state[0, r] - state_of[h].sum(0)).abs().max()) <= 2 * len(h) * 2.0 ** -24 * size
        in_use = names[flat.cpu().numpy()]
        assert len(set(in_use[in_use >= 0].tolist())) <= sum(p // page for p in prompts) + B * K * (1 + -(-steps // page) + 1)
    assert step == steps - 1
