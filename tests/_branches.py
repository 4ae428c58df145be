"""Plain 64-bit implementations (numpy, loops) of the operators that decode branches, and inputs for them."""
import numpy as np
import torch

from tests._cache import D, fork64

MAX_FP32 = float(np.finfo(np.float32).max)


def build_branches(prefix, mine, page, heads, dtype, seed, spare_rows=2, spare_pages=3):
    """A pool whose rows share prefixes: prefix[g] tokens for group g, then mine[g][i] tokens of branch i's own.  Whole
    pages are shared, the one the prefix ends in is a copy in each branch; pages and rows in random order."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.RandomState(seed)
    lens = [p + n for p, ns in zip(prefix, mine) for n in ns]
    pages = sum(p // page for p in prefix) + sum(-(-(p + n) // page) - p // page for p, ns in zip(prefix, mine) for n in ns)
    pages += spare_pages
    names = [int(x) for x in rng.permutation(pages)]
    rows, width = len(lens) + spare_rows, max([-(-n // page) for n in lens] + [0]) + 1
    slot = rng.permutation(rows)[:len(lens)]
    table, kv_len = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
    pool = torch.randn((pages, 2, heads, page, D), generator=g, device="cuda", dtype=dtype)
    b = 0
    for p, ns in zip(prefix, mine):
        shared, first = [names.pop() for _ in range(p // page)], None
        for n in ns:
            own = [names.pop() for _ in range(-(-(p + n) // page) - p // page)]
            table[slot[b], :len(shared) + len(own)] = shared + own
            kv_len[slot[b]] = p + n
            if p % page and own:
                if first is None:
                    first = own[0]
                pool[own[0], :, :, :p % page] = pool[first, :, :, :p % page]
            b += 1
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    cu = np.concatenate([[0], np.cumsum([len(ns) for ns in mine])])
    return dict(pool=pool, table=i32(table), slot=i32(slot), kv_len=i32(kv_len), cu_groups=i32(cu),
                prefix_len=i32(prefix))


def prefix64(q, c, new, scale=D ** -0.5):
    """(o, a) of kda_prefix_attention from its definition: the output and sum_j softmax_j |v_j|."""
    q = q.double().cpu().numpy()
    pool = c["pool"]
    P, _, Hkv, page, _ = pool.shape
    G = q.shape[1] // Hkv
    table, slot, kv_len, cu, prefix = (c[k].cpu().numpy() for k in ("table", "slot", "kv_len", "cu_groups", "prefix_len"))
    o, a, t, pool64 = np.zeros_like(q), np.zeros_like(q), 0, pool.double().cpu().numpy()
    for b, n in enumerate(new):
        g = int(np.searchsorted(cu, b, side="right")) - 1
        length, lp = int(kv_len[slot[b]]), int(prefix[g])
        j = np.arange(length)
        name = np.where(j < lp, table[slot[cu[g]]][j // page], table[slot[b]][j // page]) if length else np.zeros(0, int)
        mapped = (0 <= name) & (name < P)
        kv = pool64[np.where(mapped, name, 0), :, :, j % page]  # [keys, 2, heads, 128]
        for i in range(n):
            seen = mapped & (j <= length - n + i)
            for h in range(q.shape[1]):
                if not seen.any():
                    continue
                s = kv[seen, 0, h // G] @ q[t + i, h] * scale
                e = np.exp(s - s.max())
                e /= e.sum()
                o[t + i, h], a[t + i, h] = e @ kv[seen, 1, h // G], e @ np.abs(kv[seen, 1, h // G])
        t += n
    return o, a


def select64(logits, scores, choices, ended=None, end_token=-1):
    """(parent, token, score, ended) of kda_beam_select from its definition, in 64 bits."""
    x = logits.double().cpu().numpy()
    x = np.minimum(np.where(np.isnan(x), -np.inf, x), MAX_FP32)
    s = scores.double().cpu().numpy()
    s = np.where(np.isnan(s), -np.inf, s)
    over = np.zeros(s.shape, bool) if ended is None else ended.cpu().numpy().astype(bool)
    B, K, V = x.shape
    parent, token = np.full((B, choices), -1), np.full((B, choices), -1)
    score, done = np.full((B, choices), -np.inf), np.zeros((B, choices), bool)
    for b in range(B):
        found = []
        for k in range(K):
            if over[b, k]:
                found.append((-s[b, k], k, 0.0, end_token))
                continue
            top = x[b, k].max()
            if top == -np.inf:
                continue
            lse = top + np.log(np.exp(x[b, k] - top).sum())
            best = np.argsort(-x[b, k], kind="stable")[:choices]
            found += [(-(s[b, k] + (x[b, k, v] - lse)), k, -x[b, k, v], int(v)) for v in best if x[b, k, v] > -np.inf]
        for n, (t, k, _, v) in enumerate(sorted(f for f in found if f[0] < np.inf)[:choices]):
            parent[b, n], token[b, n], score[b, n], done[b, n] = k, v, -t, over[b, k] or v == end_token
    return parent, token, score, done


def beam_slots64(parent, slot, num_rows):
    """(slot, src, dst, refused prompts) of kda_beam_reorder."""
    slot, (B, K) = slot.copy(), slot.shape
    src, dst, bad = np.full((B, K), -1), np.full((B, K), -1), []
    start = slot.copy()
    flat = start.reshape(-1).tolist()
    for b in range(B):
        if any(not 0 <= r < num_rows or flat.count(r) > 1 for r in start[b].tolist()):
            bad.append(b)
            continue
        valid = [0 <= p < K for p in parent[b]]
        free = [int(start[b, k]) for k in range(K) if k not in parent[b].tolist()]
        taken = set()
        for i in range(K):
            p = int(parent[b, i])
            if valid[i] and p not in taken:
                taken.add(p)
                slot[b, i] = start[b, p]
                continue
            slot[b, i] = dst[b, i] = free.pop(0)
            src[b, i] = start[b, p] if valid[i] else -1
    return slot, src.reshape(-1), dst.reshape(-1), bad


def beam_reorder64(parent, slot, table, kv_len, pages, page):
    """The same with the cache: (slot, src, dst, refused prompts, table, kv_len, moves of pages)."""
    slot, src, dst, bad = beam_slots64(parent, slot, table.shape[0])
    move = [(int(s), int(d)) for s, d in zip(src, dst) if d >= 0]
    # a beam without a parent has no tokens: as a fork of a parent that does not exist
    t, n, moves = fork64(table, kv_len, pages, page, [s for s, _ in move], [d for _, d in move])
    for s, d in move:  # (entries past the parent's tokens are its own)
        t[d, -(-int(n[d]) // page):] = -1
    return slot, src, dst, bad, t, n, moves
