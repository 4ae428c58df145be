"""Plain 64-bit implementations (numpy, loops) of the paged-cache operators, and inputs for them."""
import numpy as np
import torch

D = 128


def build_cache(lens, page, heads, dtype, seed, spare_rows=2, spare_pages=3, pool_pages=None):
    """A pool whose rows have these lengths, pages in random order: dict of CUDA tensors."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.RandomState(seed)
    counts = [-(-n // page) for n in lens]
    rows, width = len(lens) + spare_rows, max(counts + [0]) + 1
    pages = pool_pages or sum(counts) + spare_pages
    names = rng.permutation(pages)[:sum(counts)]
    slot = rng.permutation(rows)[:len(lens)]
    table, kv_len = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
    at = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        table[slot[b], :c] = names[at:at + c]
        kv_len[slot[b]] = n
        at += c
    pool = torch.randn((pages, 2, heads, page, D), generator=g, device="cuda", dtype=dtype)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    return dict(pool=pool, table=i32(table), slot=i32(slot), kv_len=i32(kv_len))


def cu_of(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")


def queries(total, heads, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 77)
    return torch.randn((total, heads, D), generator=g, device="cuda", dtype=dtype)


def attention64(q, cache, new, window, sinks, scale=D ** -0.5):
    """(o, a): the output and sum_j softmax_j |v_j|, both [T, Hq, 128] float64."""
    q = q.double().cpu().numpy()
    pool = cache["pool"]
    P, _, Hkv, page, _ = pool.shape
    G = q.shape[1] // Hkv
    table, slot, kv_len = (cache[k].cpu().numpy() for k in ("table", "slot", "kv_len"))
    o, a, t = np.zeros_like(q), np.zeros_like(q), 0
    for b, n in enumerate(new):
        row, length = slot[b], int(kv_len[slot[b]])
        names = [int(x) for x in table[row, : -(-length // page)]]
        mapped = np.repeat([0 <= x < P for x in names], page)[:length]
        idx = torch.tensor([x if 0 <= x < P else 0 for x in names], dtype=torch.long, device=pool.device)
        kv = pool[idx].double().cpu().numpy() if len(names) else np.zeros((0, 2, Hkv, page, D))
        kv = kv.transpose(1, 2, 0, 3, 4).reshape(2, Hkv, -1, D)[:, :, :length]
        for i in range(n):
            p = length - n + i
            j = np.arange(length)
            seen = np.nonzero((j <= p) & ((j > p - window) | (j < sinks)) & mapped)[0] if length else []
            if len(seen) == 0:
                continue
            for h in range(q.shape[1]):
                s = kv[0, h // G][seen] @ q[t + i, h] * scale
                e = np.exp(s - s.max())
                e /= e.sum()
                v = kv[1, h // G][seen]
                o[t + i, h], a[t + i, h] = e @ v, e @ np.abs(v)
        t += n
    return o, a


def rope64(x, weight, table, positions, rotary, interleaved, norm, eps=1e-6):
    x = x.double().cpu().numpy().copy()
    if norm:
        x /= np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x *= weight.double().cpu().numpy()
    cs = table.double().cpu().numpy()[positions.cpu().numpy()]
    y = x.copy()
    for i in range(rotary // 2):
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        c, s = cs[:, i, 0][:, None], cs[:, i, 1][:, None]
        y[..., u], y[..., v] = x[..., u] * c - x[..., v] * s, x[..., v] * c + x[..., u] * s
    return y


def fork64(table, kv_len, pages, page, parent, child):
    """(table, kv_len, moves) of numpy int arrays; refused forks leave an empty child row."""
    table, kv_len = table.copy(), kv_len.copy()
    R, M = table.shape
    good = [0 <= p < R and 0 <= c < R and p != c and 0 <= kv_len[p] <= M * page for p, c in zip(parent, child)]
    released = {c for p, c in zip(parent, child) if 0 <= c < R and p != c}
    live = {int(x) for r in range(R) if r not in released for x in table[r] if 0 <= x < pages}
    free = [x for x in range(pages) if x not in live]
    rows, moves = {}, []
    for p, c, ok in zip(parent, child, good):
        if not (0 <= c < R) or p == c:
            continue
        row, n = np.full(M, -1, table.dtype), 0
        if ok:
            row, n = table[p].copy(), int(kv_len[p])
            old = int(row[n // page]) if n % page else -1
            if 0 <= old < pages:
                if free:
                    row[n // page] = free.pop(0)
                    moves.append((old, int(row[n // page])))
                else:
                    row, n = np.full(M, -1, table.dtype), 0
        rows[c] = (row, n)
    for c, (row, n) in rows.items():
        table[c], kv_len[c] = row, n
    return table, kv_len, moves


def release64(table, kv_len, rows, page, window, sinks):
    table, kv_len = table.copy(), kv_len.copy()
    for r in rows:
        if not 0 <= r < table.shape[0]:
            continue
        if window == 0:
            table[r], kv_len[r] = -1, 0
            continue
        for i in range(table.shape[1]):
            n = int(kv_len[r])
            # tokens n, n + 1, ... see j > p - window and j < sinks: the first of them sees most
            if not any(j > n - window or j < sinks for j in range(i * page, (i + 1) * page)):
                table[r, i] = -1
    return table, kv_len


def compact64(table, pages):
    live = sorted({int(x) for x in table.reshape(-1) if 0 <= x < pages})
    L = len(live)
    holes = [x for x in range(L) if x not in set(live)]
    moves = list(zip([x for x in live if x >= L], holes))
    to = dict(moves)
    out = np.array([[to.get(int(x), int(x)) for x in row] for row in table], np.int32)
    return out, L, moves
