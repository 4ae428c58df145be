"""Measured cases of the softmax-attention operators that stand beside the KDA layers.

Three operators over one paged cache (kv_pool [pages][2][kv heads][page_size][128], a table of
pages per row, a length per row, a row ("slot") per request):

  attention  kda_window_attention: a sliding window plus the first `sinks` tokens
  rope       kda_qk_norm_rope / kda_qk_norm_rope_append: q and k normed per head and rotated,
             k and v written to the cache in the same pass
  pages      kda_pages_fork / kda_pages_release / kda_pages_compact

`own` False runs the plain forms (elementary torch operations in 32 bits, rounded once); True
makes the calls of the package's binding.
"""
import math
import random

import torch

own = False

D = 128


# --------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------
def listed():
    att = {"op": "attention", "dtype": "bf16", "garbage": False}
    return [
        # one request generating a token: latency alone; an odd length, 12 query heads a KV head
        dict(att, name="attn_one_token", batch=1, kv_heads=8, group=12, page=64, tokens=1,
             tokens_low=1, len_low=1501, len_high=1501, window=1024, sinks=4, lens_seed=1),
        # a full decode batch at ragged lengths, some shorter than the window; the rest of each
        # last page holds what the allocation held before (NaN among it)
        dict(att, name="attn_decode_batch", batch=256, kv_heads=8, group=12, page=64, tokens=1,
             tokens_low=1, len_low=1, len_high=8192, window=1024, sinks=4, lens_seed=2,
             garbage=True),
        # long contexts with nothing out of the window, two tokens a request (a draft's verify)
        dict(att, name="attn_verify_long", batch=4, kv_heads=8, group=8, page=128, tokens=2,
             tokens_low=2, len_low=65536, len_high=131072, window=131072, sinks=0, lens_seed=3),
        # a ragged prefill of new requests in small pages, odd window and sink counts
        dict(att, name="attn_prefill_ragged", batch=9, kv_heads=4, group=6, page=16, tokens=1500,
             tokens_low=1, len_low=0, len_high=700, window=333, sinks=5, lens_seed=4),
        # the prefill workload's length and head count
        dict(att, name="attn_prefill_8k", batch=1, kv_heads=8, group=12, page=64, tokens=8192,
             tokens_low=8192, len_low=0, len_high=0, window=1024, sinks=4, lens_seed=5),
        # the largest: a chunk of a long prompt behind what the cache already holds
        dict(att, name="attn_prefill_chunk", batch=2, kv_heads=8, group=4, page=64, tokens=16384,
             tokens_low=16384, len_low=8192, len_high=32768, window=4096, sinks=16, lens_seed=6),
        # full precision: a short check run
        dict(att, name="attn_fp32", dtype="fp32", batch=3, kv_heads=2, group=3, page=32, tokens=300,
             tokens_low=40, len_low=0, len_high=500, window=257, sinks=3, lens_seed=7),
        # decode: the step's tokens into the cache
        dict(op="rope", name="rope_decode", batch=64, tokens=1, tokens_low=1, q_heads=96, kv_heads=8,
             page=64, rotary=128, interleaved=False, norm=True, weights=True, append=True,
             dtype="bf16", out="bf16", context=4096, lens_seed=8),
        # prefill: ragged requests, half the head rotated, into the cache
        dict(op="rope", name="rope_prefill", batch=5, tokens=8192, tokens_low=3000, q_heads=96,
             kv_heads=8, page=64, rotary=64, interleaved=False, norm=True, weights=True, append=True,
             dtype="bf16", out="bf16", context=20000, lens_seed=9),
        # no cache: interleaved pairs, full precision in, odd token count
        dict(op="rope", name="rope_interleaved", batch=1, tokens=2049, tokens_low=2049, q_heads=16,
             kv_heads=16, page=64, rotary=128, interleaved=True, norm=True, weights=False,
             append=False, dtype="fp32", out="fp32", context=100000, lens_seed=10),
        # all rows trimmed to what the window still sees, then four branches of two requests:
        # rows copied, the half-filled last pages duplicated in four layers
        dict(op="pages", name="pages_fork", kind="fork", rows=32, width=256, pages=6144, layers=4,
             kv_heads=8, page=16, forks=4, parents=2, len_low=500, len_high=4000, live=1.0,
             window=1024, sinks=4, lens_seed=11),
        # a fragmented cache brought together after three quarters of its requests have left
        dict(op="pages", name="pages_compact", kind="compact", rows=256, width=128, pages=8192,
             layers=1, kv_heads=8, page=64, forks=0, parents=0, len_low=500, len_high=4000,
             live=0.25, window=0, sinks=0, lens_seed=12),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prefill", "prefill", "fp32", "rope", "rope", "pages", "pages"])
    seed = rng.randrange(1 << 30)
    if kind == "decode":
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        batch, high = _log(rng, 1, 256), _log(rng, 16, 131072)
        window = rng.choice([_log(rng, 16, 8192), _log(rng, 16, 8192), 131072])
        while batch * kv * min(high, window) > 4 * 8 * 131072:  # no more than the listed reads
            batch = max(1, batch // 2)
        while batch * high * kv > 1 << 25:  # the pool itself stays under 17 GB
            high = max(16, high // 2)
        return {"op": "attention", "dtype": "bf16", "garbage": rng.random() < 0.5, "batch": batch,
                "kv_heads": kv, "group": group, "page": rng.choice([16, 32, 64, 128]),
                "tokens": rng.choice([1, 1, 2, 4, 7]), "tokens_low": 1, "len_low": max(0, high // 4 - 5),
                "len_high": high, "window": window, "sinks": rng.choice([0, 1, 4, 17, 64]), "lens_seed": seed}
    if kind == "prefill":
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 12])
        batch, tokens, window = rng.choice([1, 2, 3, 7]), _log(rng, 33, 16384), _log(rng, 64, 4096)
        while batch * tokens * kv * group * (window + 128) > 32768 * 32 * 4224:
            tokens = max(33, tokens // 2)
        low = rng.choice([0, 0, 1000])
        return {"op": "attention", "dtype": "bf16", "garbage": rng.random() < 0.5, "batch": batch,
                "kv_heads": kv, "group": group, "page": rng.choice([16, 32, 64, 128]), "tokens": tokens,
                "tokens_low": max(1, tokens // rng.choice([1, 2, 8])), "len_low": low,
                "len_high": low * 5, "window": window, "sinks": rng.choice([0, 1, 4, 33, 200]), "lens_seed": seed}
    if kind == "fp32":
        return {"op": "attention", "dtype": "fp32", "garbage": rng.random() < 0.5, "batch": rng.choice([1, 2, 5]),
                "kv_heads": rng.choice([1, 2, 4]), "group": rng.choice([1, 2, 3, 5]),
                "page": rng.choice([16, 32, 64, 128]), "tokens": _log(rng, 1, 700), "tokens_low": 1, "len_low": 0,
                "len_high": _log(rng, 1, 1500), "window": _log(rng, 16, 1000), "sinks": rng.choice([0, 2, 40]),
                "lens_seed": seed}
    if kind == "rope":
        append = rng.random() < 0.6
        batch = _log(rng, 1, 128) if append else 1
        heads, kv = rng.choice([4, 12, 32, 64, 96]), rng.choice([1, 2, 4, 8, 16])
        tokens = _log(rng, 1, 16384)
        while batch * tokens * (heads + 2 * kv) > 5 * 8192 * 112:
            tokens = max(1, tokens // 2)
            batch = max(1, batch // 2) if tokens == 1 else batch
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return {"op": "rope", "batch": batch, "tokens": tokens, "tokens_low": max(1, tokens // rng.choice([1, 3])),
                "q_heads": heads, "kv_heads": kv, "page": rng.choice([16, 32, 64, 128]),
                "rotary": rng.choice([128, 128, 64, 32, 96, 48]), "interleaved": rng.random() < 0.4,
                "norm": rng.random() < 0.8, "weights": rng.random() < 0.7, "append": append, "dtype": dtype,
                "out": "bf16" if dtype == "bf16" else rng.choice(["fp32", "bf16"]), "context": _log(rng, 64, 131072),
                "lens_seed": seed}
    rows, page, kv, layers = _log(rng, 4, 256), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 8]), rng.choice([1, 3, 8])
    high = _log(rng, 40, 8000)
    while rows * (high + page) * kv * layers > 1 << 22:
        rows, high = max(4, rows // 2), max(40, high * 3 // 4)
        layers = max(1, layers // 2)
    width = -(-high // page) + rng.choice([0, 1, 7])
    forks = rng.choice([1, 2, 3, 8, rows // 3]) or 1
    forks = min(forks, rows - 1, max(1, rows // 2))
    compact = rng.random() < 0.5
    return {"op": "pages", "kind": "compact" if compact else "fork", "rows": rows, "width": width,
            "pages": rows * width + rng.randrange(1, 50), "layers": layers, "kv_heads": kv, "page": page,
            "forks": 0 if compact else forks, "parents": 0 if compact else rng.randrange(1, max(2, min(rows - forks, 4) + 1)),
            "len_low": max(1, high // 8), "len_high": high, "live": round(rng.uniform(0.05, 0.9), 3) if compact else 1.0,
            "window": 0 if compact else rng.choice([16, 100, 1024]), "sinks": 0 if compact else rng.choice([0, 4, 40]),
            "lens_seed": seed}


# --------------------------------------------------------------------------------------
# What the program has in hand
# --------------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _lengths(case):
    """(tokens of the step, tokens before it) of each request: a case's own, the same for every seed."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "rope":
        new = [rng.randint(case["tokens_low"], case["tokens"]) for _ in range(case["batch"])]
        return new, [rng.randint(0, case["context"]) for _ in new]
    new = [rng.randint(case["tokens_low"], case["tokens"]) for _ in range(case["batch"])]
    old = [max(0, rng.randint(case["len_low"], case["len_high"]) - n) if case["len_high"] else 0 for n in new]
    return new, old


def _ints(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _table(lens, page, spare_rows, gen, device):
    """Pages of rows of these lengths, in an order without pattern: (table [R][M], pages in the pool, row of each request)."""
    counts = [-(-n // page) for n in lens]
    rows, width, pages = len(lens) + spare_rows, max(counts) + 1, sum(counts) + 3
    order = torch.randperm(pages, generator=gen, device=device, dtype=torch.int64)[: sum(counts)].to(torch.int32)
    slot = torch.randperm(rows, generator=gen, device=device)[: len(lens)].to(torch.int32)
    n = torch.tensor(counts, device=device)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=device)
    at = torch.arange(sum(counts), device=device) - torch.repeat_interleave(n.cumsum(0) - n, n)
    table[torch.repeat_interleave(slot.long(), n), at] = order
    kv_len = torch.zeros(rows, dtype=torch.int32, device=device)
    kv_len[slot.long()] = _ints(lens, device)
    return table, pages, slot, kv_len


def _prepare_attention(case, gen, device):
    new, old = _lengths(case)
    lens, dt, kv = [a + b for a, b in zip(new, old)], _dtype(case["dtype"]), case["kv_heads"]
    heads, page, total = kv * case["group"], case["page"], sum(new)
    table, pages, slot, kv_len = _table(lens, page, 2, gen, device)
    pool = torch.randn((pages, 2, kv, page, D), generator=gen, device=device, dtype=dt)
    if case["garbage"]:
        # what lies behind a row's last token has never been written by it
        for b, n in enumerate(lens):
            if n % page:
                pool[table[slot[b].long(), n // page].long(), :, :, n % page:] = float("nan")
    q = torch.randn((total, heads, D), generator=gen, device=device, dtype=dt)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return {"op": "attention", "case": case, "q": q, "pool": pool, "table": table, "slot": slot,
            "kv_len": kv_len, "cu": _ints(cu, device), "new": new, "lens": lens,
            "out": torch.empty_like(q)}


def _rope_table(positions, rotary, device):
    """(cos, sin) of base 10000 stretched four times (the NTK rule on the base), rounded from 64 bits."""
    base = 10000.0 * 4.0 ** (rotary / max(2, rotary - 2))
    inv = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=device) / rotary)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()


def _prepare_rope(case, gen, device):
    new, old = _lengths(case)
    total, hq, hkv, dt = sum(new), case["q_heads"], case["kv_heads"], _dtype(case["dtype"])
    # the projection's output: q, k and v of a token side by side
    qkv = torch.randn((total, hq + 2 * hkv, D), generator=gen, device=device, dtype=dt)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    at = torch.arange(total, device=device)
    n = torch.tensor(new, device=device)
    first = torch.repeat_interleave(torch.tensor([o - c for o, c in zip(old, cu)], device=device), n)
    positions = (at + first).to(torch.int32)
    s = {"op": "rope", "case": case, "qkv": qkv, "positions": positions,
         "rope": _rope_table(max(a + b for a, b in zip(new, old)), case["rotary"], device),
         "wq": 1 + 0.1 * torch.randn(D, generator=gen, device=device) if case["weights"] else None,
         "wk": 1 + 0.1 * torch.randn(D, generator=gen, device=device) if case["weights"] else None,
         "q_out": torch.empty((total, hq, D), dtype=_dtype(case["out"]), device=device)}
    if not case["append"]:
        s["k_out"] = torch.empty((total, hkv, D), dtype=_dtype(case["out"]), device=device)
        return s
    page = case["page"]
    # only the pages that the step writes are in the pool: those before it are mapped to no page
    lens, rows = [a + b for a, b in zip(new, old)], case["batch"] + 1
    width = max(-(-x // page) for x in lens)
    counts = [-(-x // page) - o // page for x, o in zip(lens, old)]
    pages = sum(counts) + 2
    order = torch.randperm(pages, generator=gen, device=device)[: sum(counts)].to(torch.int32)
    slot = torch.randperm(rows, generator=gen, device=device)[: case["batch"]].to(torch.int32)
    cnt = torch.tensor(counts, device=device)
    col = torch.arange(sum(counts), device=device) + torch.repeat_interleave(
        torch.tensor([o // page for o in old], device=device) - (cnt.cumsum(0) - cnt), cnt)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=device)
    table[torch.repeat_interleave(slot.long(), cnt), col] = order
    kv_len = torch.zeros(rows, dtype=torch.int32, device=device)
    kv_len[slot.long()] = _ints(lens, device)
    s |= {"pool": torch.randn((pages, 2, hkv, page, D), generator=gen, device=device, dtype=_dtype(case["out"])),
          "table": table, "slot": slot, "kv_len": kv_len, "cu": _ints(cu, device)}
    return s


def _page_rows(case):
    rng = random.Random(case["lens_seed"])
    lens = [rng.randint(case["len_low"], case["len_high"]) for _ in range(case["rows"])]
    if case["kind"] == "compact":
        stays = sorted(rng.sample(range(case["rows"]), max(1, int(case["rows"] * case["live"]))))
        return [n if r in set(stays) else 0 for r, n in enumerate(lens)], [], []
    children = rng.sample(range(case["rows"]), case["forks"])
    others = [r for r in range(case["rows"]) if r not in set(children)]
    parents = rng.sample(others, min(case["parents"], len(others)))
    return [0 if r in set(children) else n for r, n in enumerate(lens)], children, [parents[i % len(parents)] for i in range(len(children))]


def _prepare_pages(case, gen, device):
    lens, children, parents = _page_rows(case)
    page = case["page"]
    counts = torch.tensor([-(-n // page) for n in lens], device=device)
    total = int(counts.sum())
    order = torch.randperm(case["pages"], generator=gen, device=device)[:total].to(torch.int32)
    row = torch.repeat_interleave(torch.arange(case["rows"], device=device), counts)
    col = torch.arange(total, device=device) - torch.repeat_interleave(counts.cumsum(0) - counts, counts)
    table = torch.full((case["rows"], case["width"]), -1, dtype=torch.int32, device=device)
    table[row, col] = order
    pool = torch.randn((case["layers"], case["pages"], 2, case["kv_heads"], page, D), generator=gen, device=device,
                       dtype=torch.bfloat16)
    s = {"op": "pages", "case": case, "pool": pool, "table": table, "kv_len": _ints(lens, device)}
    if case["kind"] == "compact":  # the fragmented table stays: the pages move, a new table names them
        s["table_out"] = torch.empty_like(table)
    else:
        s |= {"child": _ints(children, device), "parent": _ints(parents, device),
              "rows": torch.arange(case["rows"], dtype=torch.int32, device=device)}
    return s


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed) * 1000003 + 17)
    return {"attention": _prepare_attention, "rope": _prepare_rope, "pages": _prepare_pages}[case["op"]](case, gen, device)


# --------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------
def _plain_attention(s):
    """Blocks of up to 128 consecutive tokens of a request, each with the keys that any token of it can see."""
    case, q, pool, table = s["case"], s["q"], s["pool"], s["table"]
    dev, page, window, sinks, kv, group = q.device, case["page"], case["window"], case["sinks"], case["kv_heads"], case["group"]
    block = min(128, max(s["new"]))
    cu, new = s["cu"].long(), torch.diff(s["cu"].long())
    per = (new + block - 1) // block
    count = sum(-(-n // block) for n in s["new"])
    req = torch.repeat_interleave(torch.arange(len(s["new"]), device=dev), per, output_size=count)
    start = (torch.arange(count, device=dev) - (per.cumsum(0) - per)[req]) * block
    i = start[:, None] + torch.arange(block, device=dev)
    inside = i < new[req][:, None]
    token = torch.where(inside, cu[req][:, None] + i, 0)
    row = s["slot"].long()[req]
    p = s["kv_len"].long()[row][:, None] - new[req][:, None] + i
    longest = max(s["lens"])
    if sinks + window + block > longest:
        j = torch.arange(longest, device=dev).expand(count, longest)
    else:
        base = (p[:, :1] - window + 1).clamp_min(0)
        near = base + torch.arange(window + block - 1, device=dev)
        far = torch.arange(sinks, device=dev).expand(count, sinks)
        j = torch.cat([torch.where(far < base, far, -1), near], 1)
    number = torch.gather(table[row], 1, (j.clamp(0, table.shape[1] * page - 1) // page)).long()
    there = (j >= 0) & (j < table.shape[1] * page) & (number >= 0)
    visible = there[:, None] & (j[:, None] <= p[:, :, None]) & ((j[:, None] > p[:, :, None] - window) | (j[:, None] < sinks)) & inside[:, :, None]
    seen = visible.any(1)
    number, at = number.clamp_min(0), j.clamp_min(0) % page
    k = torch.where(seen[:, :, None, None], pool[number, 0, :, at], 0).float()
    x = q[token].float().view(count, block, kv, group, D).permute(0, 2, 3, 1, 4).reshape(count, kv, group * block, D)
    score = (x @ k.permute(0, 2, 3, 1)).view(count, kv, group, block, -1)
    del k
    score = score.mul_(1 / math.sqrt(D)).masked_fill_(~visible[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = score.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    total = e.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, None, None], pool[number, 1, :, at], 0).float().permute(0, 2, 1, 3)
    o = (e.view(count, kv, group * block, -1) @ v).view(count, kv, group, block, D) / torch.where(total == 0, 1, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(count, block, kv * group, D).to(q.dtype)
    s["out"][token[inside]] = o[inside]
    return s["out"]


def _plain_rotate(x, weight, s):
    case = s["case"]
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        if weight is not None:
            x = x * weight
    r = case["rotary"]
    cs = s["rope"][s["positions"].long()][:, None]
    c, n = cs[..., 0], cs[..., 1]
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., : r // 2], x[..., r // 2: r])
    one, two = a * c - b * n, b * c + a * n
    if case["interleaved"]:
        y[..., 0:r:2], y[..., 1:r:2] = one, two
    else:
        y[..., : r // 2], y[..., r // 2: r] = one, two
    return y.to(_dtype(case["out"]))


def _plain_rope(s):
    case, hq, hkv = s["case"], s["case"]["q_heads"], s["case"]["kv_heads"]
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq: hq + hkv], s["qkv"][:, hq + hkv:]
    q, k = _plain_rotate(q, s["wq"], s), _plain_rotate(k, s["wk"], s)
    if not case["append"]:
        return q, k
    cu, page = s["cu"].long(), case["page"]
    t = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    row = s["slot"].long()[b]
    j = s["kv_len"].long()[row] - cu[b + 1] + t
    number = s["table"][row, j // page].long()
    s["pool"][number, 0, :, j % page] = k
    s["pool"][number, 1, :, j % page] = v.to(k.dtype)
    return q, s["pool"]


def _plain_fork(s):
    case, pool, pages, table, kv_len = s["case"], s["pool"], s["case"]["pages"], s["table"], s["kv_len"]
    # every row keeps the pages that a coming token can see
    rows = s["rows"].long()
    j, n = torch.arange(table.shape[1], device=table.device), kv_len[rows].long()
    gone = ((j + 1) * case["page"] <= (n - case["window"] + 1)[:, None]) & (j * case["page"] >= case["sinks"])
    table[rows] = torch.where(gone, -1, table[rows])
    parent, child = s["parent"].long(), s["child"].long()
    keep = torch.ones(table.shape[0], dtype=torch.bool, device=table.device)
    keep[child] = False
    live = torch.zeros(pages + 1, dtype=torch.int32, device=table.device)
    live[torch.where(keep[:, None] & (table >= 0), table, pages).long().view(-1)] = 1
    free = torch.argsort(live[:pages], stable=True)
    length = kv_len[parent].long()
    last = (length // case["page"]).clamp_max(table.shape[1] - 1)
    old = table[parent, last].long()
    half = (length % case["page"] != 0) & (old >= 0)
    fresh = free[(half.cumsum(0) - 1).clamp_min(0)]
    branch = table[parent]
    branch.scatter_(1, last[:, None], torch.where(half, fresh, old)[:, None].to(branch.dtype))
    table[child], kv_len[child] = branch, kv_len[parent]
    pool[:, fresh[half]] = pool[:, old[half]]
    return table, kv_len, pool


def _plain_compact(s):
    pool, pages, table = s["pool"], s["case"]["pages"], s["table"]
    live = torch.zeros(pages + 1, dtype=torch.bool, device=table.device)
    live[torch.where(table >= 0, table, pages).long().view(-1)] = True
    live = live[:pages]
    count = live.sum()
    at = torch.arange(pages, device=table.device)
    source, hole = torch.nonzero(live & (at >= count)).view(-1), torch.nonzero(~live & (at < count)).view(-1)
    to = at.clone()
    to[source] = hole
    pool[:, hole] = pool[:, source]
    s["table_out"].copy_(torch.where(table >= 0, to[table.long().clamp_min(0)].to(torch.int32), table))
    return s["table_out"], count.to(torch.int32).view(1), pool


# --------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if not own:
        if s["op"] == "attention":
            return _plain_attention(s)
        if s["op"] == "rope":
            return _plain_rope(s)
        return _plain_fork(s) if case["kind"] == "fork" else _plain_compact(s)
    from gated_delta_rule_kda_gb300 import kda
    if s["op"] == "attention":
        return kda.kda_window_attention(s["q"], s["pool"], s["table"], s["slot"], s["cu"], s["kv_len"],
                                        case["window"], case["sinks"], max_tokens=max(s["new"]), o=s["out"])
    if s["op"] == "rope":
        hq, hkv = case["q_heads"], case["kv_heads"]
        q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq: hq + hkv], s["qkv"][:, hq + hkv:]
        how = dict(norm=case["norm"], interleaved=case["interleaved"], q_out=s["q_out"])
        if not case["append"]:
            return kda.kda_qk_norm_rope(q, k, s["rope"], s["positions"], s["wq"], s["wk"], 1e-6, k_out=s["k_out"], **how)
        out = kda.kda_qk_norm_rope_append(q, k, v, s["rope"], s["positions"], s["pool"], s["table"], s["slot"], s["cu"],
                                          s["kv_len"], s["wq"], s["wk"], 1e-6, **how)
        return out, s["pool"]
    if case["kind"] == "fork":
        kda.kda_pages_release(s["table"], s["kv_len"], s["rows"], case["page"], case["window"], case["sinks"])
        kda.kda_pages_fork(s["pool"], s["table"], s["kv_len"], s["parent"], s["child"], case["page"])
        return s["table"], s["kv_len"], s["pool"]
    table, count = kda.kda_pages_compact(s["pool"], s["table"], table_out=s["table_out"])
    return table, count, s["pool"]


# --------------------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------------------
def _visible(case, n, length):
    """(pairs, keys): visible (token, key) pairs of a request, and the keys that any of its tokens sees."""
    w, sinks = case["window"], case["sinks"]
    pairs, first = 0, length - n
    # p from first to length - 1: min(p + 1, w) recent keys, and the sinks before them
    for low, high in ((first, min(length, w)), (max(first, w), length)):
        m = max(0, high - low)
        if high <= w:
            pairs += m * (low + high + 1) // 2 if m else 0
        else:
            a, b = low - w + 1, high - w  # keys before the window, over the rows: min(sinks, .)
            inner = max(0, min(b, sinks) - a + 1)
            pairs += m * w + inner * (a + a + inner - 1) // 2 + (m - inner) * sinks
    keys = length - max(0, first - w + 1) + min(sinks, max(0, first - w + 1))
    return pairs, keys


def work(case):
    if case["op"] == "attention":
        new, old = _lengths(case)
        size, heads = 2 if case["dtype"] == "bf16" else 4, case["kv_heads"] * case["group"]
        seen = [_visible(case, n, n + o) for n, o in zip(new, old)]
        return {"bytes": 2 * sum(new) * heads * D * size + sum(k for _, k in seen) * 2 * case["kv_heads"] * D * size,
                "flops": 4 * D * heads * sum(p for p, _ in seen)}
    if case["op"] == "rope":
        new, _ = _lengths(case)
        rows = case["q_heads"] + (2 if case["append"] else 1) * case["kv_heads"]
        size = (2 if case["dtype"] == "bf16" else 4) + (2 if case["out"] == "bf16" else 4)
        return {"bytes": sum(new) * (rows * D * size + case["rotary"] * 4 + 4), "flops": 8 * sum(new) * rows * D}
    lens, children, parents = _page_rows(case)
    page_bytes, entries = 2 * case["kv_heads"] * case["page"] * D * 2 * case["layers"], case["rows"] * case["width"] * 4
    if case["kind"] == "fork":
        moved = sum(1 for r in parents if lens[r] % case["page"])
        return {"bytes": 2 * moved * page_bytes + 2 * entries, "flops": 0}
    total = sum(-(-n // case["page"]) for n in lens)
    moved = int(total * (1 - total / case["pages"]))  # pages are scattered evenly
    return {"bytes": 2 * moved * page_bytes + 2 * entries, "flops": 0}


# --------------------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "pages":
        return None  # copies and whole numbers: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    q, out, page = s["q"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), case["page"]
    t0 = 0
    for b, (n, length) in enumerate(zip(s["new"], s["lens"])):
        row = s["table"][int(s["slot"][b])].long()
        for c0 in range(0, n, 1024):
            c1 = min(n, c0 + 1024)
            p = length - n + torch.arange(c0, c1, device="cuda")
            lo = max(0, length - n + c0 - case["window"] + 1)
            keys = list(range(min(case["sinks"], lo))) + list(range(lo, length - n + c1))
            j = torch.tensor(keys, device="cuda")
            kv = s["pool"][row[j // page], :, :, j % page].double()  # [keys, 2, kv heads, 128]
            hide = (j[None] > p[:, None]) | ((j[None] <= p[:, None] - case["window"]) & (j[None] >= case["sinks"]))
            for h in range(q.shape[1]):
                a = q[t0 + c0: t0 + c1, h].double() @ kv[:, 0, h // case["group"]].T / math.sqrt(D)
                out[t0 + c0: t0 + c1, h] = torch.softmax(a.masked_fill(hide, -math.inf), -1) @ kv[:, 1, h // case["group"]]
        t0 += n
    return out


def _exact_rope(s):
    case, hq, hkv, r = s["case"], s["case"]["q_heads"], s["case"]["kv_heads"], s["case"]["rotary"]
    x, pair = s["qkv"].double(), torch.view_as_complex(s["rope"].double())[s["positions"].long()]

    def turned(part, weight):
        y = part.clone()
        if case["norm"]:
            y /= (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt()
            y *= 1.0 if weight is None else weight.double()
        head = y[..., :r].reshape(*y.shape[:-1], r // 2, 2) if case["interleaved"] else y[..., :r].reshape(*y.shape[:-1], 2, r // 2).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * pair[:, None])
        y[..., :r] = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return y

    q, k = turned(x[:, :hq], s["wq"]), turned(x[:, hq: hq + hkv], s["wk"])
    if not case["append"]:
        return q, k
    pool, cu, t0 = s["pool"].double(), s["cu"].tolist(), 0
    for b, (n, old) in enumerate(zip(*_lengths(case))):
        j = old + torch.arange(n, device="cuda")
        number = s["table"][int(s["slot"][b])].long()[j // case["page"]]
        pool[number, 0, :, j % case["page"]] = k[cu[b]: cu[b + 1]]
        pool[number, 1, :, j % case["page"]] = x[cu[b]: cu[b + 1], hq + hkv:]
    return q, pool
