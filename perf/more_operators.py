"""Measured cases of the operators that decode the branches of a request (beams, samples, drafts).

Three operators beside the paged cache (kv_pool [pages][2][kv heads][page_size][128], a table of
pages per row, a length per row, a row ("slot") per request) and the pools of recurrent states:

  prefix   kda_prefix_attention: attention of requests whose rows share their first tokens, the
           shared keys read once for each group of requests
  select   kda_beam_select: the best continuations of each prompt's beams over the vocabulary
  reorder  kda_beam_reorder (and kda_pages_copy for the recurrent and convolution states): beams
           take over their parents' cache rows and states

`own` False runs the plain forms (elementary torch operations in 32 bits, rounded once; sums and
totals that decide an order in 64); True makes the calls of the package's binding.
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
    pre = {"op": "prefix", "dtype": "bf16", "garbage": False}
    sel = {"op": "select", "dtype": "bf16", "masked": 0.0, "ended": 0.0, "pad": 0}
    return [
        # two beams of one short prompt, a few tokens in: latency alone
        dict(pre, name="prefix_two_beams", groups=1, branches=2, kv_heads=8, group=12, page=64, tokens=1,
             tokens_low=1, prefix_low=501, prefix_high=501, own_low=1, own_high=20, lens_seed=1),
        # beam search over a batch of prompts of ragged lengths; what lies behind a row's last token
        # has never been written (NaN among it)
        dict(pre, name="prefix_beams", groups=16, branches=4, kv_heads=8, group=12, page=64, tokens=1,
             tokens_low=1, prefix_low=500, prefix_high=8192, own_low=1, own_high=300, lens_seed=2, garbage=True),
        # a full batch behind one system prompt, each request at its own length
        dict(pre, name="prefix_system_prompt", groups=1, branches=256, kv_heads=8, group=12, page=64, tokens=1,
             tokens_low=1, prefix_low=8192, prefix_high=8192, own_low=1, own_high=2048, lens_seed=3),
        # the largest: samples of one long context, two tokens each (a draft's verify)
        dict(pre, name="prefix_long", groups=1, branches=64, kv_heads=8, group=8, page=128, tokens=2,
             tokens_low=2, prefix_low=131072, prefix_high=131072, own_low=2, own_high=500, lens_seed=4),
        # full precision: a short check run, odd sizes
        dict(pre, name="prefix_fp32", dtype="fp32", groups=3, branches=5, kv_heads=2, group=3, page=16, tokens=3,
             tokens_low=1, prefix_low=300, prefix_high=777, own_low=3, own_high=60, lens_seed=5),
        # one prompt of four beams: latency alone
        dict(sel, name="select_one", batch=1, beams=4, choices=4, vocab=32768, lens_seed=6),
        # a large batch over a large vocabulary
        dict(sel, name="select_batch", batch=64, beams=8, choices=8, vocab=131072, lens_seed=7),
        # full precision, an odd vocabulary inside a padded row, twice as many choices as beams,
        # tokens that a constraint masks, some beams at their end
        dict(sel, name="select_masked_fp32", dtype="fp32", batch=12, beams=5, choices=10, vocab=100003, pad=61,
             masked=0.3, ended=0.2, lens_seed=8),
        # one prompt of four beams with small states: latency alone
        dict(op="reorder", name="reorder_one", batch=1, beams=4, layers=1, heads=2, attn_layers=1, kv_heads=2,
             page=64, len_low=256, len_high=600, own_high=40, lens_seed=9),
        # a batch in a stack of recurrent and attention layers: states of 6.3 MB a row and layer
        dict(op="reorder", name="reorder_states", batch=16, beams=4, layers=2, heads=96, attn_layers=1, kv_heads=8,
             page=64, len_low=500, len_high=4000, own_high=100, lens_seed=10),
        # wide beams, softmax attention in the larger share of the layers
        dict(op="reorder", name="reorder_pages", batch=32, beams=8, layers=1, heads=8, attn_layers=4, kv_heads=8,
             page=16, len_low=500, len_high=4000, own_high=64, lens_seed=11),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["prefix", "prefix", "prefix", "fp32", "select", "select", "select", "reorder", "reorder"])
    seed = rng.randrange(1 << 30)
    if kind in ("prefix", "fp32"):
        half = kind == "prefix"
        kv, group = rng.choice([1, 2, 4, 8] if half else [1, 2, 4]), rng.choice([1, 2, 3, 4, 6, 8, 12, 16] if half else [1, 2, 3, 5])
        groups, branches = (_log(rng, 1, 64), _log(rng, 1, 256)) if half else (rng.choice([1, 2, 3, 5]), _log(rng, 1, 9))
        prefix, tokens = _log(rng, 16, 131072 if half else 2000), rng.choice([1, 1, 1, 2, 4, 7])
        ownlen = _log(rng, 1, 4096 if half else 200)
        # no more than the listed largest reads and multiplies, and a pool that stays under 17 GB
        while groups * branches * tokens * kv * group * (prefix + ownlen) > 64 * 2 * 64 * 131072 // (1 if half else 64):
            groups, prefix = max(1, groups // 2), max(16, prefix * 3 // 4)
            branches = max(1, branches * 3 // 4)
        while groups * (prefix + branches * (ownlen + 128)) * kv > 1 << 23:
            groups, ownlen = max(1, groups // 2), max(1, ownlen // 2)
            prefix = max(16, prefix * 3 // 4)
        ragged = rng.random() < 0.5
        return {"op": "prefix", "dtype": "bf16" if half else "fp32", "garbage": rng.random() < 0.5, "groups": groups,
                "branches": branches, "kv_heads": kv, "group": group, "page": rng.choice([16, 32, 64, 128]),
                "tokens": tokens, "tokens_low": 1 if ragged else tokens, "prefix_low": max(0, prefix // 4 - 9) if ragged else prefix,
                "prefix_high": prefix, "own_low": 1 if ragged else max(1, ownlen // 2), "own_high": ownlen, "lens_seed": seed}
    if kind == "select":
        dtype, beams = rng.choice(["bf16", "bf16", "fp32"]), rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32])
        vocab, batch = _log(rng, 100, 262144), _log(rng, 1, 256)
        while batch * beams * vocab * (1 if dtype == "bf16" else 2) > 64 * 8 * 131072:
            batch, vocab = max(1, batch // 2), max(100, vocab * 3 // 4)
        return {"op": "select", "dtype": dtype, "batch": batch, "beams": beams,
                "choices": min(64, rng.choice([beams, beams, 2 * beams, 1, beams + 3])), "vocab": vocab,
                "pad": rng.choice([0, 0, 1, 5, 64]), "masked": rng.choice([0.0, 0.0, 0.2, 0.9]),
                "ended": rng.choice([0.0, 0.0, 0.2, 0.6]), "lens_seed": seed}
    batch, beams, layers = _log(rng, 1, 48), rng.choice([2, 3, 4, 5, 8, 16]), rng.choice([1, 1, 2, 4])
    heads, kv, attn, high = _log(rng, 1, 96), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 5]), _log(rng, 40, 6000)
    while batch * beams * layers * heads > 16 * 4 * 2 * 96:
        batch, layers, heads = max(1, batch // 2), max(1, layers // 2), max(1, heads * 3 // 4)
    while batch * (high + beams * 256) * kv * attn > 1 << 22:
        batch, high, attn = max(1, batch // 2), max(40, high * 3 // 4), max(1, attn - 1)
    return {"op": "reorder", "batch": batch, "beams": beams, "layers": layers, "heads": heads, "attn_layers": attn,
            "kv_heads": kv, "page": rng.choice([16, 32, 64, 128]), "len_low": max(1, high // 8), "len_high": high,
            "own_high": _log(rng, 1, 128), "lens_seed": seed}


# --------------------------------------------------------------------------------------
# What the program has in hand
# --------------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _ints(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _branch_lengths(case):
    """(prefix of each group; tokens of the step and tokens of its own, those included, of each request):
    a case's own, the same for every seed."""
    rng = random.Random(case["lens_seed"])
    prefix = [rng.randint(case["prefix_low"], case["prefix_high"]) for _ in range(case["groups"])]
    new = [rng.randint(case["tokens_low"], case["tokens"]) for _ in range(case["groups"] * case["branches"])]
    return prefix, new, [max(n, rng.randint(case["own_low"], case["own_high"])) for n in new]


def _branch_tables(prefix, mine, branches, page, pages, order, width):
    """Rows of a table (lists): the whole pages of the group's prefix, then pages of the request's own."""
    at, rows, first_own = 0, [], []
    for g, lp in enumerate(prefix):
        whole = order[at: at + lp // page]
        at += len(whole)
        for n in mine[g * branches: (g + 1) * branches]:
            count = -(-(lp + n) // page) - lp // page
            rows.append(whole + order[at: at + count])
            first_own.append(order[at] if count else -1)
            at += count
    return [r + [-1] * (width - len(r)) for r in rows], first_own


def _prepare_prefix(case, gen, device):
    prefix, new, mine = _branch_lengths(case)
    per, page, kv, dt = case["branches"], case["page"], case["kv_heads"], _dtype(case["dtype"])
    lens = [prefix[b // per] + n for b, n in enumerate(mine)]
    requests = len(lens)
    pages = sum(lp // page for lp in prefix) + sum(-(-n // page) - prefix[b // per] // page for b, n in enumerate(lens)) + 3
    order = torch.randperm(pages, generator=gen, device=device).tolist()
    width = max(-(-n // page) for n in lens) + 1
    rows, first_own = _branch_tables(prefix, mine, per, page, pages, order, width)
    slot = torch.randperm(requests + 2, generator=gen, device=device)[:requests]
    table = torch.full((requests + 2, width), -1, dtype=torch.int32, device=device)
    table[slot] = _ints(rows, device)
    kv_len = torch.zeros(requests + 2, dtype=torch.int32, device=device)
    kv_len[slot] = _ints(lens, device)
    pool = torch.randn((pages, 2, kv, page, D), generator=gen, device=device, dtype=dt)
    for g, lp in enumerate(prefix):  # the page that the prefix ends in: a copy in each branch
        if lp % page:
            to = torch.tensor(first_own[g * per: (g + 1) * per], device=device)
            pool[to, :, :, : lp % page] = pool[to[:1], :, :, : lp % page]
    if case["garbage"]:
        # what lies behind a row's last token has never been written by it
        for r, n in zip(rows, lens):
            if n % page:
                pool[r[n // page], :, :, n % page:] = float("nan")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], kv * case["group"], D), generator=gen, device=device, dtype=dt)
    s = {"op": "prefix", "case": case, "q": q, "pool": pool, "table": table, "slot": slot.to(torch.int32),
         "kv_len": kv_len, "cu": _ints(cu, device), "cu_groups": _ints([g * per for g in range(case["groups"] + 1)], device),
         "prefix_len": _ints(prefix, device), "prefix": prefix, "new": new, "mine": mine, "out": torch.empty_like(q)}
    if own:
        from gated_delta_rule_kda_gb300 import kda
        s["workspace"] = torch.empty(kda.kda_prefix_attention_workspace_size(dt, requests, cu[-1], case["groups"], q.shape[1], kv),
                                     dtype=torch.uint8, device=device)
    return s


def _prepare_select(case, gen, device):
    B, K, V, N = case["batch"], case["beams"], case["vocab"], case["choices"]
    dt, rng = _dtype(case["dtype"]), random.Random(case["lens_seed"])
    # logits as a projection's output of padded width; a few tokens stand out, as a model's do
    x = torch.randn((B, K, V + case["pad"]), generator=gen, device=device) * 2.5
    likely = torch.randint(V, (B, K, 12), generator=gen, device=device)
    x.scatter_add_(2, likely, 6 * torch.rand((B, K, 12), generator=gen, device=device))
    if case["masked"]:  # half of the masked tokens at the type's lowest value, half at minus infinity
        r = torch.rand((B, K, V + case["pad"]), generator=gen, device=device)
        x = x.to(dt).masked_fill_(r < case["masked"] / 2, torch.finfo(dt).min).masked_fill_(r > 1 - case["masked"] / 2, -math.inf)
    scores = torch.empty((B, K), device=device).uniform_(-12, -2, generator=gen)
    ended = torch.tensor([[rng.random() < case["ended"] for _ in range(K)] for _ in range(B)], device=device)
    s = {"op": "select", "case": case, "logits": x.to(dt)[..., :V], "scores": scores, "ended": ended if case["ended"] else None,
         "parent": torch.empty((B, N), dtype=torch.int32, device=device), "token": torch.empty((B, N), dtype=torch.int32, device=device),
         "score": torch.empty((B, N), device=device), "ended_out": torch.empty((B, N), dtype=torch.bool, device=device)}
    if own:
        from gated_delta_rule_kda_gb300 import kda
        s["workspace"] = torch.empty(kda.kda_beam_select_workspace_size(B, K, V, N), dtype=torch.uint8, device=device)
    return s


def _beam_plan(case):
    """(prompt length of each entry, tokens of its own of each beam, parent of each beam): a case's own."""
    rng = random.Random(case["lens_seed"])
    B, K = case["batch"], case["beams"]
    prompts = [rng.randint(case["len_low"], case["len_high"]) for _ in range(B)]
    steps = [rng.randint(1, case["own_high"]) for _ in range(B)]  # the beams of a prompt are of one length
    # the better a beam, the more children it has
    parents = [[min(K - 1, int(K * rng.random() ** 2)) for _ in range(K)] for _ in range(B)]
    return prompts, steps, parents


def _prepare_reorder(case, gen, device):
    prompts, steps, parents = _beam_plan(case)
    B, K, page, kv = case["batch"], case["beams"], case["page"], case["kv_heads"]
    mine = [n for n in steps for _ in range(K)]
    lens = [a + b for a, b in zip(prompts, steps) for _ in range(K)]
    used = sum(p // page for p in prompts) + sum(-(-n // page) - prompts[b // K] // page for b, n in enumerate(lens))
    pages, width, rows = used + B * K + 3, max(-(-n // page) for n in lens) + 1, B * K + 4
    order = torch.randperm(pages, generator=gen, device=device).tolist()
    slot = torch.randperm(rows, generator=gen, device=device)[: B * K]
    table = torch.full((rows, width), -1, dtype=torch.int32, device=device)
    table[slot] = _ints(_branch_tables(prompts, mine, K, page, pages, order, width)[0], device)
    kv_len = torch.zeros(rows, dtype=torch.int32, device=device)
    kv_len[slot] = _ints(lens, device)
    L, H = case["layers"], case["heads"]
    s = {"op": "reorder", "case": case, "table": table, "kv_len": kv_len, "slot": slot.to(torch.int32).view(B, K),
         "parent": _ints(parents, device), "pages": pages,
         "pool": torch.randn((case["attn_layers"], pages, 2, kv, page, D), generator=gen, device=device, dtype=torch.bfloat16),
         "S": torch.randn((L, rows, H, D, D), generator=gen, device=device),
         "conv": torch.randn((L, rows, 3, 3, H, D), generator=gen, device=device, dtype=torch.bfloat16),
         "src": torch.empty(B * K, dtype=torch.int32, device=device), "dst": torch.empty(B * K, dtype=torch.int32, device=device)}
    if own:
        from gated_delta_rule_kda_gb300 import kda
        s["workspace"] = torch.empty(kda.kda_beam_reorder_workspace_size(pages, rows), dtype=torch.uint8, device=device)
    return s


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed) * 1000003 + 29)
    return {"prefix": _prepare_prefix, "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]](case, gen, device)


# --------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------
def _keys(s, row, j, seen, part):
    """Keys (part 0) or values (1) [n][keys][kv heads][128] of rows at indices j, zeros where not seen."""
    page, table = s["case"]["page"], s["table"]
    number = torch.gather(table[row], 1, (j // page).clamp_max(table.shape[1] - 1)).long()
    there = seen & (number >= 0)
    x = s["pool"][number.clamp_min(0), part, :, j % page]
    return torch.where(there[:, :, None, None], x, 0).float(), there


def _softmax_part(q, k, hide):
    """(maximum, sum, weights) of scores [n][kv heads][rows][keys] behind a mask."""
    score = (q @ k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(D)).masked_fill_(hide, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = score.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    return top, e.sum(-1, keepdim=True), e


def _plain_prefix(s):
    """Blocks of groups: the prefix with the rows of all its branches at once, each branch with its own keys, then
    the two parts joined."""
    case, q, dev = s["case"], s["q"], s["q"].device
    per, kv, G = case["branches"], case["kv_heads"], case["group"]
    longest = max(1, max(s["prefix"]))
    tokens, own_keys = max(s["new"]), max(s["mine"])
    rows = per * tokens * G
    block = max(1, min(case["groups"], (1 << 29) // (kv * rows * (longest + own_keys))))
    cu, prefix_len = s["cu"].long(), s["prefix_len"].long()
    for g0 in range(0, case["groups"], block):
        n = min(block, case["groups"] - g0)
        b = torch.arange(g0 * per, (g0 + n) * per, device=dev)
        i = torch.arange(tokens, device=dev)
        count = cu[b + 1] - cu[b]
        inside = i < count[:, None]
        token = torch.where(inside, cu[b][:, None] + i, 0)
        row, lp = s["slot"].long()[b], prefix_len[g0: g0 + n]
        # [requests][kv heads][tokens x heads][128]
        x = q[token].float().view(n * per, tokens, kv, G, D).permute(0, 2, 1, 3, 4).reshape(n * per, kv, tokens * G, D)
        # the prefix, through the row of the group's first request
        j = torch.arange(longest, device=dev).expand(n, longest)
        shared = x.view(n, per, kv, tokens * G, D).permute(0, 2, 1, 3, 4).reshape(n, kv, rows, D)
        k, seen = _keys(s, row[::per], j, j < lp[:, None], 0)
        top1, sum1, e = _softmax_part(shared, k, ~seen[:, None, None])
        v, _ = _keys(s, row[::per], j, seen, 1)
        o1 = e @ v.permute(0, 2, 1, 3)
        del k, v, e
        part = lambda t: t.view(n, kv, per, tokens * G, -1).permute(0, 2, 1, 3, 4).reshape(n * per, kv, tokens * G, -1)
        top1, sum1, o1 = part(top1), part(sum1), part(o1)
        # what each branch added
        length = s["kv_len"].long()[row]
        j = lp.repeat_interleave(per)[:, None] + torch.arange(own_keys, device=dev)
        k, seen = _keys(s, row, j, j < length[:, None], 0)
        p = (length - count)[:, None] + i
        hide = ~seen[:, None] | (j[:, None] > p[:, :, None])  # [requests][tokens][keys]
        top2, sum2, e = _softmax_part(x, k, hide.repeat_interleave(G, 1)[:, None])
        v, _ = _keys(s, row, j, seen, 1)
        o2 = e @ v.permute(0, 2, 1, 3)
        top = torch.maximum(top1, top2)
        top = torch.where(top == -math.inf, 0, top)
        w1, w2 = (top1 - top).exp(), (top2 - top).exp()
        total = w1 * sum1 + w2 * sum2
        o = (w1 * o1 + w2 * o2) / torch.where(total == 0, 1, total)
        o = o.view(n * per, kv, tokens, G, D).permute(0, 2, 1, 3, 4).reshape(n * per, tokens, kv * G, D).to(q.dtype)
        s["out"][token[inside]] = o[inside]
    return s["out"]


def _plain_select(s):
    case, N = s["case"], s["case"]["choices"]
    B, K, V = s["logits"].shape
    x = s["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x).clamp_max_(torch.finfo(torch.float32).max)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0, top)
    lse = base.double() + (x - base).exp().sum(-1, keepdim=True, dtype=torch.float64).log()
    score = s["scores"].double()[:, :, None]
    total = torch.where(x == -math.inf, -math.inf, score + (x - lse))
    if s["ended"] is not None:
        alone = torch.full((V,), -math.inf, dtype=torch.float64, device=x.device)
        alone[END] = 0
        total = torch.where(s["ended"][:, :, None], score + alone, total)
    flat = total.view(B, K * V)
    if flat.shape[1] < N:
        flat = torch.cat([flat, flat.new_full((B, N - flat.shape[1]), -math.inf)], 1)
    best, at = torch.sort(flat, dim=1, descending=True, stable=True)  # equal ones: the lowest index first
    best, at = best[:, :N], at[:, :N]
    there = best > -math.inf
    parent, token = torch.where(there, at // V, -1).to(torch.int32), torch.where(there, at % V, -1).to(torch.int32)
    over = there & (token == END)
    if s["ended"] is not None:
        over |= there & s["ended"].gather(1, parent.long().clamp_min(0))
    return parent, token, best.float(), over


END = 2  # the token that ends a beam


def _plain_reorder(s):
    case, parent, slot, table, kv_len = s["case"], s["parent"].long(), s["slot"].long(), s["table"], s["kv_len"]
    B, K, page, dev = case["batch"], case["beams"], case["page"], s["slot"].device
    # the first child of a parent keeps its row; the others take the rows of beams without a child, in order
    i = torch.arange(K, device=dev)
    earlier = (parent[:, :, None] == parent[:, None, :]) & (i[None, None, :] < i[None, :, None])
    heir = ~earlier.any(2)
    has_child = (parent[:, :, None] == i).any(1)
    rows = slot.gather(1, torch.argsort(has_child.int(), dim=1, stable=True))
    rank = ((~heir).cumsum(1) - 1).clamp_min(0)
    held = slot.gather(1, parent)
    new = torch.where(heir, held, rows.gather(1, rank))
    src, dst = torch.where(heir, -1, held).view(-1), torch.where(heir, -1, new).view(-1)
    s["slot"].copy_(new)
    s["src"].copy_(src)
    s["dst"].copy_(dst)
    move = torch.nonzero(dst >= 0).view(-1)
    p, c = src[move], dst[move]
    # the cache: whole pages shared, a part-filled last one copied to a free page
    keep = torch.ones(table.shape[0], dtype=torch.bool, device=dev)
    keep[c] = False
    live = torch.zeros(s["pages"] + 1, dtype=torch.int32, device=dev)
    live[torch.where(keep[:, None] & (table >= 0), table, s["pages"]).long().view(-1)] = 1
    free = torch.argsort(live[: s["pages"]], stable=True)
    length = kv_len[p].long()
    last = (length // page).clamp_max(table.shape[1] - 1)
    half = length % page != 0
    old, fresh = table[p, last].long(), free[(half.cumsum(0) - 1).clamp_min(0)]
    branch = table[p]
    branch.scatter_(1, last[:, None], torch.where(half, fresh, old)[:, None].to(branch.dtype))
    at = torch.arange(table.shape[1], device=dev)
    branch = torch.where(at >= ((length + page - 1) // page)[:, None], -1, branch)
    table[c], kv_len[c] = branch, kv_len[p]
    s["pool"][:, fresh[half]] = s["pool"][:, old[half]]
    s["S"][:, c] = s["S"][:, p]
    s["conv"][:, c] = s["conv"][:, p]
    return s["slot"], s["src"], s["dst"], table, kv_len, s["pool"], s["S"], s["conv"]


# --------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if not own:
        return {"prefix": _plain_prefix, "select": _plain_select, "reorder": _plain_reorder}[s["op"]](s)
    from gated_delta_rule_kda_gb300 import kda
    if s["op"] == "prefix":
        return kda.kda_prefix_attention(s["q"], s["pool"], s["table"], s["slot"], s["cu"], s["kv_len"], s["cu_groups"],
                                        s["prefix_len"], max_tokens=case["tokens"], o=s["out"], workspace=s["workspace"])
    if s["op"] == "select":
        return kda.kda_beam_select(s["logits"], s["scores"], case["choices"], ended=s["ended"], end_token=END,
                                   parent=s["parent"], token=s["token"], score=s["score"], ended_out=s["ended_out"],
                                   workspace=s["workspace"])
    src, dst = kda.kda_beam_reorder(s["parent"], s["slot"], s["pool"], s["table"], s["kv_len"], case["page"],
                                    src=s["src"], dst=s["dst"], workspace=s["workspace"])
    kda.kda_pages_copy(s["S"], src, dst)
    kda.kda_pages_copy(s["conv"], src, dst)
    return s["slot"], src, dst, s["table"], s["kv_len"], s["pool"], s["S"], s["conv"]


# --------------------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "prefix":
        prefix, new, mine = _branch_lengths(case)
        size, heads = 2 if case["dtype"] == "bf16" else 4, case["kv_heads"] * case["group"]
        pairs = sum(n * (prefix[b // case["branches"]] + m - n) + n * (n + 1) // 2 for b, (n, m) in enumerate(zip(new, mine)))
        return {"bytes": 2 * sum(new) * heads * D * size + (sum(prefix) + sum(mine)) * 2 * case["kv_heads"] * D * size,
                "flops": 4 * D * heads * pairs}
    if case["op"] == "select":
        rng = random.Random(case["lens_seed"])
        live = sum(not rng.random() < case["ended"] for _ in range(case["batch"] * case["beams"]))
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": live * case["vocab"] * size + case["batch"] * (case["beams"] * 5 + case["choices"] * 13),
                "flops": 4 * live * case["vocab"]}
    prompts, steps, parents = _beam_plan(case)
    state = case["layers"] * case["heads"] * (D * D * 4 + 9 * D * 2)
    page_bytes = 2 * case["kv_heads"] * case["page"] * D * 2 * case["attn_layers"]
    moved = [(b, len(p) - len(set(p))) for b, p in enumerate(parents)]
    table = sum(n * -(-(prompts[b] + steps[b]) // case["page"]) for b, n in moved)
    return {"bytes": 2 * sum(n * (state + (page_bytes if (prompts[b] + steps[b]) % case["page"] else 0)) for b, n in moved) + 8 * table
            + 8 * case["batch"] * case["beams"], "flops": 0}


# --------------------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "reorder":
        return None  # copies and whole numbers: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(s)
    q, out, page, t0 = s["q"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), case["page"], 0
    for b, n in enumerate(s["new"]):  # each request by itself, through its own row
        length = s["prefix"][b // case["branches"]] + s["mine"][b]
        j = torch.arange(length, device="cuda")
        kv = s["pool"][s["table"][int(s["slot"][b])].long()[j // page], :, :, j % page].double()  # [keys, 2, kv heads, 128]
        p = length - n + torch.arange(n, device="cuda").repeat_interleave(case["group"])
        for h in range(case["kv_heads"]):
            x = q[t0: t0 + n, h * case["group"]: (h + 1) * case["group"]].double().reshape(-1, D)
            a = (x @ kv[:, 0, h].T / math.sqrt(D)).masked_fill(j > p[:, None], -math.inf)
            out[t0: t0 + n, h * case["group"]: (h + 1) * case["group"]] = (torch.softmax(a, -1) @ kv[:, 1, h]).view(n, case["group"], D)
        t0 += n
    return out


def _exact_select(s):
    case, N = s["case"], s["case"]["choices"]
    B, K, V = s["logits"].shape
    parent, token = (torch.full((B, N), -1, dtype=torch.int32) for _ in range(2))
    score, over = torch.full((B, N), -math.inf, dtype=torch.float64), torch.zeros((B, N), dtype=torch.bool)
    for b in range(B):
        found = []
        for k in range(K):
            base = float(s["scores"][b, k])
            if s["ended"] is not None and bool(s["ended"][b, k]):
                found.append((-base, k, END))
                continue
            log_p = torch.log_softmax(s["logits"][b, k].double(), -1)
            edge = torch.topk(log_p, min(N, V)).values[-1]
            at = torch.nonzero((log_p >= edge) & (log_p > -math.inf)).view(-1)
            found += [(-(base + x), k, v) for v, x in zip(at.tolist(), log_p[at].tolist())]
        for n, (t, k, v) in enumerate(sorted(found)[:N]):
            parent[b, n], token[b, n], score[b, n] = k, v, -t
            over[b, n] = v == END or (s["ended"] is not None and bool(s["ended"][b, k]))
    return parent.cuda(), token.cuda(), score.cuda(), over.cuda()
