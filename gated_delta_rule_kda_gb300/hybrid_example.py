"""A hybrid stack in miniature: one KDA layer and one softmax-attention layer side by side.

    python -m gated_delta_rule_kda_gb300.hybrid_example

A prompt is prefilled through both layers, the request is forked (the attention layer's pages are
shared, its part-filled page and the KDA layer's state rows are copied), both branches decode, the
cache is trimmed to the window, one branch leaves and the pages are brought together.  The layers'
projections are stand-ins: random tensors of the shapes they would have.
"""
from __future__ import annotations

import torch

from . import kda, synthetic

PAGE, WINDOW, SINKS = 16, 64, 4


def run(prompt: int = 150, steps: int = 24, kda_heads: int = 4, q_heads: int = 8, kv_heads: int = 2,
        seed: int = 0, device: str = "cuda"):
    """Outputs of the attention layer and of the KDA layer, [branches, steps, heads, 128] each, the
    prompt's attention output, how many pages are live at the end, and the last token's attention
    output once more, from the cache as it was brought together."""
    total, branches, rows = prompt + steps, 2, 4
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)

    # the KDA layer: pooled recurrent and convolution states, a row a request
    lin = synthetic.layer_inputs([total], kda_heads, seed=seed, s0_std=0.1, device=device)
    S_pool = torch.zeros((rows, kda_heads, 128, 128), device=device)
    conv_pool = torch.zeros((rows, 3, 3, kda_heads, 128), dtype=torch.bfloat16, device=device)
    # the attention layer: q, k, v of every token as one projection gives them, and its cache
    g = torch.Generator(device=device)
    g.manual_seed(seed + 1)
    qkv = torch.randn((total, q_heads + 2 * kv_heads, 128), generator=g, device=device, dtype=torch.bfloat16)
    q, k, v = qkv.split([q_heads, kv_heads, kv_heads], dim=1)
    wq, wk = (1 + 0.1 * torch.randn(128, generator=g, device=device) for _ in range(2))
    rope = kda.rope_table(total, 64, base=500000.0, device=device)
    width = -(-total // PAGE)
    pages = branches * width + 3
    pool = torch.zeros((1, pages, 2, kv_heads, PAGE, 128), dtype=torch.bfloat16, device=device)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=device)
    kv_len = torch.zeros(rows, dtype=torch.int32, device=device)

    def attend(t0, n, slots, pos):
        """The attention layer over tokens [t0, t0 + n), the same for each request in `slots`: its output and queries."""
        idx = torch.arange(t0, t0 + n, device=device).repeat(len(slots))
        cu, slot = i32([n * i for i in range(len(slots) + 1)]), i32(slots)
        qn = kda.kda_qk_norm_rope_append(q[idx], k[idx], v[idx], rope, pos, pool[0], table, slot, cu, kv_len, wq, wk)
        return kda.kda_window_attention(qn, pool[0], table, slot, cu, kv_len, WINDOW, SINKS, max_tokens=n), qn

    # prefill into row 2, whose pages are scattered over the pool
    row, child = 2, 0
    used = -(-total // PAGE)
    table[row, :used] = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:used].to(device, torch.int32)
    kv_len[row] = prompt
    table[row, -(-prompt // PAGE):] = -1  # pages come with the tokens
    prompt_out, _ = attend(0, prompt, [row], torch.arange(prompt, dtype=torch.int32, device=device))
    cu = i32([0, prompt])
    part = lambda t: t[:prompt].contiguous()
    _, S = kda.kda_layer_core_fused(part(lin.qp), part(lin.kp), part(lin.vp), lin.conv_w, part(lin.z), lin.A, lin.b,
                                    part(lin.beta_logit), part(lin.g), cu, lin.S0)
    S_pool[row] = S[0]
    for s, x in enumerate((lin.qp, lin.kp, lin.vp)):
        for tap in range(min(3, prompt)):  # (zeros before the first token)
            conv_pool[row, s, tap] = x[prompt - 1 - tap]

    # the branch: shared whole pages, a page of its own for the part-filled one, its own state rows
    kda.kda_pages_fork(pool, table, kv_len, i32([row]), i32([child]), PAGE)
    for states in (S_pool[None], conv_pool[None]):
        kda.kda_pages_copy(states, i32([row]), i32([child]))

    slots, att, lin_out = [row, child], [], []
    for i in range(steps):
        t = prompt + i
        if t % PAGE == 0:  # a page for each branch: any that no row names
            free = sorted(set(range(pages)) - set(table.flatten().tolist()))[:branches]
            table[slots, t // PAGE] = i32(free)
        kv_len[slots] = t + 1
        o, qn = attend(t, 1, slots, i32([t] * branches))
        att.append(o)
        pick = lambda x: x[t:t + 1].expand(branches, *x.shape[1:]).contiguous()
        lin_out.append(kda.kda_decode_layer(pick(lin.qp), pick(lin.kp), pick(lin.vp), lin.conv_w, pick(lin.z), lin.A,
                                            lin.b, pick(lin.beta_logit), pick(lin.g), i32(slots), S_pool, conv_pool,
                                            out_dtype=torch.float32))
        kda.kda_pages_release(table, kv_len, i32(slots), PAGE, WINDOW, SINKS)

    kda.kda_pages_release(table, kv_len, i32([child]), PAGE)
    _, live = kda.kda_pages_compact(pool, table)
    again = kda.kda_window_attention(qn[:1], pool[0], table, i32([row]), i32([0, 1]), kv_len, WINDOW, SINKS, max_tokens=1)
    status, detail = kda.kda_get_device_status()
    if status != 0:
        raise RuntimeError(f"device status {status} (detail {detail})")
    return torch.stack(att, 1), torch.stack(lin_out, 1), prompt_out, int(live.item()), again


if __name__ == "__main__":
    att, lin, _, live, _ = run()
    print(f"two branches of a {150}-token prompt, {att.shape[1]} steps: attention |o| {att.float().abs().mean():.4f}, "
          f"KDA |o| {lin.abs().mean():.4f}, branches equal: {torch.equal(att[0], att[1]) and torch.equal(lin[0], lin[1])}, "
          f"{live} pages live at the end")
