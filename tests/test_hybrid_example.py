"""The hybrid example end to end: prefill, fork, decode of both branches, trim, release, compact."""
import numpy as np
import pytest
import torch

from tests._cache import attention64, rope64
from tests._parity import to64

pytestmark = pytest.mark.gpu


def test_hybrid_example_against_64_bits():
    """Both branches answer alike, and as one request's attention over all tokens (tolerance: that of the
    attention tests, with q and k rounded to bf16 as the cache holds them)."""
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import hybrid_example as ex, kda
    prompt, steps, heads, kv = 150, 24, 8, 2
    att, lin, first, live, _ = ex.run(prompt, steps)
    assert torch.equal(att[0], att[1]) and torch.equal(lin[0], lin[1])
    total = prompt + steps
    # at the end one row is left: the pages of its window and of the sinks
    assert live == len({j // ex.PAGE for j in range(total) if j > total - ex.WINDOW or j < ex.SINKS})
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    qkv = torch.randn((total, heads + 2 * kv, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    wq, wk = (1 + 0.1 * torch.randn(128, generator=g, device="cuda") for _ in range(2))
    table, pos = kda.rope_table(total, 64, base=500000.0), torch.arange(total, dtype=torch.int32, device="cuda")
    turn = lambda x, w: torch.from_numpy(rope64(x, w, table, pos, 64, False, True)).to(torch.bfloat16)
    q, k = turn(qkv[:, :heads], wq), turn(qkv[:, heads:heads + kv], wk)
    pool = torch.zeros((1, 2, kv, 256, 128), dtype=torch.bfloat16)
    pool[0, 0, :, :total] = k.transpose(0, 1)
    pool[0, 1, :, :total] = qkv[:, heads + kv:].transpose(0, 1).cpu()
    cache = dict(pool=pool, table=torch.zeros((1, 1), dtype=torch.int32), slot=torch.zeros(1, dtype=torch.int32),
                 kv_len=torch.tensor([total], dtype=torch.int32))
    ref, a = attention64(q, cache, [total], ex.WINDOW, ex.SINKS)
    got = np.concatenate([to64(first), to64(att[0])])
    # k and q may round to the neighbouring bf16 where fp32 and 64 bits fall either side of a tie: one
    # ulp (2^-8) of one of 128 products, some 2^-8 |q_i k_i| scale < 2^-9 of a score unit
    assert (np.abs(got - ref) <= 2.0 ** -8 * (a + np.abs(ref)) + 2.0 ** -8 * a).all()


def test_hybrid_example_answers_alike_after_release_and_compaction():
    """The last token asked once more, of the row that is left in the compacted cache: the same keys and values in other
    pages.  Window and sinks are two key tiles, which one CTA takes whatever the batch, so the bits are the same."""
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import hybrid_example as ex
    att, _, _, _, again = ex.run(150, 24)
    assert att.float().abs().max() > 0.1
    assert torch.equal(again[0], att[0, -1])


@pytest.mark.parametrize("prompt", [150, 64])
def test_hybrid_example_recurrent_layer_against_the_oracle(prompt):
    """The KDA layer's prefill, its states handed to the pools and to the branch, and the decode of both branches: one
    run of the oracle over prompt and steps, at the layer's tolerance."""
    import oracle
    from gated_delta_rule_kda_gb300 import build, synthetic
    from tests._parity import assert_gated_close
    build.build()
    from gated_delta_rule_kda_gb300 import hybrid_example as ex
    steps, heads = 24, 4
    _, lin, _, _, _ = ex.run(prompt, steps)
    inp = synthetic.layer_inputs([prompt + steps], heads, seed=0, s0_std=0.1, device="cuda")
    conv_w = to64(inp.conv_w).reshape(3, heads * 128, 4)
    f = to64
    o, _ = oracle.kda_layer_core(f(inp.qp), f(inp.kp), f(inp.vp), conv_w, f(inp.z), f(inp.A), f(inp.b),
                                 f(inp.beta_logit), f(inp.g), inp.cu_seqlens.cpu().numpy(), f(inp.S0))
    for branch in range(2):
        assert_gated_close(to64(lin[branch]), o[prompt:], False, f"branch {branch}")


@pytest.mark.parametrize("prompt", [1, 2])
def test_hybrid_example_with_a_prompt_shorter_than_the_convolution(prompt):
    """The convolution state of a prompt of fewer than three tokens has zeros for those before its first."""
    test_hybrid_example_recurrent_layer_against_the_oracle(prompt)
