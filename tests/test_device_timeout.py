"""A device-side wait that runs out, on purpose, in the one safe form.

Every wait inside the tensor-core prefill is bounded; when one gives up, the kernel records
KDA_ERR_DEVICE_TIMEOUT with the place it waited, leaves through its normal exit (the final
barrier and the release of its tensor memory), and the context stays usable.  The debug
library (KDA_DEBUG) can arm one launch in which the warps that build a chunk's operands skip
their first "chunk ready" hand-off before anything is issued into that chunk's slot, with
every wait limited to 1 ms, so that the consuming warps' wait for the chunk runs out with no
copy or tensor-core product in flight.  Nothing faults, traps or hangs: the test checks the
reported status, then that the next prefill through the same library is correct.
"""
import ctypes
import time

import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_kda_gb300 import synthetic
from tests._parity import TOL_BF16, assert_close, to64

TIMEOUT = 5
UNSUPPORTED = 2
WAIT_FOR_READY_CHUNK = 20


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def test_normal_library_refuses_the_injection(kda):
    """Only the debug library arms anything; the normal one says so and changes nothing."""
    assert kda.library().kda_debug_inject_handoff_timeout() == UNSUPPORTED


def _prefill(lib, inp, o, S_final, stream):
    P = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None
    T, H = inp.q.shape[:2]
    N = inp.cu_seqlens.numel() - 1
    return lib.kda_prefill(0, 1, N, T, H, P(inp.q), P(inp.k), P(inp.v), P(inp.log_alpha),
                           P(inp.beta), None, P(inp.cu_seqlens), 1.0 / np.sqrt(128.0), P(o),
                           P(S_final), None, 0, stream)


@pytest.mark.gpu
def test_debug_library_reports_a_wait_that_runs_out(kda):
    from gated_delta_rule_kda_gb300 import build
    lib = ctypes.CDLL(build.build(debug=True))
    lib.kda_prefill.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int32, ctypes.c_int32,
                                ctypes.c_int32] + [ctypes.c_void_p] * 7 + [
                                ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.kda_get_device_status.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    lib.kda_debug_inject_handoff_timeout.argtypes = []
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    detail = ctypes.c_uint32(0)
    assert lib.kda_get_device_status(stream, ctypes.byref(detail)) == 0

    # two chunks (50 tokens) per (sequence, head): the skipped hand-off is the only one the
    # consuming warps wait for, and the building warps finish on their own
    inp = synthetic.prefill_inputs([50], 2, torch.bfloat16, seed=61, device="cuda")
    o = torch.zeros((50, 2, 128), dtype=torch.float32, device="cuda")
    Sf = torch.zeros((1, 2, 128, 128), dtype=torch.float32, device="cuda")
    assert lib.kda_debug_inject_handoff_timeout() == 0
    assert _prefill(lib, inp, o, Sf, stream) == 0
    assert lib.kda_get_device_status(stream, ctypes.byref(detail)) == TIMEOUT
    assert detail.value == WAIT_FOR_READY_CHUNK

    # the injection was for that launch only: the next prefill is whole and correct
    assert _prefill(lib, inp, o, Sf, stream) == 0
    assert lib.kda_get_device_status(stream, ctypes.byref(detail)) == 0
    f = to64
    ref_o, ref_S = oracle.kda_prefill(f(inp.q), f(inp.k), f(inp.v), f(inp.log_alpha),
                                      f(inp.beta), inp.cu_seqlens.cpu().numpy())
    assert_close(to64(o), ref_o, TOL_BF16, "o after the timed-out launch")
    assert_close(to64(Sf), ref_S, TOL_BF16, "S_final after the timed-out launch")


def test_normal_library_refuses_the_attention_injection(kda):
    assert kda.library().kda_debug_inject_attention_timeout() == UNSUPPORTED


# (tokens of each request, tokens before them, window, details): one token a row and a few (the kernel for short
# steps, a row over one CTA and over several), a prefill, and a short step behind a long row (CTAs that share an item)
ATTENTION = [([1], [100], 60, [97]), ([2, 1], [3000, 500], 2 ** 31 - 1, [97]), ([300, 20], [50, 0], 50, range(64, 128)),
             ([40], [3000], 2 ** 31 - 1, range(64, 128))]


@pytest.mark.gpu
@pytest.mark.parametrize("new,old,window,details", ATTENTION)
def test_debug_library_reports_attention_waits_that_run_out(kda, new, old, window, details):
    """The load warps fetch nothing, so every other warp's wait runs out: the launch leaves with the status, o as it
    was, and the next call is right."""
    _attention_gives_up(kda, new, old, window, details)


@pytest.mark.gpu
@pytest.mark.parametrize("new,old,window,details", ATTENTION)
def test_attention_that_gives_up_waits_only_for_what_is_in_flight(kda, new, old, window, details):
    """With every wait limited to 1 ms the launch is over in far less than the 2 s of one unlimited wait."""
    assert _attention_gives_up(kda, new, old, window, details) < 0.5


def _attention_gives_up(kda, new, old, window, details):
    from gated_delta_rule_kda_gb300 import build
    from tests._cache import build_cache, cu_of, queries
    c = build_cache([a + b for a, b in zip(new, old)], 32, 2, torch.bfloat16, seed=59)
    q, cu = queries(sum(new), 8, torch.bfloat16, 59), cu_of(new)
    want = kda.kda_window_attention(q, c["pool"], c["table"], c["slot"], cu, c["kv_len"], window, 4, max_tokens=max(new))
    assert kda.kda_get_device_status()[0] == 0
    lib = ctypes.CDLL(build.build(debug=True))
    lib.kda_window_attention.argtypes = kda.library().kda_window_attention.argtypes
    lib.kda_get_device_status.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    lib.kda_debug_inject_attention_timeout.argtypes = []
    stream, detail = torch.cuda.current_stream().cuda_stream, ctypes.c_uint32(0)
    o = torch.full_like(q, -7.0)

    def attend():
        R, M = c["table"].shape
        P, _, Hkv, page, _ = c["pool"].shape
        assert lib.kda_window_attention(0, len(new), sum(new), max(new), 8, Hkv, P, page, R, M, window, 4, q.data_ptr(),
                                        c["pool"].data_ptr(), c["table"].data_ptr(), c["slot"].data_ptr(), cu.data_ptr(),
                                        c["kv_len"].data_ptr(), 128 ** -0.5, o.data_ptr(), stream) == 0
        return lib.kda_get_device_status(stream, ctypes.byref(detail))

    assert lib.kda_debug_inject_attention_timeout() == 0
    t0 = time.perf_counter()
    assert attend() == TIMEOUT and detail.value in details
    taken = time.perf_counter() - t0
    assert bool((o == -7.0).all())
    assert attend() == 0 and torch.equal(o, want)
    return taken
