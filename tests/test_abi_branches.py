"""Refusals of the operators that decode branches (no GPU needed): bad arguments are turned down on the host
before any launch (nothing is dereferenced in these calls)."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced
MIS = 0x10008   # not 16-byte aligned
ODD = 0x10002   # not 4-byte aligned
BYTE = 0x10001


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def prefix(lib, **kw):
    a = dict(dt=0, batch=2, T=4, most=4, Hq=8, Hkv=2, P=8, page=64, R=3, M=5, Ng=1, q=FAKE, pool=FAKE, table=FAKE,
             slot=FAKE, cu=FAKE, kv_len=FAKE, groups=FAKE, lens=FAKE, scale=0.1, o=2 * FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.kda_prefix_attention(a["dt"], a["batch"], a["T"], a["most"], a["Hq"], a["Hkv"], a["P"], a["page"], a["R"],
                                    a["M"], a["Ng"], a["q"], a["pool"], a["table"], a["slot"], a["cu"], a["kv_len"],
                                    a["groups"], a["lens"], a["scale"], a["o"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(dt=3), dict(dt=-1), dict(batch=0), dict(T=-1), dict(most=0), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(P=0),
    dict(page=0), dict(page=-16), dict(R=0), dict(M=0), dict(Ng=0), dict(Ng=-1), dict(q=None), dict(q=MIS), dict(o=None),
    dict(o=MIS), dict(o=FAKE), dict(pool=None), dict(pool=MIS), dict(table=None), dict(table=ODD), dict(slot=None),
    dict(slot=ODD), dict(cu=None), dict(cu=ODD), dict(kv_len=None), dict(kv_len=ODD), dict(groups=None),
    dict(groups=ODD), dict(lens=None), dict(lens=ODD)])
def test_prefix_rejects_bad_arguments(kda, bad):
    assert prefix(kda.library(), **bad) == 1


@pytest.mark.parametrize("bad", [
    dict(page=48), dict(page=256), dict(page=1), dict(Hq=2 * 129), dict(Hkv=65536, Hq=65536), dict(M=1 << 26),
    dict(P=1 << 24), dict(T=1 << 29), dict(batch=(1 << 20) + 1), dict(Ng=(1 << 20) + 1)])
def test_prefix_unsupported(kda, bad):
    assert prefix(kda.library(), **bad) == 2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefix_workspace(kda, dtype):
    lib, code = kda.library(), 0 if dtype == torch.bfloat16 else 1
    need = kda.kda_prefix_attention_workspace_size(dtype, 2, 4, 1, 8, 2)
    assert need > 0
    assert prefix(lib, dt=code, ws=None) == prefix(lib, dt=code, ws=MIS) == prefix(lib, dt=code, wsb=need - 1) == 3
    for more in ((2, 4000, 1, 8, 2), (2, 4000, 1, 80, 2)):
        assert kda.kda_prefix_attention_workspace_size(dtype, *more) > need
    assert kda.kda_prefix_attention_workspace_size(dtype, 2, 4, 9, 8, 2) >= need  # (nothing is kept by group)
    for bad in ((0, 4, 1, 8, 2), (2, -1, 1, 8, 2), (2, 4, 0, 8, 2), (2, 4, 1, 9, 2), (2, 4, 1, 0, 2), (2, 4, 1, 8, 0)):
        assert kda.kda_prefix_attention_workspace_size(dtype, *bad) == 0


def select(lib, **kw):
    a = dict(dt=0, B=2, K=4, V=1000, N=4, logits=FAKE, stride=1000, scores=FAKE, ended=None, end=-1, parent=FAKE,
             token=FAKE, score=FAKE, over=None, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.kda_beam_select(a["dt"], a["B"], a["K"], a["V"], a["N"], a["logits"], a["stride"], a["scores"], a["ended"],
                               a["end"], a["parent"], a["token"], a["score"], a["over"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(dt=2), dict(B=0), dict(K=0), dict(V=0), dict(N=0), dict(N=-1), dict(stride=999), dict(end=-2), dict(end=1000),
    dict(ended=FAKE), dict(logits=None), dict(logits=BYTE), dict(dt=1, logits=ODD), dict(scores=None), dict(scores=ODD),
    dict(parent=None), dict(parent=ODD), dict(token=None), dict(token=ODD), dict(score=None), dict(score=ODD)])
def test_select_rejects_bad_arguments(kda, bad):
    assert select(kda.library(), **bad) == 1


def test_select_unsupported_and_workspace(kda):
    lib = kda.library()
    for bad in (dict(K=65), dict(N=65), dict(V=(1 << 21) + 1, stride=1 << 22), dict(B=1 << 19)):
        assert select(lib, **bad) == 2
    need = kda.kda_beam_select_workspace_size(2, 4, 1000, 4)
    assert need > 0
    assert select(lib, ws=None) == select(lib, ws=MIS) == select(lib, wsb=need - 1) == 3
    for more in ((3, 4, 1000, 4), (2, 5, 1000, 4), (2, 4, 100000, 4), (2, 4, 1000, 5)):
        assert kda.kda_beam_select_workspace_size(*more) > need
    for bad in ((0, 4, 10, 4), (2, 0, 10, 4), (2, 65, 10, 4), (2, 4, 0, 4), (2, 4, 10, 0), (2, 4, 10, 65)):
        assert kda.kda_beam_select_workspace_size(*bad) == 0


def reorder(lib, **kw):
    a = dict(B=2, K=4, R=9, parent=FAKE, slot=FAKE, src=FAKE, dst=FAKE, L=1, P=8, nbytes=64, page=16, M=3, table=FAKE,
             kv_len=FAKE, pool=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.kda_beam_reorder(a["B"], a["K"], a["R"], a["parent"], a["slot"], a["src"], a["dst"], a["L"], a["P"],
                                a["nbytes"], a["page"], a["M"], a["table"], a["kv_len"], a["pool"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(K=0), dict(R=0), dict(R=7), dict(B=1 << 30), dict(parent=None), dict(parent=ODD), dict(slot=None),
    dict(slot=ODD), dict(src=None), dict(src=ODD), dict(dst=None), dict(dst=ODD), dict(L=0), dict(P=0), dict(nbytes=0),
    dict(nbytes=24), dict(nbytes=-16), dict(page=0), dict(M=0), dict(table=ODD), dict(kv_len=None), dict(kv_len=ODD),
    dict(pool=None), dict(pool=MIS)])
def test_reorder_rejects_bad_arguments(kda, bad):
    assert reorder(kda.library(), **bad) == 1


def test_reorder_unsupported_and_workspace(kda):
    lib = kda.library()
    for bad in (dict(K=65, R=1000), dict(R=(1 << 18) + 1), dict(P=(1 << 20) + 1), dict(M=1 << 28)):
        assert reorder(lib, **bad) == 2
    need = kda.kda_beam_reorder_workspace_size(8, 9)
    assert need > 0
    assert reorder(lib, ws=None) == reorder(lib, ws=MIS) == reorder(lib, wsb=need - 1) == 3


def _arguments():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    return dict(q=torch.zeros((2, 4, 128)), pool=torch.zeros((3, 2, 2, 16, 128)), table=i32(5, 3), slot=i32(1), cu=i32(2),
                kv_len=i32(5), groups=i32(2), lens=i32(1), most=2, logits=torch.zeros((1, 2, 9)), scores=torch.zeros((1, 2)),
                choices=3, ended=None, end=-1, parent=i32(1, 2), beams=i32(1, 2), page=16,
                workspace=torch.zeros(1 << 26, dtype=torch.uint8), o=None, out=None, flags=None)


def _calls(kda, a):
    return {
        "prefix": lambda: kda.kda_prefix_attention(a["q"], a["pool"], a["table"], a["slot"], a["cu"], a["kv_len"],
                                                   a["groups"], a["lens"], max_tokens=a["most"], o=a["o"],
                                                   workspace=a["workspace"]),
        "select": lambda: kda.kda_beam_select(a["logits"], a["scores"], a["choices"], ended=a["ended"], end_token=a["end"],
                                              parent=a["out"], ended_out=a["flags"], workspace=a["workspace"]),
        "reorder": lambda: kda.kda_beam_reorder(a["parent"], a["beams"], a["pool"][None], a["table"], a["kv_len"],
                                                a["page"], workspace=a["workspace"]),
        "slots": lambda: kda.kda_beam_reorder(a["parent"], a["beams"], num_rows=9),
    }


class _NoLaunch:
    """In place of the library: takes down what a call would have launched."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, entry):
        return lambda *a: self.calls.append((entry, a)) or 0


@pytest.mark.parametrize("name", ["prefix", "select", "reorder", "slots"])
def test_binding_refuses_tensors_that_are_not_on_the_gpu(kda, name, monkeypatch):
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    with pytest.raises(ValueError, match="GPU"):
        _calls(kda, _arguments())[name]()
    assert not lib.calls


@pytest.mark.gpu
@pytest.mark.parametrize("name,arg", [("prefix", "table"), ("prefix", "groups"), ("prefix", "lens"), ("prefix", "pool"),
                                      ("prefix", "workspace"), ("select", "scores"), ("select", "workspace"),
                                      ("reorder", "parent"), ("reorder", "kv_len"), ("reorder", "pool"), ("slots", "parent")])
def test_binding_refuses_one_tensor_left_on_the_host(kda, name, arg, monkeypatch):
    a = {x: t.cuda() if isinstance(t, torch.Tensor) and x != arg else t for x, t in _arguments().items()}
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    with pytest.raises(ValueError, match="GPU"):
        _calls(kda, a)[name]()
    assert not lib.calls


I64 = torch.int64


@pytest.mark.parametrize("error,name,change", [
    (TypeError, "prefix", dict(q=torch.zeros((2, 4, 128), dtype=torch.bfloat16))),
    (ValueError, "prefix", dict(q=torch.zeros((2, 4, 64)))),
    (ValueError, "prefix", dict(q=torch.zeros((2, 4, 256))[..., ::2])),
    (ValueError, "prefix", dict(pool=torch.zeros((3, 2, 16, 128)))),
    (ValueError, "prefix", dict(groups=torch.zeros(3, dtype=torch.int32))),
    (TypeError, "prefix", dict(lens=torch.zeros(1, dtype=I64))),
    (ValueError, "prefix", dict(o=torch.zeros((2, 5, 128)))),
    (TypeError, "select", dict(logits=torch.zeros((1, 2, 9), dtype=torch.float16))),
    (ValueError, "select", dict(logits=torch.zeros((1, 2, 18))[..., ::2])),
    (ValueError, "select", dict(logits=torch.zeros((3, 4, 9))[:, :2], scores=torch.zeros((3, 2)))),
    (ValueError, "select", dict(scores=torch.zeros((2, 1)))),
    (TypeError, "select", dict(scores=torch.zeros((1, 2), dtype=torch.float64))),
    (TypeError, "select", dict(ended=torch.zeros((1, 2)), end=1)),
    (ValueError, "select", dict(ended=torch.zeros((2, 1), dtype=torch.bool), end=1)),
    (ValueError, "select", dict(out=torch.zeros((1, 2), dtype=torch.int32))),
    (TypeError, "select", dict(out=torch.zeros((1, 3), dtype=I64))),
    (ValueError, "select", dict(flags=torch.zeros((1, 2), dtype=torch.bool))),
    (ValueError, "reorder", dict(parent=torch.zeros((2, 1), dtype=torch.int32))),
    (TypeError, "reorder", dict(parent=torch.zeros((1, 2), dtype=I64))),
    (ValueError, "reorder", dict(kv_len=torch.zeros(4, dtype=torch.int32))),
    (ValueError, "slots", dict(parent=torch.zeros(2, dtype=torch.int32), beams=torch.zeros(2, dtype=torch.int32)))])
def test_binding_refuses_what_it_cannot_marshal(kda, error, name, change, monkeypatch):
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    monkeypatch.setattr(kda, "_launch", lambda stream, dev: None)  # (it refuses CPU tensors)
    with pytest.raises(error):
        _calls(kda, {**_arguments(), **change})[name]()
    assert not lib.calls
    _calls(kda, _arguments())[name]()
    assert len(lib.calls) == 1


def test_binding_of_reorder_without_a_table(kda, monkeypatch):
    """Half a cache, or no number of rows, is refused."""
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    monkeypatch.setattr(kda, "_launch", lambda stream, dev: None)
    a = _arguments()
    for kw in (dict(), dict(num_rows=9, kv_len=a["kv_len"]), dict(num_rows=9, pool=a["pool"][None]),
               dict(page_table=a["table"], kv_len=a["kv_len"], pool=a["pool"][None], num_rows=4)):
        with pytest.raises(ValueError):
            kda.kda_beam_reorder(a["parent"], a["beams"], **kw)
    assert not lib.calls


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 5, 2 ** 40])
def test_binding_does_not_wrap_large_counts(kda, big, monkeypatch):
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    monkeypatch.setattr(kda, "_launch", lambda stream, dev: None)
    calls = _calls(kda, {**_arguments(), "most": big, "page": big})
    calls["prefix"]()
    calls["reorder"]()
    (_, prefix), (_, reorder) = lib.calls
    assert prefix[3] == 2 ** 31 - 1 and reorder[10] == 2 ** 31 - 1
    for end in (big, -big):  # tokens that the call itself refuses
        _calls(kda, {**_arguments(), "end": end})["select"]()
        assert lib.calls[-1][1][9] == (2 ** 31 - 1 if end > 0 else -2)
    for choices, status in ((big, 2), (65, 2), (0, 1), (-big, 1)):
        with pytest.raises(kda.KdaError) as e:
            _calls(kda, {**_arguments(), "choices": choices})["select"]()
        assert e.value.status == status


STREAMED = ["prefix", "select", "reorder", "slots"]


@pytest.mark.parametrize("name", STREAMED)
def test_what_a_call_allocates_belongs_to_its_stream(kda, name, monkeypatch):
    """Every torch.empty of a call that is given a stream happens while that stream is the current one."""
    import contextlib
    import types
    current, made, launched = [None], [], []

    @contextlib.contextmanager
    def switch(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    real, empty, a = kda.library(), torch.empty, _arguments()

    class Lib:
        def __getattr__(self, entry):
            return getattr(real, entry) if entry.endswith("workspace_size") else lambda *x: launched.append(x[-1]) or 0

    def record(*x, **kw):
        made.append(current[0])
        return empty(*x, **kw)

    monkeypatch.setattr(kda, "_lib", Lib())
    monkeypatch.setattr(kda, "_launch", lambda s, dev: s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch, "empty", record)
    s = types.SimpleNamespace(cuda_stream=0x1230)
    {"prefix": lambda: kda.kda_prefix_attention(a["q"], a["pool"], a["table"], a["slot"], a["cu"], a["kv_len"],
                                                a["groups"], a["lens"], stream=s),
     "select": lambda: kda.kda_beam_select(a["logits"], a["scores"], stream=s),
     "reorder": lambda: kda.kda_beam_reorder(a["parent"], a["beams"], a["pool"][None], a["table"], a["kv_len"], 16, stream=s),
     "slots": lambda: kda.kda_beam_reorder(a["parent"], a["beams"], num_rows=9, stream=s)}[name]()
    assert launched == [0x1230]
    assert made and all(x is s for x in made)


def test_normal_library_refuses_the_injection(kda):
    assert kda.library().kda_debug_inject_prefix_timeout() == 2


@pytest.mark.parametrize("logits,stride", [
    (torch.zeros((6, 40))[:, :33].unsqueeze(1), 40),            # one beam a prompt, out of a padded output
    (torch.zeros((6, 4, 33))[:, :1], 4 * 33),                   # the first of several beams
    (torch.zeros((6, 4, 40))[:, 2:3, :33], 4 * 40),
    (torch.zeros((4, 6, 33)).transpose(0, 1)[:, 1:2], 33),
    (torch.zeros((6, 4, 40))[..., :33], 40),
    (torch.zeros((1, 4, 40))[..., :33], 40),
    (torch.zeros((1, 1, 40))[..., :33], None),                  # one row: any stride does
    (torch.zeros((6, 40))[:, :1].unsqueeze(1), 40)])
def test_binding_takes_rows_that_are_evenly_spaced(kda, logits, stride, monkeypatch):
    """The stride of a dimension of size 1 says nothing about where rows lie."""
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    monkeypatch.setattr(kda, "_launch", lambda stream, dev: None)
    B, K, V = logits.shape
    kda.kda_beam_select(logits, torch.zeros((B, K)), 2, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    (entry, a), = lib.calls
    assert entry == "kda_beam_select" and a[1:4] == (B, K, V) and a[6] >= V and stride in (None, a[6])


class _Cut(ctypes.Structure):
    """PrefixCut of csrc/kda_prefix_attention.cuh."""
    _fields_ = [(x, ctypes.c_int32) for x in ("by_rows", "G", "tile", "keys", "ctas", "slot_rows", "width")] + [("tile_us", ctypes.c_float)]


class _Cache(ctypes.Structure):
    """CacheArgs of csrc/kda_common.cuh."""
    _fields_ = ([(x, ctypes.c_int32) for x in ("batch", "total_tokens", "num_pages", "page_size", "table_rows", "table_width")]
                + [(x, ctypes.c_void_p) for x in ("page_table", "slot", "cu_tokens", "kv_len")])


class _Prefix(ctypes.Structure):
    """PrefixAttentionArgs of csrc/kda_common.cuh."""
    _fields_ = ([(x, ctypes.c_int32) for x in ("dtype", "max_tokens", "num_q_heads", "num_kv_heads", "num_groups")]
                + [(x, ctypes.c_void_p) for x in ("q", "kv_pool", "cu_groups", "prefix_len")]
                + [("scale", ctypes.c_float), ("o", ctypes.c_void_p), ("cache", _Cache), ("workspace", ctypes.c_void_p),
                   ("status", ctypes.c_void_p)])


@pytest.mark.parametrize("name,each", [("prefix_cut_tc", 1), ("prefix_cut_rows", 2)])
@pytest.mark.parametrize("sms", [8, 16, 100, 148, 152])
def test_prefix_launch_fits_the_gpu(kda, name, each, sms):
    """Over the prefixes there are no more CTAs than a GPU of so many SMs holds at once (the launch over the own keys only
    begins when all of them have), and a team of them is no larger than that."""
    cut = getattr(kda.library(), f"_ZN3kda{len(name)}{name}ERKNS_19PrefixAttentionArgsEi")
    cut.restype = _Cut
    for groups, tokens, width in ((1, 4, 3), (1, 4000, 4096), (3, 100000, 1 << 20)):
        a = _Prefix(num_q_heads=96, num_kv_heads=8, num_groups=groups,
                    cache=_Cache(batch=tokens, total_tokens=tokens, num_pages=1 << 20, page_size=64, table_rows=tokens, table_width=width))
        x = cut(ctypes.byref(a), sms)
        assert x.G == 12 and x.ctas == each * sms and 1 <= x.width <= x.ctas
