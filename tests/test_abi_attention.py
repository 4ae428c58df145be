"""Refusals of the paged-cache operators (no GPU needed): bad arguments are turned down on the host
before any launch (nothing is dereferenced in these calls)."""
import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced
MIS = 0x10008   # not 16-byte aligned
ODD = 0x10002   # not 4-byte aligned

OK_CACHE = dict(batch=2, T=4, P=8, page=64, R=3, M=5, table=FAKE, slot=FAKE, cu=FAKE, kv_len=FAKE)


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_kda_gb300 import build
    build.build()
    from gated_delta_rule_kda_gb300 import kda as mod
    return mod


def attention(lib, **kw):
    a = dict(OK_CACHE, dt=0, most=4, Hq=8, Hkv=2, window=16, sinks=1, q=FAKE, pool=FAKE, o=FAKE, scale=0.1)
    a.update(kw)
    return lib.kda_window_attention(a["dt"], a["batch"], a["T"], a["most"], a["Hq"], a["Hkv"], a["P"], a["page"],
                                    a["R"], a["M"], a["window"], a["sinks"], a["q"], a["pool"], a["table"],
                                    a["slot"], a["cu"], a["kv_len"], a["scale"], a["o"], None)


@pytest.mark.parametrize("bad", [
    dict(dt=3), dict(dt=-1), dict(batch=0), dict(T=-1), dict(most=0), dict(Hq=0), dict(Hkv=0), dict(Hq=7),
    dict(P=0), dict(page=0), dict(page=-16), dict(R=0), dict(M=0), dict(window=0), dict(window=-5), dict(sinks=-1),
    dict(q=None), dict(q=MIS), dict(o=None), dict(o=MIS), dict(pool=None), dict(pool=MIS), dict(table=None),
    dict(table=ODD), dict(slot=None), dict(slot=ODD), dict(cu=None), dict(cu=ODD), dict(kv_len=None), dict(kv_len=ODD)])
def test_attention_rejects_bad_arguments(kda, bad):
    assert attention(kda.library(), **bad) == 1


@pytest.mark.parametrize("bad", [
    dict(page=48), dict(page=256), dict(page=1), dict(Hq=2 * 129), dict(Hkv=65536, Hq=65536), dict(M=1 << 26),
    dict(P=1 << 24), dict(T=1 << 29)])
def test_attention_unsupported(kda, bad):
    assert attention(kda.library(), **bad) == 2


def rope(lib, append, **kw):
    a = dict(OK_CACHE, din=0, dout=0, Hq=8, Hkv=2, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, wq=FAKE, wk=None,
             eps=1e-6, norm=1, rope=FAKE, npos=10, rotary=64, inter=0, pos=FAKE, pool=FAKE, qo=FAKE, ko=FAKE)
    a.update(kw)
    if not append:
        return lib.kda_qk_norm_rope(a["din"], a["dout"], a["T"], a["Hq"], a["Hkv"], a["q"], a["qs"], a["k"], a["ks"],
                                    a["wq"], a["wk"], a["eps"], a["norm"], a["rope"], a["npos"], a["rotary"],
                                    a["inter"], a["pos"], a["qo"], a["ko"], None)
    return lib.kda_qk_norm_rope_append(
        a["din"], a["dout"], a["batch"], a["T"], a["Hq"], a["Hkv"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
        a["wq"], a["wk"], a["eps"], a["norm"], a["rope"], a["npos"], a["rotary"], a["inter"], a["pos"], a["P"],
        a["page"], a["R"], a["M"], a["table"], a["slot"], a["cu"], a["kv_len"], a["pool"], a["qo"], None)


COMMON = [dict(din=2), dict(dout=-1), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(q=None), dict(q=MIS), dict(k=MIS),
          dict(qs=1023), dict(qs=1025), dict(ks=255), dict(ks=260), dict(wq=MIS), dict(wk=MIS), dict(norm=2),
          dict(inter=-1), dict(rope=None), dict(rope=MIS), dict(npos=0), dict(rotary=-16), dict(rotary=144),
          dict(pos=None), dict(pos=ODD), dict(qo=None), dict(qo=MIS)]


@pytest.mark.parametrize("bad", COMMON + [dict(ko=None), dict(ko=MIS)])
def test_norm_rope_rejects_bad_arguments(kda, bad):
    assert rope(kda.library(), False, **bad) == 1


@pytest.mark.parametrize("bad", COMMON + [dict(v=None), dict(v=MIS), dict(vs=4), dict(pool=None), dict(pool=MIS),
                                          dict(batch=0), dict(P=0), dict(page=0), dict(R=0), dict(M=0),
                                          dict(table=None), dict(slot=ODD), dict(cu=None), dict(kv_len=None)])
def test_norm_rope_append_rejects_bad_arguments(kda, bad):
    assert rope(kda.library(), True, **bad) == 1


def test_norm_rope_unsupported(kda):
    lib = kda.library()
    assert rope(lib, False, rotary=24) == rope(lib, True, rotary=8) == 2
    assert rope(lib, False, T=1 << 30) == 2
    assert rope(lib, True, page=24) == rope(lib, True, M=1 << 27) == rope(lib, True, P=1 << 24) == 2


def copy(lib, **kw):
    a = dict(L=1, P=8, nbytes=64, n=2, src=FAKE, dst=FAKE, pool=FAKE)
    a.update(kw)
    return lib.kda_pages_copy(a["L"], a["P"], a["nbytes"], a["n"], a["src"], a["dst"], a["pool"], None)


POOL = [dict(L=0), dict(P=0), dict(nbytes=0), dict(nbytes=24), dict(nbytes=-16), dict(pool=None), dict(pool=MIS)]


@pytest.mark.parametrize("bad", POOL + [dict(n=-1), dict(src=None), dict(dst=ODD)])
def test_copy_rejects_bad_arguments(kda, bad):
    assert copy(kda.library(), **bad) == 1


def fork(lib, **kw):
    a = dict(L=1, P=8, nbytes=64, page=16, R=4, M=3, F=2, parent=FAKE, child=FAKE, table=FAKE, kv_len=FAKE, pool=FAKE,
             ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.kda_pages_fork(a["L"], a["P"], a["nbytes"], a["page"], a["R"], a["M"], a["F"], a["parent"], a["child"],
                              a["table"], a["kv_len"], a["pool"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", POOL + [dict(page=0), dict(R=0), dict(M=0), dict(F=-1), dict(F=5), dict(parent=None),
                                        dict(child=ODD), dict(table=None), dict(kv_len=ODD)])
def test_fork_rejects_bad_arguments(kda, bad):
    assert fork(kda.library(), **bad) == 1


def compact(lib, **kw):
    a = dict(L=1, P=8, nbytes=64, R=4, M=4, tin=FAKE, tout=FAKE + 64, live=FAKE, pool=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.kda_pages_compact(a["L"], a["P"], a["nbytes"], a["R"], a["M"], a["tin"], a["tout"], a["live"],
                                 a["pool"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", POOL + [dict(R=0), dict(M=0), dict(tin=None), dict(tout=ODD), dict(live=None),
                                        dict(tout=FAKE + 60)])
def test_compact_rejects_bad_arguments(kda, bad):
    assert compact(kda.library(), **bad) == 1


def test_pages_workspace_and_limits(kda):
    lib = kda.library()
    need = kda.kda_pages_workspace_size(8, 4)
    assert need > 0 and kda.kda_pages_workspace_size(8, 40) > need
    for call in (fork, compact):
        assert call(lib, ws=None) == call(lib, ws=MIS) == call(lib, wsb=need - 1) == 3
        assert call(lib, P=(1 << 20) + 1) == call(lib, R=(1 << 18) + 1, M=1, **({"tout": FAKE} if call is compact else {})) == 2
    assert fork(lib, M=1 << 28) == 2


def release(lib, **kw):
    a = dict(R=4, M=3, page=16, n=2, rows=FAKE, window=0, sinks=0, table=FAKE, kv_len=FAKE)
    a.update(kw)
    return lib.kda_pages_release(a["R"], a["M"], a["page"], a["n"], a["rows"], a["window"], a["sinks"], a["table"],
                                 a["kv_len"], None)


@pytest.mark.parametrize("bad", [dict(R=0), dict(M=0), dict(page=0), dict(n=-1), dict(rows=None), dict(window=-1),
                                 dict(sinks=-1), dict(table=None), dict(kv_len=ODD)])
def test_release_rejects_bad_arguments(kda, bad):
    assert release(kda.library(), **bad) == 1
    assert release(kda.library(), M=1 << 28) == 2


def test_binding_refuses_what_it_cannot_marshal(kda):
    """Types, layouts and lengths that the C call cannot see are refused by the binding (CPU tensors)."""
    q, pool = torch.zeros((2, 4, 128)), torch.zeros((3, 2, 2, 16, 128))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(page_table=i32(2, 3), slot=i32(1), cu_tokens=i32(2), kv_len=i32(2))
    for error, change, x, p in [
            (TypeError, {}, q.bfloat16(), pool), (ValueError, {}, q, pool[0]),
            (ValueError, dict(cu_tokens=i32(3)), q, pool), (ValueError, dict(kv_len=i32(3)), q, pool),
            (TypeError, dict(slot=torch.zeros(1, dtype=torch.int64)), q, pool),
            (ValueError, {}, torch.zeros((2, 4, 256))[..., ::2], pool)]:
        with pytest.raises(error):
            c = {**good, **change}
            kda.kda_window_attention(x, p, c["page_table"], c["slot"], c["cu_tokens"], c["kv_len"], 4)
    with pytest.raises(ValueError):  # heads that do not lie side by side
        kda.kda_qk_norm_rope(torch.zeros((2, 8, 128))[:, ::2], q, None, None)
    with pytest.raises(ValueError):
        kda.kda_qk_norm_rope(q, torch.zeros((3, 4, 128)), None, None)
    with pytest.raises(ValueError):
        kda.kda_qk_norm_rope(q, q, torch.zeros((9, 8, 2)), i32(5))
    with pytest.raises(ValueError):
        kda.kda_pages_copy(torch.zeros((1, 4, 8)), i32(2), i32(3))
    with pytest.raises(ValueError):
        kda.kda_pages_copy(torch.zeros((4, 8)), i32(2), i32(2))


def _binding_arguments():
    """Arguments that every paged-cache call of the binding takes, on the CPU."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    return dict(q=torch.zeros((2, 4, 128)), k=torch.zeros((2, 2, 128)), v=torch.zeros((2, 2, 128)),
                rope=torch.zeros((9, 8, 2)), positions=i32(2), pool=torch.zeros((3, 2, 2, 16, 128)), table=i32(2, 3),
                slot=i32(1), cu=i32(2), kv_len=i32(2), wq=torch.zeros(128), wk=torch.zeros(128), rows=i32(1),
                workspace=torch.zeros(1 << 12, dtype=torch.uint8), live=i32(1), window=16, sinks=1, most=2, page=16)


def _binding_calls(kda, a):
    cache = (a["pool"], a["table"], a["slot"], a["cu"], a["kv_len"])
    return {
        "rope": lambda: kda.kda_qk_norm_rope(a["q"], a["k"], a["rope"], a["positions"], a["wq"], a["wk"]),
        "append": lambda: kda.kda_qk_norm_rope_append(a["q"], a["k"], a["v"], a["rope"], a["positions"], *cache, a["wq"],
                                                      a["wk"]),
        "attention": lambda: kda.kda_window_attention(a["q"], *cache, a["window"], a["sinks"], max_tokens=a["most"]),
        "copy": lambda: kda.kda_pages_copy(a["pool"][None], a["rows"], a["rows"]),
        "fork": lambda: kda.kda_pages_fork(a["pool"][None], a["table"], a["kv_len"], a["rows"], a["rows"], a["page"],
                                           workspace=a["workspace"]),
        "release": lambda: kda.kda_pages_release(a["table"], a["kv_len"], a["rows"], a["page"], a["window"], a["sinks"]),
        "compact": lambda: kda.kda_pages_compact(a["pool"][None], a["table"], num_live=a["live"],
                                                 workspace=a["workspace"]),
    }


class _NoLaunch:
    """In place of the library: takes down what a call would have launched."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, entry):
        return lambda *a: self.calls.append((entry, a)) or 0


@pytest.mark.parametrize("name", ["rope", "append", "attention", "copy", "fork", "release", "compact"])
def test_binding_refuses_tensors_that_are_not_on_the_gpu(kda, name, monkeypatch):
    """Host addresses never reach a kernel."""
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    with pytest.raises(ValueError, match="GPU"):
        _binding_calls(kda, _binding_arguments())[name]()
    assert not lib.calls


@pytest.mark.gpu
@pytest.mark.parametrize("name,arg", [("rope", "rope"), ("rope", "positions"), ("rope", "wk"), ("append", "v"),
                                      ("append", "slot"), ("append", "cu"), ("attention", "table"),
                                      ("attention", "kv_len"), ("copy", "rows"), ("fork", "kv_len"),
                                      ("fork", "workspace"), ("release", "rows"), ("compact", "live")])
def test_binding_refuses_one_tensor_left_on_the_host(kda, name, arg, monkeypatch):
    a = {x: t.cuda() if isinstance(t, torch.Tensor) and x != arg else t for x, t in _binding_arguments().items()}
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    with pytest.raises(ValueError, match="GPU"):
        _binding_calls(kda, a)[name]()
    assert not lib.calls


@pytest.mark.parametrize("name,change", [
    ("rope", dict(wq=torch.zeros(127))), ("rope", dict(wk=torch.zeros(1))), ("append", dict(wq=torch.zeros(64))),
    ("append", dict(wk=torch.zeros(0))), ("rope", dict(rope=torch.zeros((9, 8, 1)))),
    ("append", dict(rope=torch.zeros((9, 16, 1)))), ("rope", dict(rope=torch.zeros((9, 4, 4)))),
    ("append", dict(rope=torch.zeros((9, 16))))])
def test_binding_refuses_weights_and_tables_of_another_shape(kda, name, change, monkeypatch):
    """The C call cannot see that a weight is not [128] or a table not [positions, rotary_dim / 2, 2]: the kernel would
    read past their ends."""
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    monkeypatch.setattr(kda, "_launch", lambda stream, dev: None)  # (it refuses CPU tensors)
    with pytest.raises(ValueError):
        _binding_calls(kda, {**_binding_arguments(), **change})[name]()
    assert not lib.calls
    _binding_calls(kda, _binding_arguments())[name]()
    assert len(lib.calls) == 1


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40])
def test_binding_does_not_wrap_large_counts(kda, big, monkeypatch):
    """A window, sink count or token bound past 2^31 - 1 means no more than that; a page size is refused by the call
    itself (which sees one that no cache has)."""
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    monkeypatch.setattr(kda, "_launch", lambda stream, dev: None)  # (it refuses CPU tensors)
    most = 2 ** 31 - 1
    calls = _binding_calls(kda, {**_binding_arguments(), "window": big, "sinks": big, "most": big, "page": big})
    for name in ("attention", "release", "fork"):
        calls[name]()
    (_, attention), (_, release), (_, fork) = lib.calls
    assert attention[3] == most and attention[10:12] == (most, most)
    assert release[2] == most and release[5:7] == (most, most)
    assert fork[3] == most
    calls = _binding_calls(kda, {**_binding_arguments(), "window": -big, "sinks": -big, "most": -big})
    for name in ("attention", "release"):
        calls[name]()
    (_, attention), (_, release) = lib.calls[3:]
    assert attention[3] < 0 and attention[10] < 0 and attention[11] < 0 and release[5] < 0 and release[6] < 0


def test_binding_refuses_more_pages_than_the_call_can_count(kda, monkeypatch):
    """[1, 2^32 + 8, 16] bytes: the page count would wrap to 8."""
    lib = _NoLaunch()
    monkeypatch.setattr(kda, "_lib", lib)
    monkeypatch.setattr(kda, "_launch", lambda stream, dev: None)
    pool = torch.zeros(16, dtype=torch.uint8).expand(1, 2 ** 32 + 8, 16)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="pages"):
        kda.kda_pages_copy(pool, one, one)
    assert not lib.calls
