"""Refusals of the cache entry points, on the CPU: the library's status codes for bad
arguments (nothing is launched) and the binding's checks of tensors."""
import pytest
import torch

from sparse_long_sequence_dilated_b200 import dilattn

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = 0, 1, 2, 3, 4
MB = 1 << 20
FAKE = 64 * MB  # fake device addresses, 16 MiB apart; never dereferenced by a refused call
A = {n: FAKE + 16 * MB * i for i, n in enumerate(
    ("k", "v", "offsets", "start", "table", "kc", "vc", "ks", "vs", "q", "seq", "pos", "out", "lse", "ws"))}

CACHE = dict(pages=6, Hkv=2, P=16, d=64, fmt=0)
BAD_CACHE = [dict(pages=0), dict(Hkv=0), dict(P=8), dict(P=48), dict(P=256), dict(fmt=2), dict(fmt=-1),
             dict(B=0), dict(max_pages=0), dict(max_pages=1 << 27), dict(pages=1 << 30),
             dict(kc=None), dict(vc=A["vc"] + 8), dict(ks=A["ks"] + 4), dict(table=A["table"] + 2),
             dict(vc=A["kc"]), dict(vs=A["ks"]), dict(ks=A["kc"] + 1024), dict(table=A["vc"])]


def _write(**kw):
    a = dict(A, **CACHE, T=3, B=3, max_pages=4, sk=128, sv=128)
    a.update(kw)
    return dilattn.load().dilattn_cache_write(
        a["k"], a["v"], a["sk"], a["sv"], a["offsets"], a["start"], a["T"], a["table"], a["B"],
        a["max_pages"], a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["Hkv"], a["P"], a["d"], a["fmt"], None)


def _read(**kw):
    a = dict(A, **CACHE, T=3, B=3, max_pages=4, sk=128, sv=128)
    a.update(kw)
    return dilattn.load().dilattn_cache_read(
        a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["Hkv"], a["P"], a["d"], a["fmt"], a["table"], a["B"],
        a["max_pages"], a["offsets"], a["start"], a["T"], a["k"], a["v"], a["sk"], a["sv"], None)


def _decode(pats=((64, 1), (128, 2)), **kw):
    a = dict(A, **CACHE, T=3, B=3, max_pages=4, H=4, sq=256, wsb=None)
    a.update(kw)
    w, r, n = dilattn._patterns(pats)
    need = dilattn.decode_workspace_size(max(a["T"], 1), max(a["H"], 2), 2, 64)
    return dilattn.load().dilattn_decode(
        a["q"], a["sq"], a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["Hkv"], a["P"], a["d"], a["fmt"],
        a["table"], a["B"], a["max_pages"], a["seq"], a["pos"], a["out"], a["lse"], a["T"], a["H"], w, r, n,
        a["ws"], need if a["wsb"] is None else a["wsb"], None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU the call would launch on fake addresses")
@pytest.mark.parametrize("call", [_write, _read, _decode])
def test_the_unchanged_call_passes_the_checks(call):
    assert call() == CUDA  # it ends at the device lookup


@pytest.mark.parametrize("call", [_write, _read, _decode])
@pytest.mark.parametrize("kw", BAD_CACHE)
def test_bad_caches(call, kw):
    assert call(**kw) == INVALID


@pytest.mark.parametrize("call", [_write, _read, _decode])
def test_head_sizes(call):
    assert call(d=96) == UNSUPPORTED


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(offsets=None, T=2), dict(offsets=A["offsets"] + 1), dict(start=None), dict(start=A["start"] + 2),
    dict(k=None), dict(v=A["v"] + 8), dict(sk=127), dict(sk=120), dict(sv=132), dict(sv=-128),
    dict(k=A["kc"]), dict(v=A["ks"]), dict(v=A["vc"] + 64)])
def test_bad_token_batches(call, kw):
    assert call(**kw) == INVALID


def test_write_and_read_overlaps():
    assert _read(v=A["k"]) == INVALID                       # two outputs
    assert _read(v=A["k"] + 128) == INVALID                 # rows of 256 bytes, 256 apart
    assert _read(v=A["k"] + 384, sk=256, sv=256) == INVALID
    assert _read(v=A["k"] + 128, sk=256, sv=256) == INVALID
    assert _read(v=A["k"] + 256, sk=256, sv=128) == INVALID
    assert _read(k=A["offsets"] - 64) == INVALID
    assert _write(start=A["vs"]) == INVALID                 # an input inside the cache
    # the first token ends before the cache, the last one lies in it
    assert _write(k=A["kc"] - 256 - 8192, sk=4096) == INVALID


@pytest.mark.parametrize("call", [_write, _read, _decode])
def test_no_tokens_is_no_work(call):
    kw = dict(T=0, k=None, v=None, q=None, pos=None, out=None, lse=None)
    assert call(**kw) == OK


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(H=3), dict(seq=None, T=4), dict(seq=A["seq"] + 1), dict(pos=None), dict(pos=A["pos"] + 2),
    dict(pats=()), dict(pats=((0, 1),)), dict(pats=((8, 0),)), dict(pats=tuple((8, 1) for _ in range(17))),
    dict(q=None), dict(q=A["q"] + 8), dict(sq=255), dict(sq=248), dict(out=None), dict(out=A["out"] + 4), dict(lse=A["lse"] + 4),
    dict(out=A["q"]), dict(out=A["kc"]), dict(lse=A["out"]), dict(lse=A["vs"]), dict(ws=A["out"] + 256), dict(ws=A["q"])])
def test_bad_decodes(kw):
    assert _decode(**kw) == INVALID


def test_decode_workspaces():
    size = dilattn.decode_workspace_size
    assert size(0, 2, 1, 64) == size(1, 3, 2, 64) == size(1, 2, 1, 96) == 0
    assert _decode(ws=None) == WORKSPACE
    assert _decode(ws=A["ws"] + 64) == WORKSPACE
    assert _decode(wsb=size(3, 4, 2, 64) - 1) == WORKSPACE


# ------------------------------------------------------------------ the binding
def _tensors(fmt=torch.int8):
    c = dilattn.Cache(torch.zeros((6, 2, 16, 64), dtype=fmt), torch.zeros((6, 2, 16, 64), dtype=fmt),
                      torch.ones((6, 2)), torch.ones((6, 2)))
    z = lambda *s: torch.zeros(s, dtype=torch.int32)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    return c, z(3, 4), z(3), x, torch.zeros((3, 4, 64), dtype=torch.bfloat16)


def test_wrappers_refuse_host_tensors():
    c, table, start, x, q = _tensors()
    for call in (lambda: dilattn.cache_write(c, x, x, table, start), lambda: dilattn.cache_read(c, table, start),
                 lambda: dilattn.decode(q, c, table, start, [(8, 1)])):
        with pytest.raises(ValueError, match="must be on a CUDA device"):
            call()


def test_new_cache_formats():
    assert dilattn.new_cache(2, 1, 16, 64, "int8", "cpu").k.dtype == torch.int8
    assert dilattn.new_cache(2, 1, 16, 64, "e4m3", "cpu").v.dtype == torch.float8_e4m3fn
    with pytest.raises(ValueError, match="fmt"):
        dilattn.new_cache(2, 1, 16, 64, "bf16", "cpu")


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_size") else 0
        return fn


@pytest.fixture
def rec(monkeypatch):
    """A recording stand-in for the library, with the device check relaxed."""
    r = _Recorder()
    orig = dilattn._need

    def need_on_host(t, name, shape, dtypes, device=None):
        try:
            orig(t, name, shape, dtypes)
        except ValueError as e:
            if "must be on" not in str(e):
                raise

    monkeypatch.setattr(dilattn, "load", lambda *a, **k: r)
    monkeypatch.setattr(dilattn, "_need", need_on_host)
    monkeypatch.setattr(dilattn, "_stream_handle", lambda s: 1234)
    return r


@pytest.mark.parametrize("fmt,code", [(torch.float8_e4m3fn, 0), (torch.int8, 1)])
def test_marshalling(rec, fmt, code):
    c, table, start, x, q = _tensors(fmt)
    offsets = torch.zeros(4, dtype=torch.int32)
    cp = (c.k.data_ptr(), c.v.data_ptr(), c.k_scale.data_ptr(), c.v_scale.data_ptr(), 6, 2, 16, 64, code)
    wide = torch.zeros((3, 6, 64), dtype=torch.bfloat16)  # a fused projection: q, k and v side by side
    k, v = wide[:, 2:4], wide[:, 4:6]
    dilattn.cache_write(c, k, v, table, start, offsets)
    assert rec.calls[-1] == ("dilattn_cache_write", (
        k.data_ptr(), v.data_ptr(), 384, 384, offsets.data_ptr(), start.data_ptr(), 3, table.data_ptr(), 3, 4,
        *cp, 1234))
    dilattn.cache_write(c, x, x, table, start)
    assert rec.calls[-1][1][2:5] == (128, 128, None)
    kk, vv = dilattn.cache_read(c, table, start, offsets, 5)
    assert kk.shape == (5, 2, 64)
    assert rec.calls[-1] == ("dilattn_cache_read", (
        *cp, table.data_ptr(), 3, 4, offsets.data_ptr(), start.data_ptr(), 5, kk.data_ptr(), vv.data_ptr(), 128, 128,
        1234))
    ws = torch.zeros(512, dtype=torch.uint8)
    out, lse = dilattn.decode(q, c, table, start, [(8, 1), (16, 2)], seq=start, workspace=ws)
    name, a = rec.calls[-1]
    assert name == "dilattn_decode"
    assert a[:20] == (q.data_ptr(), 256, *cp, table.data_ptr(), 3, 4, start.data_ptr(), start.data_ptr(),
                      out.data_ptr(), lse.data_ptr(), 3, 4)
    assert (list(a[20])[:2], list(a[21])[:2], *a[22:]) == ([8, 16], [1, 2], 2, ws.data_ptr(), 512, 1234)
    dilattn.decode(q, c, table, start, [(8, 1)])
    assert rec.calls[-2] == ("dilattn_decode_workspace_size", (3, 4, 2, 64)) and rec.calls[-1][1][14] is None


@pytest.mark.parametrize("change,match", [
    (lambda t: t.update(c=t["c"]._replace(v=t["c"].v[:5])), "cache.v: shape"),
    (lambda t: t.update(c=t["c"]._replace(v=t["c"].v.view(torch.uint8))), "cache.v: dtype"),
    (lambda t: t.update(c=t["c"]._replace(k_scale=t["c"].k_scale.double())), "cache.k_scale: dtype"),
    (lambda t: t.update(c=t["c"]._replace(v_scale=t["c"].v_scale[:, :1])), "cache.v_scale: shape"),
    (lambda t: t.update(table=t["table"].long()), "table: dtype"),
    (lambda t: t.update(table=t["table"][0]), r"expected a \[B, max_pages\] table"),
    (lambda t: t.update(table=t["table"].t()), "table must be contiguous"),
    (lambda t: t.update(start=t["start"][:2]), "(start|pos): shape"),
    (lambda t: t.update(start=t["start"].long()), "(start|pos): dtype"),
])
def test_bad_cache_tensors(rec, change, match):
    c, table, start, x, q = _tensors()
    t = dict(c=c, table=table, start=start)
    change(t)
    for call in (lambda: dilattn.cache_write(t["c"], x, x, t["table"], t["start"]),
                 lambda: dilattn.decode(q, t["c"], t["table"], t["start"], [(8, 1)])):
        with pytest.raises(ValueError, match=match):
            call()
    assert not rec.calls


def test_bad_token_tensors(rec):
    c, table, start, x, q = _tensors()
    w = dilattn.cache_write
    wide = torch.zeros((3, 260), dtype=torch.bfloat16)
    for call, match in (
            (lambda: w(c, x[:2], x, table, start), "v: shape"),
            (lambda: w(c, x[:2], x[:2], table, start), "2 tokens without offsets"),
            (lambda: w(c, x.half(), x, table, start), "k: dtype"),
            (lambda: w(c, x, x[:, :1].expand(3, 2, 64), table, start), "v must be contiguous"),
            (lambda: w(c, x[:1].expand(3, 2, 64), x, table, start), "k must be contiguous"),
            (lambda: w(c, wide[:, :128].view(3, 2, 64), x, table, start), "k must be contiguous"),
            (lambda: w(c, x.transpose(0, 1), x, table, start), "k: shape"),
            (lambda: w(c, x, x, table, start, start), "offsets: shape"),
            (lambda: dilattn.cache_read(c, table, start, torch.zeros(4, dtype=torch.int32)), "without total"),
            (lambda: dilattn.cache_read(c, table, start, k=x.float()), "k: dtype"),
            (lambda: dilattn.cache_read(c, table, start, v=x[:2]), "v: shape"),
            (lambda: dilattn.decode(q[:, :3], c, table, start, [(8, 1)]), "3 query heads over 2"),
            (lambda: dilattn.decode(q[0], c, table, start, [(8, 1)]), "expected a"),
            (lambda: dilattn.decode(q, c, table, start, [(8, 1)], seq=start[:1]), "seq: shape"),
            (lambda: dilattn.decode(q, c, table[:2], start, [(8, 1)]), "3 tokens without seq"),
            (lambda: dilattn.decode(q, c, table, start, [(8, 1)], out=q.float()), "out: dtype"),
            (lambda: dilattn.decode(q, c, table, start, [(8, 1)], lse=q[:, :, 0].float().t()), "lse: shape"),
            (lambda: dilattn.decode(q, c, table, start, [(8, 1)], workspace=q), "workspace: ")):
        with pytest.raises(ValueError, match=match):
            call()
    assert all(n.endswith("_size") for n, _ in rec.calls)
