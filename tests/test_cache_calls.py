"""The compiled marshalling of the cache calls: what it takes, and what it leaves to dilattn.py."""
import numpy as np
import pytest
import torch

from cache_util import bf16, filled, i32, normal
from sparse_long_sequence_dilated_b200 import dilattn

WRITE, READ, DECODE = "cache_write", "cache_read", "decode"


def test_host_tensors_and_other_objects_are_left():
    calls = dilattn._calls()
    t = torch.zeros(3)
    for x in (t, None, 5, "k"):
        assert calls.cache_write(*[x] * 9) is None
        assert calls.cache_read(*[x] * 8) is None
        assert calls.decode(*[x] * 12) is None
    for f, n in ((calls.cache_write, 9), (calls.cache_read, 8), (calls.decode, 12)):
        with pytest.raises(TypeError, match=f"expected {n} arguments"):
            f(t)


def _setup(fmt="e4m3"):
    rng = np.random.default_rng(31)
    pair, table = filled(rng, [70, 33, 5], 2, 16, 64, fmt)
    k, v = (bf16(normal(rng, 3, 2, 64)).cuda() for _ in range(2))
    q = bf16(normal(rng, 3, 4, 64)).cuda()
    return pair.dev, i32(table), k, v, q, i32([60, 32, 4])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_it_makes_the_call_that_python_makes(fmt):
    """The plain form through the compiled call; with a stream given, through Python: same bits."""
    dev, table, k, v, q, at = _setup(fmt)
    calls, stream = dilattn._calls(), torch.cuda.current_stream()
    other = dilattn.Cache(*(t.clone() for t in dev))
    offsets = i32([0, 1, 2, 3])
    for off in (None, offsets):
        assert calls.cache_write(*dev, table, k, v, at, off) == (0,)
        dilattn.cache_write(other, k, v, table, at, off, stream=stream)
        for a, b in zip(dev, other):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        rc, a, b = calls.cache_read(*dev, table, at, off, 3)
        want = dilattn.cache_read(dev, table, at, off, 3, stream=stream)
        assert rc == 0 and torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert calls.cache_read(*dev, table, at, None, None)[1].shape == (3, 2, 64)
    fused = torch.cat([q, k, v], 1)  # strided rows
    assert calls.cache_write(*dev, table, fused[:, 4:6], fused[:, 6:], at, None) == (0,)
    ws = dilattn.decode_workspace(3, 4, 2, 64)
    out, lse = torch.empty_like(q), torch.empty((3, 4), device="cuda")
    seq = i32([0, 1, 2])
    want = dilattn.decode(q, dev, table, at, [(32, 1), (64, 2)], stream=stream)
    for pats in ([(32, 1), (64, 2)], ((32, 1), [64, 2])):
        for args in ((None,) * 4, (seq, out, lse, ws)):
            rc, a, b = calls.decode(*dev, table, fused[:, :4], at, pats, *args)
            assert rc == 0 and torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert a.data_ptr() == out.data_ptr() and b.data_ptr() == lse.data_ptr()
    # a refusal of the library comes back as its status
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    assert calls.decode(*dev, table, q, at, [(32, 1)], None, None, None, small)[0] == 4
    with pytest.raises(dilattn.DilattnError, match="WORKSPACE"):
        dilattn.decode(q, dev, table, at, [(32, 1)], workspace=small)
    assert dilattn.device_error() == 0


@pytest.mark.gpu
def test_what_does_not_fit_is_left_and_then_refused():
    dev, table, k, v, q, at = _setup()
    calls, offsets, ok = dilattn._calls(), i32([0, 1, 2, 3]), [(32, 1)]
    bad_caches = [dev._replace(v=dev.v[:2]), dev._replace(k=dev.k.view(torch.uint8)), dev._replace(v=dev.v.view(torch.int8)),
                  dev._replace(k_scale=dev.k_scale.double()), dev._replace(v_scale=dev.v_scale.cpu()),
                  dev._replace(k=dev.k.transpose(1, 2)), dev._replace(k=dev.k[0])]
    for c in bad_caches:
        for call in (lambda: calls.cache_write(*c, table, k, v, at, None), lambda: calls.cache_read(*c, table, at, None, None),
                     lambda: calls.decode(*c, table, q, at, ok, None, None, None, None)):
            assert call() is None
        with pytest.raises(ValueError):
            dilattn.cache_write(c, k, v, table, at)
    for t in (table.long(), table[0], table.t(), table.cpu(), table[:2]):
        assert calls.cache_write(*dev, t, k, v, at, None) is None
        with pytest.raises(ValueError):
            dilattn.cache_write(dev, k, v, t, at)
    for a in ((k[:2], v, at, None), (k, v.half(), at, None), (k.cpu(), v, at, None), (k, v[:, :1].expand(3, 2, 64), at, None),
              (k, v, at.long(), None), (k, v, at[:2], None), (k, v, at, at), (k[:2], v[:2], at, None)):
        assert calls.cache_write(*dev, table, *a) is None
        with pytest.raises(ValueError):
            dilattn.cache_write(dev, a[0], a[1], table, a[2], a[3])
    for a in ((at, offsets, None), (at, None, 2)):
        assert calls.cache_read(*dev, table, *a) is None
        with pytest.raises(ValueError):
            dilattn.cache_read(dev, table, *a)
    for kw in (dict(q=q[:, :3]), dict(q=q[0]), dict(q=q.float()), dict(pos=at.long()), dict(pos=at[:2]), dict(seq=at[:2]),
               dict(out=q[:2]), dict(lse=at), dict(workspace=q)):
        a = dict(dict(q=q, pos=at, patterns=ok, seq=None, out=None, lse=None, workspace=None), **kw)
        assert calls.decode(*dev, table, *a.values()) is None
        with pytest.raises(ValueError):
            dilattn.decode(a["q"], dev, table, a["pos"], ok, seq=a["seq"], out=a["out"], lse=a["lse"], workspace=a["workspace"])
    # pairs that only Python takes apart, and numbers that no int holds
    for pats in (np.array([[32, 1]]), [(np.int64(32), 1)], [(2 ** 31, 1)], [(0, 1)], [(32, 1, 1)], [], 7):
        assert calls.decode(*dev, table, q, at, pats, None, None, None, None) is None
    a = dilattn.decode(q, dev, table, at, ok)
    b = dilattn.decode(q, dev, table, at, [(np.int64(32), np.int64(1))])
    assert torch.equal(a[0], b[0])
    assert dilattn.device_error() == 0
