"""Refusals of the heads' norm and rotation, without a GPU."""
import ctypes as C

import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
from fsdp_sharded_optimizer_step_amd import binding

EINVAL, ERANGE, EOVERLAP = binding.ZERO_EINVAL, binding.ZERO_ERANGE, binding.ZERO_EOVERLAP
T, D = 10, 24


class _View(C.Structure):
    _fields_ = [("data_dev", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class _Heads(C.Structure):
    _fields_ = [("tensor", C.c_int32), ("heads", C.c_int32), ("x", _View), ("dy", _View), ("out", _View)]


class _Rotation(C.Structure):
    _fields_ = [("positions_dev", C.c_void_p), ("freqs_dev", C.c_void_p), ("position_bytes", C.c_int32),
                ("n_axes", C.c_int32), ("sections", C.c_int32 * 4), ("interleaved", C.c_int32)]


def test_packed_structures():
    """What the binding packs is what a C client fills in."""
    h = _Heads(3, 7, _View(at(1), 11, 12), _View(at(2), 21, 22), _View(at(3), 31, 32))
    assert binding._pack_heads(3, 7, at(1), 11, 12, at(2), 21, 22, at(3), 31, 32) == bytes(h)
    r = _Rotation(at(4), at(5), 8, 3, (C.c_int32 * 4)(1, 2, 3, 0), 1)
    packed = binding._pack_rotation(at(4), at(5), 8, 3, 1, 2, 3, 0, 1)
    assert len(packed) == C.sizeof(r) and packed[:44] == bytes(r)[:44]


def at(n, off=0):
    """A host address standing in for a device pointer; never read."""
    return 0x10000000 * n + off


@pytest.fixture(scope="module")
def L():
    return z.Layout([17, D, 600, D], 0, 4, 1)


def view(n, heads, ts=None, hs=D, off=0):
    return _View(at(n, off) if n else None, heads * D if ts is None else ts, hs)


def side(tensor, heads, base, **kw):
    v = dict(x=view(base, heads), dy=view(base + 1, heads), out=view(base + 2, heads))
    v.update(kw)
    return _Heads(tensor, heads, v["x"], v["dy"], v["out"])


def turn(sections=(6, 6), freqs=at(30), positions=at(31), pbytes=4, axes=None, inter=0):
    return _Rotation(positions, freqs, pbytes, len(sections) if axes is None else axes,
                     (C.c_int32 * 4)(*sections), inter)


def call(L, grad, q="q", k="k", rot=None, params=at(32), tokens=T, d=D, eps=1e-6, scale=1.0, flags=0, acc=at(33),
         out=at(34), ws=at(35), ws_bytes=1 << 20, handle="L"):
    q = side(1, 4, 10) if q == "q" else q
    k = side(3, 2, 20) if k == "k" else k
    rot = turn() if rot is None else rot
    ref = lambda s: None if s is None else C.byref(s)  # noqa: E731
    args = [L.handle if handle == "L" else None, params, tokens, d, eps, C.byref(rot), ref(q), ref(k)]
    if grad:
        return z.load().zero_head_norm_rotate_grad(*args, scale, flags, acc, out, ws, ws_bytes, None)
    return z.load().zero_head_norm_rotate(*args, None)


INF = float("inf")
q, k = lambda **kw: side(1, 4, 10, **kw), lambda **kw: side(3, 2, 20, **kw)  # noqa: E731
BOTH = [
    (EINVAL, dict(handle=None)), (EINVAL, dict(tokens=-1)), (EINVAL, dict(d=0)), (EINVAL, dict(d=23)),
    (EINVAL, dict(eps=-1.0)), (EINVAL, dict(eps=INF)), (EINVAL, dict(eps=float("nan"))),
    (EINVAL, dict(params=None)), (EINVAL, dict(q=side(2, 4, 10))), (EINVAL, dict(q=side(-2, 4, 10))),
    (EINVAL, dict(q=side(1, -1, 10))), (ERANGE, dict(q=side(4, 4, 10))), (ERANGE, dict(k=side(3, (1 << 14) + 1, 20))),
    (ERANGE, dict(tokens=(1 << 30) + 1)), (ERANGE, dict(d=513, q=side(-1, 4, 10), k=None)),
    (EINVAL, dict(rot=turn((7, 6)))), (EINVAL, dict(rot=turn((-1, 6)))), (EINVAL, dict(rot=turn(pbytes=2))),
    (EINVAL, dict(rot=turn(axes=5))), (EINVAL, dict(rot=turn(inter=2))), (EINVAL, dict(rot=turn(freqs=None))),
    (EINVAL, dict(rot=turn(positions=None))),
    (EINVAL, dict(q=q(x=view(0, 4)))), (EINVAL, dict(q=q(out=view(0, 4)))), (EINVAL, dict(k=k(x=view(20, 2, hs=-1)))),
    (ERANGE, dict(q=q(x=view(10, 4, hs=(1 << 40) + 1)))), (ERANGE, dict(q=q(x=view(10, 4, ts=1 << 40), ), tokens=1 << 20)),
    # rows of an output that meet
    (EINVAL, dict(q=q(out=view(12, 4, hs=D - 1)))), (EINVAL, dict(q=q(out=view(12, 4, ts=4 * D - 1)))),
    (EINVAL, dict(q=q(out=view(12, 4, ts=D, hs=T * D - 1)))), (EINVAL, dict(q=q(out=view(12, 4, ts=0)))),
    # memory
    (EOVERLAP, dict(q=q(out=view(10, 4)))), (EOVERLAP, dict(q=q(out=view(20, 4)))),
    (EOVERLAP, dict(q=q(out=view(22, 4)))), (EOVERLAP, dict(k=k(out=view(32, 2, off=40)))),
    (EOVERLAP, dict(k=k(out=view(31, 2, off=40)))), (EOVERLAP, dict(k=k(out=view(30, 2, off=80)))),
    (EOVERLAP, dict(q=q(out=view(12, 4, ts=5 * D)), k=k(out=view(12, 2, ts=5 * D, off=8 * D)))),
    (EOVERLAP, dict(q=q(out=view(12, 4, ts=6 * D)), k=k(out=view(12, 2, ts=6 * D, off=8 * D - 2)))),
]
GRAD = [
    (EINVAL, dict(scale=INF)), (EINVAL, dict(flags=8)), (EINVAL, dict(flags=4)), (EINVAL, dict(acc=None)),
    (EINVAL, dict(flags=2, out=None)), (EINVAL, dict(ws=None)), (EINVAL, dict(ws_bytes=100)),
    (EINVAL, dict(ws=at(35, 8))), (EINVAL, dict(q=q(dy=view(0, 4)))),
    (EOVERLAP, dict(q=q(out=view(11, 4)))), (EOVERLAP, dict(ws=at(10))), (EOVERLAP, dict(ws=at(12))),
    (EOVERLAP, dict(flags=2, out=at(33))), (EOVERLAP, dict(acc=at(11))), (EOVERLAP, dict(acc=at(35))),
]


@pytest.mark.parametrize("grad", [False, True])
def test_an_eps_beyond_binary32_is_refused(L, grad):
    assert call(L, grad, eps=3.5e38) == EINVAL and call(L, grad, eps=1e300) == EINVAL
    assert call(L, grad, eps=3e38, tokens=0) == 0


@pytest.mark.parametrize("grad", [False, True])
def test_both_refuse(L, grad):
    for status, bad in BOTH:
        assert call(L, grad, **bad) == status, bad


def test_the_gradient_refuses(L):
    for status, bad in GRAD:
        assert call(L, True, **bad) == status, bad


def test_nothing_to_do(L):
    for grad in (False, True):
        assert call(L, grad, tokens=0, q=q(x=view(0, 4), out=view(0, 4))) == 0
        assert call(L, grad, q=None, k=None) == 0
        assert call(L, grad, q=side(-1, 0, 10), k=None, params=None, acc=None) == 0


def test_workspace(L):
    f = z.load().zero_head_norm_rotate_grad_workspace
    ref = lambda s: None if s is None else C.byref(s)  # noqa: E731
    assert f(L.handle, T, D, ref(q()), ref(k())) > 0
    assert f(L.handle, T, D, ref(side(-1, 4, 10)), None) == 0 == f(L.handle, 0, D, ref(q()), None)
    assert f(None, T, D, ref(q()), None) == EINVAL and f(L.handle, T, D, ref(side(9, 4, 10)), None) == ERANGE
    # bounded by the launch's shape, however many tokens there are
    assert f(L.handle, 1 << 30, D, ref(q()), ref(k())) <= 64 << 20


def test_wrappers_refuse(L):
    b = torch.bfloat16
    new = lambda *s, dtype=b: torch.zeros(*s, dtype=dtype)  # noqa: E731
    x, y = new(T, 4, D), new(T, 2, D)
    params = new(L.padded)
    pos, f = new(T, dtype=torch.int32), new(12, dtype=torch.float64)

    def fwd(q=x, k=y, params=params, rot=z.Rotation(pos, f), qo=x, ko=y, wq=1, wk=3):
        z.zero_head_norm_rotate(L, wq, wk, params, q, k, 1e-6, rot, qo, ko)
    for bad in (dict(q=new(T, 4, D + 1)), dict(q=None), dict(ko=None), dict(qo=None, ko=None, q=None, k=None),
                dict(q=new(T, 4, D, dtype=torch.float32)), dict(q=new(T, 4, 2 * D)[..., ::2]), dict(qo=new(T, D)),
                dict(ko=new(T + 1, 2, D)), dict(params=new(L.padded - 1)), dict(params=new(L.padded, dtype=torch.float32)),
                dict(rot=z.Rotation(pos[1:], f)), dict(rot=z.Rotation(pos.float(), f)),
                dict(rot=z.Rotation(pos, f.float())), dict(rot=z.Rotation(pos, f, [6, 6])),
                dict(rot=z.Rotation(pos, f, [11])), dict(rot=z.Rotation(new(2, T, dtype=torch.int64), f)),
                dict(rot=z.Rotation(new(5, T, dtype=torch.int64), f, [2, 2, 2, 3, 3])), dict()):
        with pytest.raises(ValueError):
            fwd(**bad)
    with pytest.raises(z.ZeroError):
        fwd(wq=7)
    acc = torch.zeros(L.padded)

    def grad(dq=x, q=x, qx=x, acc=acc, flags=0, out=None, wq=1):
        z.zero_head_norm_rotate_grad(L, wq, 3, params, dq, y, q, y, 1e-6, None, qx, y, acc, 1.0, flags, out)
    for bad in (dict(dq=None), dict(q=None), dict(qx=None), dict(acc=None), dict(acc=acc[1:]), dict(flags=2),
                dict(dq=new(T, 4, D + 1)), dict()):
        with pytest.raises(ValueError):
            grad(**bad)
